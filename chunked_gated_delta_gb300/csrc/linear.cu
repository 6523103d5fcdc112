// linear.cu -- kda_linear: y = act(x w^T, scaled, + bias) + residual, with
// 16-bit or e4m3 operands on the tcgen05 tensor cores and the whole epilogue
// in fp32 from the accumulators.
//
//     acc[m, n] = sum_k x[m, k] w[n, k]
//     y[m, n]   = act(acc * x_scale[m] * w_scale[n] + bias[n]) + residual[m, n]
//
// The scales belong to rows of x and rows of w, so they factor out of the sum
// over k and cost one product each in the epilogue.
//
// One CTA takes 128 features (rows of w: the MMA's M) and NT tokens (rows of
// x: the MMA's N) of one slice of k.  Features on the MMA's M side let a batch
// of one to a few tokens use a narrow accumulator while w, which is what such
// a call has to read, streams through a deep shared-memory ring.  With few
// tiles, a cluster of CTAs shares one tile: each takes a slice of k, and they
// join their fp32 sums through distributed shared memory, in rank order, each
// CTA finishing a part of the tokens.
//
// Bound: for few tokens HBM (w), but at these sizes the fixed parts of a call
// weigh as much: 59 tokens x 4096 x 4096 in e4m3 with residual 7.1 us (w alone
// 2.5), 16 tokens in bf16 9.4 (w 5.0).  One token has a kernel of its own
// (linear_one.cu), many have linear_wide.cu; choose() below says which and why.
#include <cmath>

#include "linear.cuh"

namespace kda {
namespace {

constexpr int kLinThreads = 256;
constexpr int kLinWarps = kLinThreads / 32;
constexpr int kEarly = 2;           // tokens of a warp whose residual is loaded before the sums are there
constexpr int kFeatures = 128;      // rows of w per tile
constexpr int kMaxStages = 12;

template <int NT>
struct LinShape {
    static constexpr int kStageBytes = (kFeatures + NT) * kRowBytes;
    static constexpr int kFit = (kSmemMax - 2048) / kStageBytes;
    static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
    static constexpr int kSmem = kStages * kStageBytes + 1024;
    // accumulators that an fp32 y sums its stages of k in turn in (see linear_wide.cu on its segments); their
    // number is set by TMEM, so their share of the error grows with k: against 64 bits, 16 tokens at K = 2048,
    // 8192 and 32768 9.7e-8, 2.4e-7, 1.0e-6 (fp32 products 1.2e-7, 2.3e-7, 4.0e-7), 200 tokens 1.3e-7, 4.8e-7, 2.1e-6
    static constexpr int kAccs = NT <= 64 ? 8 : 512 / NT;
    static_assert(kStages * kStageBytes >= kFeatures * NT * 4, "the ring holds the tile's partial sums");
};

// grid: (cluster size x feature tiles, token tiles)
template <int NT, bool F8>
__global__ void __launch_bounds__(kLinThreads) kda_linear_kernel(const __grid_constant__ LinArgs a, int log_split) {
    using Shape = LinShape<NT>;
    constexpr int kStages = Shape::kStages;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t full[kStages], empty[kStages], done;
    __shared__ uint32_t tmem_base;
    __shared__ int s_fail;
    uint8_t* ring = ptx::align_smem_1024(raw);

    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0);
    const int split = 1 << log_split;
    const int rank = log_split ? (int)cluster_rank() : 0;
    const int n0 = (int)(blockIdx.x >> log_split) * kFeatures;
    const int m0 = (int)blockIdx.y * NT;
    const int kb0 = (int)((int64_t)a.kblocks * rank >> log_split);
    const int count = (int)((int64_t)a.kblocks * (rank + 1) >> log_split) - kb0;
    const int accs = a.out == KDA_DTYPE_F32 ? min(Shape::kAccs, count) : 1;
    const uint32_t cols = a.out == KDA_DTYPE_F32 ? NT * Shape::kAccs : NT < 32 ? 32 : NT;  // a power of two >= 32

    if (tid == 0) {
        ptx::prefetch_tmap(&a.tm_w);
        ptx::prefetch_tmap(&a.tm_x);
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
        }
        ptx::mbar_init(&done, 1);
        ptx::fence_mbar_init();
        s_fail = 0;
    }
    if (warp == 2) {
        ptx::tmem_alloc(&tmem_base, cols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    ptx::grid_dep_launch();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_base;
    ptx::grid_dep_wait();

    // What the end of the tile needs besides the sums is asked for now: a warp's
    // features' bias and scales, and the residual and scale of its first tokens.
    const int log_part = (31 - __clz(NT)) - log_split, part = 1 << log_part;
    const int tokens = min(NT, a.M - m0);
    const int lane = tid & 31, n = n0 + lane * 4, live = min(4, a.N - n);
    const bool wide = a.wide && live == 4;
    float bias[4], ws[4], xs[kEarly];
    uint4 early[kEarly];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bias[i] = a.bias && i < live ? a.bias[n + i] : 0.f;
        ws[i] = F8 && i < live ? a.w_scale[n + i] : 1.f;
    }
#pragma unroll
    for (int i = 0; i < kEarly; ++i) {
        const int c = warp + i * kLinWarps, t = (rank << log_part) + c;
        xs[i] = 1.f;
        early[i] = make_uint4(0u, 0u, 0u, 0u);
        if (c < part && t < tokens) {
            if (F8) xs[i] = a.x_scale[m0 + t];
            if (a.residual && wide) early[i] = load_four(a.residual, (int64_t)(m0 + t) * a.ldr + n, a.out);
        }
    }

    if (warp == 0 && elect_one()) {
        int issued = 0;
        bool ok = true;
        for (; issued < count; ++issued) {
            const int s = issued % kStages, round = issued / kStages;
            if (round > 0 && !wait_for(&empty[s], (round - 1) & 1)) {
                ok = false;
                break;
            }
            uint8_t* w = ring + s * Shape::kStageBytes;
            const int k = (kb0 + issued) * (F8 ? kRowBytes : kRowBytes / 2);
            ptx::mbar_arrive_expect_tx(&full[s], Shape::kStageBytes);
            ptx::tma_load_2d(w, &a.tm_w, &full[s], k, n0);
            ptx::tma_load_2d(w + kFeatures * kRowBytes, &a.tm_x, &full[s], k, m0);
        }
        if (!ok) {  // let the copies in flight land before the CTA unwinds
            s_fail = 1;
            for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
                wait_for(&full[i % kStages], (i / kStages) & 1);
        }
    } else if (warp == 1 && elect_one()) {
        bool ok = true;
        for (int i = 0; i < count && ok; ++i) {
            const int s = i % kStages;
            ok = wait_for(&full[s], (i / kStages) & 1);
            if (!ok) break;
            ptx::tc_fence_after();
            const uint32_t w = ptx::smem_u32(ring + s * Shape::kStageBytes);
            const uint64_t da = ptx::smem_desc(w, 0, 1024), db = ptx::smem_desc(w + kFeatures * kRowBytes, 0, 1024);
            const uint32_t d = tmem + (uint32_t)(i % accs * NT);
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // 32 bytes of k each
                if constexpr (F8) mma_f8(d, da + 2 * j, db + 2 * j, a.idesc, i >= accs || j > 0);
                else ptx::mma_bf16(d, da + 2 * j, db + 2 * j, a.idesc, i >= accs || j > 0);
            }
            ptx::mma_commit(&empty[s]);
        }
        if (ok) ptx::mma_commit(&done);
        else s_fail = 1;
    }
    __syncwarp();
    if (!wait_for(&done, 0, 2 * kWaitLimitNs)) s_fail = 1;
    ptx::tc_fence_after();
    __syncthreads();
    bool fail = s_fail != 0;

    // The tile's sums go to shared memory as [token][feature] in fp32, in the
    // ring, which is free once the MMAs (of every CTA of the cluster) are done;
    // with split > 1 each CTA finishes NT / split tokens, and gets their sums
    // over every slice of k.  From there a warp takes a token, a lane four
    // features, so y and the residual move in 256-byte rows.
    const int quarter = warp & 3;
    if (log_split) cluster_sync_all();
    if (!fail) {
        constexpr int kWarpCols = NT < 32 ? 16 : NT / 2;  // tokens of a warp's lane quarter
        const uint32_t mine = ptx::smem_u32(ring) + (uint32_t)(quarter * 32 + lane) * 4u;
        const int c0 = (warp >> 2) * kWarpCols;
        for (int c = c0; c < min(c0 + kWarpCols, tokens); c += 16) {
            float v[16];
            const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)c;
            ptx::tmem_ld16(at, v);
            ptx::tmem_ld_wait();
            for (int g = 1; g < accs; ++g) {
                float u[16];
                ptx::tmem_ld16(at + (uint32_t)(g * NT), u);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] += u[j];
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const uint32_t to = (uint32_t)(c + j) >> log_part;
                const uint32_t row = (uint32_t)((rank << log_part) + ((c + j) & (part - 1)));
                const uint32_t addr = mine + row * (kFeatures * 4u);
                if (log_split == 0)
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v[j]) : "memory");
                else if (c + j < tokens)
                    st_cluster_f32(peer_smem(addr, to), v[j]);
            }
        }
    }
    if (log_split) cluster_sync_all();
    else __syncthreads();
    if (!fail && live > 0) {
        const float4* sums = reinterpret_cast<const float4*>(ring) + lane;
        auto finish = [&](int c, float x_scale, uint4 r, bool have_r) {
            const int t = (rank << log_part) + c;
            if (c >= part || t >= tokens) return;
            float4 f = sums[c * (kFeatures / 4)];
            for (int k = 1; k < split; ++k) {
                const float4 u = sums[((k << log_part) + c) * (kFeatures / 4)];
                f.x += u.x;
                f.y += u.y;
                f.z += u.z;
                f.w += u.w;
            }
            float v[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = (F8 ? v[i] * (x_scale * ws[i]) : v[i]) + bias[i];
            if (a.out == KDA_DTYPE_F32) activate_all<4, false>(v, a.act);
            else activate_all<4, true>(v, a.act);
            const int64_t at = (int64_t)(m0 + t) * a.ldy + n, rat = (int64_t)(m0 + t) * a.ldr + n;
            if (wide) {
                if (a.residual && !have_r) r = load_four(a.residual, rat, a.out);
                if (a.out == KDA_DTYPE_F32) {
                    *reinterpret_cast<float4*>(static_cast<float*>(a.y) + at) =
                        make_float4(v[0] + __uint_as_float(r.x), v[1] + __uint_as_float(r.y),
                                    v[2] + __uint_as_float(r.z), v[3] + __uint_as_float(r.w));
                } else {
                    const bool f16 = a.out == KDA_DTYPE_F16;
                    const float2 lo = f16 ? from_b16x2<true>(r.x) : from_b16x2<false>(r.x);
                    const float2 hi = f16 ? from_b16x2<true>(r.y) : from_b16x2<false>(r.y);
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + at) =
                        make_uint2(pack_b16x2(v[0] + lo.x, v[1] + lo.y, f16), pack_b16x2(v[2] + hi.x, v[3] + hi.y, f16));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < live) {
                        if (a.residual) v[i] += load_out(a.residual, rat + i, a.out);
                        store_out(a.y, at + i, v[i], a.out);
                    }
            }
        };
#pragma unroll
        for (int i = 0; i < kEarly; ++i) finish(warp + i * kLinWarps, xs[i], early[i], true);
        for (int c = warp + kEarly * kLinWarps; c < part; c += kLinWarps)
            finish(c, F8 && m0 + (rank << log_part) + c < a.M ? a.x_scale[m0 + (rank << log_part) + c] : 1.f,
                   make_uint4(0u, 0u, 0u, 0u), false);
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 2) ptx::tmem_dealloc(tmem, cols);
    if (fail && tid == 0 && a.status) atomicOr(a.status, kStatusTimeout);
}

template <int NT, bool F8>
cudaError_t launch(const LinArgs& a, int log_split, cudaStream_t s) {
    using Shape = LinShape<NT>;
    auto kern = kda_linear_kernel<NT, F8>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape::kSmem);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((a.N + kFeatures - 1) / kFeatures) << log_split, (unsigned)((a.M + NT - 1) / NT));
    return launch_cluster(kern, grid, dim3(kLinThreads), Shape::kSmem, 1u << log_split, s, a, log_split);
}

template <int NT>
cudaError_t launch(const LinArgs& a, bool f8, int log_split, cudaStream_t s) {
    return f8 ? launch<NT, true>(a, log_split, s) : launch<NT, false>(a, log_split, s);
}

// Which kernel takes a call, and how it cuts it: the least of the modelled
// times.  The constants (us) were measured on GB300 at K = 32 to 4096, M = 1 to
// 27367, N = 4 to 8192: what a call costs beside its stages, a stage of k, the end
// of a tile, what its slices cost to join, and a further round of CTAs; over 160
// calls of sizes drawn at random its choices took 1% more than the best ones.  E.g. at N = K = 4096, 16 bits: M = 64 in tiles of 64
// tokens takes 18.2, 13.9, 12.0, 23.0 us for 1, 2, 4, 8 slices of k; M = 256
// takes 25.3 us in tiles of 64 and two slices, 17.6 in tiles of 128 and two,
// 18.9 in the wide kernel with 128 features, 26.5 with 256; M = 2048 takes 56.7
// in the wide kernel with 128, 46.0 with 256.  Rows of y off 16 bytes: 8192 x 4095
// x 4096 takes 338 us in tiles of 128 tokens, 148 in the wide kernel; 130 x 77 x
// 4096 6.5 in tiles of 64 and eight slices, 17.2 in the wide kernel; 391 x 3136 x
// 4096 (100 tiles in four slices are three rounds) 32.0 in tiles of 128 tokens and
// four slices, 20.0 in one, 17.3 in the wide kernel with 128 features.
struct Plan {
    bool wide;
    int tokens;     // per tile; of the wide kernel: features per tile
    int log_split;  // 2^log_split slices of k
};
Plan choose(int64_t M, int64_t N, int64_t bytes, int kblocks, bool rows_on_16, bool residual, bool f32) {
    const int sms = device_sm_count();
    const double stream = (double)bytes / 6.6e6;  // x and w once from HBM
    auto cost = [&](int64_t units, int64_t slots, double stages, double per_stage, double end, double call, double wave) {
        const double waves = (double)((units + slots - 1) / slots);
        return call + fmax(waves * stages * per_stage, stream) + waves * end + (waves - 1) * wave;
    };
    // Rows off 16 bytes go element by element, and a residual is waited for: after
    // every tile of the narrow kernel, after the last one of the wide kernel, which
    // ends a tile while the next is summed.
    const double odd = rows_on_16 ? 0.0 : 1.0, slow = odd + (residual ? 0.5 : 0.0);
    Plan best{false, 16, 0};
    double least = 1e30;
    auto offer = [&](Plan p, double c) {
        if (c < least) least = c, best = p;
    };
    constexpr struct { int tokens; double stage, end, join; } kNarrow[] = {
        {16, 0.186, 0.3, 0.0}, {32, 0.19, 0.5, 0.0}, {64, 0.205, 1.0, 0.4}, {128, 0.245, 2.9, 2.6}};
    for (const auto& t : kNarrow) {
        if (t.tokens < 64 && t.tokens < M) continue;      // a second token tile would read w again
        if ((M + t.tokens - 1) / t.tokens > 65535) continue;  // (rows of the grid)
        const int64_t tiles = (M + t.tokens - 1) / t.tokens * ((N + kFeatures - 1) / kFeatures);
        for (int ls = 0; ls <= 3 && (ls == 0 || kblocks >> ls >= 4); ++ls) {
            const int slots = ls < 3 ? sms : 112;         // clusters of 8 leave SMs of a GPC over
            offer({false, t.tokens, ls}, cost(tiles << ls, slots, (double)((kblocks + (1 << ls) - 1) >> ls), t.stage,
                                              (t.end + slow * (double)min((int64_t)t.tokens, M) / 32) / (1 << ls) + (ls ? t.join : 0.0),
                                              ls ? 4.5 : M > 64 ? 3.9 : 3.3, 4.0));
        }
        if (t.tokens >= M) break;
    }
    if (M > 64) {
        const int64_t tm = (M + 255) / 256;
        // a tile's sums hide the end of the one before only as far as they last
        const double end = (f32 ? 3.0 : 1.5) * (1.0 + odd * (2.0 * slow - 1.0));
        for (int tn = 128; tn <= 256; tn *= 2) {
            const double stage = tn == 128 ? 0.2 : 0.3, tile_end = tn == 128 ? end : (f32 ? 2.5 : 1.8) * end;
            offer({true, tn, 0}, cost(tm * ((N + tn - 1) / tn), sms / 2, kblocks, stage, 0.0,
                                      (tn == 128 ? 2.7 : 2.2) + tile_end, fmax(0.0, tile_end - kblocks * stage)));
        }
    }
    return best;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_linear(const void* x, const void* w, const float* bias, const void* residual,
                                 const float* x_scale, const float* w_scale, void* y, int64_t M, int64_t N, int64_t K,
                                 const kda_linear_opts* opts, int32_t* status_word, void* stream) {
    if (!opts || M < 0 || N < 1 || K < 1) return KDA_ERR_INVALID_ARG;
    const kda_linear_opts& p = *opts;
    const bool f8 = p.io_dtype == KDA_DTYPE_E4M3;
    if (p.io_dtype != KDA_DTYPE_BF16 && p.io_dtype != KDA_DTYPE_F16 && !f8) return KDA_ERR_INVALID_ARG;
    if (p.out_dtype != KDA_DTYPE_BF16 && p.out_dtype != KDA_DTYPE_F16 && p.out_dtype != KDA_DTYPE_F32)
        return KDA_ERR_INVALID_ARG;
    if (p.act < KDA_ACT_NONE || p.act > KDA_ACT_LOGSIGMOID || p.reserved != 0) return KDA_ERR_INVALID_ARG;
    if (f8 != (x_scale != nullptr) || f8 != (w_scale != nullptr)) return KDA_ERR_INVALID_ARG;
    const int es = dtype_bytes(p.io_dtype), oes = dtype_bytes(p.out_dtype);
    int64_t ldx = p.x_stride ? p.x_stride : K, ldw = p.w_stride ? p.w_stride : K;
    const int64_t ldr = p.residual_stride ? p.residual_stride : N, ldy = p.y_stride ? p.y_stride : N;
    if (ldx < K || ldw < K || ldr < N || ldy < N) return KDA_ERR_INVALID_ARG;
    if (M > INT32_MAX / 2 || N > INT32_MAX / 2 || K > INT32_MAX / 2) return KDA_ERR_UNSUPPORTED;
    if (M == 0) return KDA_OK;
    if (!x || !w || !y) return KDA_ERR_INVALID_ARG;
    const int64_t whole = (K * es + 15) / 16 * 16 / es;  // a single row has no stride: any that a TMA map takes
    if (M == 1) ldx = whole;
    if (N == 1) ldw = whole;
    if (!is_aligned(x, 16) || !is_aligned(w, 16) || ldx * es % 16 != 0 || ldw * es % 16 != 0 ||
        !is_aligned(y, oes) || !is_aligned(residual, oes) || !is_aligned(bias, 4) || !is_aligned(x_scale, 4) ||
        !is_aligned(w_scale, 4) || !is_aligned(status_word, 4))
        return KDA_ERR_ALIGNMENT;

    const int kblocks = (int)((K * es + kRowBytes - 1) / kRowBytes);
    LinArgs a{};
    a.bias = bias;
    a.residual = residual;
    a.x_scale = x_scale;
    a.w_scale = w_scale;
    a.y = y;
    a.status = status_word;
    a.ldr = ldr;
    a.ldy = ldy;
    a.M = (int)M;
    a.N = (int)N;
    a.kblocks = kblocks;
    a.out = p.out_dtype;
    a.act = p.act;
    a.io = p.io_dtype;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool rows_on_16 = is_aligned(y, 16) && ldy * oes % 16 == 0 &&
                            (!residual || (is_aligned(residual, 16) && ldr * oes % 16 == 0));
    const int four = 4 * oes;  // bytes of a lane's features
    a.wide = is_aligned(y, four) && ldy % 4 == 0 && (!residual || (is_aligned(residual, four) && ldr % 4 == 0));
    if (M == 1) return launch_linear_one(a, x, w, K, ldw, s) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    const Plan plan = choose(M, N, (M + N) * K * es, kblocks, rows_on_16, residual != nullptr, oes == 4);
    if (plan.wide)
        return launch_linear_wide(a, plan.tokens, x, w, K, ldx, ldw, rows_on_16, s) == cudaSuccess ? KDA_OK
                                                                                                  : KDA_ERR_CUDA;
    const int nt = plan.tokens, log_split = plan.log_split;
    if (!rows_map(&a.tm_w, p.io_dtype, w, N, K, ldw, kFeatures) || !rows_map(&a.tm_x, p.io_dtype, x, M, K, ldx, nt))
        return KDA_ERR_CUDA;
    a.idesc = f8                             ? idesc_e4m3_f32(kFeatures, nt)
              : p.io_dtype == KDA_DTYPE_BF16 ? ptx::idesc_bf16_f32(kFeatures, nt, 0, 0)
                                             : ptx::idesc_f16_f32(kFeatures, nt, 0, 0);
    cudaError_t e;
    switch (nt) {
    case 16: e = launch<16>(a, f8, log_split, s); break;
    case 32: e = launch<32>(a, f8, log_split, s); break;
    case 64: e = launch<64>(a, f8, log_split, s); break;
    default: e = launch<128>(a, f8, log_split, s); break;
    }
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
