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
#include "linear.cuh"

namespace kda {
namespace {

constexpr int kLinThreads = 128;
constexpr int kFeatures = 128;      // rows of w per tile
constexpr int kMaxStages = 12;

template <int NT>
struct LinShape {
    static constexpr int kStageBytes = (kFeatures + NT) * kRowBytes;
    static constexpr int kFit = (kSmemMax - 2048) / kStageBytes;
    static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
    static constexpr int kSmem = kStages * kStageBytes + 1024;
    static constexpr int kCols = NT < 32 ? 32 : NT;  // TMEM columns (a power of two, at least 32)
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
        ptx::tmem_alloc(&tmem_base, Shape::kCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_base;

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
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // 32 bytes of k each
                if constexpr (F8) mma_f8(tmem, da + 2 * j, db + 2 * j, a.idesc, i > 0 || j > 0);
                else ptx::mma_bf16(tmem, da + 2 * j, db + 2 * j, a.idesc, i > 0 || j > 0);
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

    const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
    const int n = n0 + tid;  // a thread's feature
    const bool n_ok = n < a.N;
    const float bias = a.bias && n_ok ? a.bias[n] : 0.f;
    const float ws = F8 && n_ok ? a.w_scale[n] : 1.f;
    const int tokens = min(NT, a.M - m0);
    auto finish = [&](float v, int m) {
        if (F8) v *= a.x_scale[m] * ws;
        v += bias;
        activate_all<1, false>(&v, a.act);
        if (a.residual) v += load_out(a.residual, (int64_t)m * a.ldr + n, a.out);
        store_out(a.y, (int64_t)m * a.ldy + n, v, a.out);
    };

    if (log_split == 0) {
        for (int c = 0; c < tokens && !fail; c += 16) {
            float v[16];
            ptx::tmem_ld16(lanes + c, v);
            ptx::tmem_ld_wait();
            if (n_ok) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (c + j < tokens) finish(v[j], m0 + c + j);
            }
        }
    } else {
        // Each CTA of the cluster finishes NT / split tokens.  Their partial
        // sums from every slice of k are gathered in its ring, which is free
        // once all the cluster's MMAs are done.
        const int log_part = (31 - __clz(NT)) - log_split, part = 1 << log_part;
        cluster_sync_all();
        const uint32_t mine = ptx::smem_u32(ring) + (uint32_t)tid * 4u;
        for (int c = 0; c < tokens && !fail; c += 16) {
            float v[16];
            ptx::tmem_ld16(lanes + c, v);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                if (c + j < tokens) {
                    const int to = (c + j) >> log_part;
                    const uint32_t row = (uint32_t)((rank << log_part) + ((c + j) & (part - 1)));
                    st_cluster_f32(peer_smem(mine + row * (kFeatures * 4u), (uint32_t)to), v[j]);
                }
            }
        }
        cluster_sync_all();
        const float* sums = reinterpret_cast<const float*>(ring) + tid;
        for (int c = 0; c < part && !fail; ++c) {
            const int t = (rank << log_part) + c;
            if (t < tokens && n_ok) {
                float v = 0.f;
                for (int r = 0; r < split; ++r) v += sums[((r << log_part) + c) * kFeatures];
                finish(v, m0 + t);
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 2) ptx::tmem_dealloc(tmem, Shape::kCols);
    if (fail && tid == 0 && a.status) atomicOr(a.status, kStatusTimeout);
}

template <int NT, bool F8>
cudaError_t launch(const LinArgs& a, int log_split, cudaStream_t s) {
    using Shape = LinShape<NT>;
    auto kern = kda_linear_kernel<NT, F8>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << log_split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((a.N + kFeatures - 1) / kFeatures) << log_split, (unsigned)((a.M + NT - 1) / NT));
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = Shape::kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, log_split);
}

template <int NT>
cudaError_t launch(const LinArgs& a, bool f8, int log_split, cudaStream_t s) {
    return f8 ? launch<NT, true>(a, log_split, s) : launch<NT, false>(a, log_split, s);
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
    if (rows_on_16 && ((M + 255) / 256) * ((N + 255) / 256) >= 64)
        return launch_linear_wide(a, 256, x, w, K, ldx, ldw, s) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    const int nt = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256;
    const int64_t tiles_m = (M + nt - 1) / nt, tiles_n = (N + kFeatures - 1) / kFeatures;
    if (tiles_m > 65535) return KDA_ERR_UNSUPPORTED;
    // As many slices of k as fill the SMs with one CTA each, at least four stages of k in each.
    int log_split = 0;
    while (log_split < 3 && (tiles_m * tiles_n << (log_split + 1)) <= device_sm_count() &&
           kblocks >> (log_split + 1) >= 4)
        ++log_split;

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
    case 128: e = launch<128>(a, f8, log_split, s); break;
    default: e = launch<256>(a, f8, log_split, s); break;
    }
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
