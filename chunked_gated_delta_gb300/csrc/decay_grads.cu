// decay_grads.cu -- gradients of linear attention with a decay per head
// (formulas of the forward: decay.cuh).
//
// With S the state before a chunk and dS the gradient of the state after it,
// both kept by decay_states.cu, the chunks are independent: one CTA each per
// head. In a chunk, D_ij = exp(G_i - G_j) for j <= i (else 0),
//     P = scale D (q k^T),  dP = scale D (do v^T)
//     dq = scale exp(G_i) do S^T + dP k
//     dk = exp(G_last - G_j) v dS^T + dP^T q
//     dv = exp(G_last - G_j) k dS + P^T do
// and, g_t being the decay of every pair of tokens that it lies between,
//     dg_t = exp(G_last) <S, dS> + sum_{i >= t} q_i . far dq_i + sum_{j < t} k_j . far dk_j
//            + sum_{j < t <= i} (q_i . k_j) dP_ij
// (far: the parts through S and dS). Each of its sums stays within the chunk, so dg is right to
// fp32's own rounding wherever it is in the sequence; the usual suffix sum of q . dq - k . dk over the
// sequence takes it as a difference of ever longer sums. For the same reason S and dS are kept in
// two parts of 16 bits each, both multiplied for the far parts of dq and dk.
//
// All products are tcgen05 MMAs of 128 tokens. Their scores are computed transposed (lane j, column
// i), so that P^T and dP^T are operands out of TMEM for dv and dk; dP for dq goes through
// shared memory. The far parts are scaled by rows in registers and put back, and the near products add to them.
#include "decay.cuh"

namespace kda {
namespace {

constexpr int kWorkers = 256, kGradThreads = kWorkers + 32;

template <int KB, int VB>
struct GradShape {
    static constexpr int K = 64 * KB, V = 64 * VB;
    static constexpr int kXBytes = KB * 16384, kYBytes = VB * 16384, kPart = V * 128, kStateBytes = V * K * 2;
    static constexpr int kQ = 0, kK = kQ + kXBytes, kV = kK + kXBytes, kDo = kV + kYBytes;
    static constexpr int kDp = kDo + kYBytes;         // dP^T [j][i]
    static constexpr int kRing = kDp + 32768;         // 64 keys of S (hi, lo) and dS (hi, lo)
    static constexpr int kSmall = kRing + 4 * kPart;
    struct Small {
        ChunkDecay decay;
        float column[kDecayChunk];  // exp of the decay from the end of the 32 tokens before to a column
        float whole;
        uint32_t tmem;
        int32_t fail;
        uint64_t in_full, clean, scores, s_full, ring_read, ring_done, far, far_ok, p_ok, dv_far, dv_ok, dqk, dv;
    };
    // when everything else is done, in place of dP: the parts of dg
    struct Sums {
        float far_q[2][kDecayChunk], far_k[2][kDecayChunk], near_k[2][kDecayChunk], near_q[4][kDecayChunk], across[8];
    };
    static constexpr int kSmem = kSmall + (int)sizeof(Small);
    static_assert(sizeof(Small) >= sizeof(DecayScratch) && sizeof(Sums) <= 32768, "what shares memory fits");
    static_assert(kSmem <= 227 * 1024, "fits an SM");
};
// TMEM columns. P^T lies at 0 .. 31 and 96 .. 127 of the first scores' (each half written by those who have read what
// was there), dP^T likewise of the second's; dv in the middle of both.
constexpr uint32_t kT0 = 0, kT1 = 128, kTdq = 256, kTdk = 384;
__device__ __forceinline__ constexpr uint32_t p_column(int ks) { return (uint32_t)(ks * 8 + (ks >= 4 ? 64 : 0)); }
__device__ __forceinline__ constexpr uint32_t dv_column(int vb) { return (uint32_t)(32 + vb * 128); }

// x[0 .. 31] of each lane: lane l gets the sum over the lanes of x[l].
__device__ __forceinline__ float transposed_sum(float (&x)[32], int lane) {
#pragma unroll
    for (int n = 16; n >= 1; n >>= 1) {
        const bool up = lane & n;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float give = up ? x[i] : x[i + n], keep = up ? x[i + n] : x[i];
            x[i] = keep + __shfl_xor_sync(~0u, give, n);
        }
    }
    return x[0];
}

template <int KB, int VB, bool F16>
__global__ void __launch_bounds__(kGradThreads, 1) kda_decay_grads_kernel(const __grid_constant__ DecayGradArgs a) {
    using Shape = GradShape<KB, VB>;
    constexpr int K = Shape::K, V = Shape::V;
    extern __shared__ __align__(1024) uint8_t raw[];
    auto& sm = *reinterpret_cast<typename Shape::Small*>(raw + Shape::kSmall);
    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;

    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int item = blockIdx.x / a.H, h = blockIdx.x - item * a.H, hq = h / a.group;
    DecayPiece at;
    if (!find_piece<kGradThreads>(a.seqs, item, false, false, *reinterpret_cast<DecayScratch*>(&sm), at)) {
        if (blockIdx.x == 0 && tid == 0 && a.status) atomicOr(a.status, kStatusBadSeqlens);
        return;
    }
    if (at.n < 0) return;
    const int row0 = at.bos + at.piece * kDecayChunk, valid = min(at.len - at.piece * kDecayChunk, kDecayChunk);
    const int64_t unit = (int64_t)(at.chunk_base + at.piece) * a.H + h;
    __syncthreads();  // the search's scratch is free

    if (tid == 0) {
        for (uint64_t* b : {&sm.in_full, &sm.scores, &sm.s_full, &sm.ring_done, &sm.far, &sm.dv_far, &sm.dqk, &sm.dv})
            ptx::mbar_init(b, 1);
        for (uint64_t* b : {&sm.clean, &sm.ring_read, &sm.far_ok, &sm.p_ok, &sm.dv_ok}) ptx::mbar_init(b, kWorkers / 32);
        ptx::fence_mbar_init();
        sm.fail = 0;
    }
    if (warp == 8) {
        ptx::tmem_alloc(&sm.tmem, 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = sm.tmem;
    volatile int32_t* fail = &sm.fail;
    auto wait = [&](uint64_t& bar, uint32_t parity) {
        wait_or_note(&bar, parity, fail);
        return !*fail;
    };

    if (warp == 8) {
        if (elect_one()) {
            const uint8_t* S = a.kept + unit * 2 * Shape::kStateBytes;
            const uint8_t* dS = a.dkept + unit * 2 * Shape::kStateBytes;
            uint8_t* ring = raw + Shape::kRing;
            auto load_states = [&](int kb) {
                ptx::mbar_arrive_expect_tx(&sm.s_full, 4 * Shape::kPart);
                for (int part = 0; part < 2; ++part) {
                    const int64_t off = part * Shape::kStateBytes + kb * Shape::kPart;
                    bulk_load(ring + part * Shape::kPart, S + off, Shape::kPart, &sm.s_full);
                    bulk_load(ring + (2 + part) * Shape::kPart, dS + off, Shape::kPart, &sm.s_full);
                }
            };
            ptx::mbar_arrive_expect_tx(&sm.in_full, 2 * Shape::kXBytes + 2 * Shape::kYBytes);
            for (int b = 0; b < KB; ++b) {
                ptx::tma_load_3d(raw + Shape::kQ + b * 16384, &a.tm_q, &sm.in_full, b * 64, hq, row0);
                ptx::tma_load_3d(raw + Shape::kK + b * 16384, &a.tm_k, &sm.in_full, b * 64, hq, row0);
            }
            for (int b = 0; b < VB; ++b) {
                ptx::tma_load_3d(raw + Shape::kV + b * 16384, &a.tm_v, &sm.in_full, b * 64, h, row0);
                ptx::tma_load_3d(raw + Shape::kDo + b * 16384, &a.tm_do, &sm.in_full, b * 64, h, row0);
            }
            load_states(0);
            int loads = 1;  // fills of the ring asked for
            const uint32_t base = ptx::smem_u32(raw);
            const uint64_t q_k = ptx::smem_desc(base + Shape::kQ, 16, 1024), k_k = ptx::smem_desc(base + Shape::kK, 16, 1024);
            const uint64_t v_k = ptx::smem_desc(base + Shape::kV, 16, 1024), do_k = ptx::smem_desc(base + Shape::kDo, 16, 1024);
            const uint64_t q_mn = ptx::smem_desc(base + Shape::kQ, 16384, 1024), k_mn = ptx::smem_desc(base + Shape::kK, 16384, 1024);
            const uint64_t do_mn = ptx::smem_desc(base + Shape::kDo, 16384, 1024), dp_mn = ptx::smem_desc(base + Shape::kDp, 16384, 1024);
            const uint64_t ring_mn = ptx::smem_desc(base + Shape::kRing, 16384, 1024);
            const uint64_t ring_k = ptx::smem_desc(base + Shape::kRing, 16, 1024);
            auto step = [](int ks) { return (uint64_t)(((ks >> 2) * 16384 + (ks & 3) * 32) >> 4); };  // along rows of 64
            bool ok = false;
            do {
                if (!wait(sm.clean, 0)) break;
                ptx::tc_fence_after();
                constexpr uint32_t id_scores = idesc16<F16>(128, 128, 0, 0);
#pragma unroll 1
                for (int ks = 0; ks < 4 * KB; ++ks) ptx::mma_bf16(tmem + kT0, k_k + step(ks), q_k + step(ks), id_scores, ks > 0);
#pragma unroll 1
                for (int ks = 0; ks < 4 * VB; ++ks) ptx::mma_bf16(tmem + kT1, v_k + step(ks), do_k + step(ks), id_scores, ks > 0);
                ptx::mma_commit(&sm.scores);
                bool through = true;
#pragma unroll 1
                for (int kb = 0; kb < KB && through; ++kb) {
                    if (!(through = wait(sm.s_full, kb & 1))) break;
                    ptx::tc_fence_after();
                    constexpr uint32_t id = idesc16<F16>(128, 64, 0, 1);
#pragma unroll 1
                    for (int ks = 0; ks < 8 * VB; ++ks) {  // hi, then lo
                        const int part = ks / (4 * VB), kv = ks % (4 * VB);
                        const uint64_t at_v = (uint64_t)((part * Shape::kPart + kv * 2048) >> 4);
                        ptx::mma_bf16(tmem + kTdq + kb * 64, do_k + step(kv), ring_mn + at_v, id, ks > 0);
                        ptx::mma_bf16(tmem + kTdk + kb * 64, v_k + step(kv), ring_mn + (2 * Shape::kPart >> 4) + at_v, id, ks > 0);
                    }
                    if (kb == KB - 1) ptx::mma_commit(&sm.far);
                    ptx::mma_commit(&sm.ring_done);
                    if (!(through = wait(sm.ring_done, kb & 1) && wait(sm.ring_read, kb & 1))) break;
                    if (kb + 1 < KB) {
                        load_states(kb + 1);
                    } else {  // dS once more, its leading parts
                        ptx::mbar_arrive_expect_tx(&sm.s_full, KB * Shape::kPart);
                        for (int b = 0; b < KB; ++b)
                            bulk_load(ring + b * Shape::kPart, dS + b * Shape::kPart, Shape::kPart, &sm.s_full);
                    }
                    ++loads;
                }
                if (!through || !wait(sm.p_ok, 0) || !wait(sm.s_full, KB & 1)) break;
                ptx::tc_fence_after();
#pragma unroll 1
                for (int vb = 0; vb < VB; ++vb)
#pragma unroll 1
                    for (int ks = 0; ks < 4 * KB; ++ks)
                        ptx::mma_bf16(tmem + dv_column(vb), k_k + step(ks),
                                      ring_k + (((ks >> 2) * Shape::kPart + vb * 8192 + (ks & 3) * 32) >> 4),
                                      idesc16<F16>(128, 64, 0, 0), ks > 0);
                ptx::mma_commit(&sm.dv_far);
                if (!wait(sm.far_ok, 0)) break;
                ptx::tc_fence_after();
#pragma unroll 1
                for (int ks = 0; ks < 8; ++ks) {
                    ptx::mma_bf16(tmem + kTdq, dp_mn + ks * 128, k_mn + ks * 128, idesc16<F16>(128, K, 1, 1), 1);
                    mma_ts(tmem + kTdk, tmem + kT1 + p_column(ks), q_mn + ks * 128, idesc16<F16>(128, K, 0, 1), 1);
                }
                ptx::mma_commit(&sm.dqk);
                if (!wait(sm.dv_ok, 0)) break;
                ptx::tc_fence_after();
#pragma unroll 1
                for (int vb = 0; vb < VB; ++vb)
#pragma unroll 1
                    for (int ks = 0; ks < 8; ++ks)
                        mma_ts(tmem + dv_column(vb), tmem + kT0 + p_column(ks), do_mn + ks * 128 + vb * 1024,
                               idesc16<F16>(128, 64, 0, 1), 1);
                ptx::mma_commit(&sm.dv);
                ok = true;
            } while (false);
            if (!ok) {  // let the copies in flight land
                wait_for(&sm.in_full, 0);
                wait_for(&sm.s_full, (loads - 1) & 1);
            }
        }
    } else {
        const int quarter = warp & 3, half = warp >> 2, row = quarter * 32 + lane;
        const uint32_t t_row = tmem + ((uint32_t)(quarter * 32) << 16);
        constexpr int kCols = K / 2, kColsV = V / 2;  // columns of a thread
        auto arrive = [&](uint64_t& bar) {
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bar);
        };
        float far_q = 0.f, far_k = 0.f, near_k = 0.f, near_q[2] = {0.f, 0.f}, across = 0.f;
        {
            if (warp == 0) {
                const Pair all = sum_decay(load_g(a.g, a.g_stride, h, row0, valid, lane), sm.decay, lane);
                if (lane == 0) sm.whole = whole_decay(all);
            }
            named_sync(1, kWorkers);
            const ChunkDecay& d = sm.decay;
            const float hi = d.hi[row], lo = d.lo[row];
            if (half == 0 && quarter > 0) sm.column[row] = exp2_fast((hi - d.hi[quarter * 32 - 1]) + (lo - d.lo[quarter * 32 - 1]));
            wait(sm.in_full, 0);
            if (row >= valid) {  // rows behind the sequence: a zero factor would not hold back a NaN
                uint8_t* p = raw + (half ? Shape::kV : Shape::kQ) + row * 128;
                constexpr int kMost = KB > VB ? KB : VB;
#pragma unroll 1
                for (int c = 0; c < 16 * kMost; ++c) {
                    const int blocks = half ? VB : KB, which = c / (8 * kMost), in = c % (8 * kMost);
                    if ((in >> 3) < blocks)
                        *reinterpret_cast<uint4*>(p + (which * blocks + (in >> 3)) * 16384 + ((in & 7) << 4)) =
                            make_uint4(0u, 0u, 0u, 0u);
                }
            }
            ptx::fence_proxy_async_smem();
            arrive(sm.clean);
            named_sync(1, kWorkers);  // column is there

            // <S, dS>, 64 keys at a time: the same element of all four tiles, wherever it lies
#pragma unroll 1
            for (int kb = 0; kb < KB; ++kb) {
                wait(sm.s_full, kb & 1);
                const uint8_t* p = raw + Shape::kRing + tid * 16;
#pragma unroll 2
                for (int c = 0; c < Shape::kPart / 4096; ++c, p += 4096) {
                    uint4 w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint4*>(p + i * Shape::kPart);
                    auto dot = [&](uint32_t s, uint32_t sl, uint32_t t, uint32_t tl) {
                        const float2 x = from_b16x2<F16>(s), xl = from_b16x2<F16>(sl), y = from_b16x2<F16>(t), yl = from_b16x2<F16>(tl);
                        across = fmaf(x.x + xl.x, y.x + yl.x, across);
                        across = fmaf(x.y + xl.y, y.y + yl.y, across);
                    };
                    dot(w[0].x, w[1].x, w[2].x, w[3].x);
                    dot(w[0].y, w[1].y, w[2].y, w[3].y);
                    dot(w[0].z, w[1].z, w[2].z, w[3].z);
                    dot(w[0].w, w[1].w, w[2].w, w[3].w);
                }
                arrive(sm.ring_read);
            }
            float up_q = 1.f, up_k = 1.f;
            if (F16) up_q = a.kept_scale[unit], up_k = a.dkept_scale[unit];
            across *= up_q * up_k;

            // P^T and dP^T: row j, half of the columns i, 32 at a time, inwards from the ends (see kT0)
            wait(sm.scores, 0);
            ptx::tc_fence_after();
#pragma unroll 1
            for (int n = 0; n < 2; ++n) {
                const int b = half ? 3 - n : n;
                uint32_t p[16], dp[16];
                if (b >= quarter) {
                    float s[32], e[32];
                    ptx::tmem_ld16(t_row + kT0 + 32 * b, s);
                    ptx::tmem_ld16(t_row + kT0 + 32 * b + 16, s + 16);
                    ptx::tmem_ld16(t_row + kT1 + 32 * b, e);
                    ptx::tmem_ld16(t_row + kT1 + 32 * b + 16, e + 16);
                    ptx::tmem_ld_wait();
                    if (b > quarter) {
                        const int end = 32 * b - 1;
                        const float r = a.scale * exp2_fast((d.hi[end] - hi) + (d.lo[end] - lo));
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            const float2 f = *reinterpret_cast<const float2*>(&sm.column[32 * b + 2 * c]);
                            const float f0 = r * f.x, f1 = r * f.y;
                            p[c] = pack_b16x2(s[2 * c] * f0, s[2 * c + 1] * f1, F16);
                            e[2 * c] *= f0, e[2 * c + 1] *= f1;
                            dp[c] = pack_b16x2(e[2 * c], e[2 * c + 1], F16);
                            s[2 * c] *= e[2 * c], s[2 * c + 1] *= e[2 * c + 1];
                            near_k += s[2 * c] + s[2 * c + 1];
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            const float f = a.scale * exp2_fast((d.hi[32 * b + c] - hi) + (d.lo[32 * b + c] - lo));
                            const float x = c >= lane ? s[c] * f : 0.f;
                            e[c] = c >= lane ? e[c] * f : 0.f;
                            s[c] = c > lane ? s[c] * e[c] : 0.f;  // (a token's pair with itself has no decay)
                            near_k += s[c];
                            if (c & 1) {
                                p[c >> 1] = pack_b16x2(__uint_as_float(p[c >> 1]), x, F16);
                                dp[c >> 1] = pack_b16x2(e[c - 1], e[c], F16);
                            } else {
                                p[c >> 1] = __float_as_uint(x);
                            }
                        }
                    }
                    near_q[b & 1] = transposed_sum(s, lane);
                } else {
#pragma unroll
                    for (int c = 0; c < 16; ++c) p[c] = dp[c] = 0u;
                }
                const uint32_t column = p_column(2 * b);
                tmem_st16(t_row + kT0 + column, p);
                tmem_st16(t_row + kT1 + column, dp);
                uint8_t* to = raw + Shape::kDp + (b >> 1) * 16384 + row * 128;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    *reinterpret_cast<uint4*>(to + ((((b & 1) * 4 + c) ^ (row & 7)) << 4)) =
                        make_uint4(dp[4 * c], dp[4 * c + 1], dp[4 * c + 2], dp[4 * c + 3]);
            }
            tmem_st_wait();
            ptx::tc_fence_before();
            ptx::fence_proxy_async_smem();
            arrive(sm.p_ok);

            // the far parts of dq and dk: scaled by rows, and their products with q and k
            const float seen = exp2_fast(hi + lo), kept = exp2_fast(gap(d, kDecayChunk - 1, hi, lo));
            wait(sm.far, 0);
            ptx::tc_fence_after();
            auto scaled = [&](uint32_t column, float f, const uint8_t* x) {
                float sum = 0.f;
#pragma unroll 1
                for (int c0 = half * kCols; c0 < (half + 1) * kCols; c0 += 16) {
                    float u[16];
                    ptx::tmem_ld16(t_row + column + c0, u);
                    ptx::tmem_ld_wait();
                    const uint8_t* p = x + (c0 >> 6) * 16384 + row * 128;
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const uint4 w = *reinterpret_cast<const uint4*>(p + (((((c0 & 63) >> 3) + g) ^ (row & 7)) << 4));
                        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 y = from_b16x2<F16>(in[e]);
                            u[8 * g + 2 * e] *= f, u[8 * g + 2 * e + 1] *= f;
                            sum = fmaf(u[8 * g + 2 * e], y.x, sum);
                            sum = fmaf(u[8 * g + 2 * e + 1], y.y, sum);
                        }
                    }
                    tmem_st16(t_row + column + c0, reinterpret_cast<const uint32_t*>(u));
                }
                return sum;
            };
            far_q = scaled(kTdq, a.scale * seen * up_q, raw + Shape::kQ);
            far_k = scaled(kTdk, kept * up_k, raw + Shape::kK);
            tmem_st_wait();
            ptx::tc_fence_before();
            arrive(sm.far_ok);

            wait(sm.dv_far, 0);
            ptx::tc_fence_after();
            // (a thread's half of V: a block of 64 columns of it, or half of one)
            const uint32_t t_dv = t_row + (VB == 2 ? dv_column(half) : dv_column(0) + half * kColsV);
#pragma unroll 1
            for (int c = 0; c < kColsV; c += 16) {
                float u[16];
                ptx::tmem_ld16(t_dv + c, u);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) u[e] *= kept * up_k;
                tmem_st16(t_dv + c, reinterpret_cast<const uint32_t*>(u));
            }
            tmem_st_wait();
            ptx::tc_fence_before();
            arrive(sm.dv_ok);

            // out
            const bool live = row < valid;
            const int64_t tok = (int64_t)row0 + row;
            auto store16 = [&](uint32_t t, uint16_t* to, int count) {
#pragma unroll 1
                for (int c = 0; c < count; c += 16) {
                    float u[16];
                    ptx::tmem_ld16(t + c, u);
                    ptx::tmem_ld_wait();
                    uint32_t w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = pack_b16x2(u[2 * e], u[2 * e + 1], F16);
                    if (live) {
                        *reinterpret_cast<uint4*>(to + c) = make_uint4(w[0], w[1], w[2], w[3]);
                        *reinterpret_cast<uint4*>(to + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                    }
                }
            };
            auto store32 = [&](uint32_t t, float* to, int count) {
#pragma unroll 1
                for (int c = 0; c < count; c += 16) {
                    float u[16];
                    ptx::tmem_ld16(t + c, u);
                    ptx::tmem_ld_wait();
                    if (live)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<float4*>(to + c + 4 * e) = make_float4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]);
                }
            };
            wait(sm.dqk, 0);
            ptx::tc_fence_after();
            if (a.group == 1) {
                const int64_t to = (tok * a.H + h) * K + half * kCols;
                store16(t_row + kTdq + half * kCols, static_cast<uint16_t*>(a.dq) + to, kCols);
                store16(t_row + kTdk + half * kCols, static_cast<uint16_t*>(a.dk) + to, kCols);
            } else {
                const int64_t to = (tok * a.H + h) * K + half * kCols;
                store32(t_row + kTdq + half * kCols, static_cast<float*>(a.dq) + to, kCols);
                store32(t_row + kTdk + half * kCols, static_cast<float*>(a.dk) + to, kCols);
            }
            wait(sm.dv, 0);
            ptx::tc_fence_after();
            store16(t_dv, a.dv + (tok * a.H + h) * V + half * kColsV, kColsV);
        }
        // dg, from sums that every thread has a part of (dP has been read)
        auto& sums = *reinterpret_cast<typename Shape::Sums*>(raw + Shape::kDp);
        across += __shfl_xor_sync(~0u, across, 16);
        across += __shfl_xor_sync(~0u, across, 8);
        across += __shfl_xor_sync(~0u, across, 4);
        across += __shfl_xor_sync(~0u, across, 2);
        across += __shfl_xor_sync(~0u, across, 1);
        named_sync(1, kWorkers);
        sums.far_q[half][row] = far_q;
        sums.far_k[half][row] = far_k;
        sums.near_k[half][row] = near_k;
        sums.near_q[quarter][half * 64 + lane] = near_q[0];
        sums.near_q[quarter][half * 64 + 32 + lane] = near_q[1];
        if (lane == 0) sums.across[warp] = across;
        named_sync(1, kWorkers);
        if (warp == 0 && !sm.fail) {
            float later[4], before[4], all = 0.f;
            for (int w = 0; w < 8; ++w) all += sums.across[w];
            all *= sm.whole;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 4 * lane + i;
                const float nq = (sums.near_q[0][t] + sums.near_q[1][t]) + (sums.near_q[2][t] + sums.near_q[3][t]);
                later[i] = (sums.far_q[0][t] + sums.far_q[1][t]) + (nq - (sums.near_k[0][t] + sums.near_k[1][t]));
                before[i] = sums.far_k[0][t] + sums.far_k[1][t];
            }
            // later: sums from t on; before: sums up to t, t itself not among them
#pragma unroll
            for (int i = 2; i >= 0; --i) later[i] += later[i + 1];
#pragma unroll
            for (int i = 1; i < 4; ++i) before[i] += before[i - 1];
            float right = later[0], left = before[3];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const float r = __shfl_down_sync(~0u, right, off), l = __shfl_up_sync(~0u, left, off);
                if (lane + off < 32) right += r;
                if (lane >= off) left += l;
            }
            right = __shfl_down_sync(~0u, right, 1);
            left = __shfl_up_sync(~0u, left, 1);
            if (lane == 31) right = 0.f;
            if (lane == 0) left = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 4 * lane + i;
                if (t < valid) a.dg[((int64_t)row0 + t) * a.H + h] = all + (later[i] + right) + (left + (i ? before[i - 1] : 0.f));
            }
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 8) ptx::tmem_dealloc(tmem, 512);
    if (sm.fail && tid == 0 && a.status) atomicOr(a.status, kStatusTimeout);
}

template <int KB, int VB, bool F16>
cudaError_t launch_shape(const DecayGradArgs& a, cudaStream_t s) {
    using Shape = GradShape<KB, VB>;
    auto kern = kda_decay_grads_kernel<KB, VB, F16>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape::kSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3((unsigned)(a.seqs.pieces * a.H)), dim3(kGradThreads), (size_t)Shape::kSmem, s, a);
}

// The gradients of q and k, summed over the value heads that share them: in fp32 [rows, Hqk, group, K] each.
__global__ void __launch_bounds__(256) kda_decay_group_kernel(const float* dq32, const float* dk32, void* dq, void* dk,
                                                              int64_t fours, int K4, int group, int f16) {
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const float* in = blockIdx.y ? dk32 : dq32;
    uint2* out = static_cast<uint2*>(blockIdx.y ? dk : dq);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < fours; i += (int64_t)gridDim.x * 256) {
        const int64_t head = i / K4;
        const float4* p = reinterpret_cast<const float4*>(in) + head * group * K4 + (i - head * K4);
        float4 s = *p;
        for (int g = 1; g < group; ++g) {
            const float4 x = p[(int64_t)g * K4];
            s = make_float4(s.x + x.x, s.y + x.y, s.z + x.z, s.w + x.w);
        }
        out[i] = make_uint2(pack_b16x2(s.x, s.y, f16), pack_b16x2(s.z, s.w, f16));
    }
}

// dg of a decay per head: the sum over all tokens, 256 rows at a time and then those sums, in a fixed order.
constexpr int kGateRows = 256;
__global__ void __launch_bounds__(256) kda_decay_gate_rows_kernel(const float* dg, float* part, int64_t rows, int H) {
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int64_t r0 = (int64_t)blockIdx.x * kGateRows, r1 = min(r0 + kGateRows, rows);
    const int h = blockIdx.y * 256 + threadIdx.x;
    if (h >= H) return;
    double s = 0.0;
    for (int64_t r = r0; r < r1; ++r) s += (double)dg[r * H + h];
    part[(int64_t)blockIdx.x * H + h] = (float)s;
}
__global__ void __launch_bounds__(256) kda_decay_gate_kernel(const float* part, float* dg, int64_t parts, int H) {
    __shared__ double sums[256];
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int h = blockIdx.x;
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < parts; i += 256) s += (double)part[i * H + h];
    sums[threadIdx.x] = s;
    for (int n = 128; n > 0; n >>= 1) {
        __syncthreads();
        if (threadIdx.x < n) sums[threadIdx.x] += sums[threadIdx.x + n];
    }
    if (threadIdx.x == 0) dg[h] = (float)sums[0];
}

}  // namespace

cudaError_t launch_decay_grads(const DecayGradArgs& a, int K, int V, bool f16, cudaStream_t s) {
    if (K == 128) {
        if (V == 128) return f16 ? launch_shape<2, 2, true>(a, s) : launch_shape<2, 2, false>(a, s);
        return f16 ? launch_shape<2, 1, true>(a, s) : launch_shape<2, 1, false>(a, s);
    }
    if (V == 128) return f16 ? launch_shape<1, 2, true>(a, s) : launch_shape<1, 2, false>(a, s);
    return f16 ? launch_shape<1, 1, true>(a, s) : launch_shape<1, 1, false>(a, s);
}

cudaError_t launch_decay_group(const float* dq32, const float* dk32, void* dq, void* dk, int64_t rows, int heads, int K,
                               int group, bool f16, int sms, cudaStream_t s) {
    const int64_t fours = rows * heads * (K / 4), blocks = (fours + 255) / 256;
    return launch_dependent(kda_decay_group_kernel, dim3((unsigned)(blocks < 16 * sms ? blocks : 16 * sms), 2), dim3(256),
                            (size_t)0, s, dq32, dk32, dq, dk, fours, K / 4, group, (int)f16);
}

cudaError_t launch_decay_gate(const float* dg, float* part, float* out, int64_t rows, int H, cudaStream_t s) {
    const int64_t parts = (rows + kGateRows - 1) / kGateRows;
    if (parts > 0) {
        const cudaError_t e = launch_dependent(kda_decay_gate_rows_kernel, dim3((unsigned)parts, (unsigned)((H + 255) / 256)),
                                               dim3(256), (size_t)0, s, dg, part, rows, H);
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(kda_decay_gate_kernel, dim3((unsigned)H), dim3(256), (size_t)0, s, part, out, parts, H);
}

}  // namespace kda
