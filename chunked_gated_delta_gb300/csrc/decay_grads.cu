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
// All products are tcgen05 MMAs of 128 tokens. The scores are computed transposed (lane j, column
// i), so that P^T and dP^T are operands out of TMEM for dv and dk; dP for dq goes through
// shared memory. The far parts are scaled by rows in registers and put back, and the near products add
// to them. S and dS come 64 values at a time; outputs leave by TMA from where their inputs were.
//
// Value heads that share q and k: two of them are a cluster of two CTAs; each gives the other its fp32 dq and
// dk of half of the rows, straight into the other's shared memory, while dv and dg are made, and adds up
// the half that it keeps (4 x 4096 x 32 heads in pairs 550 us, against 635 with fp32 parts in HBM and a kernel that adds
// them up). More heads leave such parts: pairs that add up two of four or eight took 625 and 617 us against 618 and 609,
// clusters of four and eight that read one another's tiles 629 and 785.
//
// Bound: the chain of a tile's phases (one CTA of 226 KB per SM): loads 2.3 thousand cycles, scores 1.9, P and
// dP 3.1, the second half of the states until 8.9, far parts 1.7, near products and stores 6 (1.9 GHz; tensor cores
// 23% busy, issue 33%). 352 KB a tile: 4 x 8192 tokens x 32 heads of 128 x 128
// 595 us, 4.8 TB/s; the states' scan before it 370 us, 5.7 TB/s; both together 967. First as 8 warps
// with stores by threads 888 us for this kernel. A persistent form that loads the next tile's do and states early
// measured the same (1012 for both).
#include "decay.cuh"

namespace kda {
namespace {

constexpr int kWorkers = 512, kWorkerWarps = kWorkers / 32, kGradThreads = kWorkers + 32;
// Of the 16 blocks of 32 x 32 scores six lie right of the diagonal: their warps have nothing to do while the others make
// P and dP, and take <S, dS> meanwhile.
constexpr int kDotWarps = 6;

template <int KB, int VB>
struct GradShape {
    static constexpr int K = 64 * KB, V = 64 * VB;
    static constexpr int kXBytes = KB * 16384, kYBytes = VB * 16384, kPart = K * 128, kStateBytes = V * K * 2;
    static constexpr int kQ = 0, kK = kQ + kXBytes, kV = kK + kXBytes, kDo = kV + kYBytes;
    static constexpr int kDp = kDo + kYBytes;         // dP^T [j][i]
    static constexpr int kRing = kDp + 32768;         // 64 values of S (hi, lo) and dS (hi, lo), each x all keys
    static constexpr int kSmall = kRing + 4 * kPart;
    struct Small {
        ChunkDecay decay;
        float column[kDecayChunk];  // exp of the decay from the end of the 32 tokens before to a column
        float whole;
        int32_t rise;                     // fp16: see rise_of
        uint32_t top[2][kWorkerWarps];    // fp16: the largest of a warp's scores, and of do v^T
        uint32_t tmem;
        int32_t fail;
        uint64_t may_give, given;  // of a pair: the other's rows may be given to it, it has given this one's
        uint64_t in_full, clean, scores, s_full, ring_read, ring_done, far, far_ok, p_ok, dv_far, dv_ok, dqk, dv;
    };
    // when everything else is done, in place of dP: the parts of dg
    struct Sums {
        float far_q[4][kDecayChunk], far_k[4][kDecayChunk], near_k[4][kDecayChunk], near_q[4][kDecayChunk];
        float across[kDotWarps], later[4], before[4];
    };
    static constexpr int kSmem = kSmall + (int)sizeof(Small);
    static_assert(sizeof(Small) >= sizeof(DecayScratch) && sizeof(Sums) <= 32768, "what shares memory fits");
    static_assert(kSmem <= 227 * 1024, "fits an SM");
    static_assert(4 * kPart == 2 * kXBytes, "a group's fp32 dq and dk fit where q and k, and the states, were");
    // Where part `part` of 64 values of dS lies, the vb'th time.
    static __host__ __device__ constexpr int d_state(int vb, int part) {
        return vb == 0 ? kRing + (2 + part) * kPart : part == 0 ? kRing + 3 * kPart : kV;
    }
};
// TMEM columns: the scores, and when all of them have been read P^T, dP^T and dv in their place; dq and dk.
constexpr uint32_t kT0 = 0, kT1 = 128, kTp = kT0, kTdp = kT0 + 64, kTdv = kT1, kTdq = 256, kTdk = 384;

// A barrier of all threads of a cluster, in two halves: writes before the one are seen after the other.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// Where the other CTA of a pair has what lies at this one's shared address `at`.
__device__ __forceinline__ uint32_t in_cta(uint32_t at, int rank) {
    uint32_t there;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
    return there;
}
__device__ __forceinline__ void arrive_there(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// bytes of this CTA's shared memory into another's, whose barrier counts them
__device__ __forceinline__ void bulk_push(uint32_t to, uint32_t from, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to),
                 "r"(from), "r"(bytes), "r"(bar)
                 : "memory");
}

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
        for (uint64_t* b : {&sm.clean, &sm.far_ok, &sm.p_ok, &sm.dv_ok}) ptx::mbar_init(b, kWorkerWarps);
        ptx::mbar_init(&sm.ring_read, kDotWarps);
        ptx::mbar_init(&sm.may_give, 1);
        ptx::mbar_init(&sm.given, 1);
        ptx::fence_mbar_init();
        if (a.paired) ptx::mbar_arrive_expect_tx(&sm.given, 2 * 64 * K * 4);
        sm.fail = 0;
    }
    if (warp == kWorkerWarps) {
        ptx::tmem_alloc(&sm.tmem, 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    // (not before: it counts from a block's first thread that runs it, and a dependent that shares this SM could take the
    // TMEM that this block still needs)
    ptx::grid_dep_launch();
    const uint32_t tmem = sm.tmem;
    if (a.paired) cluster_arrive();  // this CTA's barriers are there
    volatile int32_t* fail = &sm.fail;
    auto wait = [&](uint64_t& bar, uint32_t parity) {
        wait_or_note(&bar, parity, &sm.fail);
        return !*fail;
    };
    auto wait_cluster = [&](uint64_t& bar, uint32_t parity) {
        wait_or_note<true>(&bar, parity, &sm.fail);
        return !*fail;
    };

    if (warp == kWorkerWarps) {
        if (elect_one()) {
            const uint8_t* S = a.kept + unit * 2 * Shape::kStateBytes;
            const uint8_t* dS = a.dkept + unit * 2 * Shape::kStateBytes;
            // 64 values of the states at a time. The second time dS's leading part has the place of the first's other
            // part (the first is kept for dv), and its own other part that of v's first half, which is done with.
            auto load_states = [&](int vb) {
                ptx::mbar_arrive_expect_tx(&sm.s_full, 4 * Shape::kPart);
                for (int part = 0; part < 2; ++part) {
                    const int64_t off = part * Shape::kStateBytes + vb * Shape::kPart;
                    bulk_load(raw + Shape::kRing + part * Shape::kPart, S + off, Shape::kPart, &sm.s_full);
                    bulk_load(raw + Shape::d_state(vb, part), dS + off, Shape::kPart, &sm.s_full);
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
            auto part_mn = [&](int at) { return ptx::smem_desc(base + at, 8192, 1024); };  // 64 values x keys, N = keys
            auto part_k = [&](int at) { return ptx::smem_desc(base + at, 16, 1024); };     // the same, N = values
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
                for (int vb = 0; vb < VB && through; ++vb) {
                    if (!(through = wait(sm.s_full, vb & 1))) break;
                    ptx::tc_fence_after();
                    constexpr uint32_t id = idesc16<F16>(128, K, 0, 1);
#pragma unroll 1
                    for (int part = 0; part < 2; ++part) {
                        const uint64_t s = part_mn(Shape::kRing + part * Shape::kPart), ds = part_mn(Shape::d_state(vb, part));
#pragma unroll 1
                        for (int ks = 0; ks < 4; ++ks) {
                            const uint32_t more = vb + part + ks > 0;
                            ptx::mma_bf16(tmem + kTdq, do_k + step(4 * vb + ks), s + ks * 128, id, more);
                            ptx::mma_bf16(tmem + kTdk, v_k + step(4 * vb + ks), ds + ks * 128, id, more);
                        }
                    }
                    if (vb == VB - 1) ptx::mma_commit(&sm.far);
                    if (vb + 1 < VB) {
                        ptx::mma_commit(&sm.ring_done);
                        if (!(through = wait(sm.ring_done, 0) && wait(sm.ring_read, 0))) break;
                        load_states(vb + 1);
                        ++loads;
                    }
                }
                // The tile that probably comes next on this SM, if it is of this sequence, into L2.
                const int ahead = (blockIdx.x + a.sms) / a.H - item, next_h = (blockIdx.x + a.sms) % a.H;
                if (at.piece + ahead < at.pieces) {
                    const int row = row0 + ahead * kDecayChunk, next_hq = next_h / a.group;
                    for (int b = 0; b < KB; ++b) {
                        ptx::tma_prefetch_3d(&a.tm_q, b * 64, next_hq, row);
                        ptx::tma_prefetch_3d(&a.tm_k, b * 64, next_hq, row);
                    }
                    for (int b = 0; b < VB; ++b) {
                        ptx::tma_prefetch_3d(&a.tm_v, b * 64, next_h, row);
                        ptx::tma_prefetch_3d(&a.tm_do, b * 64, next_h, row);
                    }
                    const int64_t next = (int64_t)(at.chunk_base + at.piece + ahead) * a.H + next_h;
                    ptx::bulk_prefetch_l2(a.kept + next * 2 * Shape::kStateBytes, 2 * Shape::kStateBytes);
                    ptx::bulk_prefetch_l2(a.dkept + next * 2 * Shape::kStateBytes, 2 * Shape::kStateBytes);
                }
                if (!through || !wait(sm.p_ok, 0)) break;
                ptx::tc_fence_after();
#pragma unroll 1
                for (int vb = 0; vb < VB; ++vb) {
                    const uint64_t ds = part_k(Shape::d_state(vb, 0));
#pragma unroll 1
                    for (int ks = 0; ks < 4 * KB; ++ks)
                        ptx::mma_bf16(tmem + kTdv + vb * 64, k_k + step(ks), ds + (((ks >> 2) * 8192 + (ks & 3) * 32) >> 4),
                                      idesc16<F16>(128, 64, 0, 0), ks > 0);
                }
                ptx::mma_commit(&sm.dv_far);
                if (!wait(sm.far_ok, 0)) break;
                ptx::tc_fence_after();
#pragma unroll 1
                for (int ks = 0; ks < 8; ++ks) {
                    ptx::mma_bf16(tmem + kTdq, dp_mn + ks * 128, k_mn + ks * 128, idesc16<F16>(128, K, 1, 1), 1);
                    mma_ts(tmem + kTdk, tmem + kTdp + ks * 8, q_mn + ks * 128, idesc16<F16>(128, K, 0, 1), 1);
                }
                ptx::mma_commit(&sm.dqk);
                if (!wait(sm.dv_ok, 0)) break;
                ptx::tc_fence_after();
#pragma unroll 1
                for (int ks = 0; ks < 8; ++ks)
                    mma_ts(tmem + kTdv, tmem + kTp + ks * 8, do_mn + ks * 128, idesc16<F16>(128, V, 0, 1), 1);
                ptx::mma_commit(&sm.dv);
                ok = true;
            } while (false);
            if (!ok) {  // let the copies in flight land
                wait_for(&sm.in_full, 0);
                wait_for(&sm.s_full, (loads - 1) & 1);
            }
        }
    } else {
        // 16 warps: a quarter of the rows each (TMEM's lanes), and a quarter of the columns.
        const int quarter = warp & 3, part = warp >> 2, row = quarter * 32 + lane;
        const uint32_t t_row = tmem + ((uint32_t)(quarter * 32) << 16), base = ptx::smem_u32(raw);
        constexpr int kCols = K / 4, kColsV = V / 4;  // columns of a thread
        auto arrive = [&](uint64_t& bar) {
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bar);
        };
        float far_q = 0.f, far_k = 0.f, near_k = 0.f, near_q = 0.f, across = 0.f;
        if (warp == 0) {
            const LoadedG g = load_g(a.g, a.g_stride, h, row0, valid, lane);
            const Pair all = sum_decay(g, sm.decay, lane);
            const int rise = F16 ? rise_of(g) : 0;
            if (lane == 0) sm.whole = whole_decay(all), sm.rise = rise;
        }
        if (F16 && lane == 0) sm.top[0][warp] = sm.top[1][warp] = 0u;  // (warps right of the diagonal have no scores)
        float up_q = 1.f, up_k = 1.f;
        if (F16) up_q = a.kept_scale[unit], up_k = a.dkept_scale[unit];
        named_sync(1, kWorkers);
        const ChunkDecay& d = sm.decay;
        const float hi = d.hi[row], lo = d.lo[row];
        if (part == 0 && quarter > 0) sm.column[row] = exp2_fast((hi - d.hi[quarter * 32 - 1]) + (lo - d.lo[quarter * 32 - 1]));
        wait(sm.in_full, 0);
        if (valid < kDecayChunk) {  // rows behind the sequence: a zero factor would not hold back a NaN
            if (row >= valid && part < 4) {
                const uint32_t to = base + (part == 0 ? Shape::kQ : part == 1 ? Shape::kK : part == 2 ? Shape::kV : Shape::kDo) + row * 128;
#pragma unroll 1
                for (int c = 0; c < 8 * (part < 2 ? KB : VB); ++c) sts128(to + (c >> 3) * 16384 + ((c & 7) << 4), 0u, 0u, 0u, 0u);
            }
        }
        ptx::fence_proxy_async_smem();
        arrive(sm.clean);

        // <S, dS>, 64 values at a time: the same element of all four tiles, wherever it lies
        const int dot_warp = part < quarter ? quarter * (quarter - 1) / 2 + part : -1;  // 0 .. 5
        auto dot_states = [&](int vb) {
            wait(sm.s_full, vb & 1);
            const uint32_t s = base + Shape::kRing, ds = base + Shape::d_state(vb, 0), dsl = base + Shape::d_state(vb, 1);
#pragma unroll 1
            for (int c = (dot_warp * 32 + lane) * 16; c < Shape::kPart; c += kDotWarps * 512) {
                const uint4 w[4] = {lds128(s + c), lds128(s + c + Shape::kPart), lds128(ds + c), lds128(dsl + c)};
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
        };
        named_sync(1, kWorkers);  // column is there

        // P and dP as fp16 have to be near the top of its range, or small ones lose their bits and large ones overflow: a
        // power of two for the chunk's P and one for its dP, which the far parts of dv, and of dq and dk, are multiplied by and
        // the outputs divided (4 x 8192 tokens x 32 heads of 128 x 128, with the scan: 1039 us, without any 1004).
        auto power = [&](int which) {
            const uint32_t top = __reduce_max_sync(~0u, sm.top[which][lane & (kWorkerWarps - 1)]);
            return score_power(__uint_as_float(top) * fabsf(a.scale), sm.rise);
        };
        // P^T and dP^T: row j, 32 columns i
        {
            const int b = part;
            uint32_t p[16], dp[16];
            if (b >= quarter) {
                wait(sm.scores, 0);
                ptx::tc_fence_after();
                float s[32], e[32];
                ptx::tmem_ld16(t_row + kT0 + 32 * b, s);
                ptx::tmem_ld16(t_row + kT0 + 32 * b + 16, s + 16);
                ptx::tmem_ld16(t_row + kT1 + 32 * b, e);
                ptx::tmem_ld16(t_row + kT1 + 32 * b + 16, e + 16);
                ptx::tmem_ld_wait();
                float up_p = 1.f, up_d = 1.f;
                if constexpr (F16) {
                    float most_s = 0.f, most_e = 0.f;
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const bool pair = b > quarter || c >= lane;
                        most_s = fmaxf(most_s, pair ? fabsf(s[c]) : 0.f);
                        most_e = fmaxf(most_e, pair ? fabsf(e[c]) : 0.f);
                    }
                    const uint32_t top_s = __reduce_max_sync(~0u, __float_as_uint(most_s));
                    const uint32_t top_e = __reduce_max_sync(~0u, __float_as_uint(most_e));
                    if (lane == 0) sm.top[0][warp] = top_s, sm.top[1][warp] = top_e;
                    named_sync(8, 32 * (kWorkerWarps - kDotWarps));
                    up_p = power_of_two(power(0)), up_d = power_of_two(power(1));
                }
                if (b > quarter) {
                    const int end = 32 * b - 1;
                    const float r = a.scale * exp2_fast((d.hi[end] - hi) + (d.lo[end] - lo));
                    const uint64_t r2 = pair_of(r, r);
                    uint64_t sum = 0;  // (two zeros)
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float2 column = *reinterpret_cast<const float2*>(&sm.column[32 * b + 2 * c]);
                        const uint64_t f = mul2(r2, pair_of(column.x, column.y)), x = pair_of(s[2 * c], s[2 * c + 1]);
                        const float2 scaled = floats_of(F16 ? mul2(mul2(x, f), pair_of(up_p, up_p)) : mul2(x, f));
                        p[c] = pack_b16x2(scaled.x, scaled.y, F16);
                        const uint64_t y = mul2(pair_of(e[2 * c], e[2 * c + 1]), f), m = mul2(x, y);
                        const float2 dscaled = floats_of(F16 ? mul2(y, pair_of(up_d, up_d)) : y), pair = floats_of(m);
                        dp[c] = pack_b16x2(dscaled.x, dscaled.y, F16);
                        s[2 * c] = pair.x, s[2 * c + 1] = pair.y;
                        sum = add2(sum, m);
                    }
                    const float2 both = floats_of(sum);
                    near_k = both.x + both.y;
                } else {
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const float f = a.scale * exp2_fast((d.hi[32 * b + c] - hi) + (d.lo[32 * b + c] - lo));
                        const float x = c >= lane ? (F16 ? up_p * (s[c] * f) : s[c] * f) : 0.f;
                        e[c] = c >= lane ? e[c] * f : 0.f;
                        s[c] = c > lane ? s[c] * e[c] : 0.f;  // (a token's pair with itself has no decay)
                        near_k += s[c];
                        if (c & 1) {
                            p[c >> 1] = pack_b16x2(__uint_as_float(p[c >> 1]), x, F16);
                            dp[c >> 1] = F16 ? pack_b16x2(up_d * e[c - 1], up_d * e[c], F16) : pack_b16x2(e[c - 1], e[c], F16);
                        } else {
                            p[c >> 1] = __float_as_uint(x);
                        }
                    }
                }
                near_q = transposed_sum(s, lane);
            } else {
                dot_states(0);
#pragma unroll
                for (int c = 0; c < 16; ++c) p[c] = dp[c] = 0u;
            }
            const uint32_t to = swizzled_row(base + Shape::kDp + (b >> 1) * 16384, row);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                sts128(to ^ (((b & 1) * 4 + c) << 4), dp[4 * c], dp[4 * c + 1], dp[4 * c + 2], dp[4 * c + 3]);
            ptx::tc_fence_before();
            named_sync(1, kWorkers);  // all scores have been read
            ptx::tc_fence_after();
            tmem_st16(t_row + kTp + 16 * b, p);
            tmem_st16(t_row + kTdp + 16 * b, dp);
        }
        tmem_st_wait();
        ptx::tc_fence_before();
        ptx::fence_proxy_async_smem();
        arrive(sm.p_ok);
#pragma unroll 1
        for (int vb = 1; vb < VB; ++vb)
            if (dot_warp >= 0) dot_states(vb);
        across *= up_q * up_k;
        float p_up = 1.f, p_down = 1.f, d_up = 1.f, d_down = 1.f;
        if constexpr (F16) {
            const int p = power(0), d = power(1);
            p_up = power_of_two(p), p_down = power_of_two(-p), d_up = power_of_two(d), d_down = power_of_two(-d);
        }

        // the far parts of dq and dk: scaled by rows, and their products with q and k
        const float seen = exp2_fast(hi + lo), kept = exp2_fast(gap(d, kDecayChunk - 1, hi, lo));
        wait(sm.far, 0);
        ptx::tc_fence_after();
        auto scaled = [&](uint32_t column, float f, uint32_t x) {
            uint64_t sum = 0;  // (two zeros)
            const uint64_t f2 = pair_of(f, f);
#pragma unroll 1
            for (int c0 = part * kCols; c0 < (part + 1) * kCols; c0 += 16) {
                float u[16];
                ptx::tmem_ld16(t_row + column + c0, u);
                const uint32_t p = swizzled_row(x + (c0 >> 6) * 16384, row);
                const uint4 w[2] = {lds128(p ^ ((c0 & 63) << 1)), lds128(p ^ (((c0 & 63) << 1) + 16))};
                ptx::tmem_ld_wait();
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const uint32_t in[4] = {w[g].x, w[g].y, w[g].z, w[g].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 y = from_b16x2<F16>(in[e]);
                        const uint64_t x = mul2(pair_of(u[8 * g + 2 * e], u[8 * g + 2 * e + 1]), f2);
                        sum = fma2(x, pair_of(y.x, y.y), sum);
                        const float2 now = floats_of(x);
                        u[8 * g + 2 * e] = now.x, u[8 * g + 2 * e + 1] = now.y;
                    }
                }
                tmem_st16(t_row + column + c0, reinterpret_cast<const uint32_t*>(u));
            }
            const float2 both = floats_of(sum);
            return both.x + both.y;
        };
        far_q = scaled(kTdq, a.scale * seen * up_q * d_up, base + Shape::kQ) * d_down;
        far_k = scaled(kTdk, kept * up_k * d_up, base + Shape::kK) * d_down;
        tmem_st_wait();
        ptx::tc_fence_before();
        arrive(sm.far_ok);

        const uint32_t t_dv = t_row + kTdv + part * kColsV;
        wait(sm.dv_far, 0);
        ptx::tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < kColsV; c += 16) {
            float u[16];
            ptx::tmem_ld16(t_dv + c, u);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) u[e] *= kept * up_k * p_up;
            tmem_st16(t_dv + c, reinterpret_cast<const uint32_t*>(u));
        }
        tmem_st_wait();
        ptx::tc_fence_before();
        arrive(sm.dv_ok);

        // Out: whole tiles by TMA, from where inputs were that have been read by then; rows of a sequence's last chunk
        // by their threads.
        const bool live = row < valid, staged = valid == kDecayChunk;
        const int64_t tok = (int64_t)row0 + row;
        auto store16 = [&](uint32_t t, int col, int count, uint32_t tile, uint16_t* to, float down) {
#pragma unroll 1
            for (int c = 0; c < count; c += 16) {
                float u[16];
                ptx::tmem_ld16(t + c, u);
                ptx::tmem_ld_wait();
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    w[e] = F16 ? pack_b16x2(down * u[2 * e], down * u[2 * e + 1], F16) : pack_b16x2(u[2 * e], u[2 * e + 1], F16);
                const int at_col = col + c;
                if (staged) {
                    const uint32_t p = swizzled_row(tile + (at_col >> 6) * 16384, row);
                    sts128(p ^ ((at_col & 63) << 1), w[0], w[1], w[2], w[3]);
                    sts128(p ^ (((at_col & 63) << 1) + 16), w[4], w[5], w[6], w[7]);
                } else if (live) {
                    *reinterpret_cast<uint4*>(to + at_col) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4*>(to + at_col + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                }
            }
        };
        auto store32 = [&](uint32_t t, uint32_t tile, float* to) {
#pragma unroll 1
            for (int c = part * kCols; c < (part + 1) * kCols; c += 16) {
                float u[16];
                ptx::tmem_ld16(t + c, u);
                ptx::tmem_ld_wait();
                if constexpr (F16) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) u[e] *= d_down;
                }
                const uint32_t* w = reinterpret_cast<const uint32_t*>(u);
                const uint32_t p = swizzled_row(tile + (c >> 5) * 16384, row) ^ ((c & 31) << 2);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (staged || a.paired) sts128(p ^ (e << 4), w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
                    else if (live) *reinterpret_cast<float4*>(to + c + 4 * e) = make_float4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]);
                }
            }
        };
        wait(sm.dqk, 0);
        ptx::tc_fence_after();
        const int64_t to = (tok * a.H + h) * K;
        const bool mine = (quarter >> 1) == (h & 1);  // (of a pair each head has half of the rows)
        if (a.paired) {
            // The other head's rows go to where that has them, which is free once its products are done.
            cluster_wait();  // its barriers are there
            const int peer = 1 - (h & 1);
            if (warp == 0 && elect_one()) arrive_there(in_cta(ptx::smem_u32(&sm.may_give), peer));
            if (!mine) {
                store32(t_row + kTdq, base + Shape::kQ, nullptr);
                store32(t_row + kTdk, base + Shape::kRing, nullptr);
                ptx::fence_proxy_async_smem();
                named_sync(7, 256);
                if (warp == 2 * peer && elect_one() && wait_cluster(sm.may_give, 0)) {
                    const uint32_t bar = in_cta(ptx::smem_u32(&sm.given), peer);
                    for (int b = 0; b < 2 * KB; ++b) {
                        const uint32_t at_rows = b * 16384 + peer * 8192;
                        bulk_push(in_cta(base + Shape::kQ + at_rows, peer), base + Shape::kQ + at_rows, 8192, bar);
                        bulk_push(in_cta(base + Shape::kRing + at_rows, peer), base + Shape::kRing + at_rows, 8192, bar);
                    }
                }
            }
        } else if (a.group == 1) {
            store16(t_row + kTdq + part * kCols, part * kCols, kCols, base + Shape::kQ, static_cast<uint16_t*>(a.dq) + to, d_down);
            store16(t_row + kTdk + part * kCols, part * kCols, kCols, base + Shape::kK, static_cast<uint16_t*>(a.dk) + to, d_down);
        } else {
            store32(t_row + kTdq, base + Shape::kQ, static_cast<float*>(a.dq) + to);
            store32(t_row + kTdk, base + Shape::kRing, static_cast<float*>(a.dk) + to);
        }
        // (the four warps of these rows: one of them sends what all have written)
        auto send = [&](auto store) {
            ptx::fence_proxy_async_smem();
            named_sync(2 + quarter, 128);
            if (staged && part == 0 && elect_one()) {
                store();
                ptx::bulk_commit();
            }
        };
        if (!a.paired) send([&] {
            // (fp32: twice the columns of 128 bytes, dq's where q and k were, dk's where the states were)
            const int blocks = a.group == 1 ? KB : 2 * KB, wide = 64 / (a.group == 1 ? 1 : 2);
            const int from_dk = a.group == 1 ? Shape::kK : Shape::kRing;
            for (int b = 0; b < blocks; ++b) {
                const int at_box = b * 16384 + quarter * 4096;
                ptx::tma_store_3d(&a.tm_dq, raw + Shape::kQ + at_box, b * wide, h, row0 + quarter * 32);
                ptx::tma_store_3d(&a.tm_dk, raw + from_dk + at_box, b * wide, h, row0 + quarter * 32);
            }
        });
        wait(sm.dv, 0);
        ptx::tc_fence_after();
        store16(t_dv, part * kColsV, kColsV, base + Shape::kV, a.dv + (tok * a.H + h) * V, p_down);
        send([&] {
            for (int b = 0; b < VB; ++b)
                ptx::tma_store_3d(&a.tm_dv, raw + Shape::kV + b * 16384 + quarter * 4096, b * 64, h, row0 + quarter * 32);
        });
        // dg, from sums that every thread has a part of (dP has been read)
        auto& sums = *reinterpret_cast<typename Shape::Sums*>(raw + Shape::kDp);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) across += __shfl_xor_sync(~0u, across, off);
        sums.far_q[part][row] = far_q;
        sums.far_k[part][row] = far_k;
        sums.near_k[part][row] = near_k;
        sums.near_q[quarter][part * 32 + lane] = near_q;
        if (lane == 0 && dot_warp >= 0) sums.across[dot_warp] = across;
        named_sync(1, kWorkers);
        if (part == 0) {  // four warps, a token a thread
            auto four = [&](const float (&x)[4][kDecayChunk]) { return (x[0][row] + x[1][row]) + (x[2][row] + x[3][row]); };
            // later: sum from this token on; before: sum up to it, itself not among them
            float later = four(sums.far_q) + (four(sums.near_q) - four(sums.near_k)), before = four(sums.far_k);
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const float l = __shfl_down_sync(~0u, later, off), b = __shfl_up_sync(~0u, before, off);
                if (lane + off < 32) later += l;
                if (lane >= off) before += b;
            }
            if (lane == 0) sums.later[quarter] = later;
            if (lane == 31) sums.before[quarter] = before;
            before = __shfl_up_sync(~0u, before, 1);
            if (lane == 0) before = 0.f;
            float all = 0.f;
#pragma unroll
            for (int i = 0; i < kDotWarps; ++i) all += sums.across[i];
            named_sync(6, 128);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i > quarter) later += sums.later[i];
                if (i < quarter) before += sums.before[i];
            }
            if (live) a.dg[tok * a.H + h] = all * sm.whole + later + before;
        }
        if (a.paired && mine) {  // what the other head had for these rows has landed where it had it itself
            wait_cluster(sm.given, 0);
            auto add = [&](uint32_t column, uint32_t tile, void* to) {
                uint32_t w[kCols / 2];
#pragma unroll
                for (int c = 0; c < kCols; c += 16) {
                    const int col = part * kCols + c;
                    float u[16];
                    ptx::tmem_ld16(t_row + column + col, u);
                    const uint32_t p = swizzled_row(tile + (col >> 5) * 16384, row) ^ ((col & 31) << 2);
                    const uint4 x[4] = {lds128(p), lds128(p ^ 16), lds128(p ^ 32), lds128(p ^ 48)};
                    ptx::tmem_ld_wait();
                    if constexpr (F16) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) u[e] *= d_down;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        w[c / 2 + 2 * e] = pack_b16x2(u[4 * e] + __uint_as_float(x[e].x), u[4 * e + 1] + __uint_as_float(x[e].y), F16);
                        w[c / 2 + 2 * e + 1] = pack_b16x2(u[4 * e + 2] + __uint_as_float(x[e].z), u[4 * e + 3] + __uint_as_float(x[e].w), F16);
                    }
                }
                named_sync(2 + quarter, 128);  // the sums of these rows have been read
                uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(to) + (tok * (a.H / 2) + hq) * K + part * kCols);
#pragma unroll
                for (int c = 0; c < kCols; c += 8) {
                    const int col = part * kCols + c;
                    const uint32_t p = swizzled_row(tile + (col >> 6) * 16384, row) ^ ((col & 63) << 1);
                    if (staged) sts128(p, w[c / 2], w[c / 2 + 1], w[c / 2 + 2], w[c / 2 + 3]);
                    else if (live) out[c / 8] = make_uint4(w[c / 2], w[c / 2 + 1], w[c / 2 + 2], w[c / 2 + 3]);
                }
            };
            add(kTdq, base + Shape::kQ, a.dq);
            add(kTdk, base + Shape::kRing, a.dk);
            send([&] {
                for (int b = 0; b < KB; ++b) {
                    const int at_box = b * 16384 + quarter * 4096;
                    ptx::tma_store_3d(&a.tm_dq, raw + Shape::kQ + at_box, b * 64, hq, row0 + quarter * 32);
                    ptx::tma_store_3d(&a.tm_dk, raw + Shape::kRing + at_box, b * 64, hq, row0 + quarter * 32);
                }
            });
        }
        if (part == 0 && elect_one()) ptx::bulk_wait_read0();
    }
    __syncwarp();
    if (a.paired) {  // what either has given has landed before one of them leaves
        if (warp == kWorkerWarps) cluster_wait();  // (the workers have been there)
        cluster_arrive();
        cluster_wait();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kWorkerWarps) ptx::tmem_dealloc(tmem, 512);
    if (sm.fail && tid == 0 && a.status) atomicOr(a.status, kStatusTimeout);
}

template <int KB, int VB, bool F16>
cudaError_t launch_shape(const DecayGradArgs& a, cudaStream_t s) {
    using Shape = GradShape<KB, VB>;
    auto kern = kda_decay_grads_kernel<KB, VB, F16>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.seqs.pieces * a.H));
    cfg.blockDim = dim3(kGradThreads);
    cfg.dynamicSmemBytes = Shape::kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = a.paired ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

// The gradients of q and k, summed over the value heads that share them: in fp32 [rows, Hqk, group, K] each. (Where the
// offsets are out of order the kernels before have written none, and this one must not write what it would find.)
__global__ void __launch_bounds__(256) kda_decay_group_kernel(const float* dq32, const float* dk32, void* dq, void* dk,
                                                              DecaySeqs seqs, int64_t fours, int K4, int group, int f16) {
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    if (!in_order<256>(seqs)) return;
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
__global__ void __launch_bounds__(256) kda_decay_gate_kernel(const float* part, float* dg, DecaySeqs seqs, int64_t parts,
                                                             int H) {
    __shared__ double sums[256];
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    if (!in_order<256>(seqs)) return;
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

cudaError_t launch_decay_group(const float* dq32, const float* dk32, void* dq, void* dk, const DecaySeqs& seqs, int64_t rows,
                               int heads, int K, int group, bool f16, int sms, cudaStream_t s) {
    const int64_t fours = rows * heads * (K / 4), blocks = (fours + 255) / 256;
    return launch_dependent(kda_decay_group_kernel, dim3((unsigned)(blocks < 16 * sms ? blocks : 16 * sms), 2), dim3(256),
                            (size_t)0, s, dq32, dk32, dq, dk, seqs, fours, K / 4, group, (int)f16);
}

cudaError_t launch_decay_gate(const float* dg, float* part, float* out, const DecaySeqs& seqs, int64_t rows, int H,
                              cudaStream_t s) {
    const int64_t parts = (rows + kGateRows - 1) / kGateRows;
    if (parts > 0) {
        const cudaError_t e = launch_dependent(kda_decay_gate_rows_kernel, dim3((unsigned)parts, (unsigned)((H + 255) / 256)),
                                               dim3(256), (size_t)0, s, dg, part, rows, H);
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(kda_decay_gate_kernel, dim3((unsigned)H), dim3(256), (size_t)0, s, part, out, seqs, parts, H);
}

}  // namespace kda
