// linear_wide.cu -- the kernel of kda_linear for many tokens.
//
// A pair of CTAs (a cluster of two, on two SMs that share a tensor-core pair)
// makes 256 tokens x 256 features at a time with cta_group::2 MMAs: each CTA
// loads 128 rows of x and 128 rows of w, its tensor core reads both CTAs' w,
// and it accumulates its own 128 tokens x 256 features in TMEM.  That halves
// the shared-memory and L2 reads of w per flop against a CTA by itself.  The
// pairs are persistent; each has two accumulators (all 512 columns of TMEM),
// so the epilogue of a tile runs beside the MMAs of the next.
//
// Roles per CTA: warp 0 loads (TMA, a ring of kStages stages), warp 1 of the
// first CTA issues the MMAs of both, warps 4-11 are the epilogue: warp w has
// the 32 tokens of TMEM lane quarter w % 4 and one half of the features.  The
// first four warps hand their registers to the epilogue's (an fp32 y keeps 128
// running sums a thread).  A thread has a token's row; 128-byte row pieces go
// through a swizzled staging box per warp, which TMA loads the residual into
// and stores y from, so global memory sees whole lines and ragged edges are
// clipped by the copy.  Rows that do not start on 16 bytes, which TMA cannot
// move, go between box and memory by the warp's own loads and stores, lanes along
// a row, still beside the next tile's MMAs: 8192 x 4095 x 4096 in bf16 148 us (338
// in the kernel for few tokens, whose rows of threads store four elements each).
//
// Bound: the tensor cores (and, seconds long, the power limit).  A stage of 64
// 16-bit k takes 0.316 us a pair, 2.0 PFLOP/s over 76 pairs: 32768 x 4096 x 4096
// with silu 545 us in a burst (cuBLAS's plain product 522 to 546), 648 to 661 kept
// up for seconds (1.66 to 1.70 PFLOP/s, of 1.73 that cuBLAS keeps up); 16361 tokens in e4m3
// 157 us (3.5 PFLOP/s).  What it took: loads and MMAs issued by an elected lane (a
// test of the lane number instead cost 713 us: the compiler then puts a loop
// around every TMA and MMA instruction).
#include "linear.cuh"

namespace kda {
namespace {

constexpr int kTileM = 256;                            // tokens per pair
constexpr int kEpilogueWarps = 8;
constexpr int kBoxBytes = 32 * 128;                    // 32 tokens x 128 bytes
constexpr int kFirstEpilogue = 4;                      // warp
constexpr int kThreads = 32 * (kFirstEpilogue + kEpilogueWarps);
// registers: 128 x 40 + 256 x 224 of the 384 x 168 that a block is launched with
constexpr int kFewRegs = 40, kManyRegs = 224;
constexpr int kGroup = 8;                              // token tiles that share a sweep over the features
constexpr int kSegment = 16;                           // stages of k per accumulator where y is fp32

// TN: features per pair, 256 or 128.
template <int TN>
struct WideShape {
    static constexpr int kXBytes = 128 * kRowBytes;                  // one CTA's part of x in a stage
    static constexpr int kStageBytes = kXBytes + TN / 2 * kRowBytes;  // and of w
    static constexpr int kStages = TN == 256 ? 6 : 8;
    static constexpr int kAccs = 512 / TN;                            // accumulators in TMEM
    static constexpr int kSmem = kStages * kStageBytes + kEpilogueWarps * kBoxBytes + 1024;
};

struct WideArgs {
    LinArgs a;
    CUtensorMap tm_y, tm_r;  // boxes of 128 bytes x 32 rows
    int direct;              // rows of y or the residual off 16 bytes: moved by the warp, not by TMA
    int tiles_m, tiles_n;
};

__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* m, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
        "[%1, {%3, %4}], [%2];" ::"r"(ptx::smem_u32(dst)),
        "l"(m), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
template <bool F8>
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
    if constexpr (F8)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::2.kind::f8f6f4 [%0], "
            "%1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::2.kind::f16 [%0], "
            "%1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
}
// Arrives on the barrier at this offset in both CTAs when the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            ptx::smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A warp has read its part of an accumulator: the first CTA may fill it again.
__device__ __forceinline__ void release(uint64_t* acc_empty, int lane) {
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) arrive_remote(peer_smem(ptx::smem_u32(acc_empty), 0));
}

// The 32 fp32 values of a lane's row in a box, two swizzled pieces at a time.
template <int ACT>
__device__ __forceinline__ void activated_row(uint8_t* row, int lane) {
#pragma unroll 1
    for (int j = 0; j < 8; j += 2) {
        float4* p[2] = {reinterpret_cast<float4*>(row + ((j ^ (lane & 7)) << 4)),
                        reinterpret_cast<float4*>(row + (((j + 1) ^ (lane & 7)) << 4))};
        float4 f[2] = {*p[0], *p[1]};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f[i].x = activated<ACT, false>(f[i].x);
            f[i].y = activated<ACT, false>(f[i].y);
            f[i].z = activated<ACT, false>(f[i].z);
            f[i].w = activated<ACT, false>(f[i].w);
            *p[i] = f[i];
        }
    }
}
__device__ __forceinline__ void activate_row(uint8_t* row, int lane, int act) {
    switch (act) {
    case KDA_ACT_SILU: activated_row<KDA_ACT_SILU>(row, lane); break;
    case KDA_ACT_GELU: activated_row<KDA_ACT_GELU>(row, lane); break;
    case KDA_ACT_SIGMOID: activated_row<KDA_ACT_SIGMOID>(row, lane); break;
    case KDA_ACT_LOGSIGMOID: activated_row<KDA_ACT_LOGSIGMOID>(row, lane); break;
    }
}

// A box and its place in memory, element by element (lanes along a row): IN fills
// the box, else it is stored.  COLS: 64 16-bit or 32 fp32 columns.  A residual's
// loads go 16 words at a time, from L2, where the tile's rows are asked for before
// its sums are waited for: 3259 x 5177 x 2048 with log-sigmoid to fp32 291 us with
// four at a time and from HBM, 104 with both (79 with 128 features a tile).
template <int COLS, bool IN>
__device__ __forceinline__ void move_box(uint8_t* box, void* p, int64_t ld, int m0, int n0, int M, int N, int lane) {
    constexpr int kSize = 128 / COLS;
    __syncwarp();
    const int rows = min(32, M - m0);
    constexpr int kBatch = IN ? 512 / COLS : 4;  // rows whose loads are in flight together
    for (int r0 = 0; r0 < rows; r0 += kBatch) {
        uint32_t got[kBatch][COLS / 32];
        const int64_t to = (int64_t)(m0 + r0) * ld + n0 + lane;
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
            for (int h = 0; h < COLS / 32; ++h) {
                const int r = r0 + i, c = h * 32 + lane;
                const int at = r * 128 + ((((c * kSize) >> 4) ^ (r & 7)) << 4) + ((c * kSize) & 15);
                const bool live = r < rows && n0 + c < N;
                if constexpr (kSize == 2) {
                    uint16_t* g = static_cast<uint16_t*>(p) + to + i * ld + h * 32;
                    if (IN) got[i][h] = live ? *g : 0;
                    else if (live) *g = *reinterpret_cast<uint16_t*>(box + at);
                } else {
                    uint32_t* g = static_cast<uint32_t*>(p) + to + i * ld + h * 32;
                    if (IN) got[i][h] = live ? *g : 0;
                    else if (live) *g = *reinterpret_cast<uint32_t*>(box + at);
                }
            }
        if constexpr (IN) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
#pragma unroll
                for (int h = 0; h < COLS / 32; ++h) {
                    const int r = r0 + i, c = h * 32 + lane;
                    const int at = r * 128 + ((((c * kSize) >> 4) ^ (r & 7)) << 4) + ((c * kSize) & 15);
                    if constexpr (kSize == 2) *reinterpret_cast<uint16_t*>(box + at) = (uint16_t)got[i][h];
                    else *reinterpret_cast<uint32_t*>(box + at) = got[i][h];
                }
        }
    }
    __syncwarp();
}

// Tile t of the sweep: groups of kGroup token tiles, the features outside, the group's tokens inside.
__device__ __forceinline__ void tile_at(int t, int tiles_m, int tiles_n, int* tm, int* tn) {
    const int per = kGroup * tiles_n;
    const int g = t / per, first = g * kGroup, rows = min(kGroup, tiles_m - first);
    const int in = t - g * per;
    *tn = in / rows;
    *tm = first + in - *tn * rows;
}

// OUT16: y is bf16 or fp16 (64 columns a box), else fp32 (32 columns a box).  An
// fp32 y gets more of the sum's accuracy: the tensor cores' own additions drop
// bits below the running sum, so k is cut into segments of kSegment stages,
// each in an accumulator of its own, that the epilogue adds in registers (1.0e-6
// against 64 bits for K = 2048 to 32768).  A 16-bit y takes all of k in one: the
// rounding is all of its error (0.001675 either way for 32768 x 4096 x 4096), but
// 0.25% of its elements round to the neighbour of what fp32 products would give.
template <int TN, bool F8, bool OUT16>
__global__ void __launch_bounds__(kThreads, 1) kda_linear_wide_kernel(const __grid_constant__ WideArgs p) {
    using Shape = WideShape<TN>;
    constexpr int kStages = Shape::kStages, kStageBytes = Shape::kStageBytes, kAccs = Shape::kAccs;
    constexpr bool kSegments = !OUT16;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t full[kStages], empty[kStages], acc_full[kAccs], acc_empty[kAccs];
    __shared__ __align__(8) uint64_t res[kEpilogueWarps];
    __shared__ uint32_t tmem_base;
    __shared__ int s_fail;
    uint8_t* ring = ptx::align_smem_1024(raw);
    const LinArgs& a = p.a;

    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
    const int tiles = p.tiles_m * p.tiles_n;

    if (tid == 0) {
        ptx::prefetch_tmap(&a.tm_w);
        ptx::prefetch_tmap(&a.tm_x);
        if (!p.direct) ptx::prefetch_tmap(&p.tm_y);
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < kAccs; ++b) {
            ptx::mbar_init(&acc_full[b], 1);
            ptx::mbar_init(&acc_empty[b], 2 * kEpilogueWarps);
        }
        for (int w = 0; w < kEpilogueWarps; ++w) ptx::mbar_init(&res[w], 1);
        ptx::fence_mbar_init();
        s_fail = 0;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         ptx::smem_u32(&tmem_base)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    ptx::tc_fence_before();
    ptx::grid_dep_launch();
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers are set before either signals the other's
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_base;
    ptx::grid_dep_wait();

    if (warp < kFirstEpilogue) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
        if (warp == 0 && elect_one()) {
            int it = 0;  // stages issued
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                int tm, tn;
                tile_at(t, p.tiles_m, p.tiles_n, &tm, &tn);
                const int m = tm * kTileM + (int)rank * 128, n = tn * TN + (int)rank * (TN / 2);
                for (int kb = 0; kb < a.kblocks; ++kb, ++it) {
                    const int s = it % kStages, round = it / kStages;
                    if (round > 0 && !(ok = wait_for(&empty[s], (round - 1) & 1))) break;
                    uint8_t* x = ring + s * kStageBytes;
                    const int k = kb * (F8 ? kRowBytes : kRowBytes / 2);
                    // the first CTA's barrier counts the bytes of both
                    if (rank == 0) ptx::mbar_arrive_expect_tx(&full[s], 2 * kStageBytes);
                    const uint32_t bar = peer_smem(ptx::smem_u32(&full[s]), 0);
                    tma_load_pair(x, &a.tm_x, bar, k, m);
                    tma_load_pair(x + Shape::kXBytes, &a.tm_w, bar, k, n);
                }
            }
            if (!ok) {  // let the copies in flight land (the first CTA sees both CTAs' bytes)
                s_fail = 1;
                if (rank == 0)
                    for (int i = max(0, it - kStages); i < it; ++i)
                        wait_for(&full[i % kStages], (i / kStages) & 1);
            }
        }
        if (warp == 1 && rank == 0 && elect_one()) {
            int it = 0, n_acc = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                for (int kb = 0; kb < a.kblocks; ++kb, ++it) {
                    const bool opens = kSegments ? kb % kSegment == 0 : kb == 0;
                    const int b = n_acc % kAccs, round = n_acc / kAccs;
                    if (opens) {
                        if (round > 0 && !(ok = wait_for<true>(&acc_empty[b], (round - 1) & 1))) break;
                        ptx::tc_fence_after();
                    }
                    const int s = it % kStages;
                    if (!(ok = wait_for(&full[s], (it / kStages) & 1))) break;
                    ptx::tc_fence_after();
                    const uint32_t x = ptx::smem_u32(ring + s * kStageBytes);
                    const uint64_t da = ptx::smem_desc(x, 0, 1024), db = ptx::smem_desc(x + Shape::kXBytes, 0, 1024);
#pragma unroll
                    for (int j = 0; j < 4; ++j)  // 32 bytes of k each
                        mma_pair<F8>(tmem + (uint32_t)(b * TN), da + 2 * j, db + 2 * j, a.idesc, !opens || j > 0);
                    commit_pair(&empty[s]);
                    if (kb + 1 == a.kblocks || (kSegments && (kb + 1) % kSegment == 0)) {
                        commit_pair(&acc_full[b]);
                        ++n_acc;
                    }
                }
            }
            if (!ok) s_fail = 1;
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        constexpr int kCols = TN / 2;  // features of a warp
        constexpr int kBoxCols = OUT16 ? 64 : 32;
        constexpr int kBoxes = kCols / kBoxCols;
        const int e = warp - kFirstEpilogue, quarter = warp & 3, half = e >> 2;
        uint8_t* box = ring + kStages * kStageBytes + e * kBoxBytes;
        uint8_t* row = box + lane * 128;
        const bool f16 = a.out == KDA_DTYPE_F16;
        const int segments = kSegments ? (a.kblocks + kSegment - 1) / kSegment : 1;
        int n_acc = 0;
        uint32_t loads = 0, asked = 0;  // residual boxes that arrived, and that were asked for (lane 0)
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs) {
            int tm, tn;
            tile_at(t, p.tiles_m, p.tiles_n, &tm, &tn);
            const int m0 = tm * kTileM + (int)rank * 128 + quarter * 32, n0 = tn * TN + half * kCols;
            float bias[kCols / 32], scale[kCols / 32];  // of features n0 + 32 i + lane, handed round by shuffles
            float xs = 1.f;
#pragma unroll
            for (int i = 0; i < kCols / 32; ++i) {
                const int n = n0 + 32 * i + lane;
                bias[i] = a.bias && n < a.N ? a.bias[n] : 0.f;
                scale[i] = F8 && n < a.N ? a.w_scale[n] : 1.f;
            }
            if (F8 && m0 + lane < a.M) xs = a.x_scale[m0 + lane];
            const bool rows = m0 < a.M;
            auto load_residual = [&](int n) {
                if (lane == 0 && !p.direct) {
                    ptx::bulk_wait_read0();  // the box's last store has read it
                    ptx::mbar_arrive_expect_tx(&res[e], kBoxBytes);
                    ptx::tma_load_2d(box, &p.tm_r, &res[e], n, m0);
                    ++asked;
                }
            };
            if (a.residual && rows && n0 < a.N) load_residual(n0);
            if (a.residual && p.direct && m0 + lane < a.M && n0 < a.N) {  // into L2 by the time it is asked for
                constexpr int kSize = OUT16 ? 2 : 4;
                const uint8_t* from = static_cast<const uint8_t*>(a.residual) + ((int64_t)(m0 + lane) * a.ldr + n0) * kSize;
                const int bytes = min(kCols, a.N - n0) * kSize;
                for (int at = 0; at < bytes; at += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(from + at));
            }
            float sum[kSegments ? kCols : 1];
            uint32_t acc = 0;
            for (int g = 0; g < segments; ++g, ++n_acc) {
                const int b = n_acc % kAccs;
                ok = __all_sync(~0u, wait_for(&acc_full[b], (n_acc / kAccs) & 1, 2 * kWaitLimitNs));
                if (!ok) break;
                ptx::tc_fence_after();
                acc = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(b * TN + half * kCols);
                if constexpr (kSegments) {
#pragma unroll
                    for (int c = 0; c < kCols; c += 16) {
                        float v[16];
                        ptx::tmem_ld16(acc + c, v);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j) sum[c + j] = g ? sum[c + j] + v[j] : v[j];
                    }
                    release(&acc_empty[b], lane);
                }
            }
            if (!ok) break;
            // One box of the row piece after another.  (Running sums are in registers, so
            // their boxes are unrolled; from TMEM it is a loop, whose code is shorter.)
#pragma unroll(kSegments ? kBoxes : 1)
            for (int q = 0; q < kBoxes; ++q) {
                const int n = n0 + q * kBoxCols;
                const bool live = rows && n < a.N;
                float fresh[kSegments ? 1 : kBoxCols];
                float* v = kSegments ? sum + q * kBoxCols : fresh;  // (registers: every index is known)
                if constexpr (!kSegments) {
#pragma unroll
                    for (int c = 0; c < kBoxCols; c += 16) ptx::tmem_ld16(acc + q * kBoxCols + c, v + c);
                    ptx::tmem_ld_wait();
                    if (q == kBoxes - 1) release(&acc_empty[(n_acc - 1) % kAccs], lane);
                }
                if (!live) continue;
#pragma unroll
                for (int h = 0; h < kBoxCols / 32; ++h) {
                    float box_bias = bias[h], box_scale = scale[h];
#pragma unroll
                    for (int i = 1; i < kBoxes; ++i)
                        if (q == i) box_bias = bias[i * (kBoxCols / 32) + h], box_scale = scale[i * (kBoxCols / 32) + h];
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        if (F8) v[32 * h + c] *= xs * __shfl_sync(~0u, box_scale, c);
                        v[32 * h + c] += __shfl_sync(~0u, box_bias, c);
                    }
                }
                if (p.direct) {
                    if (a.residual) move_box<kBoxCols, true>(box, const_cast<void*>(a.residual), a.ldr, m0, n, a.M, a.N, lane);
                } else if (a.residual) {
                    ok = __all_sync(~0u, wait_for(&res[e], loads & 1));
                    if (!ok) break;
                    ++loads;
                } else {
                    if (lane == 0) ptx::bulk_wait_read0();
                    __syncwarp();
                }
                if constexpr (OUT16) {
                    activate_all<kBoxCols, true>(v, a.act);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {  // 16-byte pieces of the row, swizzled
                        uint4* at = reinterpret_cast<uint4*>(row + ((j ^ (lane & 7)) << 4));
                        float* f = v + 8 * j;
                        if (a.residual) {
                            const uint4 u = *at;
                            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 r = f16 ? from_b16x2<true>(w[i]) : from_b16x2<false>(w[i]);
                                f[2 * i] += r.x;
                                f[2 * i + 1] += r.y;
                            }
                        }
                        *at = make_uint4(pack_b16x2(f[0], f[1], f16), pack_b16x2(f[2], f[3], f16),
                                         pack_b16x2(f[4], f[5], f16), pack_b16x2(f[6], f[7], f16));
                    }
                } else {
                    // The activation runs over the row in the box, in a loop: unrolled over the
                    // registers its code alone, once per tile, took longer than its arithmetic
                    // (4096 x 2048 x 2048 with log-sigmoid 40 us, without it 30).
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float4* at = reinterpret_cast<float4*>(row + ((j ^ (lane & 7)) << 4));
                        float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (a.residual) r = *at;
                        float4 f = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                        if (a.act == KDA_ACT_NONE) f = make_float4(f.x + r.x, f.y + r.y, f.z + r.z, f.w + r.w);
                        *at = f;
                        v[4 * j] = r.x, v[4 * j + 1] = r.y, v[4 * j + 2] = r.z, v[4 * j + 3] = r.w;
                    }
                    if (a.act != KDA_ACT_NONE) {
                        activate_row(row, lane, a.act);
                        if (a.residual) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                float4* at = reinterpret_cast<float4*>(row + ((j ^ (lane & 7)) << 4));
                                const float4 f = *at;
                                *at = make_float4(f.x + v[4 * j], f.y + v[4 * j + 1], f.z + v[4 * j + 2],
                                                  f.w + v[4 * j + 3]);
                            }
                        }
                    }
                }
                if (p.direct) {
                    move_box<kBoxCols, false>(box, a.y, a.ldy, m0, n, a.M, a.N, lane);
                    continue;
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    ptx::tma_store_2d(&p.tm_y, box, n, m0);
                    ptx::bulk_commit();
                }
                if (a.residual && q + 1 < kBoxes && n + kBoxCols < a.N) load_residual(n + kBoxCols);
            }
        }
        if (!ok) s_fail = 1;
        if (lane == 0) {
            if (asked != loads) wait_for(&res[e], loads & 1);
            ptx::bulk_wait0();
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // neither CTA leaves while the other may still signal or read it
    ptx::tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    if (s_fail && tid == 0 && a.status) atomicOr(a.status, kStatusTimeout);
}

bool box_map(CUtensorMap* m, int dtype, const void* base, int64_t M, int64_t N, int64_t ld) {
    const int es = dtype_bytes(dtype);
    const uint64_t dims[2] = {(uint64_t)N, (uint64_t)M};
    const uint64_t strides[1] = {(uint64_t)ld * es};
    const uint32_t box[2] = {(uint32_t)(128 / es), 32};
    const CUtensorMapDataType dt = dtype == KDA_DTYPE_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : dtype == KDA_DTYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                            : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return make_tensormap(m, dt, 2, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int TN, bool F8, bool OUT16>
cudaError_t launch(WideArgs& p, const void* w, int64_t K, int64_t ldw, cudaStream_t s) {
    LinArgs& a = p.a;
    if (!rows_map(&a.tm_w, a.io, w, a.N, K, ldw, TN / 2)) return cudaErrorInvalidValue;
    a.idesc = F8                        ? idesc_e4m3_f32(kTileM, TN)
              : a.io == KDA_DTYPE_BF16 ? ptx::idesc_bf16_f32(kTileM, TN, 0, 0)
                                       : ptx::idesc_f16_f32(kTileM, TN, 0, 0);
    p.tiles_n = (a.N + TN - 1) / TN;
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n, pairs = device_sm_count() / 2;
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;
    auto kern = kda_linear_wide_kernel<TN, F8, OUT16>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, WideShape<TN>::kSmem);
    if (e != cudaSuccess) return e;
    return launch_cluster(kern, dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))), dim3(kThreads),
                          WideShape<TN>::kSmem, 2, s, p);
}

template <int TN, bool F8>
cudaError_t launch(WideArgs& p, bool out16, const void* w, int64_t K, int64_t ldw, cudaStream_t s) {
    return out16 ? launch<TN, F8, true>(p, w, K, ldw, s) : launch<TN, F8, false>(p, w, K, ldw, s);
}

}  // namespace

cudaError_t launch_linear_wide(const LinArgs& a, int tn, const void* x, const void* w, int64_t K, int64_t ldx,
                               int64_t ldw, bool rows_on_16, cudaStream_t s) {
    WideArgs p{};
    p.a = a;
    p.tiles_m = (a.M + kTileM - 1) / kTileM;
    p.direct = !rows_on_16;
    if (!rows_map(&p.a.tm_x, a.io, x, a.M, K, ldx, 128)) return cudaErrorInvalidValue;
    if (rows_on_16 && (!box_map(&p.tm_y, a.out, a.y, a.M, a.N, a.ldy) ||
                       (a.residual && !box_map(&p.tm_r, a.out, a.residual, a.M, a.N, a.ldr))))
        return cudaErrorInvalidValue;
    const bool f8 = a.io == KDA_DTYPE_E4M3;
    const bool out16 = a.out != KDA_DTYPE_F32;
    if (tn == 128) return f8 ? launch<128, true>(p, out16, w, K, ldw, s) : launch<128, false>(p, out16, w, K, ldw, s);
    return f8 ? launch<256, true>(p, out16, w, K, ldw, s) : launch<256, false>(p, out16, w, K, ldw, s);
}

}  // namespace kda
