// decay_scan.cuh -- the state scan of linear attention with a decay per head
// (formulas: decay.cuh), with its output (decay_out.cu) or by itself
// (decay_states.cu).
//
// One CTA walks the chunks of a piece of one (sequence, head), with the state in
// the registers of one warpgroup, transposed (thread v has S[:, v]), in fp32.
// Per chunk of 128 tokens, all as tcgen05 MMAs with M = 128:
//     scores   q k^T                      token x token, TMEM
//     far      q S                        S rounded to 16 bits as the operand
//     near     P v                        P = scale exp(G_i - G_j) scores, 16 bits, from TMEM
//     added    v^T (exp(G_last - G_j) k)  value x key, in two products
// and o = scale exp(G_i) far + near; S = exp(G_last) S + added.  The scaled k of
// the last product does not fit 16 bits as k does, so it is split in two parts,
// hi = k w rounded and lo = what hi lost, whose products add up: what is added keeps
// 2^-17 of itself (fp16: 2^-22) instead of 2^-8, and the states, which are fp32 outputs and
// sums over all tokens, come out 2.3e-6 (4e-7) from 64 bits.  far is scaled by
// rows in TMEM, where near then adds to it, so that o needs one accumulator and can have two in turn.
//
// Warps: 0 loads (TMA), 1 issues MMAs, 2 sums the chunk's decays; two warpgroups scale
// k, one each holds the state, turns scores into P, and writes o, so that
// those of neighbouring chunks overlap. Their registers are shared out by what they
// hold. With its output a chunk's q, k and v have one buffer each, free again as
// soon as they have been read (k when it has been scaled, into buffers of its own).
//
// Bound: HBM and, close behind it, shared memory. A chunk's 96 KB in and 32 KB out take
// 4800 cycles of an SM's share of HBM (128 CTAs), and the 576 KB that its loads, products and
// operands move through shared memory 4500. 4 x 8192 tokens x 32 heads of 128 x 128 in bf16: 205 to
// 208 us, 5.3 TB/s (79 to 80% of what a copy reaches); in fp16 231. Steps on the way (us): k scaled in
// place, hi after lo, o by its threads' stores 345; registers spilled beside what is left of L1, each a
// trip to L2, brought down 311; loops instead of unrolled code (five roles' code has to fit the instruction
// cache together) 277; o by TMA and k, v, q in single buffers 212; waits of a few instructions, far
// before added, k read before it is scaled 195.
#pragma once
#include "decay.cuh"

namespace kda {
namespace {

template <int KB, int VB, bool OUT>
struct DecayScanShape {
    static constexpr int K = 64 * KB, V = 64 * VB;
    static constexpr int kKeyWarps = 8;  // (a thread has half of a token's row)
    static constexpr int kFirstState = 4 + kKeyWarps;
    static constexpr int kThreads = 32 * (kFirstState + 4 + (OUT ? 8 : 0));
    static constexpr int kXBytes = KB * 16384, kYBytes = VB * 16384, kStateBytes = V * K * 2;
    // Stages: every tensor's tile is read early in a chunk (the scaled parts of k have buffers of their own, and so has
    // o), so one of each is enough where two do not fit.
    static constexpr int kOne = kXBytes * (OUT ? 2 : 1) + kYBytes;
    static constexpr int kFixed = 2 * kXBytes + (OUT ? 1 : 2) * kStateBytes + (OUT ? kYBytes : 0);
    static constexpr int kStages = kFixed + 2 * kOne <= 224 * 1024 ? 2 : 1;
    static constexpr int kY = 0, kX = kStages * kYBytes, kQ = kX + kStages * kXBytes;
    // (where V = 64 the MMAs with v^T read 128 columns, the second half from what follows, into lanes nobody reads)
    static constexpr int kHi = OUT ? kQ + kStages * kXBytes : kQ, kLo = kHi + kXBytes, kS = kLo + kXBytes;
    static constexpr int kO = kS + (OUT ? 1 : 2) * kStateBytes;
    static constexpr int kSmall = kO + (OUT ? kYBytes : 0);
    struct Small {
        ChunkDecay decay[2];
        float column[OUT ? kDecayChunk : 1];  // exp of the decay from a column to the end of its 32
        float whole[2], unscale[2], key_unscale[2];
        uint32_t top[4], key_top[2][8];
        // fp16: see rise_of; the largest of the keys as they are; what 32 rows' scores are multiplied by, as a power of two
        int32_t rise[2];
        uint32_t plain_top[2][8];
        int8_t score_powers[2][4];
        uint64_t x_full[2], x_empty[2], q_full[2], q_empty[2], y_full[2], y_empty[2], g_ready[2], g_free[2];
        uint64_t plain[2], scaled[2];  // plain_top and score_powers are there
        uint64_t scores, p_ready, s_ready, keys, keys_read, added, added_read, far, far_ok, o_full, o_free[2];
        uint32_t tmem;
        int32_t fail;
        // The piece: first token row, tokens from there to the sequence's end, chunks, index of the first one, sequence,
        // head, and whether it starts and ends its direction. (Here and not in registers, which the roles are short of.)
        int32_t row, left, chunks, chunk, n, head, first, last;
    };
    static constexpr int kSmem = kSmall + (int)sizeof(Small);
    static_assert(sizeof(Small) >= sizeof(DecaySortScratch), "the search's scratch fits");
    static_assert(kSmem <= 227 * 1024, "fits an SM");
    static constexpr uint32_t kScores = 0, kAdded = OUT ? 128 : 0, kOut = 256;  // TMEM columns (kOut: twice 128)
    static constexpr uint32_t kTmem = OUT ? 512 : 128;
};

// Registers: those that the block is launched with, handed out as control, keys, state, scores, output. (fp16 with its
// output: its scores' and outputs' powers of two spill with bf16's split: 237 instead of 231 us, K = 64 23.9 instead of 20.6.)
template <bool F16, bool OUT>
struct DecayScanRegs {
    static constexpr bool kPowers = F16 && OUT;
    static constexpr int kControl = kPowers ? 40 : OUT ? 56 : 96, kKeys = kPowers ? 56 : OUT ? 64 : 88;
    static constexpr int kState = kPowers ? 176 : OUT ? 168 : 240, kScores = kPowers ? 80 : 64, kOut = kPowers ? 72 : 64;
    static_assert(OUT ? kControl + 2 * kKeys + kState + kScores + kOut <= 6 * 80 : kControl + 2 * kKeys + kState <= 4 * 128,
                  "within what the block is launched with");
};

// The largest in size of PIECES 16-byte pieces of fp16 in a swizzled row, from piece c0 on (NaN counts as nothing).
template <int PIECES>
__device__ __forceinline__ float largest_half(uint32_t row, int c0) {
    __half2 most[4];  // (one would be a chain of as many steps as there are words)
#pragma unroll
    for (int e = 0; e < 4; ++e) most[e] = __half2half2(__ushort_as_half(0));
#pragma unroll 2
    for (int c = c0; c < c0 + PIECES; ++c) {
        const uint4 x = lds128((row ^ ((c & 7) << 4)) + (c >> 3) * 16384);
        const uint32_t in[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) most[e] = __hmax2(most[e], __habs2(*reinterpret_cast<const __half2*>(&in[e])));
    }
    const __half2 all = __hmax2(__hmax2(most[0], most[1]), __hmax2(most[2], most[3]));
    return fmaxf(__low2float(all), __high2float(all));
}

template <int KB, int VB, bool F16, bool OUT>
__global__ void __launch_bounds__(DecayScanShape<KB, VB, OUT>::kThreads, 1)
    kda_decay_scan_kernel(const __grid_constant__ DecayScanArgs a) {
    using Shape = DecayScanShape<KB, VB, OUT>;
    using Regs = DecayScanRegs<F16, OUT>;
    constexpr int K = Shape::K, V = Shape::V, NS = Shape::kStages;
    extern __shared__ __align__(1024) uint8_t raw[];
    auto& sm = *reinterpret_cast<typename Shape::Small*>(raw + Shape::kSmall);
    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31, quarter = warp & 3;
    const DecayScanDir& dir = a.dir[blockIdx.y];
    const bool reverse = !OUT && dir.reverse;

    ptx::grid_dep_wait();
    {
        const int item = blockIdx.x / a.H;
        DecayPiece at;
        auto& scratch = *reinterpret_cast<DecaySortScratch*>(&sm);
        if (!find_piece<Shape::kThreads>(a.seqs, item, false, true, scratch, at, a.seqs.whole ? scratch.len : nullptr)) {
            if (blockIdx.x == 0 && tid == 0 && a.status) atomicOr(a.status, kStatusBadSeqlens);
            return;
        }
        const bool first = at.piece == 0, last = at.piece == at.pieces - 1;
        if (at.n < 0 || (a.totals_only && (reverse ? first : last))) return;  // (nothing follows a direction's last piece)
        __syncthreads();  // the search's scratch is free
        if (tid == 0) {
            const int c0 = at.piece * a.seqs.seg_chunks;
            sm.row = at.bos + c0 * kDecayChunk;
            sm.left = at.len - c0 * kDecayChunk;
            sm.chunks = min(ceil_div(at.len, kDecayChunk) - c0, a.seqs.seg_chunks);
            sm.chunk = at.chunk_base + c0;
            sm.n = at.n;
            sm.head = blockIdx.x - item * a.H;
            sm.first = reverse ? last : first;
            sm.last = reverse ? first : last;
        }
    }

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(&sm.x_full[s], 1);
            ptx::mbar_init(&sm.x_empty[s], Shape::kKeyWarps + (OUT ? 1 : 0) + (OUT && F16 ? 4 : 0));
            ptx::mbar_init(&sm.q_full[s], 1);
            ptx::mbar_init(&sm.q_empty[s], F16 ? 5 : 1);
            ptx::mbar_init(&sm.plain[s], 1);
            ptx::mbar_init(&sm.scaled[s], 4);
            ptx::mbar_init(&sm.y_full[s], 1);
            ptx::mbar_init(&sm.y_empty[s], 1);
            ptx::mbar_init(&sm.g_ready[s], 1);
            ptx::mbar_init(&sm.g_free[s], Shape::kKeyWarps + (OUT ? 8 : 0) + 2 * VB);
            ptx::mbar_init(&sm.o_free[s], 4);
        }
        for (uint64_t* b : {&sm.scores, &sm.keys_read, &sm.added, &sm.far, &sm.o_full}) ptx::mbar_init(b, 1);
        for (uint64_t* b : {&sm.p_ready, &sm.far_ok}) ptx::mbar_init(b, 4);
        ptx::mbar_init(&sm.keys, Shape::kKeyWarps);
        for (uint64_t* b : {&sm.s_ready, &sm.added_read}) ptx::mbar_init(b, 2 * VB);
        ptx::fence_mbar_init();
        sm.fail = 0;
    }
    if (warp == 1) {
        ptx::tmem_alloc(&sm.tmem, Shape::kTmem);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    // (not before: it counts from a block's first thread that runs it, and a dependent that shares this SM could take the
    // TMEM that this block still needs)
    ptx::grid_dep_launch();
    const uint32_t tmem = sm.tmem, base = ptx::smem_u32(raw);
    const int chunks = sm.chunks;
    // tokens of the piece before the it'th chunk that is taken
    auto offset = [&](int it) { return (reverse ? chunks - 1 - it : it) * kDecayChunk; };
    volatile int32_t* fail = &sm.fail;
    auto wait = [&](uint64_t& bar, uint32_t parity) { wait_or_note(&bar, parity, &sm.fail); };
    auto arrive = [&](uint64_t& bar) {  // once per warp
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bar);
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs::kControl));
        if (warp == 0 && elect_one()) {
            // ---------------------------------------------------------- loads
            const int h = sm.head, hq = h / a.group;
            int it = 0;
            for (; it < chunks; ++it) {
                const int sx = it % NS, row = sm.row + offset(it);
                const uint32_t px = ((it / NS) & 1) ^ 1;  // of the stage's last use
                if (it >= NS) wait(sm.x_empty[sx], px);
                if (*fail) break;
                ptx::mbar_arrive_expect_tx(&sm.x_full[sx], Shape::kXBytes);
                for (int b = 0; b < KB; ++b)
                    ptx::tma_load_3d(raw + Shape::kX + sx * Shape::kXBytes + b * 16384, &dir.tm_x, &sm.x_full[sx], b * 64,
                                     hq, row);
                if constexpr (OUT) {
                    if (it >= NS) wait(sm.q_empty[sx], px);
                    ptx::mbar_arrive_expect_tx(&sm.q_full[sx], Shape::kXBytes);
                    for (int b = 0; b < KB; ++b)
                        ptx::tma_load_3d(raw + Shape::kQ + sx * Shape::kXBytes + b * 16384, &a.tm_q, &sm.q_full[sx],
                                         b * 64, hq, row);
                }
                if (it >= NS) wait(sm.y_empty[sx], px);
                ptx::mbar_arrive_expect_tx(&sm.y_full[sx], Shape::kYBytes);
                for (int b = 0; b < VB; ++b)
                    ptx::tma_load_3d(raw + Shape::kY + sx * Shape::kYBytes + b * 16384, &dir.tm_y, &sm.y_full[sx], b * 64,
                                     h, row);
            }
            if (*fail)  // let the copies in flight land
                for (int i = max(0, it - NS); i < it; ++i) {
                    wait_for(&sm.x_full[i % NS], (i / NS) & 1);
                    if (OUT) wait_for(&sm.q_full[i % NS], (i / NS) & 1);
                    wait_for(&sm.y_full[i % NS], (i / NS) & 1);
                }
        } else if (warp == 1 && elect_one()) {
            // ---------------------------------------------------------- MMAs
            constexpr uint32_t id_scores = idesc16<F16>(128, 128, 0, 0), id_far = idesc16<F16>(128, V, 0, 0),
                               id_near = idesc16<F16>(128, V, 0, 1), id_added = idesc16<F16>(128, K, 1, 1);
            for (int it = 0; it < chunks && !*fail; ++it) {
                const int sx = it % NS;
                const uint32_t ph = it & 1, px = (it / NS) & 1;
                const uint32_t y_mn = desc_lo(base + Shape::kY + sx * Shape::kYBytes, 16384);
                const uint32_t q_k = desc_lo(base + Shape::kQ + sx * Shape::kXBytes, 16);
                if constexpr (OUT) {
                    const uint32_t x_k = desc_lo(base + Shape::kX + sx * Shape::kXBytes, 16);
                    wait(sm.x_full[sx], px);
                    wait(sm.q_full[sx], px);
                    ptx::tc_fence_after();
#pragma unroll 1
                    for (uint32_t ks = 0; ks < 4 * KB; ++ks) {
                        const uint32_t off = (ks & 3) * 2 + (ks >> 2) * 1024;
                        mma_lo(tmem + Shape::kScores, q_k + off, x_k + off, id_scores, ks);
                    }
                    ptx::mma_commit(&sm.scores);
                    ptx::mma_commit(&sm.x_empty[sx]);
                }
                if constexpr (OUT) {
                    const uint32_t t_out = tmem + Shape::kOut + ph * 128, s_k = desc_lo(base + Shape::kS, 16);
                    wait(sm.s_ready, ph);
                    if (it >= 2) wait(sm.o_free[ph], ((it >> 1) - 1) & 1);
                    ptx::tc_fence_after();
#pragma unroll 1
                    for (uint32_t ks = 0; ks < 4 * KB; ++ks)
                        mma_lo(t_out, q_k + (ks & 3) * 2 + (ks >> 2) * 1024, s_k + (ks & 3) * 2 + (ks >> 2) * (V * 8), id_far, ks);
                    ptx::mma_commit(&sm.far);
                    ptx::mma_commit(&sm.q_empty[sx]);
                }
                if (it > 0) wait(sm.added_read, ph ^ 1);
                wait(sm.y_full[sx], px);
                wait(sm.keys, ph);
                ptx::tc_fence_after();
                const uint32_t hi_mn = desc_lo(base + Shape::kHi, 16384);
#pragma unroll 1
                for (uint32_t ks = 0; ks < 16; ++ks)  // hi, then lo
                    mma_lo(tmem + Shape::kAdded, y_mn + (ks & 7) * 128, hi_mn + (ks & 7) * 128 + (ks >> 3) * (Shape::kXBytes >> 4),
                           id_added, ks);
                ptx::mma_commit(&sm.added);
                ptx::mma_commit(&sm.keys_read);
                if constexpr (OUT) {
                    const uint32_t t_out = tmem + Shape::kOut + ph * 128;
                    wait(sm.p_ready, ph);
                    wait(sm.far_ok, ph);
                    ptx::tc_fence_after();
#pragma unroll 1
                    for (uint32_t ks = 0; ks < 8; ++ks)
                        mma_ts_lo(t_out, tmem + Shape::kScores + ks * 8, y_mn + ks * 128, id_near);
                    ptx::mma_commit(&sm.o_full);
                }
                ptx::mma_commit(&sm.y_empty[sx]);
            }
        } else if (warp == 2) {
            // ---------------------------------------------------------- decays
            auto loaded = [&](int it) {
                return load_g(a.g, a.g_stride, sm.head, (int64_t)sm.row + offset(it), sm.left - offset(it), lane);
            };
            LoadedG next;
            if (chunks > 0) next = loaded(0);
            for (int it = 0; it < chunks; ++it) {
                const int st = it & 1;
                const LoadedG now = next;
                if (it + 1 < chunks) next = loaded(it + 1);
                if (it >= 2) wait(sm.g_free[st], ((it >> 1) - 1) & 1);
                const Pair all = sum_decay(now, sm.decay[st], lane);
                const int rise = OUT && F16 ? rise_of(now) : 0;
                if (lane == 0) sm.whole[st] = whole_decay(all), sm.rise[st] = rise;
                arrive(sm.g_ready[st]);
            }
        }
    } else if (warp < Shape::kFirstState) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs::kKeys));
        // ---------------------------------------------------------- keys: scaled, in two parts
        // the token whose row this thread has, and 16-byte pieces from c_first on (all of it, or half)
        constexpr int kPieces = K / 8 / (Shape::kKeyWarps / 4);
        const int j = quarter * 32 + lane, c_first = ((warp - 4) >> 2) * kPieces;
        const uint32_t to = swizzled_row(base + Shape::kHi, j);
        for (int it = 0; it < chunks; ++it) {
            const int st = it & 1, sx = it % NS;
            const bool live = j < sm.left - offset(it);
            wait(sm.g_ready[st], (it >> 1) & 1);
            const ChunkDecay& d = sm.decay[st];
            float w = dir.weight * exp2_fast(reverse ? d.hi[j] + d.lo[j]
                                                     : gap(d, kDecayChunk - 1, d.hi[j], d.lo[j]));
            arrive(sm.g_free[st]);
            wait(sm.x_full[sx], (it / NS) & 1);
            const uint32_t row = swizzled_row(base + Shape::kX + sx * Shape::kXBytes, j);
            float up = 1.f;
            if constexpr (F16) {
                // The scaled keys may be far below fp16's normal range, where a part keeps no relative precision: a
                // power of two for all of the chunk's brings the largest near the top of it.
                const float plain = live ? largest_half<kPieces>(row, c_first) : 0.f, m = plain * fabsf(w);
                const uint32_t top = __reduce_max_sync(~0u, __float_as_uint(m));
                const uint32_t plain_top = OUT ? __reduce_max_sync(~0u, __float_as_uint(plain)) : 0u;
                if (lane == 0) sm.key_top[st][warp - 4] = top, sm.plain_top[st][warp - 4] = plain_top;
                named_sync(4, 32 * Shape::kKeyWarps);
                if (OUT && j == 0 && c_first == 0) ptx::mbar_arrive(&sm.plain[st]);
                uint32_t all = sm.key_top[st][0];
#pragma unroll
                for (int i = 1; i < Shape::kKeyWarps; ++i) all = max(all, sm.key_top[st][i]);
                up = scale_to_f16(all);
                w *= up;
            }
            if (it > 0) wait(sm.keys_read, st ^ 1);
            if (F16 && j == 0 && c_first == 0) sm.key_unscale[st] = 1.f / up;
            const uint64_t w2 = pair_of(w, w), minus = pair_of(-1.f, -1.f);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                constexpr int kHalf = kPieces / 2;
                uint4 x[kHalf];
#pragma unroll
                for (int i = 0; i < kHalf; ++i) {
                    const int c = c_first + half * kHalf + i;
                    x[i] = lds128((row ^ ((c & 7) << 4)) + (c >> 3) * 16384);
                }
                if (half == 1) arrive(sm.x_empty[sx]);
#pragma unroll
                for (int i = 0; i < kHalf; ++i) {
                    const int c = c_first + half * kHalf + i;
                    if (!live) x[i] = make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t in[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float2 f = from_b16x2<F16>(in[e]);
                        const uint64_t p = mul2(pair_of(f.x, f.y), w2);
                        f = floats_of(p);
                        hi[e] = pack_b16x2(f.x, f.y, F16);
                        f = from_b16x2<F16>(hi[e]);
                        f = floats_of(fma2(pair_of(f.x, f.y), minus, p));
                        lo[e] = pack_b16x2(f.x, f.y, F16);
                    }
                    const uint32_t p = (to ^ ((c & 7) << 4)) + (c >> 3) * 16384;
                    sts128(p, hi[0], hi[1], hi[2], hi[3]);
                    sts128(p + Shape::kXBytes, lo[0], lo[1], lo[2], lo[3]);
                }
            }
            if (sm.left - offset(it) < kDecayChunk) {
                // rows behind the sequence are another's, or nobody's: a zero weight would not hold back a NaN
                wait(sm.y_full[sx], (it / NS) & 1);
                if (!live && c_first == 0) {
                    const uint32_t y = base + Shape::kY + sx * Shape::kYBytes + j * 128;
#pragma unroll 1
                    for (int c = 0; c < V / 8; ++c) sts128(y + (c >> 3) * 16384 + ((c & 7) << 4), 0u, 0u, 0u, 0u);
                }
            }
            ptx::fence_proxy_async_smem();
            arrive(sm.keys);
        }
    } else if (warp < Shape::kFirstState + 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Regs::kState));
        // ---------------------------------------------------------- the state, transposed: column v of S
        const int v = quarter * 32 + lane;
        constexpr int kThreads = 64 * VB;
        if (quarter < 2 * VB) {
            float S[K];
            const bool first = sm.first;
            const int64_t unit = blockIdx.x, seq = (int64_t)sm.n * a.H + sm.head;
            float* piece = dir.totals + unit * K * V + v;  // (null without pieces: not used then)
            const uint16_t* start16 = static_cast<const uint16_t*>(dir.start.p) + seq * K * V + v;
            const float* start = first ? static_cast<const float*>(dir.start.p) + seq * K * V + v : piece;
            const bool none = a.totals_only || (first && !dir.start.p), b16 = first && dir.start.b16;
            if (none) {
#pragma unroll
                for (int k = 0; k < K; ++k) S[k] = 0.f;
            } else if (!b16) {  // (all loads in flight: one after the other in sixteens they took 6 us)
#pragma unroll
                for (int k = 0; k < K; ++k) S[k] = __ldcg(start + k * V);
            } else {
#pragma unroll
                for (int k = 0; k < K; ++k) S[k] = from_b16<false>(__ldcg(start16 + k * V));
            }
            const bool keep = !OUT && dir.kept;
            float decay = 1.f;
            for (int it = 0; it < chunks; ++it) {
                const int st = it & 1, ph = it & 1;
                if (OUT || keep) {
                    // S as 16 bits (and, kept, what that lost), in rows of 128 bytes as the MMAs read them
                    if (OUT && it > 0) wait(sm.far, ph ^ 1);  // (the far products have read the last one)
                    if (!OUT && it > 0) {
                        if (quarter == 0 && elect_one()) ptx::bulk_wait_read0();  // the last chunk's copy has left
                        named_sync(1, kThreads);
                    }
                    float up = 1.f;
                    if constexpr (F16) {  // fp16's range is kept by a power of two for the whole state
                        uint32_t top = 0;
#pragma unroll
                        for (int k = 0; k < K; ++k) top = max(top, __float_as_uint(S[k]) & 0x7fffffffu);
                        top = __reduce_max_sync(~0u, top);
                        if (lane == 0) sm.top[quarter] = top;
                        named_sync(2, kThreads);
                        for (int i = 0; i < 2 * VB; ++i) top = max(top, sm.top[i]);
                        up = scale_to_f16(top);
                        named_sync(1, kThreads);  // (top is written again in the next chunk)
                    }
                    // (kept: 64 values x all keys after another, as the gradients take them)
                    const uint32_t row = OUT ? swizzled_row(base + Shape::kS, v)
                                             : swizzled_row(base + Shape::kS + (v >> 6) * KB * 8192, v & 63);
#pragma unroll
                    for (int c = 0; c < K / 8; ++c) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x = S[8 * c + 2 * e] * up, y = S[8 * c + 2 * e + 1] * up;
                            hi[e] = pack_b16x2(x, y, F16);
                            const float2 back = from_b16x2<F16>(hi[e]);
                            lo[e] = pack_b16x2(x - back.x, y - back.y, F16);
                        }
                        const uint32_t p = (row ^ ((c & 7) << 4)) + (c >> 3) * (OUT ? V * 128 : 8192);
                        sts128(p, hi[0], hi[1], hi[2], hi[3]);
                        if (!OUT) sts128(p + Shape::kStateBytes, lo[0], lo[1], lo[2], lo[3]);
                    }
                    ptx::fence_proxy_async_smem();
                    if (OUT) {
                        if (v == 0) sm.unscale[st] = 1.f / up;
                    } else {
                        named_sync(2, kThreads);
                        if (quarter == 0 && elect_one()) {
                            const int64_t chunk = (int64_t)(sm.chunk + offset(it) / kDecayChunk) * a.H + sm.head;
                            bulk_store_async(dir.kept + chunk * 2 * Shape::kStateBytes, raw + Shape::kS,
                                             2 * Shape::kStateBytes);
                            ptx::bulk_commit();
                            if (F16) dir.kept_scale[chunk] = 1.f / up;
                        }
                    }
                }
                if (OUT) arrive(sm.s_ready);
                wait(sm.g_ready[st], (it >> 1) & 1);
                const float whole = sm.whole[st];
                arrive(sm.g_free[st]);
                decay *= whole;
                wait(sm.added, ph);
                ptx::tc_fence_after();
                const float back = F16 ? sm.key_unscale[st] : 1.f;
#pragma unroll
                for (int c = 0; c < K / 16; ++c) {
                    float u[16];
                    ptx::tmem_ld16(tmem + Shape::kAdded + ((uint32_t)(quarter * 32) << 16) + c * 16, u);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        float* s = S + 16 * c + e;
                        const uint64_t w = pair_of(whole, whole), now = pair_of(s[0], s[1]), more = pair_of(u[e], u[e + 1]);
                        const float2 r = floats_of(F16 ? fma2(more, pair_of(back, back), mul2(w, now)) : fma2(w, now, more));
                        s[0] = r.x, s[1] = r.y;
                    }
                }
                ptx::tc_fence_before();
                arrive(sm.added_read);
            }
            if (a.totals_only) {
#pragma unroll
                for (int k = 0; k < K; ++k) piece[k * V] = S[k];
                if (v == 0) dir.decays[unit] = decay;
            } else if (sm.last && dir.end.p) {
                const int64_t seq = (int64_t)sm.n * a.H + sm.head;
                if (dir.end.b16) {
                    uint16_t* p = static_cast<uint16_t*>(dir.end.p) + seq * K * V + v;
#pragma unroll
                    for (int k = 0; k < K; ++k) p[k * V] = to_b16(S[k], false);
                } else {
                    float* p = static_cast<float*>(dir.end.p) + seq * K * V + v;
#pragma unroll
                    for (int k = 0; k < K; ++k) p[k * V] = S[k];
                }
            }
            if (quarter == 0 && keep && elect_one()) ptx::bulk_wait0();
        }
    } else if (warp < Shape::kFirstState + 8) {
        if constexpr (OUT) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs::kScores));  // (or none: 80)
            // ------------------------------------------------------ P: row i of the scores
            const int i = quarter * 32 + lane;
            const uint32_t t_row = tmem + Shape::kScores + ((uint32_t)(quarter * 32) << 16);
            for (int it = 0; it < chunks; ++it) {
                const int st = it & 1, sx = it % NS;
                float scale = a.scale;
                wait(sm.g_ready[st], (it >> 1) & 1);
                const ChunkDecay& d = sm.decay[st];
                const float hi = d.hi[i], lo = d.lo[i];
                named_sync(3, 128);  // the last chunk's factors have been read
                sm.column[i] = exp2_fast(gap(d, quarter * 32 + 31, hi, lo));
                named_sync(3, 128);
                if constexpr (F16) {
                    // Scores as fp16 have to be near the top of its range, or small ones lose their bits and large ones
                    // overflow: a power of two for each 32 rows, which their far parts are multiplied by and o divided. It
                    // is found before the scores are there, from what they can be at most, K max |q| max |k| (of random
                    // rows 2^5 times their largest). 4 x 8192 tokens x 32 heads of 128 x 128 take 231 us, without any power
                    // 219; found from the scores themselves, which it has to wait for, 255 where this was 243, by the two
                    // warps with the least to do 268.
                    wait(sm.q_full[sx], (it / NS) & 1);
                    const float mine = largest_half<K / 8>(swizzled_row(base + Shape::kQ + sx * Shape::kXBytes, i), 0);
                    const uint32_t q_top = __reduce_max_sync(~0u, i < sm.left - offset(it) ? __float_as_uint(mine) : 0u);
                    arrive(sm.q_empty[sx]);
                    wait(sm.plain[st], (it >> 1) & 1);
                    const uint32_t k_top = __reduce_max_sync(~0u, sm.plain_top[st][lane & 7]);
                    arrive(sm.x_empty[sx]);  // (plain_top has been read: the keys after the next may come)
                    const float most = (float)K * fabsf(scale) * __uint_as_float(q_top) * __uint_as_float(k_top);
                    const int n = score_power(most, sm.rise[st]);
                    if (lane == 0) sm.score_powers[st][quarter] = (int8_t)n;
                    scale *= power_of_two(n);
                    arrive(sm.scaled[st]);
                }
                wait(sm.scores, it & 1);
                ptx::tc_fence_after();
                // Left of the diagonal's 32 x 32 block a pair's decay is taken in two steps, from the token to
                // the end of its 32 and from there to i, both at most one: one multiplication each
                // instead of an exponential per pair.
#pragma unroll 1
                for (int b = 0; b < quarter; ++b) {
                    const int end = 32 * b + 31;
                    const float r = scale * exp2_fast((hi - d.hi[end]) + (lo - d.lo[end]));
                    const uint64_t r2 = pair_of(r, r);
                    float s[32];
                    uint32_t p[16];
                    ptx::tmem_ld16(t_row + 32 * b, s);
                    ptx::tmem_ld16(t_row + 32 * b + 16, s + 16);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float4 c = *reinterpret_cast<const float4*>(&sm.column[32 * b + 2 * e]);
                        const float2 u = floats_of(mul2(pair_of(s[2 * e], s[2 * e + 1]), mul2(r2, pair_of(c.x, c.y))));
                        const float2 v = floats_of(mul2(pair_of(s[2 * e + 2], s[2 * e + 3]), mul2(r2, pair_of(c.z, c.w))));
                        p[e] = pack_b16x2(u.x, u.y, F16);
                        p[e + 1] = pack_b16x2(v.x, v.y, F16);
                    }
                    tmem_st16(t_row + 16 * b, p);  // (over scores that have been read)
                }
#pragma unroll 1
                for (int c = 0; c < 32; c += 16) {  // the diagonal's block
                    float s[16];
                    uint32_t p[8];
                    ptx::tmem_ld16(t_row + 32 * quarter + c, s);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float2 h2 = *reinterpret_cast<const float2*>(&d.hi[32 * quarter + c + e]);
                        const float2 l2 = *reinterpret_cast<const float2*>(&d.lo[32 * quarter + c + e]);
                        const float u = s[e] * (scale * exp2_fast((hi - h2.x) + (lo - l2.x)));
                        const float v = s[e + 1] * (scale * exp2_fast((hi - h2.y) + (lo - l2.y)));
                        p[e >> 1] = pack_b16x2(c + e <= lane ? u : 0.f, c + e + 1 <= lane ? v : 0.f, F16);
                    }
                    tmem_st8(t_row + 16 * quarter + (c >> 1), p);
                }
#pragma unroll 1
                for (int c = 16 * quarter + 16; c < 64; c += 8) {
                    const uint32_t none[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
                    tmem_st8(t_row + c, none);
                }
                tmem_st_wait();
                ptx::tc_fence_before();
                arrive(sm.g_free[st]);
                arrive(sm.p_ready);
            }
        }
    } else {
        if constexpr (OUT) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs::kOut));
            // ------------------------------------------------------ o: row i
            // A warp's 32 rows leave by TMA out of a swizzled copy (rows stored by their threads are 32 lines a store);
            // where the sequence ends among them, by their threads.
            const int i = quarter * 32 + lane;
            const uint32_t t_row = tmem + ((uint32_t)(quarter * 32) << 16), box = base + Shape::kO + quarter * 4096;
            const uint32_t to = swizzled_row(box, lane);
            for (int it = 0; it < chunks; ++it) {
                const int st = it & 1, tok = offset(it) + i;
                const bool whole = tok - lane + 32 <= sm.left;
                const uint32_t t_out = t_row + Shape::kOut + st * 128;
                wait(sm.g_ready[st], (it >> 1) & 1);
                float f = a.scale * exp2_fast(sm.decay[st].hi[i] + sm.decay[st].lo[i]), down = 1.f;
                arrive(sm.g_free[st]);
                if constexpr (F16) {
                    wait(sm.scaled[st], (it >> 1) & 1);
                    const int n = sm.score_powers[st][quarter];
                    f *= power_of_two(n);
                    down = power_of_two(-n);
                }
                // the far part, scaled by rows: the near products add to it
                wait(sm.far, st);
                ptx::tc_fence_after();
                if (F16) f *= sm.unscale[st];
#pragma unroll 1
                for (int c = 0; c < V; c += 32) {
                    float u[32];
                    ptx::tmem_ld16(t_out + c, u);
                    ptx::tmem_ld16(t_out + c + 16, u + 16);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 r = floats_of(mul2(pair_of(f, f), pair_of(u[e], u[e + 1])));
                        u[e] = r.x, u[e + 1] = r.y;
                    }
                    tmem_st16(t_out + c, reinterpret_cast<const uint32_t*>(u));
                    tmem_st16(t_out + c + 16, reinterpret_cast<const uint32_t*>(u + 16));
                }
                tmem_st_wait();
                ptx::tc_fence_before();
                arrive(sm.far_ok);
                if (elect_one()) ptx::bulk_wait_read0();  // the last chunk's rows have left
                wait(sm.o_full, st);
                ptx::tc_fence_after();
                __syncwarp();
                uint16_t* o = a.o + (((int64_t)sm.row + tok) * a.H + sm.head) * V;
#pragma unroll 1
                for (int c = 0; c < V; c += 32) {
                    float u[32];
                    ptx::tmem_ld16(t_out + c, u);
                    ptx::tmem_ld16(t_out + c + 16, u + 16);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        uint32_t y[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float2 x = make_float2(u[8 * g + 2 * e], u[8 * g + 2 * e + 1]);
                            if constexpr (F16) x = floats_of(mul2(pair_of(x.x, x.y), pair_of(down, down)));
                            y[e] = pack_b16x2(x.x, x.y, F16);
                        }
                        if (whole) sts128((to ^ (((c & 63) << 1) + g * 16)) + (c >> 6) * 16384, y[0], y[1], y[2], y[3]);
                        else if (tok < sm.left) *reinterpret_cast<uint4*>(o + c + 8 * g) = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
                ptx::tc_fence_before();
                ptx::fence_proxy_async_smem();
                arrive(sm.o_free[st]);
                if (elect_one() && whole) {
#pragma unroll
                    for (int b = 0; b < VB; ++b)
                        ptx::tma_store_3d(&a.tm_o, raw + Shape::kO + quarter * 4096 + b * 16384, b * 64, sm.head, sm.row + tok);
                    ptx::bulk_commit();
                }
            }
            if (elect_one()) ptx::bulk_wait0();
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc(tmem, Shape::kTmem);
    if (sm.fail && tid == 0 && a.status) atomicOr(a.status, kStatusTimeout);
}

template <int KB, int VB, bool F16, bool OUT>
cudaError_t launch_scan_shape(const DecayScanArgs& a, int dirs, cudaStream_t s) {
    using Shape = DecayScanShape<KB, VB, OUT>;
    auto kern = kda_decay_scan_kernel<KB, VB, F16, OUT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape::kSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3((unsigned)(a.seqs.pieces * a.H), (unsigned)dirs), dim3(Shape::kThreads),
                            (size_t)Shape::kSmem, s, a);
}
template <bool OUT>
cudaError_t launch_scan_any(const DecayScanArgs& a, int K, int V, bool f16, int dirs, cudaStream_t s) {
    if (K == 128) {
        if (V == 128) return f16 ? launch_scan_shape<2, 2, true, OUT>(a, dirs, s) : launch_scan_shape<2, 2, false, OUT>(a, dirs, s);
        return f16 ? launch_scan_shape<2, 1, true, OUT>(a, dirs, s) : launch_scan_shape<2, 1, false, OUT>(a, dirs, s);
    }
    if (V == 128) return f16 ? launch_scan_shape<1, 2, true, OUT>(a, dirs, s) : launch_scan_shape<1, 2, false, OUT>(a, dirs, s);
    return f16 ? launch_scan_shape<1, 1, true, OUT>(a, dirs, s) : launch_scan_shape<1, 1, false, OUT>(a, dirs, s);
}

}  // namespace
}  // namespace kda
