// decay.cuh -- what the kernels of linear attention with a decay per head share
// (decay_scan.cuh: states and output; decay_grads.cu: gradients; decay_api.cu:
// the C entries).
//
// With S the K x V state of one (sequence, head) and g_t <= 0 its log decay,
//     S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t.
// In chunks of 128 tokens, G_i the sum of g over the chunk's tokens up to i and
// S the state before the chunk:
//     o_i = scale (exp(G_i) S^T q_i + sum_{j <= i} exp(G_i - G_j) (q_i . k_j) v_j)
//     S'  = exp(G_last) S + sum_j exp(G_last - G_j) k_j v_j^T
// The decay is one number per token, so it never has to be factored over the
// key dimension: it multiplies rows and columns of products.
#pragma once
#include <cuda.h>

#include "internal.h"
#include "layer_ops.cuh"
#include "ptx.cuh"
#include "tensormap.h"
#include "waits.cuh"

namespace kda {

constexpr int kDecayChunk = 128;  // tokens: one row of a tcgen05 accumulator each

// Sequences of one call, and how they are cut: `cu` null means B = N sequences
// of T tokens each.  A piece is a run of seg_chunks chunks of one sequence.
struct DecaySeqs {
    const int32_t* cu;   // int32 [N + 1] or null
    int32_t N, T;        // T: tokens of a sequence, or (packed) of all
    int32_t seg_chunks;  // chunks per piece
    int32_t pieces;      // grid size in pieces: exact, or (packed) an upper bound
    int32_t whole;       // no sequence is cut: a piece is a sequence
};

// Where a state's memory is fp32 or bf16.
struct DecayState {
    void* p;      // [N, H, K, V] or null
    int32_t b16;  // bf16
};

// One direction of the state scan: S over (k, v) forwards, or dS over (q, do) backwards.
struct DecayScanDir {
    CUtensorMap tm_x, tm_y;  // 3-D {dim, heads, rows}: k or q, v or do
    DecayState start, end;   // h0 and ht, or dht and dh0
    float* totals;           // fp32 [pieces, H, K, V]: what a piece adds, then (joined) the state that enters it
    float* decays;           // fp32 [pieces, H]: exp of a piece's whole decay
    uint8_t* kept;           // [chunks, H]: the state before each chunk, two parts of 16 bits (see scan), or null
    float* kept_scale;       // fp32 [chunks, H]: what the parts are multiplied by (fp16)
    float weight;            // of the products that are added: 1, or scale
    int32_t reverse;
};

struct DecayScanArgs {
    DecayScanDir dir[2];
    CUtensorMap tm_q;    // the output pass
    DecaySeqs seqs;
    const float* g;      // fp32: g[row * g_stride + h] (g_stride 0: one decay per head)
    int64_t g_stride;
    uint16_t* o;         // [rows, H, V]
    CUtensorMap tm_o;    // the same, 3-D {V, H, rows}, boxes of 64 x 32 rows
    int32_t* status;     // or null
    float scale;
    int32_t H, group;    // value heads, value heads per q/k head
    int32_t totals_only; // the pass before a join: pieces' totals, nothing else
};

struct DecayJoinArgs {
    DecayScanDir dir[2];
    DecaySeqs seqs;
    int32_t H, state;    // state: K V
};

struct DecayGradArgs {
    CUtensorMap tm_q, tm_k, tm_v, tm_do;
    CUtensorMap tm_dq, tm_dk, tm_dv;  // boxes of 128 bytes x 32 rows (dq, dk: as they are written)
    DecaySeqs seqs;      // seg_chunks = 1
    const float* g;
    int64_t g_stride;
    const uint8_t *kept, *dkept;
    const float *kept_scale, *dkept_scale;
    void *dq, *dk;       // [rows, Hqk, K] 16 bits, or (groups of three and more) fp32 [rows, H, K]
    uint16_t* dv;        // [rows, H, V]
    float* dg;           // fp32 [rows, H]
    int32_t* status;
    float scale;
    int32_t H, group, sms;
    int32_t paired;      // groups of two: their value heads are a cluster and add dq and dk up themselves
};

cudaError_t launch_decay_out(const DecayScanArgs& a, int K, int V, bool f16, cudaStream_t s);
cudaError_t launch_decay_states(const DecayScanArgs& a, int K, int V, bool f16, int dirs, cudaStream_t s);
cudaError_t launch_decay_join(const DecayJoinArgs& a, int dirs, cudaStream_t s);
cudaError_t launch_decay_grads(const DecayGradArgs& a, int K, int V, bool f16, cudaStream_t s);
// dq, dk [rows, heads, K] in 16 bits from fp32 [rows, heads, group, K] (nothing if the offsets of seqs are out of order)
cudaError_t launch_decay_group(const float* dq32, const float* dk32, void* dq, void* dk, const DecaySeqs& seqs, int64_t rows,
                               int heads, int K, int group, bool f16, int sms, cudaStream_t s);
// out [H]: dg [rows, H] summed over the rows (likewise); part: fp32 [(rows + 255) / 256, H]
cudaError_t launch_decay_gate(const float* dg, float* part, float* out, const DecaySeqs& seqs, int64_t rows, int H,
                              cudaStream_t s);

namespace {

// ------------------------------------------------------------------ which piece
struct DecayPiece {
    int32_t n, piece, pieces;    // sequence (-1: none), piece of it, its pieces
    int32_t bos, len;            // of the sequence
    int32_t chunk_base;          // chunks of the sequences before it
    int32_t piece_base;          // pieces of the sequences before it
};
__host__ __device__ __forceinline__ int32_t ceil_div(int32_t a, int32_t b) { return (a + b - 1) / b; }

constexpr int kMostSorted = 512;  // sequences that are taken longest first
struct DecayScratch {
    int32_t warp_pieces[32], warp_chunks[32];
    DecayPiece found;
};
struct DecaySortScratch : DecayScratch {
    int32_t len[kMostSorted];
};

// cu[n] and cu[n + 1] are no sequence's bounds.
__device__ __forceinline__ bool out_of_order(int bos, int eos, int n, int N, int T) {
    return bos < 0 || eos < bos || eos > T || (n == 0 && bos != 0) || (n == N - 1 && eos != T);
}
// cu is 0 = c0 <= c1 <= ... <= cN = T. Called by all THREADS threads.
template <int THREADS>
__device__ __forceinline__ bool in_order(const DecaySeqs& s) {
    if (!s.cu) return true;
    bool bad = false;
    for (int n = threadIdx.x; n < s.N; n += THREADS) bad |= out_of_order(s.cu[n], s.cu[n + 1], n, s.N, s.T);
    return !__syncthreads_or(bad);
}

// The piece with this index, or the first of sequence `by_seq` (index then a sequence).  Called by
// all THREADS threads.  A sequence without tokens has one piece where `empty` says so.  Returns
// false if cu is not 0 = c0 <= c1 <= ... <= cN = T.  With `len` (kMostSorted, if there are not more sequences, uncut) the
// index'th longest sequence: CTAs start in the order of their index, and a long one that starts last is waited for alone.
template <int THREADS>
__device__ __forceinline__ bool find_piece(const DecaySeqs& s, int index, bool by_seq, bool empty, DecayScratch& sm,
                                           DecayPiece& out, int32_t* len = nullptr) {
    if (!s.cu) {
        const int nc = ceil_div(s.T, kDecayChunk);
        const int per = max(ceil_div(nc, s.seg_chunks), empty ? 1 : 0);
        out.n = by_seq ? index : per > 0 ? index / per : -1;
        if (out.n >= s.N) out.n = -1;
        out.piece = by_seq ? 0 : per > 0 ? index % per : 0;
        out.pieces = per;
        out.bos = out.n * s.T;
        out.len = s.T;
        out.chunk_base = out.n * nc;
        out.piece_base = out.n * per;
        return true;
    }
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (len && s.N <= kMostSorted) {
        for (int n = tid; n < s.N; n += THREADS) len[n] = s.cu[n + 1] - s.cu[n];
        if (tid == 0) sm.found.n = 0;
        __syncthreads();
        for (int n = tid; n < s.N; n += THREADS) {
            int ahead = 0;
            for (int m = 0; m < s.N; ++m) ahead += len[m] > len[n] || (len[m] == len[n] && m < n);
            if (ahead == index) sm.found.n = n;
        }
        __syncthreads();
        index = sm.found.n;
        by_seq = true;
        __syncthreads();
    }
    const int each = (s.N + THREADS - 1) / THREADS;
    const int first = min(tid * each, s.N), last = min(first + each, s.N);
    int pieces = 0, chunks = 0;
    bool bad = false;
    for (int n = first; n < last; ++n) {
        const int bos = s.cu[n], eos = s.cu[n + 1];
        bad |= out_of_order(bos, eos, n, s.N, s.T);
        const int nc = ceil_div(max(eos - bos, 0), kDecayChunk);
        chunks += nc;
        pieces += max(ceil_div(nc, s.seg_chunks), empty ? 1 : 0);
    }
    int sp = pieces, sc = chunks;  // inclusive sums over the warp
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int p = __shfl_up_sync(~0u, sp, off), c = __shfl_up_sync(~0u, sc, off);
        if (lane >= off) sp += p, sc += c;
    }
    if (lane == 31) sm.warp_pieces[warp] = sp, sm.warp_chunks[warp] = sc;
    if (tid == 0) sm.found.n = -1;
    if (__syncthreads_or(bad)) return false;
    for (int w = 0; w < warp; ++w) sp += sm.warp_pieces[w], sc += sm.warp_chunks[w];
    sp -= pieces, sc -= chunks;  // before this thread's sequences
    if (by_seq ? (index >= first && index < last) : (index >= sp && index < sp + pieces)) {
        for (int n = first; n < last; ++n) {
            const int bos = s.cu[n], len = s.cu[n + 1] - bos;
            const int nc = ceil_div(len, kDecayChunk), per = max(ceil_div(nc, s.seg_chunks), empty ? 1 : 0);
            if (by_seq ? n == index : index < sp + per) {
                sm.found = DecayPiece{n, by_seq ? 0 : index - sp, per, bos, len, sc, sp};
                break;
            }
            sp += per, sc += nc;
        }
    }
    __syncthreads();
    out = sm.found;
    return true;
}

// ------------------------------------------------------------------ decays
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// A sum of two floats: hi + lo exactly what was added.
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ Pair add_pairs(Pair a, Pair b) {
    const float s = a.hi + b.hi, t = s - a.hi;
    const float e = (a.hi - (s - t)) + (b.hi - t) + (a.lo + b.lo);
    const float hi = s + e;
    return {hi, e - (hi - s)};
}
// g in powers of two, to 2^-45 of itself.  A decay below 2^-200 per token leaves nothing of a state
// in fp32 either way; cutting it there keeps -inf out of the differences.
__device__ __forceinline__ Pair log2_decay(float g) {
    constexpr float kLog2e = 1.44269504f, kRest = (float)(1.4426950408889634 - (double)kLog2e);
    g = g < -140.f ? -140.f : g;
    const float hi = g * kLog2e;
    return {hi, fmaf(g, kRest, fmaf(g, kLog2e, -hi))};
}

// The decays of one chunk up to each of its tokens, in powers of two: differences of these sums are
// right to 2^-24 of themselves and 2^-43 of the sums (up to 15 additions of pairs, 2^-47 each), since what the
// leading parts lost is kept in the second ones.
struct ChunkDecay {
    float hi[kDecayChunk], lo[kDecayChunk];
};
__device__ __forceinline__ float gap(const ChunkDecay& d, int i, float hi_j, float lo_j) {
    return (d.hi[i] - hi_j) + (d.lo[i] - lo_j);
}

// A warp's four tokens per lane of a chunk's g; rows behind the sequence decay by nothing.
struct LoadedG {
    float v[4];
};
__device__ __forceinline__ LoadedG load_g(const float* g, int64_t stride, int h, int64_t row0, int valid, int lane) {
    LoadedG r;
    const float* p = g + (row0 + lane * 4) * stride + h;
#pragma unroll
    for (int i = 0; i < 4; ++i, p += stride) r.v[i] = lane * 4 + i < valid ? *p : 0.f;
    return r;
}
// One warp: the sums of a chunk; the last one is returned to all lanes.
__device__ __forceinline__ Pair sum_decay(const LoadedG& g, ChunkDecay& out, int lane) {
    Pair run = log2_decay(g.v[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) run = add_pairs(run, log2_decay(g.v[i]));
#pragma unroll 1
    for (int off = 1; off < 32; off <<= 1) {
        const Pair up{__shfl_up_sync(~0u, run.hi, off), __shfl_up_sync(~0u, run.lo, off)};
        if (lane >= off) run = add_pairs(up, run);
    }
    Pair s{__shfl_up_sync(~0u, run.hi, 1), __shfl_up_sync(~0u, run.lo, 1)};
    if (lane == 0) s = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s = add_pairs(s, log2_decay(g.v[i]));
        out.hi[lane * 4 + i] = s.hi;
        out.lo[lane * 4 + i] = s.lo;
    }
    return {__shfl_sync(~0u, s.hi, 31), __shfl_sync(~0u, s.lo, 31)};
}
// n for a chunk whose decays between two tokens are at most 2^n: 0 unless some g are above zero.
__device__ __forceinline__ int rise_of(const LoadedG& g) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) s += fmaxf(g.v[i], 0.f);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(~0u, s, off);
    return (int)fminf(ceilf(s * 1.44269504f), 126.f);
}
// exp of a chunk's whole decay, to less than its last bit: a state of thousands of chunks is multiplied by
// one after the other, so their errors add up. 2^n times the power series of exp(x), |x| <= ln(2) / 2, to its
// ninth term (what is left is below 2^-33); only the last addition rounds at the size of the result.
__device__ __forceinline__ float whole_decay(Pair p) {
    const float n = rintf(p.hi);
    const float x = ((p.hi - n) + p.lo) * 0.693147181f;
    float r = fmaf(x, 1.f / 362880, 1.f / 40320);
    r = fmaf(x, r, 1.f / 5040);
    r = fmaf(x, r, 1.f / 720);
    r = fmaf(x, r, 1.f / 120);
    r = fmaf(x, r, 1.f / 24);
    r = fmaf(x, r, 1.f / 6);
    r = fmaf(x, r, 0.5f);
    return ldexpf(1.f + fmaf(x * x, r, x), (int)n);
}

// ------------------------------------------------------------------ two fp32 at a time
__device__ __forceinline__ uint64_t pair_of(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 floats_of(uint64_t p) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// ------------------------------------------------------------------ shared memory by 32-bit address
// (What little L1 is left beside these kernels' shared memory makes a spilled register a trip to L2, so the
// addresses that loops keep are single registers, and a swizzled row's pieces are one xor away from it.)
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// Row `row` of a tile of 128-byte swizzled rows: its 16-byte piece c is at this ^ (c << 4).
__device__ __forceinline__ uint32_t swizzled_row(uint32_t tile, int row) {
    return tile + (uint32_t)row * 128u + (uint32_t)((row & 7) << 4);
}

// ------------------------------------------------------------------ waits
// A wait that runs out (after kDecayWaitCycles) is noted in `fail`, and from then on nobody waits: every warp still goes
// through all of its barriers, so none is left standing at one. Results are then incomplete, and the status says so.
// Few instructions, since every role has many of these in its loop: the roles of a scan run side by side, and what they
// go through once per chunk has to fit the SM's instruction cache together (with 45 KB of it a prefill took 255 us).
constexpr uint32_t kDecayWaitCycles = 4000000000u;  // about two seconds; the counter wraps around above it
__device__ __forceinline__ uint32_t clock_lo() {
    uint32_t t;
    asm volatile("mov.u32 %0, %%clock;" : "=r"(t));
    return t;
}
// CLUSTER: the arrivals come from the other CTA of a pair.
template <bool CLUSTER = false>
__device__ __forceinline__ void wait_or_note(uint64_t* bar, uint32_t parity, int32_t* fail) {
    const uint32_t t0 = clock_lo(), at = ptx::smem_u32(fail);
#pragma unroll 1
    while (!try_wait<CLUSTER>(bar, parity)) {
        int32_t failed;
        asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(failed) : "r"(at) : "memory");
        if (failed) break;
        if (clock_lo() - t0 > kDecayWaitCycles) asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(at), "r"(1) : "memory");
    }
}

// ------------------------------------------------------------------ tcgen05
// D (+)= A B with A in TMEM: lane i, 32-bit column c hold A's row i, elements 2 c and 2 c + 1.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], "
        "[%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// The same with descriptors by their lower words (address and leading offset; of all operands here groups of rows are
// 1024 bytes apart): the issuing thread's registers are few.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo_bytes) {
    return ((saddr & 0x3FFFFu) >> 4) | ((lbo_bytes >> 4) & 0x3FFFu) << 16;
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ void mma_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void mma_ts_lo(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .b64 b;\n\t.reg .pred p;\n\tsetp.eq.b32 p, 0, 0;\n\tmov.b64 b, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "n"(kDescHi)
        : "memory");
}
// 32 lanes x 32 bits, 16 columns (see tmem_ld16).
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* u) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15};" ::"r"(u[0]),
        "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]), "r"(u[10]),
        "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* u) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(u[0]), "r"(u[1]),
                 "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
template <bool F16>
__host__ __device__ constexpr uint32_t idesc16(int M, int N, int a_mn, int b_mn) {
    return F16 ? ptx::idesc_f16_f32(M, N, a_mn, b_mn) : ptx::idesc_bf16_f32(M, N, a_mn, b_mn);
}

// A barrier of `threads` threads of the block.
__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bulk_store_async(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(ptx::smem_u32(src)),
                 "r"(bytes)
                 : "memory");
}

// A multiplier 2^n that brings values of up to `top` in size to 2^13 .. 2^14 (1 for zero, infinities and NaN).
__device__ __forceinline__ float scale_to_f16(uint32_t top_bits) {
    const int e = (int)(top_bits >> 23) - 127;
    if (top_bits == 0 || e == 128) return 1.f;
    const int n = min(max(13 - e, -126), 126);
    return __uint_as_float((uint32_t)(n + 127) << 23);
}
__device__ __forceinline__ float power_of_two(int n) { return __uint_as_float((uint32_t)(n + 127) << 23); }
// n for scores in fp16: times 2^n the largest, `top`, is 2^13 .. 2^14 after decays of at most 2^rise, so that those down to
// 2^-27 of it are in fp16's normal range. At most 40: scores below 2^-54 add less than half of fp16's smallest number
// to any output, and what the state adds to the same sum is multiplied by 2^n too.
__device__ __forceinline__ int score_power(float top, int rise) {
    const uint32_t bits = __float_as_uint(top);
    const int e = (int)(bits >> 23) - 127;
    return bits == 0 || e == 128 ? 0 : min(max(13 - e - rise, -126), 40);
}

}  // namespace
}  // namespace kda
