// step.cu -- kda_step: the gated delta rule for the few new tokens of a decode
// step, on a cache of states addressed by slot and updated in place.
//
// Per token, with S [K, V] the state of one (sequence, head):
//     S <- Diag(exp g) S
//     delta = beta (v - S^T k);   S <- S + k delta^T;   o = scale S^T q.
// Both products with the decayed S are taken in one pass over it, since
//     S_new^T q = S^T q + (k . q) delta,
// so a token costs one sum over the K rows (and one exchange between warps)
// instead of two dependent ones.
//
// Bound: each state is read and written once per call, 2 K V 4 bytes (128 KB at
// K = V = 128 in fp32) against ~7 K V flops, so HBM for a token or two; a few
// tokens per state of 128 x 64 are bound by the issue of their arithmetic.
//
// Two kernels.  This one, for few (sequence, head) pairs: one CTA takes VT
// columns of one pair (the columns are independent given q, k, g, beta).  It
// holds its K x VT part in registers as float4 (a warp's load covers whole
// 128-byte lines), in fp32 whatever the cache's type, across all the tokens.
// From two pairs per SM on the streaming kernel below takes over.  Measured at
// K = V = 128 in fp32, this kernel against that one: 32 pairs 2.9 us, 5.0;
// 128 pairs 4.3, 5.4; 256 pairs 9.7, 10.5; 512 pairs 17, 14; 16384 pairs 490,
// 341 (6.3 TB/s, 94% of what a copy reaches).
#include "internal.h"
#include "layer_ops.cuh"
#include "waits.cuh"

namespace kda {
namespace {

constexpr int kStepThreads = 256, kStepWarps = kStepThreads / 32;
constexpr int kTokens = 4;  // tokens whose inputs are loaded together (even: the exchange buffers alternate)

struct StepArgs {
    const uint16_t *q, *k, *v, *beta;  // bf16 or fp16 bits
    const float* g;
    void* state;                       // fp32 or bf16 [slots, H, K, V]
    const int32_t* slots;              // or null
    const int32_t* cu;                 // or null
    uint16_t* o;
    int32_t* status;                   // or null
    int64_t q_stride, k_stride, v_stride, g_stride, beta_stride;
    float scale;
    int N, T, H, V, group, num_slots, logits;
    int vec;  // q, k, v and g rows take loads of four elements
};

__device__ __forceinline__ void report(int32_t* status, int bit) {
    if (status) atomicOr(status, bit);
}

// Whether sequence n's offsets are not those of 0 = c0 <= c1 <= ... <= cN = T.
__device__ __forceinline__ bool bad_offsets(const StepArgs& a, int n, int bos, int eos) {
    return bos < 0 || eos < bos || eos > a.T || (n == 0 && bos != 0) || (n == a.N - 1 && eos != a.T);
}
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(ptx::smem_u32(src)),
                 "r"(bytes)
                 : "memory");
}

// A token's inputs in shared memory.
template <int K, int COLS>
struct Token {
    float4 kqe[K];  // per row: k, q, exp(g)
    float v[COLS];
    float beta, kq, unused[2];  // kq: k . q
};

// What the warps of THREADS threads exchange of a token: S^T k and S^T q of their rows.
template <int COLS, int THREADS>
struct Sums {
    float4 k[THREADS / 32][COLS / 4], q[THREADS / 32][COLS / 4];
};

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(~0u, x, off);
    return x;
}
__device__ __forceinline__ void add4(float4& a, const float4 b) {
    a.x += b.x;
    a.y += b.y;
    a.z += b.z;
    a.w += b.w;
}
__device__ __forceinline__ void fma4(float4& a, float k, const float4 b) {
    a.x = fmaf(k, b.x, a.x);
    a.y = fmaf(k, b.y, a.y);
    a.z = fmaf(k, b.z, a.z);
    a.w = fmaf(k, b.w, a.w);
}
__device__ __forceinline__ float4 shuffle4(const float4 a, int off) {
    return make_float4(__shfl_xor_sync(~0u, a.x, off), __shfl_xor_sync(~0u, a.y, off), __shfl_xor_sync(~0u, a.z, off),
                       __shfl_xor_sync(~0u, a.w, off));
}

// One token on the K x COLS part of a state that THREADS threads hold, each
// kRows rows (THREADS / (COLS / 4) apart) of four columns.  sums: not those of
// the token before (a thread may still read them); sync: a barrier of these
// threads, false to give up.  o points at the thread's columns of the token's
// output.
template <int K, int COLS, bool F16, int kRows, int THREADS, typename Sync>
__device__ __forceinline__ bool step_token(float4 (&S)[kRows], const Token<K, COLS>& in, Sums<COLS, THREADS>& sums,
                                           float scale, uint16_t* o, int tid, Sync sync) {
    constexpr int kColGroups = COLS / 4, kRowLanes = THREADS / kColGroups, kWarps = THREADS / 32;
    const int cg = tid % kColGroups, rl = tid / kColGroups, warp = tid >> 5, lane = tid & 31;
    float4 pk = make_float4(0.f, 0.f, 0.f, 0.f), pq = pk;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const float4 r = in.kqe[rl + i * kRowLanes];
        S[i].x *= r.z;
        S[i].y *= r.z;
        S[i].z *= r.z;
        S[i].w *= r.z;
        fma4(pk, r.x, S[i]);
        fma4(pq, r.y, S[i]);
    }
#pragma unroll
    for (int off = kColGroups; off < 32; off <<= 1) {  // row lanes of the same columns in this warp
        add4(pk, shuffle4(pk, off));
        add4(pq, shuffle4(pq, off));
    }
    if (lane < kColGroups) {
        sums.k[warp][cg] = pk;
        sums.q[warp][cg] = pq;
    }
    if (!sync()) return false;
    float4 d = sums.k[0][cg];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) add4(d, sums.k[w][cg]);
    const float beta = in.beta;
    const float4 v = *reinterpret_cast<const float4*>(in.v + cg * 4);
    d = make_float4(beta * (v.x - d.x), beta * (v.y - d.y), beta * (v.z - d.z), beta * (v.w - d.w));
    if (rl == 0) {
        float4 y = sums.q[0][cg];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) add4(y, sums.q[w][cg]);
        fma4(y, in.kq, d);
        *reinterpret_cast<uint2*>(o) =
            make_uint2(pack_b16x2(scale * y.x, scale * y.y, F16), pack_b16x2(scale * y.z, scale * y.w, F16));
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) fma4(S[i], in.kqe[rl + i * kRowLanes].x, d);
    return true;
}
// Four elements of a state, in fp32 or bf16, at p[index of 4].
template <bool STATE16>
__device__ __forceinline__ float4 load_state(const void* p, int64_t four) {
    if constexpr (STATE16) {
        const uint2 w = static_cast<const uint2*>(p)[four];
        const float2 lo = from_b16x2<false>(w.x), hi = from_b16x2<false>(w.y);
        return make_float4(lo.x, lo.y, hi.x, hi.y);
    } else {
        return static_cast<const float4*>(p)[four];
    }
}
template <bool STATE16>
__device__ __forceinline__ void store_state(void* p, int64_t four, float4 s) {
    if constexpr (STATE16)
        static_cast<uint2*>(p)[four] = make_uint2(pack_b16x2(s.x, s.y, false), pack_b16x2(s.z, s.w, false));
    else
        static_cast<float4*>(p)[four] = s;
}

// PER_SM: CTAs that an SM has room for, and so the registers of a thread, which hold
// its part of the state and the loads in flight.
template <int K, int VT, bool F16, bool STATE16, int PER_SM>
__global__ void __launch_bounds__(kStepThreads, PER_SM) kda_step_kernel(const StepArgs a) {
    constexpr int kColGroups = VT / 4;                      // threads across a row, 4 columns each
    constexpr int kRowLanes = kStepThreads / kColGroups;    // rows in flight per step of i
    constexpr int kRows = K / kRowLanes;                    // rows a thread holds
    static_assert(kRows >= 1 && kRows * kRowLanes == K, "the threads tile the K rows");
    __shared__ Token<K, VT> s_token[kTokens];
    __shared__ Sums<VT, kStepThreads> s_sums[2];

    const int tid = threadIdx.x;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int tiles = a.V / VT;
    const int tile = blockIdx.x % tiles;
    const int h = (blockIdx.x / tiles) % a.H;
    const int n = blockIdx.x / tiles / a.H;
    const bool first = tile == 0 && h == 0 && tid == 0;

    int64_t row0 = (int64_t)n * a.T;
    int len = a.T;
    if (a.cu) {
        const int bos = a.cu[n], eos = a.cu[n + 1];
        if (bad_offsets(a, n, bos, eos)) {
            if (first) report(a.status, kStatusBadSeqlens);
            return;
        }
        row0 = bos;
        len = eos - bos;
    }
    if (len == 0) return;
    const int slot = a.slots ? a.slots[n] : n;
    const bool in_cache = slot >= 0 && slot < a.num_slots;

    const int cg = tid % kColGroups, rl = tid / kColGroups;
    // (a state's elements in fours)
    const int64_t at = in_cache ? ((((int64_t)slot * a.H + h) * K + rl) * a.V + tile * VT) / 4 + cg : 0;
    const int64_t row_step = (int64_t)kRowLanes * a.V / 4;
    float4 S[kRows];
    if (in_cache) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) S[i] = load_state<STATE16>(a.state, at + i * row_step);
    }

    // Inputs of kTokens tokens at a time, whose loads are in flight together: k
    // and g rows by the first K threads, q by the next 128, v by the first VT.  They
    // are turned into fp32 when they are staged: a load's first use waits for it,
    // and there each token's waited before the next token's was asked for.
    const int hq = h / a.group;
    const int kr = tid & 127;
    uint16_t in_k[kTokens], in_q[kTokens], in_v[kTokens], in_b[kTokens];
    float in_g[kTokens];
    auto load_tokens = [&](int t0) {
#pragma unroll
        for (int j = 0; j < kTokens; ++j) {
            if (t0 + j >= len) break;
            const int64_t row = row0 + t0 + j;
            if (tid < K) {
                in_k[j] = a.k[row * a.k_stride + (int64_t)hq * K + tid];
                in_g[j] = a.g[row * a.g_stride + (int64_t)h * K + tid];
            }
            if (tid >= 128 && kr < K) in_q[j] = a.q[row * a.q_stride + (int64_t)hq * K + kr];
            if (tid < VT) in_v[j] = a.v[row * a.v_stride + (int64_t)h * a.V + tile * VT + tid];
            if (tid == 0) in_b[j] = a.beta[row * a.beta_stride + h];
        }
    };
    auto stage_tokens = [&](int t0) {
#pragma unroll
        for (int j = 0; j < kTokens; ++j) {
            if (t0 + j >= len) break;
            if (tid < K) {
                s_token[j].kqe[tid].x = from_b16<F16>(in_k[j]);
                s_token[j].kqe[tid].z = expf(in_g[j]);
            }
            if (tid >= 128 && kr < K) s_token[j].kqe[kr].y = from_b16<F16>(in_q[j]);
            if (tid < VT) s_token[j].v[tid] = from_b16<F16>(in_v[j]);
            if (tid == 0) {
                const float b = from_b16<F16>(in_b[j]);
                s_token[j].beta = a.logits ? 1.f / (1.f + expf(-b)) : b;
            }
        }
    };
    load_tokens(0);

    // The same slot twice would race: the first sequence that names it has it.
    bool taken = false;
    if (in_cache && a.slots)
        for (int j = tid; j < n; j += kStepThreads) taken |= a.slots[j] == slot;
    stage_tokens(0);
    taken = __syncthreads_or(taken);

    uint16_t* o = a.o + (row0 * a.H + h) * a.V + tile * VT + cg * 4;
    const int64_t o_step = (int64_t)a.H * a.V;
    if (!in_cache || taken) {
        if (first && (taken || slot >= a.num_slots)) report(a.status, kStatusBadSlots);
        for (int t = rl; t < len; t += kRowLanes) *reinterpret_cast<uint2*>(o + t * o_step) = make_uint2(0u, 0u);
        return;
    }

    for (int t0 = 0; t0 < len; t0 += kTokens) {
        if (t0 > 0) {
            __syncthreads();  // the tokens before have been read
            stage_tokens(t0);
            __syncthreads();
        }
        const int count = min(kTokens, len - t0), of = (tid >> 5) - kStepWarps / 2;
        if (of >= 0 && of < count) {  // k . q, read after the first token's barrier
            float kq = 0.f;
#pragma unroll
            for (int r = tid & 31; r < K; r += 32) kq += s_token[of].kqe[r].x * s_token[of].kqe[r].y;
            kq = warp_sum(kq);
            if (tid % 32 == 0) s_token[of].kq = kq;
        }
        if (t0 + kTokens < len) load_tokens(t0 + kTokens);
        for (int j = 0; j < count; ++j)
            step_token<K, VT, F16, kRows, kStepThreads>(S, s_token[j], s_sums[j & 1], a.scale, o + (t0 + j) * o_step, tid,
                                                        [] {
                                                            __syncthreads();
                                                            return true;
                                                        });
    }

#pragma unroll
    for (int i = 0; i < kRows; ++i) store_state<STATE16>(a.state, at + i * row_step, S[i]);
}

// ------------------------------------------------------------------ many sequences
// With states enough to fill the GPU the call is a stream through them, and the
// kernel above spends its time between a CTA's load, its sums and its store.
// Here CTAs are persistent: a warp loads whole states (K V elements are
// contiguous) into a ring in shared memory with bulk copies, groups of threads
// (two of 256, or four of 128 where V is 64, so that a thread has 16 rows for K =
// 128 and 8 for 64; three groups of 256 with half the rows measured 11% slower)
// take them in turn, and a warp stores them back from the ring, so loads, sums
// and stores of different states overlap on every SM.
//
// The tokens' inputs (k, q, g, v, beta) come through a small ring for each group,
// filled by one of two warps that have several tokens' loads in flight: one
// token's inputs are a kilobyte that nothing else has touched, and waiting for
// them token by token cost about 2 us each.  The units (a sequence and head)
// are published ahead of the loads so that it can run ahead.
constexpr int kComputeWarps = 16, kInputWarps = 2;
constexpr int kLoadWarp = kComputeWarps, kStoreWarp = kLoadWarp + 1, kFirstInputWarp = kLoadWarp + 2;
constexpr int kStreamThreads = (kFirstInputWarp + kInputWarps) * 32;
constexpr int kUnits = 60;  // published units kept
// Packed sequences are taken longest first, up to this many: the CTAs and groups
// take units in turn, so neighbours in that order share out evenly (96 sequences
// of 0 to 5 tokens in their own order: 31.8 us, the last group 1.7 times the
// mean; sorted: 30.1).  More sequences even out by their number.
constexpr int kMostSorted = 512;
// Tokens of a sequence (of all, where packed) that the streaming kernel takes: a
// few tenths of a second at most, well under what its waits allow.
constexpr int kMostStreamed = 1 << 16;
// Barriers of the loads, one per unit in turn, more of them than slots of the
// ring: copies land in any order, so a group can wait for its next unit while
// the other group's unit in the same slot is still on its way.  With a barrier
// per slot that wait would be two phases early, which its parity cannot tell
// from a phase that is over.  Units up to kRing + 2 before one that is waited
// for are done, so kFull barriers are never more than one phase behind.
constexpr int kFull = 16;
constexpr int kDepth = 3;   // tokens an input warp has in flight
// Units published before a load is waited for.  An input warp takes every second
// unit, and may look kDepth of them ahead of the one that holds the ring up.
constexpr int kAhead = kInputWarps * (kDepth + 1) + 2;

struct Unit {
    int64_t row0, state;           // first token row; first element of the state
    int len, head, qk_head, unused;  // tokens; < 0: no more units
};

template <int K, int V, bool STATE16>
struct StreamShape {
    static constexpr int kThreads = 2 * V;                       // of a group
    static constexpr int kWarps = kThreads / 32;
    static constexpr int kGroups = kComputeWarps / kWarps;
    static constexpr int kBytes = K * V * (STATE16 ? 2 : 4);
    static constexpr bool kLarge = kBytes > 32768;
    static constexpr int kRing = kLarge ? 3 : kBytes == 32768 ? 5 : 8;
    static constexpr int kSlots = kLarge ? 3 : 4;   // tokens in a group's input ring
    static constexpr int kSums = kLarge ? 1 : 2;    // exchange buffers: with one, a second barrier per token
    struct Group {
        Sums<V, kThreads> sums[kSums];
        Token<K, V> token[kSlots];
        uint64_t token_full[kSlots], token_empty[kSlots];
    };
    struct Shared {
        uint8_t ring[kRing][kBytes];
        Group group[kGroups];
        Unit unit[kUnits];
        uint16_t order[kMostSorted];
        uint64_t known[kUnits], full[kFull], done[kRing], empty[kRing];
    };
    static constexpr int kSmem = (int)sizeof(Shared) + 128;
    static_assert(kSmem <= 227 * 1024, "fits an SM");
    static_assert(kRing >= kGroups + 1 && kFull >= kRing + kGroups && kUnits >= kRing + kAhead + 32 + kGroups,
                  "barriers and published units outlive their use");
    static_assert(kGroups % kInputWarps == 0, "a group's tokens come from one warp");
};

// Named barrier of one group; true if `ok` holds for all its threads.
template <int THREADS>
__device__ __forceinline__ bool group_sync(int group, bool ok) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.and.pred q, %1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"(group + 1), "n"(THREADS), "r"((uint32_t)ok)
        : "memory");
    return all != 0;
}

// COUNT (2 or 4) consecutive 16-bit elements as they come from memory: two in a
// word where vec says that they are aligned together, else one.  Taken apart only
// when they are used: a load's first use is where its latency is waited for.
template <int COUNT>
struct Raw16 {
    uint32_t w[COUNT];
    __device__ __forceinline__ void load(const uint16_t* p, bool vec) {
        if (vec) {
            if constexpr (COUNT == 4) {
                const uint2 x = *reinterpret_cast<const uint2*>(p);
                w[0] = x.x, w[1] = x.y;
            } else {
                w[0] = *reinterpret_cast<const uint32_t*>(p);
            }
        } else {
#pragma unroll
            for (int i = 0; i < COUNT; ++i) w[i] = p[i];
        }
    }
    template <bool F16>
    __device__ __forceinline__ float at(int i, bool vec) const {
        return from_b16<F16>((uint16_t)(vec ? w[i / 2] >> (16 * (i & 1)) : w[i]));
    }
};
template <int COUNT>
__device__ __forceinline__ void load_f32(const float* p, bool vec, float (&w)[COUNT]) {
    if (vec) {
        if constexpr (COUNT == 4) {
            const float4 x = *reinterpret_cast<const float4*>(p);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        } else {
            const float2 x = *reinterpret_cast<const float2*>(p);
            w[0] = x.x, w[1] = x.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) w[i] = p[i];
    }
}

template <int K, int V, bool F16, bool STATE16>
__global__ void __launch_bounds__(kStreamThreads, 1) kda_step_stream_kernel(const StepArgs a) {
    using Shape = StreamShape<K, V, STATE16>;
    constexpr int kRing = Shape::kRing, kSlots = Shape::kSlots, kGroups = Shape::kGroups;
    constexpr int kThreads = Shape::kThreads, kWarps = Shape::kWarps;
    constexpr int kColGroups = V / 4;
    constexpr int kRowLanes = kThreads / kColGroups;
    constexpr int kRows = K / kRowLanes;
    extern __shared__ uint8_t raw[];
    auto& sm = *reinterpret_cast<typename Shape::Shared*>(raw + ((128u - (ptx::smem_u32(raw) & 127u)) & 127u));

    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
    if (tid < kUnits) ptx::mbar_init(&sm.known[tid], 1);
    if (tid < kFull) ptx::mbar_init(&sm.full[tid], 1);
    if (tid < kRing) {
        ptx::mbar_init(&sm.done[tid], kWarps);
        ptx::mbar_init(&sm.empty[tid], 1);
    }
    if (tid < kGroups * kSlots) {
        ptx::mbar_init(&sm.group[tid / kSlots].token_full[tid % kSlots], 1);
        ptx::mbar_init(&sm.group[tid / kSlots].token_empty[tid % kSlots], kWarps);
    }
    ptx::fence_mbar_init();
    ptx::grid_dep_launch();
    __syncthreads();
    ptx::grid_dep_wait();
    const bool sorted = a.cu && a.N <= kMostSorted;
    if (sorted) {
        // place of a sequence: those that are longer, and those as long before it
        uint8_t* len = sm.ring[0];  // (not in use yet; up to 255)
        const int n = tid;
        int mine = 0;
        if (n < kMostSorted) {
            if (n < a.N) {
                const int bos = a.cu[n], eos = a.cu[n + 1];
                mine = bad_offsets(a, n, bos, eos) ? 0 : min(eos - bos, 255);
            }
            len[n] = (uint8_t)mine;
        }
        __syncthreads();
        if (n < a.N) {
            int place = 0;
            const uint32_t all = (uint32_t)mine * 0x01010101u;
            for (int j = 0; j < a.N; j += 4) {
                const uint32_t four = *reinterpret_cast<const uint32_t*>(len + j);
                uint32_t ahead = __vcmpgtu4(four, all);
                if (j < n) ahead |= __vcmpeq4(four, all) & (n - j >= 4 ? ~0u : (1u << (8 * (n - j))) - 1u);
                place += __popc(ahead) >> 3;
            }
            sm.order[place] = (uint16_t)n;
        }
        ptx::fence_proxy_async_smem();  // (copies write there next)
        __syncthreads();
    }

    if (warp == kLoadWarp) {
        const int total = a.N * a.H;
        int u = blockIdx.x, published = 0, issued = 0, batch = kAhead + 1;
        bool end = false, ok = true;
        while (ok) {
            if (!end && published <= issued + kAhead) {
                // A batch of units, one per lane, so that their offsets and slots, and the
                // look through the earlier sequences' slots, are waited for once.  (The
                // first batch is small: the first loads wait for it.)
                const int64_t mine = u + (int64_t)lane * gridDim.x;
                const bool here = lane < batch && mine < total;
                const int at = here ? (int)mine / a.H : 0, h = here ? (int)mine - at * a.H : 0;
                const int n = sorted ? sm.order[at] : at;
                Unit unit{(int64_t)n * a.T, 0, here ? a.T : 0, h, h / a.group, 0};
                if (here && a.cu) {
                    const int bos = a.cu[n], eos = a.cu[n + 1];
                    const bool bad = bad_offsets(a, n, bos, eos);
                    if (bad && h == 0) report(a.status, kStatusBadSeqlens);
                    unit.row0 = bos;
                    unit.len = bad ? 0 : eos - bos;
                }
                const int slot = here && a.slots ? a.slots[n] : n;
                bool taken = false;
                if (a.slots) {
                    // 128 earlier slots at a time, handed round by shuffles: one after the
                    // other they are loads to wait for, while no state is asked for
                    const int most = __reduce_max_sync(~0u, here ? n : 0);
                    for (int j0 = 0; j0 < most; j0 += 128) {
                        int others[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) others[i] = j0 + 32 * i + lane < most ? a.slots[j0 + 32 * i + lane] : -1;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (j0 + 32 * i >= most) break;
#pragma unroll 8
                            for (int l = 0; l < 32; ++l)
                                taken |= __shfl_sync(~0u, others[i], l) == slot && j0 + 32 * i + l < n;
                        }
                    }
                }
                const bool refused = unit.len > 0 && (slot < 0 || slot >= a.num_slots || taken);
                if (refused) {
                    if (h == 0 && slot >= 0) report(a.status, kStatusBadSlots);
                    uint16_t* o = a.o + (unit.row0 * a.H + h) * V;
                    for (int t = 0; t < unit.len; ++t, o += (int64_t)a.H * V)
                        for (int c = 0; c < V; c += 8) *reinterpret_cast<uint4*>(o + c) = make_uint4(0u, 0u, 0u, 0u);
                }
                unit.state = ((int64_t)slot * a.H + h) * (K * V);
                const uint32_t live = __ballot_sync(~0u, unit.len > 0 && !refused);
                if ((live >> lane) & 1u) {
                    const int i = (published + __popc(live & ((1u << lane) - 1u))) % kUnits;
                    sm.unit[i] = unit;
                    ptx::mbar_arrive(&sm.known[i]);
                }
                published += __popc(live);
                u = (int)min((int64_t)total, u + (int64_t)batch * gridDim.x);
                batch = 32;
                if (u >= total) {
                    end = true;
                    if (lane < kGroups) {  // the end, once for each group
                        const int i = (published + lane) % kUnits;
                        sm.unit[i].len = -1;
                        ptx::mbar_arrive(&sm.known[i]);
                    }
                }
                __syncwarp();
            } else if (issued < published) {
                const int s = issued % kRing, round = issued / kRing;
                if (round > 0) ok = __all_sync(~0u, wait_for(&sm.empty[s], (round - 1) & 1));
                if (!ok) break;
                if (elect_one()) {
                    uint64_t* full = &sm.full[issued % kFull];
                    ptx::mbar_arrive_expect_tx(full, Shape::kBytes);
                    bulk_load(sm.ring[s],
                              static_cast<const uint8_t*>(a.state) + sm.unit[issued % kUnits].state * (STATE16 ? 2 : 4),
                              Shape::kBytes, full);
                }
                __syncwarp();
                ++issued;
            } else {
                break;
            }
        }
        if (!ok && lane == 0) report(a.status, kStatusTimeout);
        for (int i = max(0, issued - kRing); i < issued; ++i) wait_for(&sm.full[i % kFull], (i / kFull) & 1);
    } else if (warp == kStoreWarp) {
        if (elect_one()) {
            for (int i = 0;; ++i) {
                const int s = i % kRing;
                if (!wait_for(&sm.known[i % kUnits], (i / kUnits) & 1)) break;
                const Unit unit = sm.unit[i % kUnits];
                if (unit.len < 0 || !wait_for(&sm.done[s], (i / kRing) & 1)) break;
                bulk_store(static_cast<uint8_t*>(a.state) + unit.state * (STATE16 ? 2 : 4), sm.ring[s],
                           Shape::kBytes);
                ptx::bulk_commit();
                ptx::bulk_wait_read0();
                ptx::mbar_arrive(&sm.empty[s]);
            }
            ptx::bulk_wait0();
        }
    } else if (warp >= kFirstInputWarp) {
        constexpr int kk = K / 32, vv = V / 32;  // elements of a lane
        Raw16<kk> rk[kDepth], rq[kDepth];
        Raw16<vv> rv[kDepth];
        uint16_t rb[kDepth];
        float rg[kDepth][kk];
        bool has[kDepth];
        int i = warp - kFirstInputWarp, t = 0;  // the next token to ask for
        int to_group[kDepth], sent[kGroups / kInputWarps] = {};  // tokens sent to each of its groups
        bool ok = __all_sync(~0u, wait_for(&sm.known[i], 0));
        Unit unit = sm.unit[i];
        const uint16_t *pk = nullptr, *pq = nullptr, *pv = nullptr, *pb = nullptr;  // this lane's part of the next token
        const float* pg = nullptr;
        // Where a unit's five inputs start: one lane computes each, and hands it round.
        const int64_t my_stride = lane == 0 ? a.k_stride : lane == 1 ? a.q_stride : lane == 2 ? a.g_stride
                                                       : lane == 3 ? a.v_stride : a.beta_stride;
        const int my_dim = lane < 3 ? K : lane == 3 ? V : 1;
        auto open = [&] {
            const int64_t at = unit.row0 * my_stride + (int64_t)(lane < 2 ? unit.qk_head : unit.head) * my_dim;
            pk = a.k + __shfl_sync(~0u, at, 0) + lane * kk;
            pq = a.q + __shfl_sync(~0u, at, 1) + lane * kk;
            pg = a.g + __shfl_sync(~0u, at, 2) + lane * kk;
            pv = a.v + __shfl_sync(~0u, at, 3) + lane * vv;
            pb = a.beta + __shfl_sync(~0u, at, 4);
        };
        open();
        auto ask = [&](int d) {
            has[d] = ok && unit.len > 0;
            if (!has[d]) return;
            to_group[d] = i % kGroups;
            rk[d].load(pk, a.vec);
            rq[d].load(pq, a.vec);
            load_f32<kk>(pg, a.vec, rg[d]);
            rv[d].load(pv, a.vec);
            rb[d] = *pb;
            pk += a.k_stride;
            pq += a.q_stride;
            pg += a.g_stride;
            pv += a.v_stride;
            pb += a.beta_stride;
            if (++t == unit.len) {
                t = 0;
                i += kInputWarps;
                ok = __all_sync(~0u, wait_for(&sm.known[i % kUnits], (i / kUnits) & 1));
                unit = sm.unit[i % kUnits];
                open();
            }
        };
#pragma unroll
        for (int d = 0; d < kDepth; ++d) ask(d);
        bool more = true;
        while (more) {
#pragma unroll
            for (int d = 0; d < kDepth; ++d) {
                more = more && has[d];
                if (!more) break;
                auto& gr = sm.group[to_group[d]];
                int c = 0;  // the token's number in its group (the array stays in registers)
#pragma unroll
                for (int x = 0; x < kGroups / kInputWarps; ++x)
                    if (to_group[d] / kInputWarps == x) c = sent[x]++;
                const int s = c % kSlots, round = c / kSlots;
                if (round > 0 && !__all_sync(~0u, wait_for(&gr.token_empty[s], (round - 1) & 1))) {
                    more = false;
                    break;
                }
                auto& to = gr.token[s];
                float kq = 0.f;
#pragma unroll
                for (int x = 0; x < kk; ++x) {
                    const float fk = rk[d].template at<F16>(x, a.vec), fq = rq[d].template at<F16>(x, a.vec);
                    to.kqe[lane * kk + x] = make_float4(fk, fq, expf(rg[d][x]), 0.f);
                    kq = fmaf(fk, fq, kq);
                }
                kq = warp_sum(kq);
#pragma unroll
                for (int x = 0; x < vv; ++x) to.v[lane * vv + x] = rv[d].template at<F16>(x, a.vec);
                if (lane == 0) {
                    const float x = from_b16<F16>(rb[d]);
                    to.beta = a.logits ? 1.f / (1.f + expf(-x)) : x;
                    to.kq = kq;
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&gr.token_full[s]);  // (32 arrivals would queue up at the barrier)
                ask(d);
            }
        }
    } else {
        const int group = warp / kWarps, gt = tid - group * kThreads;
        const int cg = gt % kColGroups, rl = gt / kColGroups;
        auto& gr = sm.group[group];
        bool ok = true;
        int c = 0;  // tokens done
        for (int i = group;; i += kGroups) {
            ok = wait_for(&sm.known[i % kUnits], (i / kUnits) & 1);
            const Unit unit = sm.unit[i % kUnits];
            if (ok && unit.len < 0) {  // (a thread that gave up waits for the others once)
                ok = group_sync<kThreads>(group, true);
                break;
            }
            const int s = i % kRing;
            void* tile = sm.ring[s];
            ok = ok && wait_for(&sm.full[i % kFull], (i / kFull) & 1);
            float4 S[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) S[r] = load_state<STATE16>(tile, (rl + r * kRowLanes) * kColGroups + cg);
            uint16_t* o = a.o + (unit.row0 * a.H + unit.head) * V + cg * 4;
            int t = 0;
            do {  // (once with ok false, to give up together)
                const int ts = c % kSlots, b = c % Shape::kSums;
                ok = ok && wait_for(&gr.token_full[ts], (c / kSlots) & 1);
                // with one exchange buffer: the sums before have been read
                if (Shape::kSums == 1 && c > 0 && !(ok = group_sync<kThreads>(group, ok))) break;
                ok = step_token<K, V, F16, kRows, kThreads>(S, gr.token[ts], gr.sums[b], a.scale, o, gt,
                                                            [&] { return group_sync<kThreads>(group, ok); });
                if (!ok) break;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&gr.token_empty[ts]);
                ++c;
                o += (int64_t)a.H * V;
            } while (++t < unit.len);
            if (!ok) break;
#pragma unroll
            for (int r = 0; r < kRows; ++r) store_state<STATE16>(tile, (rl + r * kRowLanes) * kColGroups + cg, S[r]);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&sm.done[s]);
        }
        if (!ok && gt == 0) report(a.status, kStatusTimeout);
    }
}

template <int K, int V, bool F16, bool STATE16>
cudaError_t launch_stream(const StepArgs& a, int sms, cudaStream_t s) {
    auto kern = kda_step_stream_kernel<K, V, F16, STATE16>;
    constexpr int kSmem = StreamShape<K, V, STATE16>::kSmem;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3((unsigned)min((int64_t)sms, (int64_t)a.N * a.H)), dim3(kStreamThreads), kSmem, s,
                            a);
}

template <int K, int V>
cudaError_t launch_stream(const StepArgs& a, bool f16, bool state16, int sms, cudaStream_t s) {
    if (f16) return state16 ? launch_stream<K, V, true, true>(a, sms, s) : launch_stream<K, V, true, false>(a, sms, s);
    return state16 ? launch_stream<K, V, false, true>(a, sms, s) : launch_stream<K, V, false, false>(a, sms, s);
}

template <int K, int VT, int PER_SM>
cudaError_t launch(const StepArgs& a, bool f16, bool state16, unsigned grid, cudaStream_t s) {
    auto kern = f16 ? (state16 ? kda_step_kernel<K, VT, true, true, PER_SM> : kda_step_kernel<K, VT, true, false, PER_SM>)
                    : (state16 ? kda_step_kernel<K, VT, false, true, PER_SM> : kda_step_kernel<K, VT, false, false, PER_SM>);
    return launch_dependent(kern, dim3(grid), dim3(kStepThreads), 0, s, a);
}

// Calls whose CTAs have an SM each get all its registers where K = 128 (140 a thread
// instead of 128): 32 pairs with V = 128 2.9 us, for 3.4 with room for two; with more
// CTAs than SMs 128 pairs take 5.5 us, for 4.3.  K = 64 uses 126 either way (3.2 us for
// 256 pairs; 3.8 with the 80 that the compiler takes unasked).
template <int K, int VT>
cudaError_t launch(const StepArgs& a, bool f16, bool state16, int sms, cudaStream_t s) {
    const unsigned grid = (unsigned)((int64_t)a.N * a.H * (a.V / VT));
    if constexpr (K == 128)
        if (grid <= (unsigned)sms) return launch<K, VT, 1>(a, f16, state16, grid, s);
    return launch<K, VT, 2>(a, f16, state16, grid, s);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_step(const void* q, const void* k, const void* v, const float* g, const void* beta,
                               float scale, void* state, const int32_t* slots, const int32_t* cu_seqlens, void* o,
                               const kda_dims* dims, const kda_step_opts* opts, int32_t* status_word, void* stream) {
    if (!dims || !opts) return KDA_ERR_INVALID_ARG;
    const kda_dims& d = *dims;
    const bool packed = cu_seqlens != nullptr;
    if (packed != (d.num_seqs > 0) || d.num_seqs < 0 || d.B < 1 || d.T < 0 || d.H < 1 || (packed && d.B != 1))
        return KDA_ERR_INVALID_ARG;
    if ((d.K != 64 && d.K != 128) || (d.V != 64 && d.V != 128)) return KDA_ERR_UNSUPPORTED;
    const kda_step_opts& p = *opts;
    if ((p.io_dtype != KDA_IO_BF16 && p.io_dtype != KDA_IO_F16) ||
        (p.state_dtype != KDA_STATE_F32 && p.state_dtype != KDA_STATE_BF16) ||
        (p.beta_logits != 0 && p.beta_logits != 1) || p.reserved != 0 || p.num_slots < 1 || p.qk_heads < 0 ||
        (p.qk_heads > 0 && (p.qk_heads > d.H || d.H % p.qk_heads != 0)))
        return KDA_ERR_INVALID_ARG;
    const int N = packed ? d.num_seqs : d.B;
    if (!slots && N > p.num_slots) return KDA_ERR_INVALID_ARG;
    const int64_t rows = (int64_t)d.B * d.T;
    if (rows > INT32_MAX / 2 || (int64_t)N * d.H * (d.V / 32) > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    const int hq = p.qk_heads > 0 ? p.qk_heads : d.H;
    const int64_t wq = (int64_t)hq * d.K, wv = (int64_t)d.H * d.V, wg = (int64_t)d.H * d.K;
    StepArgs a{};
    a.q_stride = p.q_stride ? p.q_stride : wq;
    a.k_stride = p.k_stride ? p.k_stride : wq;
    a.v_stride = p.v_stride ? p.v_stride : wv;
    a.g_stride = p.g_stride ? p.g_stride : wg;
    a.beta_stride = p.beta_stride ? p.beta_stride : d.H;
    if (a.q_stride < wq || a.k_stride < wq || a.v_stride < wv || a.g_stride < wg || a.beta_stride < d.H)
        return KDA_ERR_INVALID_ARG;
    if ((slots && !is_aligned(slots, 4)) || (packed && !is_aligned(cu_seqlens, 4)) ||
        (status_word && !is_aligned(status_word, 4)))
        return KDA_ERR_ALIGNMENT;
    if (rows > 0) {
        if (!q || !k || !v || !g || !beta || !state || !o) return KDA_ERR_INVALID_ARG;
        if (!is_aligned(q, 2) || !is_aligned(k, 2) || !is_aligned(v, 2) || !is_aligned(beta, 2) ||
            !is_aligned(g, 4) || !is_aligned(o, 16) || !is_aligned(state, 16))
            return KDA_ERR_ALIGNMENT;
    }
    if (!packed && rows == 0) return KDA_OK;
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.beta = static_cast<const uint16_t*>(beta);
    a.g = g;
    a.state = state;
    a.slots = slots;
    a.cu = cu_seqlens;
    a.o = static_cast<uint16_t*>(o);
    a.status = status_word;
    a.scale = scale;
    a.N = N;
    a.T = d.T;
    a.H = d.H;
    a.V = d.V;
    a.group = d.H / hq;
    a.num_slots = p.num_slots;
    a.logits = p.beta_logits;
    a.vec = is_aligned(q, 8) && is_aligned(k, 8) && is_aligned(v, 8) && is_aligned(g, 16) && a.q_stride % 4 == 0 &&
            a.k_stride % 4 == 0 && a.v_stride % 4 == 0 && a.g_stride % 4 == 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f16 = p.io_dtype == KDA_IO_F16, s16 = p.state_dtype == KDA_STATE_BF16;
    const int sms = device_sm_count();
    cudaError_t e;
    // (Tokens of one sequence follow one another: its waits must not run out over a very long one.)
    if ((int64_t)N * d.H >= 2 * sms && d.T <= kMostStreamed) {
        if (d.K == 128)
            e = d.V == 128 ? launch_stream<128, 128>(a, f16, s16, sms, s) : launch_stream<128, 64>(a, f16, s16, sms, s);
        else
            e = d.V == 128 ? launch_stream<64, 128>(a, f16, s16, sms, s) : launch_stream<64, 64>(a, f16, s16, sms, s);
    } else {
        e = d.K == 128 ? launch<128, 64>(a, f16, s16, sms, s) : launch<64, 64>(a, f16, s16, sms, s);
    }
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
