// decay_step.cu -- kda_decay_step: linear attention with a decay per head for the
// few new tokens of a decode step, on a cache of states addressed by slot and
// updated in place:  S <- exp(g) S + k v^T,  o = scale S^T q.
//
// Unlike the delta rule's, a token's update does not depend on what the state
// answers, so the tokens of a batch follow one another in registers and only
// their outputs, which sum over the rows that the threads share, meet in shared memory.
//
// Bound: each state is read and written once per call, 2 K V 4 bytes (128 KB at
// K = V = 128 in fp32) against 5 K V flops a token: HBM, or for a handful of states the
// launch and one trip to memory. Few threads with many columns each spend the least on a token's
// shared loads and sums over rows, so five CTAs (K = 64: eight) of 128 threads an SM, in different stages of
// load, sums and store, keep HBM busy without a ring, and sums are taken two floats at a time: 512 requests x
// 32 heads of 128 x 128 in fp32 307 us (7 TB/s; a copy reaches 6.7), 96 x 3 tokens x 32 heads of 128 x 64 in
// bf16 25.6, of 64 x 64 15.5. One float at a time in 256 threads, four an SM, 315, 32.9 and 20.4;
// columns by 32 in 128 threads, eight an SM, 310, 28.5 and 18 to 20; 128 columns 388.
#include "decay.cuh"

namespace kda {
namespace {

constexpr int kStepTokens = 8;  // tokens whose inputs are loaded together

struct DecayStepArgs {
    const uint16_t *q, *k, *v;
    const float* g;
    void* state;
    const int32_t* slots;  // or null
    const int32_t* cu;     // or null
    uint16_t* o;
    int32_t* status;       // or null
    int64_t q_stride, k_stride, v_stride, g_stride;
    float scale;
    int32_t N, T, H, V, group, num_slots;
    int32_t vec;  // rows of q, k and v take loads of four elements
};

// Four columns of a state as two pairs of floats.
template <bool STATE16>
__device__ __forceinline__ void load_four(const void* p, int64_t four, uint64_t (&s)[2]) {
    if constexpr (STATE16) {
        const uint2 w = static_cast<const uint2*>(p)[four];
        const float2 a = from_b16x2<false>(w.x), b = from_b16x2<false>(w.y);
        s[0] = pair_of(a.x, a.y);
        s[1] = pair_of(b.x, b.y);
    } else {
        const ulonglong2 w = static_cast<const ulonglong2*>(p)[four];
        s[0] = w.x;
        s[1] = w.y;
    }
}
template <bool STATE16>
__device__ __forceinline__ void store_four(void* p, int64_t four, const uint64_t (&s)[2]) {
    if constexpr (STATE16) {
        const float2 a = floats_of(s[0]), b = floats_of(s[1]);
        static_cast<uint2*>(p)[four] = make_uint2(pack_b16x2(a.x, a.y, false), pack_b16x2(b.x, b.y, false));
    } else {
        static_cast<ulonglong2*>(p)[four] = make_ulonglong2(s[0], s[1]);
    }
}

// Four 16-bit elements; vec: together.
template <bool F16>
__device__ __forceinline__ float4 load_inputs(const uint16_t* p, bool vec) {
    if (vec) {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
        const float2 x = from_b16x2<F16>(w.x), y = from_b16x2<F16>(w.y);
        return make_float4(x.x, x.y, y.x, y.y);
    }
    return make_float4(from_b16<F16>(p[0]), from_b16<F16>(p[1]), from_b16<F16>(p[2]), from_b16<F16>(p[3]));
}

// One CTA has VT columns of one (sequence, head): THREADS threads, each kRows rows of four columns.
template <int K, int VT, int THREADS, bool F16, bool STATE16, int PER_SM>
__global__ void __launch_bounds__(THREADS, PER_SM) kda_decay_step_kernel(const DecayStepArgs a) {
    constexpr int kColGroups = VT / 4, kRowLanes = THREADS / kColGroups, kRows = K / kRowLanes;
    constexpr int kWarps = THREADS / 32, kParts = kColGroups >= 32 ? kRowLanes : kWarps;
    static_assert(kRows >= 1 && kRows * kRowLanes == K, "the threads tile the K rows");
    __shared__ __align__(16) float s_k[kStepTokens][K], s_q[kStepTokens][K];
    __shared__ float4 s_v[kStepTokens][kColGroups];
    __shared__ float s_decay[kStepTokens];
    __shared__ __align__(16) int s_bad[kWarps];  // packed: whether a warp has found offsets out of order
    __shared__ float4 s_o[kStepTokens][kParts][kColGroups];

    const int tid = threadIdx.x;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int tiles = a.V / VT;
    const int tile = blockIdx.x % tiles, h = (blockIdx.x / tiles) % a.H, n = blockIdx.x / tiles / a.H;
    const bool first = tile == 0 && h == 0 && tid == 0;

    int64_t row0 = (int64_t)n * a.T;
    int len = a.T;
    const int slot = a.slots ? a.slots[n] : n;  // (asked for together with the bounds)
    if (a.cu) {
        const int bos = a.cu[n], eos = a.cu[n + 1];
        if (out_of_order(bos, eos, n, a.N, a.T)) {
            if (first && a.status) atomicOr(a.status, kStatusBadSeqlens);
            return;
        }
        row0 = bos;
        len = eos - bos;
        if (len == 0) return;
        // Others out of order may have the same rows (0, 3, 1, 4 gives two sequences rows 1 and 2): with any that are nothing is
        // done. Every CTA looks for itself: 96 sequences of 32 heads of 128 x 64 take 35.3 us, by their own offsets alone
        // 34.3; 2048 of 2 heads of 64 x 64 20.8 and 17.5. (What was found waits in shared memory, registers being short; a
        // barrier of its own 35.6 and 21.5; offsets asked for ahead of the own ones 35.2 and 21.7, by fours 38 and 26.)
        bool bad = (a.cu[0] != 0) | (a.cu[a.N] != a.T);
#pragma unroll 4
        for (int j = tid; j < a.N; j += THREADS) bad |= a.cu[j + 1] < a.cu[j];
        bad = __any_sync(~0u, bad);
        if ((tid & 31) == 0) s_bad[tid >> 5] = bad;
    }
    if (len == 0) return;
    const bool in_cache = slot >= 0 && slot < a.num_slots;

    const int cg = tid % kColGroups, rl = tid / kColGroups;
    const int64_t at = in_cache ? ((((int64_t)slot * a.H + h) * K + rl) * a.V + tile * VT) / 4 + cg : 0;
    const int64_t row_step = (int64_t)kRowLanes * a.V / 4;
    uint64_t S[kRows][2];  // two floats each
    if (in_cache) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) load_four<STATE16>(a.state, at + i * row_step, S[i]);
    }
    const int hq = h / a.group;
    // Inputs of kStepTokens tokens, four elements a thread where rows allow it: one trip to memory.
    auto stage = [&](int t0) {
        constexpr int kEach = K / 4, kEachV = VT / 4;
#pragma unroll
        for (int e0 = 0; e0 < kStepTokens * kEach; e0 += THREADS) {
            const int j = (e0 + tid) / kEach, r = (e0 + tid) % kEach * 4;
            if (j < kStepTokens && t0 + j < len) {
                const int64_t row = row0 + t0 + j;
                const uint16_t* k = a.k + row * a.k_stride + (int64_t)hq * K + r;
                const uint16_t* q = a.q + row * a.q_stride + (int64_t)hq * K + r;
                *reinterpret_cast<float4*>(&s_k[j][r]) = load_inputs<F16>(k, a.vec);
                *reinterpret_cast<float4*>(&s_q[j][r]) = load_inputs<F16>(q, a.vec);
            }
        }
#pragma unroll
        for (int e0 = 0; e0 < kStepTokens * kEachV; e0 += THREADS) {
            const int j = (e0 + tid) / kEachV, c = (e0 + tid) % kEachV;
            if (j < kStepTokens && t0 + j < len)
                s_v[j][c] = load_inputs<F16>(a.v + (row0 + t0 + j) * a.v_stride + (int64_t)h * a.V + tile * VT + c * 4, a.vec);
        }
        if (tid < kStepTokens && t0 + tid < len) s_decay[tid] = expf(a.g[(row0 + t0 + tid) * a.g_stride + h]);
    };
    // The same slot twice would race: the first sequence that names it has it.
    bool taken = false;
    if (in_cache && a.slots)
        for (int j = tid; j < n; j += THREADS) taken |= a.slots[j] == slot;
    stage(0);
    taken = __syncthreads_or(taken);
    if (a.cu) {
        bool bad = false;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) bad |= s_bad[w] != 0;
        if (bad) return;
    }

    uint16_t* o = a.o + (row0 * a.H + h) * a.V + tile * VT;
    const int64_t o_step = (int64_t)a.H * a.V;
    if (!in_cache || taken) {
        if (first && (taken || slot >= a.num_slots) && a.status) atomicOr(a.status, kStatusBadSlots);
        for (int t = rl; t < len; t += kRowLanes) *reinterpret_cast<uint2*>(o + t * o_step + cg * 4) = make_uint2(0u, 0u);
        return;
    }
    for (int t0 = 0; t0 < len; t0 += kStepTokens) {
        if (t0 > 0) {
            __syncthreads();  // the tokens before, and their sums, have been read
            stage(t0);
            __syncthreads();
        }
        const int count = min(kStepTokens, len - t0);
        for (int j = 0; j < count; ++j) {
            const uint64_t d = pair_of(s_decay[j], s_decay[j]);
            const float4 v = s_v[j][cg];
            const uint64_t v01 = pair_of(v.x, v.y), v23 = pair_of(v.z, v.w);
            uint64_t y01 = 0, y23 = 0;
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const uint64_t k = pair_of(s_k[j][rl + i * kRowLanes], s_k[j][rl + i * kRowLanes]);
                const uint64_t q = pair_of(s_q[j][rl + i * kRowLanes], s_q[j][rl + i * kRowLanes]);
                S[i][0] = fma2(d, S[i][0], mul2(k, v01));
                S[i][1] = fma2(d, S[i][1], mul2(k, v23));
                y01 = fma2(q, S[i][0], y01);
                y23 = fma2(q, S[i][1], y23);
            }
            const float2 ya = floats_of(y01), yb = floats_of(y23);
            float4 y = make_float4(ya.x, ya.y, yb.x, yb.y);
#pragma unroll
            for (int off = kColGroups; off < 32; off <<= 1) {  // row lanes of the same columns in this warp
                y.x += __shfl_xor_sync(~0u, y.x, off);
                y.y += __shfl_xor_sync(~0u, y.y, off);
                y.z += __shfl_xor_sync(~0u, y.z, off);
                y.w += __shfl_xor_sync(~0u, y.w, off);
            }
            if (kColGroups >= 32) s_o[j][rl][cg] = y;
            else if ((tid & 31) < kColGroups) s_o[j][tid >> 5][cg] = y;
        }
        if (t0 + count >= len) {  // (the stores leave while the outputs are summed)
#pragma unroll
            for (int i = 0; i < kRows; ++i) store_four<STATE16>(a.state, at + i * row_step, S[i]);
        }
        __syncthreads();
        for (int e = tid; e < count * kColGroups; e += THREADS) {
            const int j = e / kColGroups, c = e % kColGroups;
            float4 y = s_o[j][0][c];
#pragma unroll
            for (int w = 1; w < kParts; ++w) {
                const float4 x = s_o[j][w][c];
                y = make_float4(y.x + x.x, y.y + x.y, y.z + x.z, y.w + x.w);
            }
            *reinterpret_cast<uint2*>(o + (t0 + j) * o_step + c * 4) =
                make_uint2(pack_b16x2(a.scale * y.x, a.scale * y.y, F16), pack_b16x2(a.scale * y.z, a.scale * y.w, F16));
        }
    }
}

template <int K, int VT, int THREADS, int PER_SM>
cudaError_t launch(const DecayStepArgs& a, bool f16, bool s16, cudaStream_t s) {
    const dim3 grid((unsigned)((int64_t)a.N * a.H * (a.V / VT)));
    if (f16)
        return s16 ? launch_dependent(kda_decay_step_kernel<K, VT, THREADS, true, true, PER_SM>, grid, dim3(THREADS), 0, s, a)
                   : launch_dependent(kda_decay_step_kernel<K, VT, THREADS, true, false, PER_SM>, grid, dim3(THREADS), 0, s, a);
    return s16 ? launch_dependent(kda_decay_step_kernel<K, VT, THREADS, false, true, PER_SM>, grid, dim3(THREADS), 0, s, a)
               : launch_dependent(kda_decay_step_kernel<K, VT, THREADS, false, false, PER_SM>, grid, dim3(THREADS), 0, s, a);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_decay_step(const void* q, const void* k, const void* v, const float* g, float scale,
                                     void* state, const int32_t* slots, const int32_t* cu_seqlens, void* o,
                                     const kda_dims* dims, const kda_decay_opts* opts, int32_t* status_word,
                                     void* stream) {
    if (!dims || !opts) return KDA_ERR_INVALID_ARG;
    const kda_dims& d = *dims;
    const bool packed = cu_seqlens != nullptr;
    if (packed != (d.num_seqs > 0) || d.num_seqs < 0 || d.B < 1 || d.T < 0 || d.H < 1 || (packed && d.B != 1))
        return KDA_ERR_INVALID_ARG;
    if ((d.K != 64 && d.K != 128) || (d.V != 64 && d.V != 128)) return KDA_ERR_UNSUPPORTED;
    const kda_decay_opts& p = *opts;
    if ((p.io_dtype != KDA_IO_BF16 && p.io_dtype != KDA_IO_F16) ||
        (p.state_dtype != KDA_STATE_F32 && p.state_dtype != KDA_STATE_BF16) || (p.head_gate != 0 && p.head_gate != 1) ||
        p.reserved != 0 || p.num_slots < 1 || p.do_stride != 0 || p.qk_heads < 0 ||
        (p.qk_heads > 0 && (p.qk_heads > d.H || d.H % p.qk_heads != 0)))
        return KDA_ERR_INVALID_ARG;
    const int N = packed ? d.num_seqs : d.B;
    if (!slots && N > p.num_slots) return KDA_ERR_INVALID_ARG;
    const int64_t rows = (int64_t)d.B * d.T;
    if (rows > INT32_MAX / 2 || (int64_t)N * d.H * (d.V / 32) > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    const int hq = p.qk_heads > 0 ? p.qk_heads : d.H;
    const int64_t wq = (int64_t)hq * d.K, wv = (int64_t)d.H * d.V;
    DecayStepArgs a{};
    a.q_stride = p.q_stride ? p.q_stride : wq;
    a.k_stride = p.k_stride ? p.k_stride : wq;
    a.v_stride = p.v_stride ? p.v_stride : wv;
    a.g_stride = p.head_gate ? 0 : p.g_stride ? p.g_stride : d.H;
    if (a.q_stride < wq || a.k_stride < wq || a.v_stride < wv || (p.head_gate ? p.g_stride != 0 : a.g_stride < d.H))
        return KDA_ERR_INVALID_ARG;
    if ((slots && !is_aligned(slots, 4)) || (packed && !is_aligned(cu_seqlens, 4)) ||
        (status_word && !is_aligned(status_word, 4)))
        return KDA_ERR_ALIGNMENT;
    if (rows == 0 && !packed) return KDA_OK;
    if (rows > 0) {
        if (!q || !k || !v || !g || !state || !o) return KDA_ERR_INVALID_ARG;
        if (!is_aligned(q, 2) || !is_aligned(k, 2) || !is_aligned(v, 2) || !is_aligned(g, 4) || !is_aligned(o, 16) ||
            !is_aligned(state, 16))
            return KDA_ERR_ALIGNMENT;
    }
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
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
    a.vec = is_aligned(q, 8) && is_aligned(k, 8) && is_aligned(v, 8) && a.q_stride % 4 == 0 && a.k_stride % 4 == 0 &&
            a.v_stride % 4 == 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f16 = p.io_dtype == KDA_IO_F16, s16 = p.state_dtype == KDA_STATE_BF16;
    const cudaError_t e = d.K == 128 ? launch<128, 64, 128, 5>(a, f16, s16, s) : launch<64, 64, 128, 8>(a, f16, s16, s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
