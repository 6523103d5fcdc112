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
// K = V = 128 in fp32) against ~7 K V flops, so HBM.  One CTA takes VT columns
// of one (sequence, head): the columns are independent given q, k, g, beta.  It
// holds its K x VT part in registers as float4 (a warp's load covers whole
// 128-byte lines), in fp32 whatever the cache's type, across all the tokens.
#include "layer_ops.cuh"

namespace kda {
namespace {

constexpr int kStepThreads = 256;

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
};

__device__ __forceinline__ void report(int32_t* status, int bit) {
    if (status) atomicOr(status, bit);
}

template <int K, int VT, bool F16, bool STATE16>
__global__ void __launch_bounds__(kStepThreads) kda_step_kernel(const StepArgs a) {
    constexpr int kColGroups = VT / 4;                      // threads across a row, 4 columns each
    constexpr int kRowLanes = kStepThreads / kColGroups;    // rows in flight per step of i
    constexpr int kRows = K / kRowLanes;                    // rows a thread holds
    constexpr int kWarps = kStepThreads / 32;
    static_assert(kRows >= 1 && kRows * kRowLanes == K, "the threads tile the K rows");
    __shared__ float4 s_kqe[2][K];   // per row: k, q, exp(g)
    __shared__ float s_v[2][VT];
    __shared__ float s_beta[2];
    __shared__ float4 s_sum[2][kWarps][kColGroups];  // per warp: S^T k, S^T q
    __shared__ float s_kq[kWarps];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tiles = a.V / VT;
    const int tile = blockIdx.x % tiles;
    const int h = (blockIdx.x / tiles) % a.H;
    const int n = blockIdx.x / tiles / a.H;
    const bool first = tile == 0 && h == 0 && tid == 0;

    int64_t row0 = (int64_t)n * a.T;
    int len = a.T;
    if (a.cu) {
        const int bos = a.cu[n], eos = a.cu[n + 1];
        const bool bad = bos < 0 || eos < bos || eos > a.T || (n == 0 && bos != 0) || (n == a.N - 1 && eos != a.T);
        if (bad) {
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
    const int64_t at = in_cache ? (((int64_t)slot * a.H + h) * K + rl) * a.V + tile * VT + cg * 4 : 0;
    float4 S[kRows];
    if (in_cache) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t off = at + (int64_t)i * kRowLanes * a.V;
            if constexpr (STATE16) {
                const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.state) + off);
                const float2 lo = from_b16x2<false>(w.x), hi = from_b16x2<false>(w.y);
                S[i] = make_float4(lo.x, lo.y, hi.x, hi.y);
            } else {
                S[i] = *reinterpret_cast<const float4*>(static_cast<const float*>(a.state) + off);
            }
        }
    }

    // A token's inputs: k and g rows by the first K threads, q by the next 128,
    // v by the first VT; loaded one token ahead of their use.
    const int hq = h / a.group;
    const int kr = tid & 127;
    float in_k = 0.f, in_g = 0.f, in_q = 0.f, in_v = 0.f, in_b = 0.f;
    auto load_token = [&](int64_t row) {
        if (tid < K) {
            in_k = from_b16<F16>(a.k[row * a.k_stride + (int64_t)hq * K + tid]);
            in_g = a.g[row * a.g_stride + (int64_t)h * K + tid];
        }
        if (tid >= 128 && kr < K) in_q = from_b16<F16>(a.q[row * a.q_stride + (int64_t)hq * K + kr]);
        if (tid < VT) in_v = from_b16<F16>(a.v[row * a.v_stride + (int64_t)h * a.V + tile * VT + tid]);
        if (tid == 0) in_b = from_b16<F16>(a.beta[row * a.beta_stride + h]);
    };
    auto stage_token = [&](int b) {
        if (tid < K) {
            s_kqe[b][tid].x = in_k;
            s_kqe[b][tid].z = expf(in_g);
        }
        if (tid >= 128 && kr < K) s_kqe[b][kr].y = in_q;
        if (tid < VT) s_v[b][tid] = in_v;
        if (tid == 0) s_beta[b] = a.logits ? 1.f / (1.f + expf(-in_b)) : in_b;
    };
    load_token(row0);

    // The same slot twice would race: the first sequence that names it has it.
    bool taken = false;
    if (in_cache && a.slots)
        for (int j = tid; j < n; j += kStepThreads) taken |= a.slots[j] == slot;
    stage_token(0);
    taken = __syncthreads_or(taken);

    uint16_t* o = a.o + (row0 * a.H + h) * a.V + tile * VT + cg * 4;
    const int64_t o_step = (int64_t)a.H * a.V;
    if (!in_cache || taken) {
        if (first && (taken || slot >= a.num_slots)) report(a.status, kStatusBadSlots);
        for (int t = rl; t < len; t += kRowLanes) *reinterpret_cast<uint2*>(o + t * o_step) = make_uint2(0u, 0u);
        return;
    }

    for (int t = 0; t < len; ++t) {
        const int b = t & 1;
        if (t + 1 < len) load_token(row0 + t + 1);
        float4 pk = make_float4(0.f, 0.f, 0.f, 0.f), pq = pk;
        float kq = 0.f;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const float4 r = s_kqe[b][rl + i * kRowLanes];
            S[i].x *= r.z;
            S[i].y *= r.z;
            S[i].z *= r.z;
            S[i].w *= r.z;
            pk.x += r.x * S[i].x;
            pk.y += r.x * S[i].y;
            pk.z += r.x * S[i].z;
            pk.w += r.x * S[i].w;
            pq.x += r.y * S[i].x;
            pq.y += r.y * S[i].y;
            pq.z += r.y * S[i].z;
            pq.w += r.y * S[i].w;
            kq += r.x * r.y;
        }
#pragma unroll
        for (int off = kColGroups; off < 32; off <<= 1) {  // row lanes of the same columns in this warp
            pk.x += __shfl_xor_sync(~0u, pk.x, off);
            pk.y += __shfl_xor_sync(~0u, pk.y, off);
            pk.z += __shfl_xor_sync(~0u, pk.z, off);
            pk.w += __shfl_xor_sync(~0u, pk.w, off);
            pq.x += __shfl_xor_sync(~0u, pq.x, off);
            pq.y += __shfl_xor_sync(~0u, pq.y, off);
            pq.z += __shfl_xor_sync(~0u, pq.z, off);
            pq.w += __shfl_xor_sync(~0u, pq.w, off);
            kq += __shfl_xor_sync(~0u, kq, off);
        }
        if (lane < kColGroups) {
            s_sum[0][warp][cg] = pk;
            s_sum[1][warp][cg] = pq;
        }
        if (lane == 0) s_kq[warp] = kq;
        __syncthreads();
        float4 d = s_sum[0][0][cg];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            const float4 x = s_sum[0][w][cg];
            d.x += x.x;
            d.y += x.y;
            d.z += x.z;
            d.w += x.w;
        }
        const float beta = s_beta[b];
        const float4 v = *reinterpret_cast<const float4*>(&s_v[b][cg * 4]);
        d = make_float4(beta * (v.x - d.x), beta * (v.y - d.y), beta * (v.z - d.z), beta * (v.w - d.w));
        if (rl == 0) {
            float4 y = s_sum[1][0][cg];
            float c = s_kq[0];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) {
                const float4 x = s_sum[1][w][cg];
                y.x += x.x;
                y.y += x.y;
                y.z += x.z;
                y.w += x.w;
                c += s_kq[w];
            }
            *reinterpret_cast<uint2*>(o + t * o_step) =
                make_uint2(pack_b16x2(a.scale * (y.x + c * d.x), a.scale * (y.y + c * d.y), F16),
                           pack_b16x2(a.scale * (y.z + c * d.z), a.scale * (y.w + c * d.w), F16));
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const float kk = s_kqe[b][rl + i * kRowLanes].x;
            S[i].x += kk * d.x;
            S[i].y += kk * d.y;
            S[i].z += kk * d.z;
            S[i].w += kk * d.w;
        }
        if (t + 1 < len) {
            stage_token(b ^ 1);  // last read before the barrier above, in token t - 1's update
            __syncthreads();
        }
    }

#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t off = at + (int64_t)i * kRowLanes * a.V;
        if constexpr (STATE16)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.state) + off) =
                make_uint2(pack_b16x2(S[i].x, S[i].y, false), pack_b16x2(S[i].z, S[i].w, false));
        else
            *reinterpret_cast<float4*>(static_cast<float*>(a.state) + off) = S[i];
    }
}

template <int K, int VT>
cudaError_t launch(const StepArgs& a, bool f16, bool state16, cudaStream_t s) {
    const unsigned grid = (unsigned)((int64_t)a.N * a.H * (a.V / VT));
    if (f16) {
        if (state16) kda_step_kernel<K, VT, true, true><<<grid, kStepThreads, 0, s>>>(a);
        else kda_step_kernel<K, VT, true, false><<<grid, kStepThreads, 0, s>>>(a);
    } else {
        if (state16) kda_step_kernel<K, VT, false, true><<<grid, kStepThreads, 0, s>>>(a);
        else kda_step_kernel<K, VT, false, false><<<grid, kStepThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
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
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f16 = p.io_dtype == KDA_IO_F16, s16 = p.state_dtype == KDA_STATE_BF16;
    const cudaError_t e = d.K == 128 ? launch<128, 64>(a, f16, s16, s) : launch<64, 64>(a, f16, s16, s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
