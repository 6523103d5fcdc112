// rotary.cu -- kda_rotary: the positions of q and k. Pairs (x, y) of a head's first
// 2 * pairs elements are turned by the angle position * freq:
//     x' = amplitude (x cos - y sin),  y' = amplitude (x sin + y cos),
// the rest of the head is copied.
//
// The angle of a far position is hundreds of thousands of radians, of which fp32 would
// keep a few hundredths. It is taken in turns, as a fraction of 64 bits: position times
// that fraction, as integers, wraps around where the angle does, so little is lost to its size (2^-65 of a turn
// for each position, beside the frequency's own 53 bits), without any 64-bit float arithmetic per token. Of the product's
// leading 32 bits an fp32 number has 24; the other eight turn its sine and cosine by what they are worth.
//
// Bound: q and k read and written once. A CTA goes through groups of tokens (one, or as many as its loads hold);
// its threads make their cosines and sines once for all heads, in shared memory, while
// the rows are on their way, 16 bytes a load, from places that a thread works out once. 32768 tokens x 64 heads of
// 128 in bf16 164 us (6.5 TB/s, 98% of a copy) in both layouts; 59 tokens x 40 heads 5 us, the call. Two loads side by
// side for the interleaved layout 190, and places worked out for every token 114 instead of 110 us for
// 40 heads of which half is turned.
#include "internal.h"
#include "layer_ops.cuh"
#include "ptx.cuh"

namespace kda {
namespace {

constexpr int kRotaryThreads = 128;
constexpr int kMostPairs = 512;
constexpr int kItems = 4;  // pieces of a row that a thread has in flight

struct RotaryArgs {
    const void *q, *k;
    void *q_out, *k_out;
    const void* positions;  // int64 or int32
    const double* freqs;
    int64_t tokens, q_stride, k_stride, q_out_stride, k_out_stride;  // in elements
    int32_t q_heads, k_heads, dim, pairs, positions64, inverse;
    int32_t group;   // consecutive tokens that a CTA takes together
    uint32_t magic;  // e / per_head is the upper half of e * magic (0: divide)
    float amplitude;
};

template <int IO>
struct Io;
template <>
struct Io<KDA_DTYPE_BF16> {
    using T = uint16_t;
    static __device__ __forceinline__ float get(T x) { return from_b16<false>(x); }
    static __device__ __forceinline__ T put(float x) { return to_b16(x, false); }
};
template <>
struct Io<KDA_DTYPE_F16> {
    using T = uint16_t;
    static __device__ __forceinline__ float get(T x) { return from_b16<true>(x); }
    static __device__ __forceinline__ T put(float x) { return to_b16(x, true); }
};
template <>
struct Io<KDA_DTYPE_F32> {
    using T = float;
    static __device__ __forceinline__ float get(T x) { return x; }
    static __device__ __forceinline__ T put(float x) { return x; }
};

// C elements (16 bytes, or one) in a register block.
template <typename T, int C>
struct alignas(sizeof(T) * C) Piece {
    T x[C];
};

// C: elements of a load. A row of a head is items: those of pairs (two loads of C elements: in the half layout the
// x and the y of C pairs, else C / 2 pairs in the first half of the turned elements and C / 2 in the second, so that
// a warp's loads and stores are of whole lines in both; C = 1 is a pair either way), then those that are copied (two
// loads of C elements next to each other).
template <int IO, int C, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotaryThreads, C > 1 ? 6 : 8) kda_rotary_kernel(const RotaryArgs a) {
    using T = typename Io<IO>::T;
    using P = Piece<T, C>;
    __shared__ __align__(16) float2 s_turn[2][kMostPairs];  // cos, sin
    __shared__ uint64_t s_share[kMostPairs];  // one position's share of a turn, times 2^64
    __shared__ int16_t s_of[kMostPairs];      // which of the tokens taken together
    const int tid = threadIdx.x;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int own = a.group * a.pairs;
    for (int p = tid; p < own; p += kRotaryThreads) {  // (each read by the thread that wrote it)
        const int of = p / a.pairs;
        double t = a.freqs[p - of * a.pairs] * 0.15915494309189535;
        t -= floor(t);
        s_share[p] = __double2ull_rn(t * 18446744073709551616.0);
        s_of[p] = (int16_t)of;
    }
    const int turned = a.pairs / C;                               // items of pairs in a head
    const int copied = (a.dim - 2 * a.pairs + 2 * C - 1) / (2 * C);
    const int per_head = turned + copied, heads = a.q_heads + a.k_heads, items = heads * per_head;

    auto angles = [&](int64_t tok, int count, float2* to) {
        for (int p = tid; p < count * a.pairs; p += kRotaryThreads) {
            const int64_t at = tok + s_of[p];
            const uint64_t pos = a.positions64 ? static_cast<const uint64_t*>(a.positions)[at]
                                               : (uint64_t)(int64_t)static_cast<const int32_t*>(a.positions)[at];
            // (the leading 32 bits of the fraction, as half turns in -1 .. 1: 24 of them, and the angle that the rest is)
            const uint32_t turn = (uint32_t)((pos * s_share[p]) >> 32);
            const float half_turns = (float)(int32_t)(turn & ~0xffu) * 0x1p-31f, rest = (float)(turn & 0xffu) * (3.14159265f * 0x1p-31f);
            float s, c;
            sincospif(half_turns, &s, &c);
            const float s0 = s;
            s = fmaf(c, rest, s);
            c = fmaf(-s0, rest, c);
            to[p] = make_float2(a.amplitude * c, a.inverse ? -a.amplitude * s : a.amplitude * s);
        }
    };
    constexpr int kOneLoad = -1, kTwoLoads = -2;  // of an item that is copied
    struct Item {
        const T* in;
        T* out;
        int pair;   // the turn of its first pair, or how it is copied
        bool of_q;
    };
    auto item_at = [&](int64_t tok, int e) {
        const int t = a.group == 1 ? 0 : e / items;
        e -= t * items;
        tok += t;
        const int head = a.magic ? (int)__umulhi((uint32_t)e, a.magic) : e / per_head, i = e - head * per_head;
        Item r;
        r.of_q = head < a.q_heads;
        int first;
        if (i < turned) {
            r.pair = t * a.pairs + (INTERLEAVED && C > 1 ? i * (C / 2) : i * C);
            first = INTERLEAVED && C == 1 ? 2 * i : i * C;
        } else {
            first = 2 * a.pairs + (i - turned) * 2 * C;
            r.pair = first + C < a.dim ? kTwoLoads : kOneLoad;
        }
        if (r.of_q) {
            r.in = static_cast<const T*>(a.q) + tok * a.q_stride + (int64_t)head * a.dim + first;
            r.out = static_cast<T*>(a.q_out) + tok * a.q_out_stride + (int64_t)head * a.dim + first;
        } else {
            r.in = static_cast<const T*>(a.k) + tok * a.k_stride + (int64_t)(head - a.q_heads) * a.dim + first;
            r.out = static_cast<T*>(a.k_out) + tok * a.k_out_stride + (int64_t)(head - a.q_heads) * a.dim + first;
        }
        return r;
    };
    const int apart = INTERLEAVED && C == 1 ? 1 : a.pairs;  // the two loads of a turned item

    const int64_t first_token = (int64_t)blockIdx.x * a.group, ahead = (int64_t)gridDim.x * a.group;
    const bool once = a.group * items <= kItems * kRotaryThreads;  // then a thread has the same items of every token
    Item item[kItems];
    if (once) {
#pragma unroll
        for (int i = 0; i < kItems; ++i) item[i] = item_at(first_token, tid + i * kRotaryThreads);
    }
    int buf = 0;
    for (int64_t tok = first_token; tok < a.tokens; tok += ahead, buf ^= 1) {
        const int count = a.tokens - tok < a.group ? (int)(a.tokens - tok) : a.group, all = count * items;
        for (int e0 = tid; e0 - tid < all; e0 += kItems * kRotaryThreads) {
            P x[kItems], y[kItems];
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                const int e = e0 + i * kRotaryThreads;
                if (e < all) {
                    if (!once) item[i] = item_at(tok, e);
                    const Item at = item[i];
                    x[i] = *reinterpret_cast<const P*>(at.in);
                    if (at.pair != kOneLoad) y[i] = *reinterpret_cast<const P*>(at.in + (at.pair >= 0 ? apart : C));
                }
            }
            if (e0 == tid) {  // (one barrier per group: the buffer before last has been read by all)
                angles(tok, count, s_turn[buf]);
                __syncthreads();
            }
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                const int e = e0 + i * kRotaryThreads;
                if (e >= all) break;
                const Item at = item[i];
                if (at.pair >= 0) {
                    if constexpr (C == 8) {  // 16 bits: words of two elements
                        const float4* turns = reinterpret_cast<const float4*>(&s_turn[buf][at.pair]);  // two pairs' each
                        const int half = a.pairs >> 2;  // between the turns of an item's two loads
                        uint32_t* u = reinterpret_cast<uint32_t*>(&x[i]);
                        uint32_t* w = reinterpret_cast<uint32_t*>(&y[i]);
                        constexpr bool kF16 = IO == KDA_DTYPE_F16;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const float4 t = turns[INTERLEAVED && c >= 2 ? half + c - 2 : c];
                            if constexpr (INTERLEAVED) {
                                uint32_t* v = c < 2 ? u + 2 * c : w + 2 * c - 4;
                                const float2 m = from_b16x2<kF16>(v[0]), n = from_b16x2<kF16>(v[1]);
                                v[0] = pack_b16x2(m.x * t.x - m.y * t.y, m.x * t.y + m.y * t.x, kF16);
                                v[1] = pack_b16x2(n.x * t.z - n.y * t.w, n.x * t.w + n.y * t.z, kF16);
                            } else {
                                const float2 m = from_b16x2<kF16>(u[c]), n = from_b16x2<kF16>(w[c]);
                                u[c] = pack_b16x2(m.x * t.x - n.x * t.y, m.y * t.z - n.y * t.w, kF16);
                                w[c] = pack_b16x2(m.x * t.y + n.x * t.x, m.y * t.w + n.y * t.z, kF16);
                            }
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < C; ++c) {
                            const int late = INTERLEAVED && C > 1 && 2 * c >= C ? (a.pairs - C) / 2 : 0;
                            const float2 t = s_turn[buf][at.pair + c + late];
                            T *u, *w;
                            if constexpr (INTERLEAVED) {
                                u = 2 * c < C ? &x[i].x[2 * c % C] : &y[i].x[2 * c % C];
                                w = 2 * c + 1 < C ? &x[i].x[(2 * c + 1) % C] : &y[i].x[(2 * c + 1) % C];
                            } else {
                                u = &x[i].x[c];
                                w = &y[i].x[c];
                            }
                            const float m = Io<IO>::get(*u), n = Io<IO>::get(*w);
                            *u = Io<IO>::put(m * t.x - n * t.y);
                            *w = Io<IO>::put(m * t.y + n * t.x);
                        }
                    }
                } else if (at.in == at.out) {
                    continue;
                }
                *reinterpret_cast<P*>(at.out) = x[i];
                if (at.pair != kOneLoad) *reinterpret_cast<P*>(at.out + (at.pair >= 0 ? apart : C)) = y[i];
            }
        }
        if (once) {
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                item[i].in += ahead * (item[i].of_q ? a.q_stride : a.k_stride);
                item[i].out += ahead * (item[i].of_q ? a.q_out_stride : a.k_out_stride);
            }
        }
    }
}

template <int IO, int C>
cudaError_t launch(const RotaryArgs& a, bool interleaved, unsigned grid, cudaStream_t s) {
    return interleaved ? launch_dependent(kda_rotary_kernel<IO, C, true>, dim3(grid), dim3(kRotaryThreads), 0, s, a)
                       : launch_dependent(kda_rotary_kernel<IO, C, false>, dim3(grid), dim3(kRotaryThreads), 0, s, a);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_rotary(const void* q, const void* k, const void* positions, const double* freqs, void* q_out,
                                 void* k_out, int64_t tokens, int32_t q_heads, int32_t k_heads, int32_t dim,
                                 const kda_rotary_opts* opts, void* stream) {
    if (!opts) return KDA_ERR_INVALID_ARG;
    const kda_rotary_opts& p = *opts;
    if (tokens < 0 || q_heads < 1 || k_heads < 0 || dim < 1 || p.pairs < 1 || p.pairs > dim / 2 ||
        (p.io_dtype != KDA_DTYPE_BF16 && p.io_dtype != KDA_DTYPE_F16 && p.io_dtype != KDA_DTYPE_F32) ||
        (p.positions_i64 != 0 && p.positions_i64 != 1) || (p.interleaved != 0 && p.interleaved != 1) ||
        (p.inverse != 0 && p.inverse != 1) || p.reserved != 0)
        return KDA_ERR_INVALID_ARG;
    if (p.pairs > kMostPairs || (int64_t)(q_heads + (int64_t)k_heads) * dim > INT32_MAX / 2) return KDA_ERR_UNSUPPORTED;
    const int64_t wq = (int64_t)q_heads * dim, wk = (int64_t)k_heads * dim;
    RotaryArgs a{};
    a.q_stride = p.q_stride ? p.q_stride : wq;
    a.k_stride = p.k_stride ? p.k_stride : wk;
    a.q_out_stride = p.q_out_stride ? p.q_out_stride : wq;
    a.k_out_stride = p.k_out_stride ? p.k_out_stride : wk;
    if (a.q_stride < wq || a.k_stride < wk || a.q_out_stride < wq || a.k_out_stride < wk) return KDA_ERR_INVALID_ARG;
    if (tokens == 0) return KDA_OK;
    if (!q || !q_out || !positions || !freqs || (k_heads > 0 && (!k || !k_out))) return KDA_ERR_INVALID_ARG;
    // in place, rows as they lie, or apart
    if (k_heads > 0 && (q_out == k_out || q_out == k || k_out == q)) return KDA_ERR_INVALID_ARG;
    if ((q == q_out && a.q_stride != a.q_out_stride) || (k_heads > 0 && k == k_out && a.k_stride != a.k_out_stride))
        return KDA_ERR_INVALID_ARG;
    const int es = dtype_bytes(p.io_dtype);
    if (!is_aligned(q, es) || !is_aligned(q_out, es) || (k_heads > 0 && (!is_aligned(k, es) || !is_aligned(k_out, es))) ||
        !is_aligned(positions, p.positions_i64 ? 8 : 4) || !is_aligned(freqs, 8))
        return KDA_ERR_ALIGNMENT;
    a.q = q;
    a.k = k;
    a.q_out = q_out;
    a.k_out = k_out;
    a.positions = positions;
    a.freqs = freqs;
    a.tokens = tokens;
    a.q_heads = q_heads;
    a.k_heads = k_heads;
    a.dim = dim;
    a.pairs = p.pairs;
    a.positions64 = p.positions_i64;
    a.inverse = p.inverse;
    a.amplitude = p.amplitude;
    const int C = 16 / es;
    bool wide = dim % C == 0 && p.pairs % C == 0;
    for (const void* x : {q, static_cast<const void*>(q_out)}) wide = wide && is_aligned(x, 16);
    for (int64_t x : {a.q_stride, a.q_out_stride}) wide = wide && x % C == 0;
    if (k_heads > 0) {
        for (const void* x : {k, static_cast<const void*>(k_out)}) wide = wide && is_aligned(x, 16);
        for (int64_t x : {a.k_stride, a.k_out_stride}) wide = wide && x % C == 0;
    }
    const int W = wide ? C : 1;
    const uint32_t per_head = (uint32_t)(p.pairs / W + (dim - 2 * p.pairs + 2 * W - 1) / (2 * W));
    // (floor(2^32 / d) + 1 divides e by d where e * d < 2^32)
    if (per_head > 1 && (uint64_t)(q_heads + k_heads) * per_head * per_head < (1ull << 32)) a.magic = (uint32_t)((1ull << 32) / per_head) + 1;
    // Tokens of few heads are taken together, as far as their loads and turns fit, and every CTA has some.
    const int64_t most = (int64_t)device_sm_count() * 6, items = (int64_t)(q_heads + k_heads) * per_head;
    int64_t group = kItems * kRotaryThreads / items;
    if (group > kMostPairs / p.pairs) group = kMostPairs / p.pairs;
    if (group > tokens / most) group = tokens / most;
    a.group = group > 1 ? (int32_t)group : 1;
    const int64_t groups = (tokens + a.group - 1) / a.group;
    // Four times the CTAs that fit balance the end of a long call (64 heads of 128, 32768 tokens, pairs side by side:
    // 164 us, else 183), where each has four groups for its start (9 heads of 256, 16384 tokens: 39 us with more, 35).
    const int64_t ctas = groups >= 16 * most ? 4 * most : most;
    const unsigned grid = (unsigned)(groups < ctas ? groups : ctas);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (p.io_dtype == KDA_DTYPE_F32)
        e = wide ? launch<KDA_DTYPE_F32, 4>(a, p.interleaved, grid, s) : launch<KDA_DTYPE_F32, 1>(a, p.interleaved, grid, s);
    else if (p.io_dtype == KDA_DTYPE_F16)
        e = wide ? launch<KDA_DTYPE_F16, 8>(a, p.interleaved, grid, s) : launch<KDA_DTYPE_F16, 1>(a, p.interleaved, grid, s);
    else
        e = wide ? launch<KDA_DTYPE_BF16, 8>(a, p.interleaved, grid, s) : launch<KDA_DTYPE_BF16, 1>(a, p.interleaved, grid, s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
