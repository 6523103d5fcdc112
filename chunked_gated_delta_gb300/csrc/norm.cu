// norm.cu -- kda_rms_norm: root-mean-square norm of rows, with the residual's
// addition before it and an output in 16, 32 or 8 bits (e4m3 with one scale a
// row).
//
//     s = x + r;   y = s * (1 / sqrt(mean(s^2) + eps)) * w
//     8 bits: a = max(max |y|, 1e-30), code = e4m3(y * (448 / a)), scale = a / 448
//
// Bound: HBM; every element is read once and written once.  A row stays in the
// registers of its threads between the load and the store, so the statistics
// cost exchanges but no second read: the sum of squares and, for 8 bits, the
// largest |s w|, which times 1 / sqrt(...) is the largest |y| (to a rounding),
// so that both are joined at once.  A row is taken by a team: 2 to 32 lanes of a
// warp for short rows (head norms), so that its sums are shuffles and many rows
// share a CTA, or a whole CTA for long ones, with one barrier.  Measured: 1.07 M
// rows of 128 81 us (6.7 TB/s, what a copy reaches), with residual to e4m3 6.9
// TB/s; 32768 rows of 4096 82 us (6.5), with residual to e4m3 135 (7.0); 16384
// fp32 rows of 4096 87 us (6.2), with residual 157 (6.8).
#include <type_traits>

#include "internal.h"
#include "layer_ops.cuh"
#include "ptx.cuh"

namespace kda {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 1e-30f;  // keeps 448 / a finite for a row of zeros

struct NormArgs {
    const void *x, *r, *w;
    void *y, *sum;
    float* y_scale;
    int64_t rows, x_stride, r_stride, sum_stride;
    int dim, out, w_f32;
    int y_with_x;  // SHIFT: y's rows lie off 16 bytes as x's do
    int exchange;  // SHIFT: they do not, and y goes through shared memory (a code's byte gains nothing by it)
    float eps, inv_dim;
};

// VEC elements of type IO (a KDA_DTYPE) as fp32: one 16-byte load (two for
// fp32) where VEC is 8, else one element.
template <int IO, int VEC>
__device__ __forceinline__ void load_vec(const void* p, int64_t at, float* f) {
    if constexpr (VEC == 8 && IO == KDA_DTYPE_F32) {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
        const float4 a = q[0], b = q[1];
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else if constexpr (VEC == 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = from_b16x2<IO == KDA_DTYPE_F16>(w[i]);
            f[2 * i] = v.x, f[2 * i + 1] = v.y;
        }
    } else if constexpr (IO == KDA_DTYPE_F32) {
        f[0] = static_cast<const float*>(p)[at];
    } else {
        f[0] = from_b16<IO == KDA_DTYPE_F16>(static_cast<const uint16_t*>(p)[at]);
    }
}
template <int VEC>
__device__ __forceinline__ void store_vec(void* p, int64_t at, const float* f, int dtype) {
    if constexpr (VEC == 8) {
        if (dtype == KDA_DTYPE_F32) {
            float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
            q[0] = make_float4(f[0], f[1], f[2], f[3]);
            q[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else if (dtype == KDA_DTYPE_E4M3) {
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p) + at) =
                make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3]), pack_e4m3x4(f[4], f[5], f[6], f[7]));
        } else {
            const bool h = dtype == KDA_DTYPE_F16;
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) =
                make_uint4(pack_b16x2(f[0], f[1], h), pack_b16x2(f[2], f[3], h), pack_b16x2(f[4], f[5], h),
                           pack_b16x2(f[6], f[7], h));
        }
    } else {
        if (dtype == KDA_DTYPE_F32) static_cast<float*>(p)[at] = f[0];
        else if (dtype == KDA_DTYPE_E4M3) static_cast<uint8_t*>(p)[at] = (uint8_t)pack_e4m3x2(f[0], 0.f);
        else static_cast<uint16_t*>(p)[at] = to_b16(f[0], dtype == KDA_DTYPE_F16);
    }
}

// Joins the sum and the largest over the team: lanes of a warp (TEAM <= 32), or
// the whole CTA (TEAM = 0) through s[32].
template <int TEAM>
__device__ __forceinline__ float2 team_join(float2 v, float2* s, bool with_max) {
    auto join = [&](int off) {
        v.x += __shfl_xor_sync(~0u, v.x, off);
        if (with_max) v.y = max_nan(v.y, __shfl_xor_sync(~0u, v.y, off));
    };
    constexpr int kLanes = TEAM ? TEAM : 32;
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) join(off);
    if constexpr (TEAM == 0) {
        const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) s[threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < warps ? s[lane] : make_float2(0.f, 0.f);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) join(off);
    }
    return v;
}

// Eight elements as they come from memory.
template <int IO>
struct Raw {
    uint4 v[IO == KDA_DTYPE_F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* p, int64_t at) {
        constexpr int kSize = IO == KDA_DTYPE_F32 ? 4 : 2;
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + at * kSize);
#pragma unroll
        for (int i = 0; i < kSize / 2; ++i) v[i] = q[i];
    }
    __device__ __forceinline__ void unpack(float* f) const {
        if constexpr (IO == KDA_DTYPE_F32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f[4 * i] = __uint_as_float(v[i].x), f[4 * i + 1] = __uint_as_float(v[i].y);
                f[4 * i + 2] = __uint_as_float(v[i].z), f[4 * i + 3] = __uint_as_float(v[i].w);
            }
        } else {
            const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 u = from_b16x2<IO == KDA_DTYPE_F16>(w[i]);
                f[2 * i] = u.x, f[2 * i + 1] = u.y;
            }
        }
    }
};
// Elements c .. c + 7 of a row of `dim`, of which some may lie outside it (SHIFT).
template <int IO, int VEC, bool SHIFT>
__device__ __forceinline__ void load_part(const void* p, int64_t row, int c, int dim, float* f) {
    if (!SHIFT || (c >= 0 && c + VEC <= dim)) {
        load_vec<IO, VEC>(p, row + c, f);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            f[j] = 0.f;
            if (c + j >= 0 && c + j < dim) load_vec<IO, 1>(p, row + c + j, f + j);
        }
    }
}
template <int VEC, bool SHIFT>
__device__ __forceinline__ void store_part(void* p, int64_t row, int c, int dim, const float* f, int dtype, bool vector) {
    if (!SHIFT || (vector && c >= 0 && c + VEC <= dim)) {
        store_vec<VEC>(p, row + c, f, dtype);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            if (c + j >= 0 && c + j < dim) store_vec<1>(p, row + c + j, f + j, dtype);
    }
}

// SHIFT: rows that do not start on 16 bytes, but x, the residual and the sum all
// off by the same: vectors start before the row, at its 16-byte boundary, and
// only a row's first and last vector go by elements.
template <int IO, int VEC, int NV, int TEAM, bool SHIFT>
__global__ void __launch_bounds__(TEAM ? 256 : SHIFT ? 576 : 1024) kda_norm_kernel(const NormArgs a) {
    __shared__ float2 s_join[32];
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int per = TEAM ? (int)(blockDim.x / TEAM) : 1;  // rows a CTA takes
    const int lane = TEAM ? (int)(threadIdx.x % TEAM) : (int)threadIdx.x;
    const int width = TEAM ? TEAM : (int)blockDim.x;
    const int64_t row = (int64_t)blockIdx.x * per + (TEAM ? (int)(threadIdx.x / TEAM) : 0);
    const bool live = row < a.rows;  // (teams past the last row still take part in the shuffles)
    const bool f8 = a.out == KDA_DTYPE_E4M3;
    int off = 0;  // elements from the 16-byte boundary before the row to its start
    if constexpr (SHIFT) {
        constexpr int kSize = IO == KDA_DTYPE_F32 ? 4 : 2;
        off = (int)((reinterpret_cast<uintptr_t>(a.x) / kSize + (uint64_t)(row * a.x_stride)) % (16 / kSize));
    }
    auto column = [&](int i) { return (lane + i * width) * VEC - off; };
    auto inside = [&](int c) { return c < a.dim && (!SHIFT || c + VEC > 0); };
    float s[NV][VEC];
    // Whole vectors of x and the residual are all asked for first, and only then taken
    // apart, which waits for them: residual rows to e4m3 152 -> 137 us for 32768 x 4096
    // (a ring in shared memory filled ahead by bulk copies was at 152, each vector
    // waited for by itself 170).  Small teams off 16 bytes do better without.
    constexpr bool kRaw = VEC == 8 && (!SHIFT || TEAM == 0);
    if constexpr (kRaw) {
        Raw<IO> rx[NV], rr[NV];
        auto whole = [&](int c) { return live && c + (SHIFT ? VEC - 1 : 0) < a.dim && (!SHIFT || c >= 0); };
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (whole(column(i))) rx[i].load(a.x, row * a.x_stride + column(i));
        if (a.r) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (whole(column(i))) rr[i].load(a.r, row * a.r_stride + column(i));
        }
        auto take = [&](int i, const Raw<IO>& raw, const void* p, int64_t stride, float* f) {
            const int c = column(i);
            if (whole(c)) {
                raw.unpack(f);
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    f[j] = 0.f;
                    if (SHIFT && live && c + j >= 0 && c + j < a.dim) load_vec<IO, 1>(p, row * stride + c + j, f + j);
                }
            }
        };
#pragma unroll
        for (int i = 0; i < NV; ++i) take(i, rx[i], a.x, a.x_stride, s[i]);
        if (a.r) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float r[VEC];
                take(i, rr[i], a.r, a.r_stride, r);
#pragma unroll
                for (int j = 0; j < VEC; ++j) s[i][j] += r[j];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = column(i);
#pragma unroll
            for (int j = 0; j < VEC; ++j) s[i][j] = 0.f;
            if (live && inside(c)) load_part<IO, VEC, SHIFT>(a.x, row * a.x_stride, c, a.dim, s[i]);
        }
        if (a.r) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = column(i);
                float r[VEC] = {};
                if (live && inside(c)) load_part<IO, VEC, SHIFT>(a.r, row * a.r_stride, c, a.dim, r);
#pragma unroll
                for (int j = 0; j < VEC; ++j) s[i][j] += r[j];
            }
        }
    }
    if (a.sum) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = column(i);
            if (live && inside(c)) store_part<VEC, SHIFT>(a.sum, row * a.sum_stride, c, a.dim, s[i], IO, true);
        }
    }
    // s becomes s w; the scale of a row follows its statistics
    float2 stat = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = column(i);
#pragma unroll
        for (int j = 0; j < VEC; ++j) stat.x += s[i][j] * s[i][j];
        if (a.w && inside(c)) {
            float w[VEC];
            if constexpr (SHIFT) {  // (the weight has its own boundary)
                const bool words = (TEAM == 0 || TEAM == 32) && IO != KDA_DTYPE_F32 && !a.w_f32 && c >= 1 && c + VEC < a.dim;
                if (words) {
                    const uint16_t* at = static_cast<const uint16_t*>(a.w) + c;
                    const int odd = (int)(reinterpret_cast<uintptr_t>(at) >> 1) & 1;
                    const uint32_t* from = reinterpret_cast<const uint32_t*>(at - odd);
                    uint32_t u[VEC / 2 + 1];
#pragma unroll
                    for (int j = 0; j < VEC / 2; ++j) u[j] = from[j];
                    u[VEC / 2] = odd ? from[VEC / 2] : 0u;
#pragma unroll
                    for (int j = 0; j < VEC / 2; ++j) {
                        const float2 v = from_b16x2<IO == KDA_DTYPE_F16>(__funnelshift_r(u[j], u[j + 1], 16 * odd));
                        w[2 * j] = v.x, w[2 * j + 1] = v.y;
                    }
                }
#pragma unroll
                for (int j = 0; j < VEC && !words; ++j) {
                    w[j] = 0.f;
                    if (c + j >= 0 && c + j < a.dim) {
                        if (a.w_f32) load_vec<KDA_DTYPE_F32, 1>(a.w, c + j, w + j);
                        else load_vec<IO, 1>(a.w, c + j, w + j);
                    }
                }
            } else {
                if (a.w_f32) load_vec<KDA_DTYPE_F32, VEC>(a.w, c, w);
                else load_vec<IO, VEC>(a.w, c, w);
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) s[i][j] *= w[j];
        }
        if (f8) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) stat.y = max_nan(stat.y, fabsf(s[i][j]));
        }
    }
    stat = team_join<TEAM>(stat, s_join, f8);
    const float rstd = 1.f / sqrtf(stat.x * a.inv_dim + a.eps);
    float inv = 1.f;
    if (f8) {
        const float amax = max_nan(kAmaxFloor, stat.y * rstd);
        inv = kE4m3Max / amax;
        if (live && lane == 0) a.y_scale[row] = amax / kE4m3Max;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = column(i);
        if (live && inside(c)) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) s[i][j] = s[i][j] * rstd * inv;
        }
        if constexpr (SHIFT) {
            if (a.exchange) {
                // y's own boundary: the lanes of a team, or of a warp, exchange their vectors so
                // that neighbours store neighbours
                extern __shared__ __align__(16) float s_row[];
                constexpr int kLanes = TEAM ? TEAM : 32;
                const int in_team = lane % kLanes, c0 = c - in_team * VEC;
                if ((lane - in_team + i * width) * VEC >= a.dim + 8) break;  // (all teams of a warp do)
                float* piece = s_row + (threadIdx.x - in_team) * VEC;
                __syncwarp();
#pragma unroll
                for (int j = 0; j < VEC; j += 4)
                    *reinterpret_cast<float4*>(piece + in_team * VEC + j) =
                        make_float4(s[i][j], s[i][j + 1], s[i][j + 2], s[i][j + 3]);
                __syncwarp();
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const int e = j * kLanes + in_team;
                    if (live && c0 + e >= 0 && c0 + e < a.dim) store_vec<1>(a.y, row * a.dim + c0 + e, piece + e, a.out);
                }
                continue;
            }
        }
        if (live && inside(c)) store_part<VEC, SHIFT>(a.y, row * a.dim, c, a.dim, s[i], a.out, a.y_with_x);
    }
}

template <int IO, int VEC, int NV, int TEAM, bool SHIFT = false>
cudaError_t launch(const NormArgs& a, int threads, cudaStream_t s) {
    const int64_t per = TEAM ? threads / TEAM : 1;
    return launch_dependent(kda_norm_kernel<IO, VEC, NV, TEAM, SHIFT>, dim3((unsigned)((a.rows + per - 1) / per)),
                            dim3((unsigned)threads), SHIFT && a.exchange ? threads * VEC * 4 : 0, s, a);
}

template <int IO, int VEC>
cudaError_t pick(const NormArgs& a, cudaStream_t s) {
    const int vecs = (a.dim + VEC - 1) / VEC;
    auto threads = [&](int nv) { return (vecs + nv * 32 - 1) / (nv * 32) * 32; };
    if constexpr (VEC == 8) {
        if (vecs > 32 && vecs <= 1024 && a.rows <= 2 * device_sm_count())
            return launch<IO, VEC, 1, 0>(a, threads(1), s);
        if (a.r) {
            if (vecs <= 4) return launch<IO, VEC, 2, 2>(a, 256, s);
            if (vecs <= 8) return launch<IO, VEC, 2, 4>(a, 256, s);
            if (vecs <= 16) return launch<IO, VEC, 2, 8>(a, 256, s);
            if (vecs <= 32) return launch<IO, VEC, 2, 16>(a, 256, s);
            if (vecs <= 64) return launch<IO, VEC, 2, 32>(a, 256, s);
        } else {
            if (vecs <= 8) return launch<IO, VEC, 4, 2>(a, 256, s);
            if (vecs <= 16) return launch<IO, VEC, 4, 4>(a, 256, s);
            if (vecs <= 32) return launch<IO, VEC, 4, 8>(a, 256, s);
            if (vecs <= 64) return launch<IO, VEC, 4, 16>(a, 256, s);
        }
        if (vecs <= 128) return launch<IO, VEC, 4, 32>(a, 256, s);
        // (an fp32 vector is two loads: 16384 rows of 4096 with residual 158 us, 180 in fours)
        if (IO == KDA_DTYPE_F32 && a.r && vecs <= 2048) return launch<IO, VEC, 2, 0>(a, threads(2), s);
        return launch<IO, VEC, 4, 0>(a, threads(4), s);
    } else {
        if (vecs <= 32) return launch<IO, VEC, 4, 8>(a, 256, s);
        if (vecs <= 128) return launch<IO, VEC, 4, 32>(a, 256, s);
        if (vecs <= 512) return launch<IO, VEC, 16, 32>(a, 256, s);
        if (vecs <= 16384) return launch<IO, VEC, 16, 0>(a, threads(16), s);
        return launch<IO, VEC, 32, 0>(a, threads(32), s);
    }
}

// Rows off 16 bytes.  (26000 rows of 5003 with residual, to e4m3: 466 us element by
// element, 243 in vectors from the boundary before the row; to fp32, whose rows lie
// off 16 bytes otherwise than x's, 471 us stored from where the vectors are, 233
// through shared memory.)
template <int IO>
cudaError_t pick_shifted(const NormArgs& a, cudaStream_t s) {
    const int vecs = a.dim / 8 + 2;  // at most
    if (vecs <= 32) return launch<IO, 8, 4, 8, true>(a, 256, s);
    if (vecs <= 64) return launch<IO, 8, 4, 16, true>(a, 256, s);
    if (vecs <= 128) return launch<IO, 8, 4, 32, true>(a, 256, s);
    if (vecs <= 2048) return launch<IO, 8, 4, 0, true>(a, (vecs + 127) / 128 * 32, s);
    return launch<IO, 8, 8, 0, true>(a, (vecs + 255) / 256 * 32, s);  // (at most 4097, 544 threads)
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_rms_norm(const void* x, const void* residual, const void* weight, void* y, float* y_scale,
                                   void* sum, int64_t rows, int64_t dim, const kda_norm_opts* opts, void* stream) {
    if (!opts || rows < 0 || dim < 1) return KDA_ERR_INVALID_ARG;
    const kda_norm_opts& p = *opts;
    if (p.io_dtype != KDA_DTYPE_BF16 && p.io_dtype != KDA_DTYPE_F16 && p.io_dtype != KDA_DTYPE_F32)
        return KDA_ERR_INVALID_ARG;
    if (p.out_dtype != p.io_dtype && p.out_dtype != KDA_DTYPE_F32 && p.out_dtype != KDA_DTYPE_E4M3)
        return KDA_ERR_INVALID_ARG;
    if ((p.weight_f32 != 0 && p.weight_f32 != 1) || !(p.eps >= 0.f)) return KDA_ERR_INVALID_ARG;
    if ((p.out_dtype == KDA_DTYPE_E4M3) != (y_scale != nullptr)) return KDA_ERR_INVALID_ARG;
    if (dim > 32768) return KDA_ERR_UNSUPPORTED;
    NormArgs a{};
    a.x_stride = p.x_stride ? p.x_stride : dim;
    a.r_stride = p.residual_stride ? p.residual_stride : dim;
    a.sum_stride = p.sum_stride ? p.sum_stride : dim;
    if (a.x_stride < dim || a.r_stride < dim || a.sum_stride < dim) return KDA_ERR_INVALID_ARG;
    if (rows == 0) return KDA_OK;
    if (rows > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (!x || !y) return KDA_ERR_INVALID_ARG;
    const int es = dtype_bytes(p.io_dtype), wes = p.weight_f32 ? 4 : es, oes = dtype_bytes(p.out_dtype);
    if (!is_aligned(x, es) || !is_aligned(residual, es) || !is_aligned(sum, es) || !is_aligned(weight, wes) ||
        !is_aligned(y, oes) || !is_aligned(y_scale, 4))
        return KDA_ERR_ALIGNMENT;
    a.x = x;
    a.r = residual;
    a.w = weight;
    a.y = y;
    a.sum = sum;
    a.y_scale = y_scale;
    a.rows = rows;
    a.dim = (int)dim;
    a.out = p.out_dtype;
    a.w_f32 = p.weight_f32;
    a.eps = p.eps;
    a.inv_dim = 1.f / (float)dim;
    const bool wide = dim % 8 == 0 && is_aligned(x, 16) && is_aligned(residual, 16) && is_aligned(sum, 16) &&
                      is_aligned(weight, 16) && is_aligned(y, 8 * oes < 16 ? 8 : 16) && a.x_stride * es % 16 == 0 &&
                      (!residual || a.r_stride * es % 16 == 0) && (!sum || a.sum_stride * es % 16 == 0);
    // the same distance from a 16-byte boundary as x's in every row
    auto with_x = [&](const void* t, int64_t stride) {
        return (reinterpret_cast<uintptr_t>(t) - reinterpret_cast<uintptr_t>(x)) % 16 == 0 &&
               (stride - a.x_stride) * es % 16 == 0;
    };
    const bool shifted = !wide && dim >= 32 && (!residual || with_x(residual, a.r_stride)) &&
                         (!sum || with_x(sum, a.sum_stride));
    a.y_with_x = p.out_dtype == p.io_dtype && with_x(y, dim);
    a.exchange = !a.y_with_x && p.out_dtype != KDA_DTYPE_E4M3;
    auto run = [&](auto io) {
        constexpr int kIo = decltype(io)::value;
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        return wide ? pick<kIo, 8>(a, s) : shifted ? pick_shifted<kIo>(a, s) : pick<kIo, 1>(a, s);
    };
    cudaError_t e;
    if (p.io_dtype == KDA_DTYPE_BF16) e = run(std::integral_constant<int, KDA_DTYPE_BF16>{});
    else if (p.io_dtype == KDA_DTYPE_F16) e = run(std::integral_constant<int, KDA_DTYPE_F16>{});
    else e = run(std::integral_constant<int, KDA_DTYPE_F32>{});
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
