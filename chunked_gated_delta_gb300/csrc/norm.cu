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
// share a CTA, or a whole CTA for long ones, with one barrier; long rows with a
// residual go through a ring in shared memory instead (below).  Measured: 1.07 M
// rows of 128 82 us (6.7 TB/s, what a copy reaches), with residual to e4m3 6.9
// TB/s; 32768 rows of 4096 84 us (6.4), with residual to e4m3 152 (6.2).
#include <type_traits>

#include "internal.h"
#include "layer_ops.cuh"
#include "waits.cuh"

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
__global__ void __launch_bounds__(TEAM ? 256 : 1024) kda_norm_kernel(const NormArgs a) {
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
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = column(i);
        if (live && inside(c)) {
            load_part<IO, VEC, SHIFT>(a.x, row * a.x_stride, c, a.dim, s[i]);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) s[i][j] = 0.f;
        }
    }
    if (a.r) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = column(i);
            if (live && inside(c)) {
                float r[VEC];
                load_part<IO, VEC, SHIFT>(a.r, row * a.r_stride, c, a.dim, r);
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
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
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
            store_part<VEC, SHIFT>(a.y, row * a.dim, c, a.dim, s[i], a.out, a.y_with_x);
        }
    }
}

template <int IO, int VEC, int NV, int TEAM, bool SHIFT = false>
cudaError_t launch(const NormArgs& a, int threads, cudaStream_t s) {
    const int64_t per = TEAM ? threads / TEAM : 1;
    return launch_dependent(kda_norm_kernel<IO, VEC, NV, TEAM, SHIFT>, dim3((unsigned)((a.rows + per - 1) / per)),
                            dim3((unsigned)threads), 0, s, a);
}

// ------------------------------------------------------------------ long rows with a residual
// Two rows to load, two to store, and a barrier between: with a CTA per row (the
// kernel above) an SM's loads stop while its rows wait for their sums.  Here CTAs
// are persistent: a warp loads rows of x and the residual into a ring in shared
// memory with bulk copies, and groups of 128 threads take them in turn, so the
// loads never stop.  Measured, to e4m3: 32768 rows of 4096 170 -> 152 us (6.2 TB/s,
// 93% of a copy), 16384 of 8192 175 -> 158; rows of 2048 gain nothing (163, 167).
constexpr int kRingThreads = 128;  // of a group
constexpr int kRingGroups = 4;
constexpr int kRingAll = kRingGroups * kRingThreads + 32;
constexpr int kMostSlots = 24;
constexpr int kRingBytes = 200 * 1024;

// Slots of the ring: a multiple of the groups, so that a slot's barriers belong
// to one group (a group that waits a phase ahead of another's would misread
// their parity).
inline int ring_slots(int slot_bytes) {
    const int n = kRingBytes / slot_bytes / kRingGroups * kRingGroups;
    return n < kMostSlots ? n : kMostSlots;
}

template <int IO, int NV>
__global__ void __launch_bounds__(kRingAll, 1) kda_norm_ring_kernel(const NormArgs a, int slots) {
    constexpr int kSize = IO == KDA_DTYPE_F32 ? 4 : 2;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ __align__(8) uint64_t full[kMostSlots], empty[kMostSlots];
    __shared__ float2 s_join[kRingGroups][2][kRingThreads / 32];
    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
    const int row_bytes = a.dim * kSize, slot_bytes = 2 * row_bytes;
    if (tid < slots) {
        ptx::mbar_init(&full[tid], 1);
        ptx::mbar_init(&empty[tid], kRingThreads / 32);
    }
    ptx::fence_mbar_init();
    ptx::grid_dep_launch();
    __syncthreads();
    ptx::grid_dep_wait();

    const int count = (int)((a.rows - blockIdx.x + gridDim.x - 1) / gridDim.x);  // rows of this CTA
    if (warp == kRingGroups * (kRingThreads / 32)) {
        if (elect_one()) {
            int i = 0;
            for (; i < count; ++i) {
                const int s = i % slots, round = i / slots;
                if (round > 0 && !wait_for(&empty[s], (round - 1) & 1)) break;
                const int64_t row = blockIdx.x + (int64_t)i * gridDim.x;
                uint8_t* to = ring + s * slot_bytes;
                ptx::mbar_arrive_expect_tx(&full[s], (uint32_t)slot_bytes);
                bulk_load(to, static_cast<const uint8_t*>(a.x) + row * a.x_stride * kSize, (uint32_t)row_bytes, &full[s]);
                bulk_load(to + row_bytes, static_cast<const uint8_t*>(a.r) + row * a.r_stride * kSize,
                          (uint32_t)row_bytes, &full[s]);
            }
            // (every copy is waited for by the group that takes its row, or here if that gave up)
            for (int j = max(0, i - slots); j < i; ++j) wait_for(&full[j % slots], (j / slots) & 1);
        }
        return;
    }
    const int group = warp / (kRingThreads / 32), gt = tid - group * kRingThreads;
    const bool f8 = a.out == KDA_DTYPE_E4M3;
    bool ok = true;
    for (int i = group, k = 0; i < count; i += kRingGroups, ++k) {
        const int slot = i % slots;
        const int64_t row = blockIdx.x + (int64_t)i * gridDim.x;
        const uint8_t* x = ring + slot * slot_bytes;
        ok = ok && wait_for(&full[slot], (i / slots) & 1);
        float s[NV][8];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (gt + v * kRingThreads) * 8;
            if (c < a.dim) {
                float r[8];
                load_vec<IO, 8>(x, c, s[v]);
                load_vec<IO, 8>(x + row_bytes, c, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[v][j] += r[j];
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) s[v][j] = 0.f;
            }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&empty[slot]);
        float2 stat = make_float2(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (gt + v * kRingThreads) * 8;
            if (c < a.dim && a.sum && ok) store_vec<8>(a.sum, row * a.sum_stride + c, s[v], IO);
#pragma unroll
            for (int j = 0; j < 8; ++j) stat.x += s[v][j] * s[v][j];
            if (c < a.dim && a.w) {
                float w[8];
                if (a.w_f32) load_vec<KDA_DTYPE_F32, 8>(a.w, c, w);
                else load_vec<IO, 8>(a.w, c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[v][j] *= w[j];
            }
            if (f8) {
#pragma unroll
                for (int j = 0; j < 8; ++j) stat.y = max_nan(stat.y, fabsf(s[v][j]));
            }
        }
        stat = team_join<32>(stat, nullptr, f8);
        if (lane == 0) s_join[group][k & 1][gt >> 5] = stat;
        asm volatile("barrier.cta.sync %0, %1;" ::"r"(group + 1), "n"(kRingThreads) : "memory");
        stat = s_join[group][k & 1][0];
#pragma unroll
        for (int w = 1; w < kRingThreads / 32; ++w) {
            const float2 o = s_join[group][k & 1][w];
            stat.x += o.x;
            stat.y = max_nan(stat.y, o.y);
        }
        const float rstd = 1.f / sqrtf(stat.x * a.inv_dim + a.eps);
        float inv = 1.f;
        if (f8) {
            const float amax = max_nan(kAmaxFloor, stat.y * rstd);
            inv = kE4m3Max / amax;
            if (gt == 0 && ok) a.y_scale[row] = amax / kE4m3Max;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (gt + v * kRingThreads) * 8;
            if (c < a.dim && ok) {
#pragma unroll
                for (int j = 0; j < 8; ++j) s[v][j] = s[v][j] * rstd * inv;
                store_vec<8>(a.y, row * a.dim + c, s[v], a.out);
            }
        }
    }
}

template <int IO, int NV>
cudaError_t launch_ring(const NormArgs& a, cudaStream_t s) {
    const int slot_bytes = 2 * a.dim * (IO == KDA_DTYPE_F32 ? 4 : 2), slots = ring_slots(slot_bytes);
    auto kern = kda_norm_ring_kernel<IO, NV>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3((unsigned)device_sm_count()), dim3(kRingAll), (size_t)(slots * slot_bytes), s, a,
                            slots);
}

// Whether a call takes the ring: 16-byte rows long enough for a group of threads
// and many enough for every SM's ring.
template <int IO>
bool ring_fits(const NormArgs& a) {
    return a.r && a.dim > 2048 && a.dim <= 8192 && ring_slots(2 * a.dim * (IO == KDA_DTYPE_F32 ? 4 : 2)) >= kRingGroups &&
           a.rows >= 16 * (int64_t)device_sm_count();
}

// The team for a row of `vecs` vectors.  Four 16-byte loads a thread, whatever
// the row (two vectors of x and two of the residual, or four of x), are in flight
// together and keep the sums short.  Measured, of the 6.67 TB/s that a copy
// reaches: 1.07 M rows of 128 with one vector a thread 5.3 TB/s, with four 6.6;
// 260000 rows of 512 with residual, e4m3, two vectors 6.1, four 5.4; 32768 rows
// of 4096 without residual one vector 4.4, two 5.3, four 6.4, eight 4.8.  Few
// rows leave most SMs idle and take the shortest path instead: one vector a
// thread (one row of 4096: 2.6 us against 3.9).
template <int IO, int VEC>
cudaError_t pick(const NormArgs& a, cudaStream_t s) {
    const int vecs = (a.dim + VEC - 1) / VEC;
    auto threads = [&](int nv) { return (vecs + nv * 32 - 1) / (nv * 32) * 32; };
    if constexpr (VEC == 8) {
        if (ring_fits<IO>(a)) {
            if (a.dim <= 4096) return launch_ring<IO, 4>(a, s);
            return launch_ring<IO, 8>(a, s);
        }
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
        return launch<IO, VEC, 4, 0>(a, threads(4), s);
    } else {
        if (vecs <= 32) return launch<IO, VEC, 4, 8>(a, 256, s);
        if (vecs <= 128) return launch<IO, VEC, 4, 32>(a, 256, s);
        if (vecs <= 512) return launch<IO, VEC, 16, 32>(a, 256, s);
        if (vecs <= 16384) return launch<IO, VEC, 16, 0>(a, threads(16), s);
        return launch<IO, VEC, 32, 0>(a, threads(32), s);
    }
}

// Rows off 16 bytes.  (26000 rows of 5003, residual, e4m3: 466 us element by
// element, 272 in vectors from the boundary before the row.)
template <int IO>
cudaError_t pick_shifted(const NormArgs& a, cudaStream_t s) {
    const int vecs = a.dim / 8 + 2;  // at most
    if (vecs <= 32) return launch<IO, 8, 4, 8, true>(a, 256, s);
    if (vecs <= 128) return launch<IO, 8, 4, 32, true>(a, 256, s);
    if (vecs <= 4096) return launch<IO, 8, 4, 0, true>(a, (vecs + 127) / 128 * 32, s);
    return pick<IO, 1>(a, s);
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
