// layer_ops.cuh -- what the kernels around the recurrence share (the decode
// step, the RMS norm, the projection): element types and their conversions to
// and from fp32, warp sums, and the status bits they add.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/kda.h"
#include "common.cuh"

namespace kda {

// Status bit of kda_step (beside those of common.cuh).
constexpr int kStatusBadSlots = 4;

inline bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int dtype_bytes(int dtype) { return dtype == KDA_DTYPE_F32 ? 4 : dtype == KDA_DTYPE_E4M3 ? 1 : 2; }

namespace {

// fp32 -> two e4m3 codes (lo in the low byte), to nearest even, saturating at +-448.
__device__ __forceinline__ uint16_t pack_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
    return (uint32_t)pack_e4m3x2(a, b) | ((uint32_t)pack_e4m3x2(c, d) << 16);
}
__device__ __forceinline__ uint32_t pack_b16x2(float lo, float hi, bool f16) {
    uint32_t r;
    if (f16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint16_t to_b16(float x, bool f16) {
    return f16 ? __half_as_ushort(__float2half_rn(x)) : __bfloat16_as_ushort(__float2bfloat16_rn(x));
}
template <bool F16>
__device__ __forceinline__ float from_b16(uint16_t w) {
    if constexpr (F16) return __half2float(__ushort_as_half(w));
    else return __uint_as_float((uint32_t)w << 16);
}
template <bool F16>
__device__ __forceinline__ float2 from_b16x2(uint32_t w) {
    return make_float2(from_b16<F16>((uint16_t)(w & 0xFFFFu)), from_b16<F16>((uint16_t)(w >> 16)));
}
// max that returns NaN if either is NaN (fmaxf would drop it)
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

}  // namespace
}  // namespace kda
