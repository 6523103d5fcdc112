// linear.cuh -- what the kernels of kda_linear share (linear_one.cu: one token;
// linear.cu: few tokens; linear_wide.cu: many): arguments,
// cluster and tcgen05 wrappers, the activations.
#pragma once
#include <cuda.h>

#include "internal.h"
#include "layer_ops.cuh"
#include "ptx.cuh"
#include "tensormap.h"
#include "waits.cuh"

namespace kda {

constexpr int kRowBytes = 128;  // bytes of k per stage: 64 16-bit or 128 8-bit elements
constexpr int kSmemMax = 227 * 1024;

struct LinArgs {
    CUtensorMap tm_w, tm_x;  // 2-D {k, rows}
    const float* bias;       // or null
    const void* residual;    // out type, or null
    const float *x_scale, *w_scale;  // e4m3 only
    void* y;
    int32_t* status;         // or null
    int64_t ldr, ldy;        // elements between rows
    int M, N, kblocks;
    uint32_t idesc;
    int out, act, io;
    int wide;  // rows of y and residual take loads and stores of four elements
};

// The kernel for one token (linear_one.cu).
cudaError_t launch_linear_one(const LinArgs& a, const void* x, const void* w, int64_t K, int64_t ldw, cudaStream_t s);
// The kernel for many tokens (linear_wide.cu), tn features (128 or 256) a tile.
// tm_w, tm_x and idesc are set there; x, w are the operands and ldx, ldw their
// row strides; rows_on_16: all rows of y and the residual start on 16 bytes.
cudaError_t launch_linear_wide(const LinArgs& a, int tn, const void* x, const void* w, int64_t K, int64_t ldx,
                               int64_t ldw, bool rows_on_16, cudaStream_t s);

// launch_dependent (internal.h) with a cluster of `size` CTAs along x.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_cluster(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, unsigned size,
                                  cudaStream_t stream, const Args&... args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = size;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

namespace {

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], "
        "%1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Instruction descriptor with e4m3 A and B (format 0), fp32 D, both K-major.
constexpr uint32_t idesc_e4m3_f32(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_smem(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// exp(-|v|) to about 2^-22: 2^t with t = -|v| log2 e in fp32, times one plus what
// that product lost (its rounding and the rest of log2 e) times ln 2.  Below
// 2^-126 (|v| > 87.3) it is zero.  With `back`, exp(-|v|) is the result times
// *back, 2^-64 where t < -64 (adding 64 to such a t is exact), so a product with
// it can be right where exp(-|v|) by itself is too small.
__device__ __forceinline__ float exp_minus_abs(float v, float* back = nullptr) {
    constexpr float kLog2e = 1.44269504f, kLog2eRest = (float)(1.4426950408889634 - (double)kLog2e), kLn2 = 0.693147181f;
    const float x = fmaxf(-fabsf(v), -200.f);
    float t = x * kLog2e;
    const float lost = fmaf(x, kLog2eRest, fmaf(x, kLog2e, -t));
    if (back) {
        const bool deep = t < -64.f;
        *back = deep ? 0x1p-64f : 1.f;
        t = deep ? t + 64.f : t;
    }
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    return fmaf(e * kLn2, lost, e);
}
// FAST: y has 16 bits, whose rounding (2^-9 or 2^-12) hides the approximate
// exponential's error, which grows with |v|; SiLU below v = -87 (1e-36 in size)
// is zero then.  Else SiLU, sigmoid and log-sigmoid are within about 2^-21 of
// themselves (and zero below 2^-126 at the latest), GELU within 2^-22 |v|, as
// 1 + erf gives it: all the epilogue's threads do this for every element, so the
// library's exact forms would hold up the tiles behind.
template <int ACT, bool FAST>
__device__ __forceinline__ float activated(float v) {
    if constexpr (ACT == KDA_ACT_GELU) return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
    if constexpr (ACT == KDA_ACT_SILU || ACT == KDA_ACT_SIGMOID) {
        if constexpr (FAST) return __fdividef(ACT == KDA_ACT_SILU ? v : 1.f, 1.f + __expf(-v));
        float y;
        if constexpr (ACT == KDA_ACT_SILU) {  // v exp(v) is a normal number down to -92, exp(v) to -87
            float back;
            const float e = exp_minus_abs(v, &back);
            y = __fdividef(v < 0.f ? v * e : v, fmaf(e, back, 1.f)) * (v < 0.f ? back : 1.f);
        } else {
            const float e = exp_minus_abs(v);
            y = __fdividef(v < 0.f ? e : 1.f, 1.f + e);
        }
        return v == v ? y : v;
    }
    if constexpr (ACT == KDA_ACT_LOGSIGMOID) {
        // min(v, 0) - log(1 + e), e = exp(-|v|): log(1 + e) = 2 artanh(s) with s = e / (2 + e) <= 1/3, and
        // artanh(s) = s (1 + z p(z)), z = s^2, with p fitted to sum z^k / (2 k + 3) on [0, 1/9] (to 5e-9 of z p)
        const float e = FAST ? __expf(-fabsf(v)) : exp_minus_abs(v);
        const float s = __fdividef(e, 2.f + e), z = s * s;
        float p = 0.14012229f;
        p = fmaf(p, z, 0.13999571f);
        p = fmaf(p, z, 0.2001085f);
        p = fmaf(p, z, 0.33333207f);
        return (v > 0.f ? 0.f : v) - 2.f * fmaf(s * z, p, s);
    }
    return v;
}
template <int ACT, int COUNT, bool FAST>
__device__ __forceinline__ void activated_all(float* v) {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) v[i] = activated<ACT, FAST>(v[i]);
}
// One branch for all of a thread's values.
template <int COUNT, bool FAST>
__device__ __forceinline__ void activate_all(float* v, int act) {
    switch (act) {
    case KDA_ACT_SILU: activated_all<KDA_ACT_SILU, COUNT, FAST>(v); break;
    case KDA_ACT_GELU: activated_all<KDA_ACT_GELU, COUNT, FAST>(v); break;
    case KDA_ACT_SIGMOID: activated_all<KDA_ACT_SIGMOID, COUNT, FAST>(v); break;
    case KDA_ACT_LOGSIGMOID: activated_all<KDA_ACT_LOGSIGMOID, COUNT, FAST>(v); break;
    }
}
__device__ __forceinline__ float load_out(const void* p, int64_t at, int dtype) {
    if (dtype == KDA_DTYPE_F32) return static_cast<const float*>(p)[at];
    const uint16_t w = static_cast<const uint16_t*>(p)[at];
    return dtype == KDA_DTYPE_F16 ? from_b16<true>(w) : from_b16<false>(w);
}
// Four elements as they lie in memory (16-bit ones in x and y).
__device__ __forceinline__ uint4 load_four(const void* p, int64_t at, int dtype) {
    if (dtype == KDA_DTYPE_F32) return *reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at);
    return make_uint4(u.x, u.y, 0u, 0u);
}
__device__ __forceinline__ void store_out(void* p, int64_t at, float v, int dtype) {
    if (dtype == KDA_DTYPE_F32) static_cast<float*>(p)[at] = v;
    else static_cast<uint16_t*>(p)[at] = to_b16(v, dtype == KDA_DTYPE_F16);
}

inline bool rows_map(CUtensorMap* m, int io, const void* base, int64_t rows, int64_t k, int64_t ld, int box_rows) {
    const int es = dtype_bytes(io);
    const uint64_t dims[2] = {(uint64_t)k, (uint64_t)rows};
    const uint64_t strides[1] = {(uint64_t)ld * es};
    const uint32_t box[2] = {(uint32_t)(kRowBytes / es), (uint32_t)box_rows};
    const CUtensorMapDataType dt = io == KDA_DTYPE_E4M3  ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : io == KDA_DTYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                         : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return make_tensormap(m, dt, 2, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace
}  // namespace kda
