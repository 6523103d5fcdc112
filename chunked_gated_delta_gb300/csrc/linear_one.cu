// linear_one.cu -- the kernel of kda_linear for one token.
//
// Such a call reads w once (N K elements) for 2 N K flops: it is bound by HBM,
// and the tensor-core kernels' fixed parts (tensor maps, TMEM, a ring to fill, a
// cluster to join) are a third of its time.  Here the CUDA cores do the products
// in fp32.  A warp has four rows of w and a share of k: each lane loads 16 bytes
// of every row and of the token at the same k, so the token's elements are
// converted once for four rows, and two such chunks a lane are in flight (with
// four, a CTA's registers would leave room for one CTA on an SM instead of two).
// The 16 warps of a CTA are 1, 2 or 4 groups of rows times 16, 8 or 4 shares of
// k (fewer rows where N is small, to have CTAs for every SM); the shares are
// joined through shared memory in order.
//
// Measured over weights that L2 does not hold (bf16; the tensor-core kernel in
// brackets): 4096 x 4096 7.2 us (9.1), 4.7 TB/s, and 6.6 us a call where a part
// of w is still in L2; 2048 x 2048 2.6 (4.8); 32 x 4096 2.3 (4.3).  In e4m3 4096 x
// 4096 takes 5.7 us: half the bytes, and as many conversions and products.  For
// two tokens the same scheme took 10.8 us against 9.1, so it ends at one.
#include "linear.cuh"

namespace kda {
namespace {

constexpr int kOneWarps = 16, kOneThreads = kOneWarps * 32;
constexpr int kRowsPerWarp = 4;
constexpr int kInFlight = 2;  // chunks of a lane

struct OneArgs {
    LinArgs a;  // (no tensor maps)
    const uint8_t *x, *w;
    int64_t ldw;       // bytes between rows of w
    int K, groups;     // groups of rows in a CTA
};

// 16 bytes as fp32.
template <int IO>
struct Chunk {
    static constexpr int kElems = IO == KDA_DTYPE_E4M3 ? 16 : 8;
    static constexpr int kBytes = IO == KDA_DTYPE_E4M3 ? 1 : 2;
    static __device__ __forceinline__ void open(const uint4& u, float (&f)[kElems]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (IO == KDA_DTYPE_E4M3) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t h;
                    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w[i] >> (16 * j))));
                    const float2 v = from_b16x2<true>(h);
                    f[4 * i + 2 * j] = v.x;
                    f[4 * i + 2 * j + 1] = v.y;
                }
            } else {
                const float2 v = from_b16x2<IO == KDA_DTYPE_F16>(w[i]);
                f[2 * i] = v.x;
                f[2 * i + 1] = v.y;
            }
        }
    }
    // the first `live` elements of the chunk at p, the others zero
    static __device__ __forceinline__ uint4 part(const uint8_t* p, int live) {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        for (int i = 0; i < live; ++i) {
            const uint32_t e = kBytes == 1 ? (uint32_t)p[i] : (uint32_t) reinterpret_cast<const uint16_t*>(p)[i];
            const int at = i * kBytes;
            const uint32_t v = e << (8 * (at & 3));
            if (at < 4) w[0] |= v;
            else if (at < 8) w[1] |= v;
            else if (at < 12) w[2] |= v;
            else w[3] |= v;
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <int IO>
__global__ void __launch_bounds__(kOneThreads, 2) kda_linear_one_kernel(const OneArgs p) {
    using C = Chunk<IO>;
    __shared__ float s_part[kOneWarps][kRowsPerWarp];
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const LinArgs& a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = warp % p.groups, share = warp / p.groups, shares = kOneWarps / p.groups;
    const int row0 = (int)(blockIdx.x * p.groups + group) * kRowsPerWarp;
    const uint8_t* w[kRowsPerWarp];
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) w[r] = p.w + (int64_t)min(row0 + r, a.N - 1) * p.ldw;
    const uint8_t* x = p.x;

    float acc[kRowsPerWarp] = {};
    auto add = [&](const uint4 (&wu)[kRowsPerWarp], const uint4& xu) {
        float xf[C::kElems];
        C::open(xu, xf);
#pragma unroll
        for (int r = 0; r < kRowsPerWarp; ++r) {
            float wf[C::kElems];
            C::open(wu[r], wf);
#pragma unroll
            for (int e = 0; e < C::kElems; ++e) acc[r] = fmaf(wf[e], xf[e], acc[r]);
        }
    };

    const int chunks = p.K / C::kElems, step = shares * 32;
    int c = share * 32 + lane;
    for (; c + (kInFlight - 1) * step < chunks; c += kInFlight * step) {
        uint4 wu[kInFlight][kRowsPerWarp], xu[kInFlight];
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            const int64_t at = (int64_t)(c + i * step) * 16;
#pragma unroll
            for (int r = 0; r < kRowsPerWarp; ++r) wu[i][r] = *reinterpret_cast<const uint4*>(w[r] + at);
            xu[i] = *reinterpret_cast<const uint4*>(x + at);
        }
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) add(wu[i], xu[i]);
    }
    for (; c < chunks; c += step) {
        const int64_t at = (int64_t)c * 16;
        uint4 wu[kRowsPerWarp];
#pragma unroll
        for (int r = 0; r < kRowsPerWarp; ++r) wu[r] = *reinterpret_cast<const uint4*>(w[r] + at);
        add(wu, *reinterpret_cast<const uint4*>(x + at));
    }
    const int rest = p.K - chunks * C::kElems;
    if (rest > 0 && c == chunks) {  // the one lane whose next chunk is the broken one
        const int64_t at = (int64_t)c * 16;
        uint4 wu[kRowsPerWarp];
#pragma unroll
        for (int r = 0; r < kRowsPerWarp; ++r) wu[r] = C::part(w[r] + at, rest);
        add(wu, C::part(x + at, rest));
    }

#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
        float v = acc[r];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(~0u, v, off);
        if (lane == 0) s_part[warp][r] = v;
    }
    __syncthreads();
    const int rows = p.groups * kRowsPerWarp, n = (int)blockIdx.x * rows + tid;
    if (tid < rows && n < a.N) {
        float v = 0.f;
        for (int s = 0; s < shares; ++s) v += s_part[s * p.groups + tid / kRowsPerWarp][tid % kRowsPerWarp];
        if (IO == KDA_DTYPE_E4M3) v *= a.x_scale[0] * a.w_scale[n];
        if (a.bias) v += a.bias[n];
        if (a.out == KDA_DTYPE_F32) activate_all<1, false>(&v, a.act);
        else activate_all<1, true>(&v, a.act);
        if (a.residual) v += load_out(a.residual, n, a.out);
        store_out(a.y, n, v, a.out);
    }
}

}  // namespace

cudaError_t launch_linear_one(const LinArgs& a, const void* x, const void* w, int64_t K, int64_t ldw, cudaStream_t s) {
    OneArgs p{};
    p.a = a;
    p.x = static_cast<const uint8_t*>(x);
    p.w = static_cast<const uint8_t*>(w);
    p.ldw = ldw * dtype_bytes(a.io);
    p.K = (int)K;
    const int64_t quads = ((int64_t)a.N + kRowsPerWarp - 1) / kRowsPerWarp;
    p.groups = quads >= 4 * device_sm_count() ? 4 : quads >= 2 * device_sm_count() ? 2 : 1;
    const unsigned grid = (unsigned)((quads + p.groups - 1) / p.groups);
    auto kern = a.io == KDA_DTYPE_E4M3   ? kda_linear_one_kernel<KDA_DTYPE_E4M3>
                : a.io == KDA_DTYPE_BF16 ? kda_linear_one_kernel<KDA_DTYPE_BF16>
                                         : kda_linear_one_kernel<KDA_DTYPE_F16>;
    return launch_dependent(kern, dim3(grid), dim3(kOneThreads), 0, s, p);
}

}  // namespace kda
