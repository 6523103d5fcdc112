// decay_states.cu -- the scan of linear attention with a decay per head by
// itself: the states before every chunk, forwards and backwards at once (for the
// gradients), or what each piece of a cut sequence adds to its state; and the
// kernel that joins the pieces.
#include "decay_scan.cuh"

namespace kda {
namespace {

constexpr int kJoinThreads = 256;

// The state that enters each piece of a sequence, from what the pieces before it add (in place of
// that): S <- decay S + total.  One CTA has 1024 elements of one (sequence, head).
__global__ void __launch_bounds__(kJoinThreads) kda_decay_join_kernel(const __grid_constant__ DecayJoinArgs a) {
    __shared__ DecayScratch scratch;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int n = blockIdx.x / a.H, h = blockIdx.x - n * a.H;
    const DecayScanDir& dir = a.dir[blockIdx.z];
    DecayPiece at;
    if (!find_piece<kJoinThreads>(a.seqs, n, true, true, scratch, at) || at.n < 0 || at.pieces < 2) return;
    const int e = (blockIdx.y * kJoinThreads + threadIdx.x) * 4;
    if (e >= a.state) return;
    float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
    const int64_t seq = ((int64_t)n * a.H + h) * a.state + e;
    if (dir.start.p) {
        if (dir.start.b16) {
            const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(dir.start.p) + seq);
            const float2 x = from_b16x2<false>(w.x), y = from_b16x2<false>(w.y);
            S = make_float4(x.x, x.y, y.x, y.y);
        } else {
            S = *reinterpret_cast<const float4*>(static_cast<const float*>(dir.start.p) + seq);
        }
    }
    // Eight pieces' totals are asked for together: one after the other, each would wait for memory.
    constexpr int kBatch = 8;
    auto unit_at = [&](int i) { return (int64_t)(at.piece_base + (dir.reverse ? at.pieces - 1 - i : i)) * a.H + h; };
    for (int i0 = 0; i0 < at.pieces; i0 += kBatch) {
        float4 t[kBatch];
        float d[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (i0 + i + 1 < at.pieces) {
                t[i] = *reinterpret_cast<const float4*>(dir.totals + unit_at(i0 + i) * a.state + e);
                d[i] = dir.decays[unit_at(i0 + i)];
            }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (i0 + i >= at.pieces) break;
            if (i0 + i > 0) *reinterpret_cast<float4*>(dir.totals + unit_at(i0 + i) * a.state + e) = S;
            if (i0 + i + 1 < at.pieces)
                S = make_float4(fmaf(d[i], S.x, t[i].x), fmaf(d[i], S.y, t[i].y), fmaf(d[i], S.z, t[i].z), fmaf(d[i], S.w, t[i].w));
        }
    }
}

}  // namespace

cudaError_t launch_decay_states(const DecayScanArgs& a, int K, int V, bool f16, int dirs, cudaStream_t s) {
    return launch_scan_any<false>(a, K, V, f16, dirs, s);
}

cudaError_t launch_decay_join(const DecayJoinArgs& a, int dirs, cudaStream_t s) {
    const dim3 grid((unsigned)(a.seqs.N * a.H), (unsigned)((a.state + 4 * kJoinThreads - 1) / (4 * kJoinThreads)),
                    (unsigned)dirs);
    return launch_dependent(kda_decay_join_kernel, grid, dim3(kJoinThreads), (size_t)0, s, a);
}

}  // namespace kda
