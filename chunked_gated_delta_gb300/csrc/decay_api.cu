// decay_api.cu -- the C entries of linear attention with a decay per head for
// prompts and their gradients: checks, the plan, the workspace and the launches.
#include "decay.cuh"

namespace kda {
namespace {

// How sequences are cut. The scan walks a piece's chunks one after the other; pieces are worth a pass over k
// and v (what each adds to the state) where uncut sequences leave SMs idle. The model, in measured microseconds: a
// CTA's start and each of its chunks, with output, without, and keeping the states (backward); CTAs in
// rounds of the SMs (packed: their work shared out, and the longest); and the join. It depends on the dims
// alone, as the workspace does.
constexpr int kDecaySMs = 152;
struct PassUs {
    double start, chunk;
};
constexpr PassUs kOutUs{8.0, 3.0}, kTotalsUs{6.0, 2.0}, kKeepUs{7.0, 2.9};
constexpr double kJoinUs = 7.0;
constexpr int kUncut = 1 << 23;   // chunks per piece: more than any sequence has
constexpr int kMostPieces = 64;   // per sequence

struct DecayPlan {
    int32_t N, seg_chunks;
    int64_t pieces;  // bound for packed sequences
    int64_t chunks;  // of 128 tokens, likewise
    bool cut() const { return seg_chunks != kUncut; }
};

DecayPlan decay_plan(const kda_dims& d, bool backward) {
    const bool packed = d.num_seqs > 0;
    const int64_t N = packed ? d.num_seqs : d.B, all = ceil_div(d.T, kDecayChunk);
    // packed lengths are not known here: the longest is taken for twice their mean (as evenly spread ones have it). One that
    // is far longer is walked alone at the end: of 65536 tokens x 32 heads in 16 sequences, one of 64000 makes 361 us 1493.
    const int64_t mean = (all + N - 1) / N, nc = !packed ? all : all < 2 * mean ? all : 2 * mean;
    const int dirs = backward ? 2 : 1;
    const PassUs pass = backward ? kKeepUs : kOutUs;
    const int64_t units = N * d.H * dirs;
    auto pieces_of = [&](int64_t len) { return packed ? all / len + N : N * ((all + len - 1) / len); };
    auto time_of = [&](const PassUs& us, int64_t ctas, int64_t len) {
        if (packed) {
            const double work = (us.start * (double)ctas + us.chunk * (double)(all * d.H * dirs)) / kDecaySMs;
            const double longest = us.start + us.chunk * (double)len;
            return work > longest ? work : longest;
        }
        return (us.start + us.chunk * (double)len) * (double)((ctas + kDecaySMs - 1) / kDecaySMs);
    };
    DecayPlan p{};
    p.N = (int32_t)N;
    p.seg_chunks = kUncut;
    p.chunks = packed ? d.T / kDecayChunk + N : N * all;
    double best = 0.9 * time_of(pass, units, nc);
    for (int64_t S = 2; S <= kMostPieces && 2 * S <= nc; ++S) {
        const int64_t len = (nc + S - 1) / S, n = pieces_of(len) * d.H * dirs;
        const double cost = time_of(kTotalsUs, n - units, len) + time_of(pass, n, len) + kJoinUs;
        if (cost < best) best = cost, p.seg_chunks = (int32_t)len;
    }
    p.pieces = p.cut() ? pieces_of(p.seg_chunks) : N;
    return p;
}

struct DecayWs {
    size_t totals[2], decays[2], kept[2], kept_scale[2], dq32, dk32, dg, dg_part, total;
};
DecayWs decay_ws(const kda_dims& d, const kda_decay_opts& o, const DecayPlan& p, bool backward) {
    DecayWs w{};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + bytes, 1024);
        return at;
    };
    const size_t H = (size_t)d.H, KV = (size_t)d.K * d.V, rows = (size_t)d.B * d.T;
    for (int i = 0; i < (backward ? 2 : 1); ++i) {
        if (p.cut()) {
            w.totals[i] = take((size_t)p.pieces * H * KV * 4);
            w.decays[i] = take((size_t)p.pieces * H * 4);
        }
        if (backward) {
            w.kept[i] = take((size_t)p.chunks * H * KV * 4);
            w.kept_scale[i] = take((size_t)p.chunks * H * 4);
        }
    }
    if (backward && o.qk_heads > 0 && d.H > 2 * o.qk_heads) {
        w.dq32 = take(rows * H * d.K * 4);
        w.dk32 = take(rows * H * d.K * 4);
    }
    if (backward && o.head_gate) {
        w.dg = take(rows * H * 4);
        w.dg_part = take((rows + 255) / 256 * H * 4);
    }
    w.total = off;
    return w;
}

kda_status check_dims_opts(const kda_dims* dims, const kda_decay_opts* opts) {
    if (!dims || !opts) return KDA_ERR_INVALID_ARG;
    const kda_dims& d = *dims;
    if (d.num_seqs < 0 || d.B < 1 || d.T < 0 || d.H < 1 || (d.num_seqs > 0 && d.B != 1)) return KDA_ERR_INVALID_ARG;
    if ((d.K != 64 && d.K != 128) || (d.V != 64 && d.V != 128)) return KDA_ERR_UNSUPPORTED;
    const kda_decay_opts& p = *opts;
    if ((p.io_dtype != KDA_IO_BF16 && p.io_dtype != KDA_IO_F16) ||
        (p.state_dtype != KDA_STATE_F32 && p.state_dtype != KDA_STATE_BF16) || (p.head_gate != 0 && p.head_gate != 1) ||
        p.num_slots != 0 || p.reserved != 0 || p.qk_heads < 0 ||
        (p.qk_heads > 0 && (p.qk_heads > d.H || d.H % p.qk_heads != 0)))
        return KDA_ERR_INVALID_ARG;
    const int64_t rows = (int64_t)d.B * d.T, N = d.num_seqs > 0 ? d.num_seqs : d.B;
    if (rows > INT32_MAX / 2 || (rows / kDecayChunk + N) * (int64_t)d.H > INT32_MAX / 2 ||
        (rows + 255) / 256 * (int64_t)d.H > INT32_MAX)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

struct Strides {
    int64_t q, k, v, g, d_o;
};
kda_status strides_of(const kda_dims& d, const kda_decay_opts& p, bool backward, Strides* s) {
    const int hq = p.qk_heads > 0 ? p.qk_heads : d.H;
    const int64_t wq = (int64_t)hq * d.K, wv = (int64_t)d.H * d.V;
    *s = {p.q_stride ? p.q_stride : wq, p.k_stride ? p.k_stride : wq, p.v_stride ? p.v_stride : wv,
          p.head_gate ? 0 : p.g_stride ? p.g_stride : d.H, p.do_stride ? p.do_stride : wv};
    if (s->q < wq || s->k < wq || s->v < wv || s->d_o < wv || (p.head_gate ? p.g_stride != 0 : s->g < d.H) ||
        (!backward && p.do_stride != 0))
        return KDA_ERR_INVALID_ARG;
    for (int64_t x : {s->q, s->k, s->v, s->d_o})
        if (x % 8 != 0) return KDA_ERR_ALIGNMENT;
    return KDA_OK;
}

bool token_map(CUtensorMap* m, const void* base, int dim, int heads, int64_t rows, int64_t stride, int box_rows = kDecayChunk) {
    if (rows == 0) return true;  // (never read)
    const uint64_t dims[3] = {(uint64_t)dim, (uint64_t)heads, (uint64_t)rows};
    const uint64_t strides[2] = {(uint64_t)dim * 2, (uint64_t)stride * 2};
    const uint32_t box[3] = {64, 1, (uint32_t)box_rows};
    return make_tensormap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// fp32 parts of a group's dq and dk [rows, H, K]: boxes of 32 x 32 rows
bool group_map(CUtensorMap* m, const void* base, int dim, int heads, int64_t rows) {
    if (rows == 0) return true;
    const uint64_t dims[3] = {(uint64_t)dim, (uint64_t)heads, (uint64_t)rows};
    const uint64_t strides[2] = {(uint64_t)dim * 4, (uint64_t)dim * 4 * heads};
    const uint32_t box[3] = {32, 1, 32};
    return make_tensormap(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

DecaySeqs seqs_of(const kda_dims& d, const int32_t* cu, int64_t pieces, int32_t seg_chunks, int32_t N) {
    return DecaySeqs{cu, N, d.T, seg_chunks, (int32_t)pieces, seg_chunks == kUncut};
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" size_t kda_decay_workspace_size(const kda_dims* dims, const kda_decay_opts* opts, int32_t backward) {
    if (check_dims_opts(dims, opts) != KDA_OK || (backward != 0 && backward != 1)) return (size_t)-1;
    return decay_ws(*dims, *opts, decay_plan(*dims, backward), backward).total;
}

extern "C" kda_status kda_decay_fwd(const void* q, const void* k, const void* v, const float* g, float scale,
                                    const void* h0, const int32_t* cu_seqlens, void* o, void* ht, const kda_dims* dims,
                                    const kda_decay_opts* opts, int32_t* status_word, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    kda_status st = check_dims_opts(dims, opts);
    if (st != KDA_OK) return st;
    const kda_dims& d = *dims;
    if ((cu_seqlens != nullptr) != (d.num_seqs > 0)) return KDA_ERR_INVALID_ARG;
    Strides sd;
    if ((st = strides_of(d, *opts, false, &sd)) != KDA_OK) return st;
    const int64_t rows = (int64_t)d.B * d.T;
    if (rows > 0 && (!q || !k || !v || !g || !o)) return KDA_ERR_INVALID_ARG;
    if (h0 && h0 == ht) return KDA_ERR_INVALID_ARG;  // (pieces of one sequence read and write them in any order)
    for (const void* p : {q, k, v, h0, static_cast<const void*>(o), static_cast<const void*>(ht)})
        if (!is_aligned(p, 16)) return KDA_ERR_ALIGNMENT;
    if (!is_aligned(g, 4) || !is_aligned(cu_seqlens, 4) || !is_aligned(status_word, 4)) return KDA_ERR_ALIGNMENT;
    const DecayPlan plan = decay_plan(d, false);
    const DecayWs ws = decay_ws(d, *opts, plan, false);
    if (ws.total > 0 && (!workspace || !is_aligned(workspace, 256) || workspace_bytes < ws.total)) return KDA_ERR_WORKSPACE;
    if (rows == 0 && !ht) return KDA_OK;
    const int hq = opts->qk_heads > 0 ? opts->qk_heads : d.H;
    const bool f16 = opts->io_dtype == KDA_IO_F16;
    DecayScanArgs a{};
    if (!token_map(&a.dir[0].tm_x, k, d.K, hq, rows, sd.k) || !token_map(&a.dir[0].tm_y, v, d.V, d.H, rows, sd.v) ||
        !token_map(&a.tm_q, q, d.K, hq, rows, sd.q) || !token_map(&a.tm_o, o, d.V, d.H, rows, (int64_t)d.H * d.V, 32))
        return KDA_ERR_CUDA;
    const int32_t b16 = opts->state_dtype == KDA_STATE_BF16;
    a.dir[0].start = {const_cast<void*>(h0), b16};
    a.dir[0].end = {ht, b16};
    uint8_t* w = static_cast<uint8_t*>(workspace);
    if (plan.cut()) {
        a.dir[0].totals = reinterpret_cast<float*>(w + ws.totals[0]);
        a.dir[0].decays = reinterpret_cast<float*>(w + ws.decays[0]);
    }
    a.dir[0].weight = 1.f;
    a.seqs = seqs_of(d, cu_seqlens, plan.pieces, plan.seg_chunks, plan.N);
    a.g = g;
    a.g_stride = sd.g;
    a.o = static_cast<uint16_t*>(o);
    a.status = status_word;
    a.scale = scale;
    a.H = d.H;
    a.group = d.H / hq;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (plan.cut()) {
        a.totals_only = 1;
        e = launch_decay_states(a, d.K, d.V, f16, 1, s);
        a.totals_only = 0;
        DecayJoinArgs j{{a.dir[0], a.dir[1]}, a.seqs, d.H, d.K * d.V};
        if (e == cudaSuccess) e = launch_decay_join(j, 1, s);
    }
    if (e == cudaSuccess) e = launch_decay_out(a, d.K, d.V, f16, s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status kda_decay_bwd(const void* q, const void* k, const void* v, const float* g, const void* d_o,
                                    float scale, const void* h0, const void* dht, const int32_t* cu_seqlens, void* dq,
                                    void* dk, void* dv, float* dg, void* dh0, const kda_dims* dims,
                                    const kda_decay_opts* opts, int32_t* status_word, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    kda_status st = check_dims_opts(dims, opts);
    if (st != KDA_OK) return st;
    const kda_dims& d = *dims;
    if ((cu_seqlens != nullptr) != (d.num_seqs > 0)) return KDA_ERR_INVALID_ARG;
    Strides sd;
    if ((st = strides_of(d, *opts, true, &sd)) != KDA_OK) return st;
    const int64_t rows = (int64_t)d.B * d.T;
    if (rows > 0 && (!q || !k || !v || !g || !d_o || !dq || !dk || !dv || !dg)) return KDA_ERR_INVALID_ARG;
    if ((opts->head_gate && !dg) || (dh0 && (dh0 == h0 || dh0 == dht))) return KDA_ERR_INVALID_ARG;
    for (const void* p : {q, k, v, d_o, h0, dht, static_cast<const void*>(dq), static_cast<const void*>(dk),
                          static_cast<const void*>(dv), static_cast<const void*>(dh0)})
        if (!is_aligned(p, 16)) return KDA_ERR_ALIGNMENT;
    if (!is_aligned(g, 4) || !is_aligned(dg, 4) || !is_aligned(cu_seqlens, 4) || !is_aligned(status_word, 4))
        return KDA_ERR_ALIGNMENT;
    const DecayPlan plan = decay_plan(d, true);
    const DecayWs ws = decay_ws(d, *opts, plan, true);
    if (ws.total > 0 && (!workspace || !is_aligned(workspace, 256) || workspace_bytes < ws.total)) return KDA_ERR_WORKSPACE;
    const int hq = opts->qk_heads > 0 ? opts->qk_heads : d.H;
    const bool f16 = opts->io_dtype == KDA_IO_F16, paired = d.H == 2 * hq, parts = d.H > 2 * hq;
    DecayGradArgs a{};
    if (!token_map(&a.tm_q, q, d.K, hq, rows, sd.q) || !token_map(&a.tm_k, k, d.K, hq, rows, sd.k) ||
        !token_map(&a.tm_v, v, d.V, d.H, rows, sd.v) || !token_map(&a.tm_do, d_o, d.V, d.H, rows, sd.d_o) ||
        (!parts && (!token_map(&a.tm_dq, dq, d.K, hq, rows, (int64_t)hq * d.K, 32) ||
                    !token_map(&a.tm_dk, dk, d.K, hq, rows, (int64_t)hq * d.K, 32))) ||
        (parts && (!group_map(&a.tm_dq, static_cast<uint8_t*>(workspace) + ws.dq32, d.K, d.H, rows) ||
                   !group_map(&a.tm_dk, static_cast<uint8_t*>(workspace) + ws.dk32, d.K, d.H, rows))) ||
        !token_map(&a.tm_dv, dv, d.V, d.H, rows, (int64_t)d.H * d.V, 32))
        return KDA_ERR_CUDA;
    DecayScanArgs c{};
    const int32_t b16 = opts->state_dtype == KDA_STATE_BF16;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    for (int i = 0; i < 2; ++i) {
        DecayScanDir& r = c.dir[i];
        r.tm_x = i ? a.tm_q : a.tm_k;
        r.tm_y = i ? a.tm_do : a.tm_v;
        r.start = {const_cast<void*>(i ? dht : h0), b16};
        r.end = {i ? dh0 : nullptr, b16};
        if (plan.cut()) {
            r.totals = reinterpret_cast<float*>(w + ws.totals[i]);
            r.decays = reinterpret_cast<float*>(w + ws.decays[i]);
        }
        r.kept = w + ws.kept[i];
        r.kept_scale = reinterpret_cast<float*>(w + ws.kept_scale[i]);
        r.weight = i ? scale : 1.f;
        r.reverse = i;
    }
    c.seqs = seqs_of(d, cu_seqlens, plan.pieces, plan.seg_chunks, plan.N);
    c.g = g;
    c.g_stride = sd.g;
    c.status = status_word;
    c.scale = scale;
    c.H = d.H;
    c.group = d.H / hq;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (plan.cut()) {
        DecayScanArgs t = c;
        t.totals_only = 1;
        t.dir[0].kept = t.dir[1].kept = nullptr;
        e = launch_decay_states(t, d.K, d.V, f16, 2, s);
        DecayJoinArgs j{{c.dir[0], c.dir[1]}, c.seqs, d.H, d.K * d.V};
        if (e == cudaSuccess) e = launch_decay_join(j, 2, s);
    }
    if (e == cudaSuccess) e = launch_decay_states(c, d.K, d.V, f16, 2, s);
    if (rows > 0) {
        a.seqs = seqs_of(d, cu_seqlens, plan.chunks, 1, plan.N);
        a.g = g;
        a.g_stride = sd.g;
        a.kept = c.dir[0].kept;
        a.dkept = c.dir[1].kept;
        a.kept_scale = c.dir[0].kept_scale;
        a.dkept_scale = c.dir[1].kept_scale;
        a.dq = parts ? static_cast<void*>(w + ws.dq32) : dq;
        a.dk = parts ? static_cast<void*>(w + ws.dk32) : dk;
        a.dv = static_cast<uint16_t*>(dv);
        a.dg = opts->head_gate ? reinterpret_cast<float*>(w + ws.dg) : dg;
        a.status = status_word;
        a.scale = scale;
        a.H = d.H;
        a.group = d.H / hq;
        a.sms = device_sm_count();
        a.paired = paired;
        if (e == cudaSuccess) e = launch_decay_grads(a, d.K, d.V, f16, s);
        if (e == cudaSuccess && parts)
            e = launch_decay_group(static_cast<const float*>(a.dq), static_cast<const float*>(a.dk), dq, dk, c.seqs, rows, hq,
                                   d.K, a.group, f16, device_sm_count(), s);
    }
    if (e == cudaSuccess && opts->head_gate)
        e = launch_decay_gate(a.dg, reinterpret_cast<float*>(w + ws.dg_part), dg, c.seqs, rows, d.H, s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
