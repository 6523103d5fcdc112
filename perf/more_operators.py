"""Linear attention with one decay per head, as measured cases.

The operators of a layer whose state decays by one factor per head and token
(instead of one per key dimension, and without the delta rule), each in a plain
form (elementary torch operations in 32 bits, sums of logarithms in 64, rounded
once at the end) and as the framework's own call:

* fwd:    S_t = exp(g_t) S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t  over whole
          prompts, with the state before and after them;
* bwd:    its gradients: of q, k, v, g and of the state before the prompt;
* step:   the same recurrence for one or a few new tokens per request, on a
          cache of states addressed by slot, updated in place;
* rotary: the positions of q and k: pairs of a head's elements turned by
          position x frequency, in both layouts, on part of the head, with the
          frequencies scaled for long contexts; and the inverse turn (gradients).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CHUNK = 128  # tokens that the plain form takes together


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one short prompt of a server that answers at once: 16 heads, an odd length, nothing before it
        dict(name="fwd short prompt", op="fwd", N=1, T=509, packed=False, heads=16, qk_heads=16, K=128, V=128,
             io="bf16", state="f32", h0=False, gate="token", mean=3.0),
        # the framework's middle workload: one sequence of 4096 tokens with a state before it; a fixed decay per head
        dict(name="fwd one sequence", op="fwd", N=1, T=4096, packed=False, heads=16, qk_heads=16, K=128, V=128,
             io="f16", state="f32", h0=True, gate="head", mean=3.0),
        # the framework's headline workload: prefill (or a training step's forward) of 4 x 8192 tokens, 32 heads
        dict(name="fwd prefill", op="fwd", N=4, T=8192, packed=False, heads=32, qk_heads=32, K=128, V=128,
             io="bf16", state="f32", h0=True, gate="token", mean=3.0),
        # 16 prompts packed in one row, lengths over 1 .. 8192, two value heads to a query head
        dict(name="fwd packed", op="fwd", N=16, T=8192, packed=True, heads=32, qk_heads=16, K=128, V=128,
             io="bf16", state="f32", h0=True, gate="token", mean=5.0),
        # a small model's training step on short ragged rows: 64-wide keys, fp16
        dict(name="bwd short rows", op="bwd", N=2, T=777, packed=False, heads=8, qk_heads=8, K=64, V=128,
             io="f16", state="f32", h0=False, gate="token", mean=3.0),
        # training on packed documents with grouped heads and states carried over
        dict(name="bwd packed", op="bwd", N=7, T=4096, packed=True, heads=16, qk_heads=8, K=128, V=128,
             io="bf16", state="f32", h0=True, gate="token", mean=5.0),
        # a training step at the headline shape
        dict(name="bwd training", op="bwd", N=4, T=8192, packed=False, heads=32, qk_heads=32, K=128, V=128,
             io="bf16", state="f32", h0=True, gate="token", mean=3.0),
        # one request, one token: the latency of a decode step
        dict(name="step one request", op="step", N=1, T=1, pad=0, slots=8, packed=False, heads=32, qk_heads=32,
             K=128, V=128, io="bf16", state="f32", gate="token", mean=3.0),
        # checking drafted tokens: 0 to 5 per request, packed, grouped heads, 16-bit states
        dict(name="step drafts", op="step", N=96, T=5, pad=0, slots=101, packed=True, heads=32, qk_heads=16,
             K=128, V=64, io="f16", state="bf16", gate="token", mean=3.0),
        # a full server: 512 requests, 1.07 GB of states read and written, a fixed decay per head
        dict(name="step full server", op="step", N=512, T=1, pad=5, slots=512, packed=False, heads=32, qk_heads=32,
             K=128, V=128, io="bf16", state="f32", gate="head", mean=3.0),
        # the positions of a decode batch far into long contexts, half of each head
        dict(name="rotary decode", op="rotary", B=59, T=1, heads=32, qk_heads=8, dim=128, part=64, io="bf16",
             interleaved=False, scaling="yarn", factor=32.0, base=1e6, far=1000000, inverse=False, extra=0),
        # the positions of 32768 tokens in prefill, pairs next to each other, out of a wider projection's rows
        dict(name="rotary prefill", op="rotary", B=4, T=8192, heads=32, qk_heads=32, dim=128, part=128, io="bf16",
             interleaved=True, scaling="linear", factor=4.0, base=1e4, far=100000, inverse=False, extra=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("fwd", "fwd", "bwd", "bwd", "step", "rotary"))
    if op == "rotary":
        dim = rng.choice((64, 96, 128, 128, 256, 2 * _log(rng, 8, 128)))
        heads, qk = rng.choice(((32, 32), (32, 8), (16, 16), (8, 1), (3, 3)))
        B, T = rng.choice(((1, 1), (_log(rng, 2, 512), 1), (_log(rng, 1, 4), _log(rng, 2, 8192))))
        part = rng.choice((dim, dim, 2 * max(1, dim // 4), 2 * rng.randint(1, dim // 2)))
        return dict(op=op, B=B, T=T, heads=heads, qk_heads=qk, dim=dim, part=part,
                    io=rng.choice(("bf16", "bf16", "f16", "f32")) if B * T <= 8192 else rng.choice(("bf16", "f16")),
                    interleaved=rng.random() < 0.5, scaling=rng.choice(("none", "linear", "ntk", "yarn")),
                    factor=rng.choice((2.0, 8.0, 32.0)), base=rng.choice((1e4, 5e5, 1e6)),
                    far=rng.choice((0, 4096, 1000000)), inverse=rng.random() < 0.3, extra=rng.choice((0, 0, 24, 128)))
    K, V = rng.choice((64, 128, 128)), rng.choice((64, 128, 128))
    qk_heads = rng.choice((1, 2, 3, 8, 16, 32))
    heads = qk_heads * rng.choice((1, 2, 4)) if qk_heads <= 8 else qk_heads * rng.choice((1, 32 // qk_heads))
    gate, mean = rng.choice(("token", "token", "head")), rng.choice((1.0, 3.0, 5.0))
    io = rng.choice(("bf16", "bf16", "f16"))
    if op == "step":
        T = rng.choice((1, 1, 2, 3, 5, 8))
        N = _log(rng, 1, max(1, 512 // T))
        return dict(op=op, N=N, T=T, pad=rng.randint(0, N // 4), slots=N + rng.randint(0, 9),
                    packed=T > 1 and rng.random() < 0.6, heads=heads, qk_heads=qk_heads, K=K, V=V, io=io,
                    state=rng.choice(("f32", "f32", "bf16")), gate=gate, mean=mean)
    T = _log(rng, 1, 32768)
    N = _log(rng, 1, max(1, min(16, (4 * 8192 * 32) // (T * heads))))
    return dict(op=op, N=N, T=T, packed=rng.random() < 0.4, heads=heads, qk_heads=qk_heads, K=K, V=V, io=io,
                state=rng.choice(("f32", "f32", "bf16")), h0=rng.random() < 0.6, gate=gate, mean=mean)


# ------------------------------------------------------------------ inputs
def _lengths(case, seed):
    """Tokens of each sequence: T each, or (packed) spread evenly over 1 .. T (a step: 0 .. T), in an order of the seed's."""
    N, T = case["N"], case["T"]
    if not case["packed"]:
        return [T] * N
    order = torch.randperm(N, generator=torch.Generator().manual_seed(1000003 * seed + 17)).tolist()
    if case["op"] == "step":
        return [(T + i) % (T + 1) for i in order]
    return [max(1, T * (2 * i + 1) // (2 * N)) for i in order]


def _frequencies(case):
    """Angle per position of each pair, in 64 bits, and the factor of the cosines and sines."""
    R, base, f = case["part"], case["base"], case["factor"]
    pair = torch.arange(R // 2, dtype=torch.float64)
    if case["scaling"] == "ntk":  # a larger base: the slowest pair is slowed down by the factor, the fastest is kept
        return (base * f ** (R / (R - 2)) if R > 2 else base) ** (-2.0 * pair / R), 1.0
    freq = base ** (-2.0 * pair / R)
    if case["scaling"] == "linear":
        return freq / f, 1.0
    if case["scaling"] == "yarn":  # pairs that turn often over 4096 positions are kept, those that turn seldom slowed down
        def at(turns):
            return R * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), R - 1)
        slow = ((pair - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
        return freq * (1.0 - slow) + freq / f * slow, 0.1 * math.log(f) + 1.0
    return freq, 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    s = dict(case=dict(case))
    io = DTYPES[case["io"]]
    if case["op"] == "rotary":
        B, T, D = case["B"], case["T"], case["dim"]

        def rows(heads):
            return randn(B, T, heads * D + case["extra"]).to(io)[..., : heads * D].unflatten(-1, (heads, D))

        first = torch.randint(0, case["far"] + 1, (B, 1), generator=gen, device="cuda")
        s.update(q=rows(case["heads"]), k=rows(case["qk_heads"]), positions=first + torch.arange(T, device="cuda"))
        s["freq"], s["amplitude"] = _frequencies(case)
        s["freq"] = s["freq"].cuda()
        return s
    H, Hq, K, V, N = case["heads"], case["qk_heads"], case["K"], case["V"], case["N"]
    lens = _lengths(case, seed)
    B, T = (1, sum(lens)) if case["packed"] else (N, case["T"])

    def unit(x):
        return (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-12)).to(io)

    gate = randn(H) if case["gate"] == "head" else randn(B, T, H)
    s.update(q=unit(randn(B, T, Hq, K)), k=unit(randn(B, T, Hq, K)), v=randn(B, T, H, V).to(io),
             g=torch.nn.functional.logsigmoid(gate + case["mean"]), cu=None, lens=lens)
    if case["packed"]:
        s["cu"] = torch.tensor([0] + lens).cumsum(0).to(device="cuda", dtype=torch.int32)
    if case["op"] == "step":
        order = torch.randperm(case["slots"], generator=gen, device="cuda")[:N].to(torch.int32)
        if case["pad"]:
            order[N - case["pad"]:] = -1  # padding of the batch: no state, o is zero
        s.update(state=(0.1 * randn(case["slots"], H, K, V)).to(DTYPES[case["state"]]), slots=order,
                 live=N - case["pad"])
        return s
    state = DTYPES[case["state"]]
    s["h0"] = (0.1 * randn(N, H, K, V)).to(state) if case["h0"] else None
    if case["op"] == "bwd":
        s["do"], s["dht"] = randn(B, T, H, V).to(io), (0.1 * randn(N, H, K, V)).to(state)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if op == "fwd":
        return _own_fwd(s) if own else _plain_fwd(s)
    if op == "bwd":
        return _own_bwd(s) if own else _plain_bwd(s)
    if op == "step":
        return _own_step(s) if own else _plain_step(s)
    return _own_rotary(s) if own else _plain_rotary(s)


def _own_fwd(s):
    import chunked_gated_delta_gb300 as kda
    o, ht = kda.decay_fwd(s["q"], s["k"], s["v"], s["g"], h0=s["h0"], cu_seqlens=s["cu"],
                          state_dtype=DTYPES[s["case"]["state"]])
    return {"o": o, "ht": ht}


def _own_bwd(s):
    import chunked_gated_delta_gb300 as kda
    dq, dk, dv, dg, dh0 = kda.decay_bwd(s["q"], s["k"], s["v"], s["g"], s["do"], h0=s["h0"], dht=s["dht"],
                                        cu_seqlens=s["cu"])
    return {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dh0": dh0}


def _own_step(s):
    import chunked_gated_delta_gb300 as kda
    o = kda.decay_step(s["q"], s["k"], s["v"], s["g"], s["state"], slots=s["slots"], cu_seqlens=s["cu"])
    return {"o": o, "state": s["state"]}


def _own_rotary(s):
    import chunked_gated_delta_gb300 as kda
    c = s["case"]
    q, k = kda.rotary(s["q"], s["k"], s["positions"], s["freq"], amplitude=s["amplitude"],
                      interleaved=c["interleaved"], inverse=c["inverse"])
    return {"q": q, "k": k}


def _rows(s):
    """The token row of each place of [N, padded length], and whether it is one."""
    lens = torch.tensor(s["lens"], device="cuda")
    length = max(1, -(-max(s["lens"]) // CHUNK)) * CHUNK
    place = torch.arange(length, device="cuda")
    live = place < lens[:, None]
    first = torch.arange(len(s["lens"]), device="cuda") * s["case"]["T"] if s["cu"] is None else s["cu"][:-1].long()
    return torch.where(live, first[:, None] + place, 0), live


def _chunks(x, rows, live, heads):
    """x [B, T, H', ...] as fp32 [N, H, chunks, CHUNK, ...], zero where there is no token."""
    x = x.flatten(0, 1)[rows].float()
    x = torch.where(live.view(live.shape + (1,) * (x.dim() - 2)), x, 0.0)
    if x.shape[2] != heads:
        x = x.repeat_interleave(heads // x.shape[2], 2)
    return x.unflatten(1, (-1, CHUNK)).permute(0, 3, 1, 2, *range(4, x.dim() + 1)).contiguous()


def _tokens(s, y, rows, live, group=1):
    """[N, H, chunks, CHUNK, ...] back as [B, T, H / group, ...], summed over the heads of a group, in fp32."""
    y = y.permute(0, 2, 3, 1, *range(4, y.dim())).flatten(1, 2)
    if group > 1:
        y = y.unflatten(2, (-1, group)).sum(3)
    out = torch.empty((s["q"].shape[0] * s["q"].shape[1],) + y.shape[2:], dtype=y.dtype, device=y.device)
    out[rows[live]] = y[live]
    return out.unflatten(0, s["q"].shape[:2])


def _decays(s, rows, live):
    """The logarithms in 64 bits: within a chunk up to each token [N, H, chunks, CHUNK], and to each chunk's start [N, H, chunks + 1]."""
    H = s["case"]["heads"]
    g = s["g"] if s["case"]["gate"] == "token" else s["g"].expand(s["q"].shape[:2] + (H,))
    inner = _chunks(g, rows, live, H).double().cumsum(-1)
    return inner, torch.nn.functional.pad(inner[..., -1].cumsum(-1), (1, 0))


def _states(inner, outer, k, v, h0):
    """The state before each chunk and after the last [N, H, chunks + 1, K, V]."""
    weight = torch.exp(inner[..., -1:] - inner).float()
    added = (k * weight[..., None]).transpose(-1, -2) @ v
    n = outer.shape[-1]
    before = torch.arange(n, device="cuda")[:, None] > torch.arange(n - 1, device="cuda")
    gap = torch.where(before, outer[..., :, None] - outer[..., None, 1:], -math.inf)
    states = (torch.exp(gap).float() @ added.flatten(-2)).unflatten(-1, added.shape[-2:])
    if h0 is not None:
        states = states + torch.exp(outer).float()[..., None, None] * h0.float()[:, :, None]
    return states


def _inside(inner):
    """exp of the decay from token j to token i of a chunk, zero for j > i."""
    n = torch.arange(CHUNK, device="cuda")
    gap = torch.where(n[:, None] >= n, inner[..., :, None] - inner[..., None, :], -math.inf)
    return torch.exp(gap).float()


def _plain_fwd(s):
    c = s["case"]
    rows, live = _rows(s)
    q, k, v = (_chunks(s[n], rows, live, c["heads"]) for n in ("q", "k", "v"))
    inner, outer = _decays(s, rows, live)
    states = _states(inner, outer, k, v, s["h0"])
    o = (q @ k.transpose(-1, -2) * _inside(inner)) @ v
    o = o + torch.exp(inner).float()[..., None] * (q @ states[:, :, :-1])
    return {"o": _tokens(s, c["K"] ** -0.5 * o, rows, live).to(s["v"].dtype),
            "ht": states[:, :, -1].to(DTYPES[c["state"]])}


def _plain_bwd(s):
    c = s["case"]
    scale, group = c["K"] ** -0.5, c["heads"] // c["qk_heads"]
    rows, live = _rows(s)
    q, k, v, do = (_chunks(s[n], rows, live, c["heads"]) for n in ("q", "k", "v", "do"))
    inner, outer = _decays(s, rows, live)
    states = _states(inner, outer, k, v, s["h0"])[:, :, :-1]
    # the states' gradients after each chunk, and before the first
    added = scale * (q * torch.exp(inner).float()[..., None]).transpose(-1, -2) @ do
    n = outer.shape[-1]
    after = torch.arange(n - 1, device="cuda") >= torch.arange(n, device="cuda")[:, None]
    gap = torch.where(after, outer[..., None, :-1] - outer[..., :, None], -math.inf)
    back = (torch.exp(gap).float() @ added.flatten(-2)).unflatten(-1, added.shape[-2:])
    back = back + torch.exp(outer[..., -1:] - outer).float()[..., None, None] * s["dht"].float()[:, :, None]
    dh0, back = back[:, :, 0], back[:, :, 1:]
    # within the chunk, and through the states
    inside = scale * _inside(inner)
    scores = q @ k.transpose(-1, -2)
    dscores = do @ v.transpose(-1, -2) * inside
    seen = torch.exp(inner).float()[..., None]
    kept = torch.exp(inner[..., -1:] - inner).float()[..., None]
    dq_far = scale * seen * (do @ states.transpose(-1, -2))
    dk_far = kept * (v @ back.transpose(-1, -2))
    dv = (scores * inside).transpose(-1, -2) @ do + kept * (k @ back)
    pairs = (scores * dscores).double()
    later = (q * dq_far).sum(-1).double() + pairs.sum(-1)
    across = torch.exp(inner[..., -1]) * (states * back).sum((-1, -2)).double()
    earlier = (k * dk_far).sum(-1).double()
    dg = (later - pairs.sum(-2)).flip(-1).cumsum(-1).flip(-1) + earlier.cumsum(-1) - earlier + across[..., None]
    io = s["q"].dtype
    dg = _tokens(s, dg, rows, live)
    if c["gate"] == "head":
        dg = dg.sum((0, 1))
    return {"dq": _tokens(s, dscores @ k + dq_far, rows, live, group).to(io),
            "dk": _tokens(s, dscores.transpose(-1, -2) @ q + dk_far, rows, live, group).to(io),
            "dv": _tokens(s, dv, rows, live).to(io), "dg": dg.float(),
            "dh0": dh0.to(DTYPES[c["state"]])}


def _plain_step(s):
    c = s["case"]
    live, T, device = s["live"], c["T"], s["q"].device
    group = c["heads"] // c["qk_heads"]
    slots = s["slots"][:live].long()
    S = s["state"].index_select(0, slots).float()
    if s["cu"] is None:
        first, count = torch.arange(live, device=device) * T, torch.full((live,), T, device=device)
    else:
        first = s["cu"][:live].long()
        count = s["cu"][1: live + 1].long() - first
    q, k, v = (s[n].flatten(0, 1) for n in ("q", "k", "v"))
    g = s["g"].flatten(0, 1) if c["gate"] == "token" else s["g"].expand(q.shape[0], -1)
    o = torch.zeros((q.shape[0] + 1,) + v.shape[1:], device=device)  # the last row takes what no request has
    for t in range(T):
        has = t < count
        row = (first + t).clamp_max(q.shape[0] - 1)
        kt, qt = (x[row].float().repeat_interleave(group, 1) for x in (k, q))
        new = S * torch.exp(g[row])[..., None, None] + kt[..., None] * v[row].float()[..., None, :]
        S = torch.where(has[:, None, None, None], new, S) if c["packed"] else new
        o[torch.where(has, row, q.shape[0])] = (S * qt[..., None]).sum(-2) * c["K"] ** -0.5
    s["state"].index_copy_(0, slots, S.to(s["state"].dtype))
    return {"o": o[:-1].view(s["v"].shape).to(s["v"].dtype), "state": s["state"]}


def _plain_rotary(s):
    c = s["case"]
    angle = (s["positions"].double()[..., None] * s["freq"])[:, :, None]
    cos, sin = (s["amplitude"] * torch.cos(angle)).float(), (s["amplitude"] * torch.sin(angle)).float()
    sin = -sin if c["inverse"] else sin

    def turned(x):
        y, R = x.float(), c["part"]
        a, b = (y[..., 0:R:2], y[..., 1:R:2]) if c["interleaved"] else (y[..., : R // 2], y[..., R // 2: R])
        new = (a * cos - b * sin, a * sin + b * cos)
        new = torch.stack(new, -1).flatten(-2) if c["interleaved"] else torch.cat(new, -1)
        return torch.cat((new, y[..., R:]), -1).to(x.dtype)

    return {"q": turned(s["q"]), "k": turned(s["k"])}


# ------------------------------------------------------------------ what a pass cannot do without
def _total(case):
    """Tokens of all sequences (those that hold a request, for a step)."""
    if not case["packed"]:
        return (case["N"] - case.get("pad", 0)) * case["T"]
    return sum(_lengths(case, 0)) if case["op"] != "step" else (case["N"] - case["pad"]) * case["T"] // 2


def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4}
    b = size[case["io"]]
    if case["op"] == "rotary":
        n = case["B"] * case["T"] * (case["heads"] + case["qk_heads"]) * case["dim"]
        return {"bytes": 2 * n * b + 8 * case["B"] * case["T"], "flops": 3.0 * n * case["part"] / case["dim"]}
    H, Hq, K, V, N = case["heads"], case["qk_heads"], case["K"], case["V"], case["N"]
    tokens, state = _total(case), H * K * V * size[case["state"]]
    gate = 4 * H * tokens if case["gate"] == "token" else 4 * H
    qk, vo = tokens * Hq * K * b, tokens * H * V * b
    if case["op"] == "step":
        return {"bytes": 2 * qk + 2 * vo + gate + 2 * (N - case["pad"]) * state, "flops": 5.0 * tokens * H * K * V}
    # per token and head: the state's update and its product with q (4 K V), in chunks or one by one
    if case["op"] == "fwd":
        return {"bytes": 2 * qk + 2 * vo + gate + (1 + case["h0"]) * N * state, "flops": 4.0 * tokens * H * K * V}
    return {"bytes": 4 * qk + 3 * vo + 2 * gate + (2 + case["h0"]) * N * state, "flops": 12.0 * tokens * H * K * V}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(case, s)
    if max(s["lens"]) * (2 if case["op"] == "bwd" else 1) > 70000:
        return None
    return _exact_recurrence(case, s)


def _exact_rotary(case, s):
    """Pairs as complex numbers times amplitude e^(+-i angle)."""
    angle = torch.einsum("bt,f->btf", s["positions"].to(torch.float64), s["freq"])
    turn = torch.polar(torch.full_like(angle, s["amplitude"]), -angle if case["inverse"] else angle).unsqueeze(2)
    out = {}
    for name in ("q", "k"):
        y = s[name].double().clone()
        half = case["part"] // 2
        first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else half)
        z = torch.complex(y.index_select(-1, first), y.index_select(-1, second)) * turn
        y.index_copy_(-1, first, z.real.contiguous())
        y.index_copy_(-1, second, z.imag.contiguous())
        out[name] = y
    return out


def _exact_recurrence(case, s):
    """Token by token, all sequences at once: forwards for the states, o and dq, backwards for dk and dv; dg_t is
    what q_u dq_u - k_u dk_u of the tokens u >= t sum to, and the last state times its gradient."""
    H, K, V, N = case["heads"], case["K"], case["V"], case["N"]
    scale, which = 1.0 / math.sqrt(K), torch.arange(H, device="cuda") // (H // case["qk_heads"])
    B, T = s["q"].shape[:2]
    flat = {n: s[n].reshape(B * T, -1, s[n].shape[-1]) for n in ("q", "k", "v", "do") if n in s}
    flat["q"], flat["k"] = flat["q"][:, which], flat["k"][:, which]
    gate = s["g"].double().expand(B, T, H).reshape(B * T, H)
    lens = torch.tensor(s["lens"], device="cuda")
    starts = lens.cumsum(0) - lens
    step = case["op"] == "step"
    alive = torch.arange(N, device="cuda") < s["live"] if step else torch.ones(N, dtype=torch.bool, device="cuda")
    if step:
        S = s["state"].double()[s["slots"].long().clamp_min(0)]
    else:
        S = s["h0"].double() if s["h0"] is not None else torch.zeros((N, H, K, V), dtype=torch.float64, device="cuda")
    back = "do" in s
    o = torch.zeros((B * T + 1, H, V), dtype=torch.float64, device="cuda")
    dq = torch.zeros((B * T + 1, H, K), dtype=torch.float64, device="cuda") if back else None
    uneven = case["packed"] or step

    def tokens(t):
        has = alive & (t < lens)
        at = torch.where(has, starts + t, torch.zeros_like(starts))
        return has, at, torch.where(has, at, torch.full_like(at, B * T))

    for t in range(max(s["lens"])):
        has, at, into = tokens(t)
        k, v, q = (flat[n][at].double() for n in ("k", "v", "q"))
        new = gate[at].exp()[..., None, None] * S
        new += torch.einsum("nhk,nhv->nhkv", k, v)
        S = torch.where(has.view(N, 1, 1, 1), new, S) if uneven else new
        if back:
            dq[into] = scale * torch.matmul(S, flat["do"][at].double()[..., None])[..., 0]
        else:
            o[into] = scale * torch.matmul(q[..., None, :], S)[..., 0, :]
    if step:
        state = s["state"].double()
        used = alive & (lens > 0)
        state[s["slots"].long()[used]] = S[used]
        return {"o": o[:-1].view(s["v"].shape), "state": state}
    if not back:
        return {"o": o[:-1].view(s["v"].shape), "ht": S}
    dk, dv, ends = torch.zeros_like(dq), o, (S * s["dht"].double()).sum((-1, -2))
    dS = s["dht"].double()
    for t in range(max(s["lens"]) - 1, -1, -1):
        has, at, into = tokens(t)
        k, v, q, do = (flat[n][at].double() for n in ("k", "v", "q", "do"))
        new = dS + torch.einsum("nhk,nhv->nhkv", scale * q, do)
        dk[into] = torch.matmul(new, v[..., None])[..., 0]
        dv[into] = torch.matmul(k[..., None, :], new)[..., 0, :]
        new = gate[at].exp()[..., None, None] * new
        dS = torch.where(has.view(N, 1, 1, 1), new, dS) if uneven else new
    term = (flat["q"].double() * dq[:-1]).sum(-1) - (flat["k"].double() * dk[:-1]).sum(-1)
    run = term.flip(0).cumsum(0).flip(0)
    run = torch.cat((run, torch.zeros_like(run[:1])))
    owner = torch.repeat_interleave(torch.arange(N, device="cuda"), lens)
    dg = run[:-1] - run[(starts + lens)[owner]] + ends[owner]
    dg = dg.view(B, T, H)
    groups = (B, T, case["qk_heads"], H // case["qk_heads"], K)
    return {"dq": dq[:-1].view(groups).sum(3), "dk": dk[:-1].view(groups).sum(3), "dv": dv[:-1].view(s["v"].shape),
            "dg": dg.sum((0, 1)) if case["gate"] == "head" else dg, "dh0": dS}
