"""The operators around the recurrence in a served KDA layer, as measured cases.

Three operators, each in a plain form (elementary torch operations in 32 bits,
rounded once at the end) and as the framework's own call:

* step:   the gated delta rule for one or a few new tokens per request, on a
          cache of recurrent states addressed by slot, updated in place;
* norm:   root-mean-square norm over rows, with the residual's addition before
          it and an output in the input's type or in e4m3 with one scale a row;
* linear: x @ w^T with row and column scales (8-bit operands), bias,
          activation and residual applied before the one rounding.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "f8": torch.float8_e4m3fn}
F8_MAX = 448.0
AMAX_FLOOR = 1e-30


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one request, one token: the latency of a decode step (32 heads of 128 x 128, as at the headline shape)
        dict(name="step one request", op="step", reqs=1, pad=0, slots=8, tokens=1, packed=False, heads=32, qk_heads=32,
             K=128, V=128, io="bf16", state="f32", logits=False),
        # a decode batch of a served model with 16 heads, padded to a graph's size, in a cache with free slots
        dict(name="step batch", op="step", reqs=64, pad=5, slots=80, tokens=1, packed=False, heads=16, qk_heads=16,
             K=128, V=128, io="bf16", state="f32", logits=False),
        # a full server: 512 requests, 1.07 GB of states read and written
        dict(name="step full server", op="step", reqs=512, pad=0, slots=512, tokens=1, packed=False, heads=32,
             qk_heads=32, K=128, V=128, io="bf16", state="f32", logits=False),
        # checking drafted tokens: 0 to 5 new tokens per request (packed), grouped heads, 16-bit states, beta as logits
        dict(name="step drafts", op="step", reqs=96, pad=0, slots=101, tokens=5, packed=True, heads=32, qk_heads=16,
             K=128, V=64, io="f16", state="bf16", logits=True),
        # the norm before the projections in a decode step of one token
        dict(name="norm one token", op="norm", rows=1, dim=4096, io="bf16", out="f8", residual=True, weight=True,
             extra=0),
        # the same in prefill, at the headline's 32768 tokens
        dict(name="norm prefill", op="norm", rows=32768, dim=4096, io="bf16", out="f8", residual=True, weight=True,
             extra=0),
        # the norm of every head's output (33333 tokens x 32 heads of 128)
        dict(name="norm heads", op="norm", rows=33333 * 32, dim=128, io="bf16", out="bf16", residual=False,
             weight=True, extra=0),
        # a projection of one token
        dict(name="linear one token", op="linear", M=1, N=4096, K=4096, io="bf16", out="bf16", act="silu", bias=True,
             residual=False, extra=0),
        # the output projection of an odd decode batch, 8-bit operands, the residual added
        dict(name="linear batch f8", op="linear", M=59, N=4096, K=4096, io="f8", out="bf16", act="none", bias=False,
             residual=True, extra=0),
        # the decay gate of 4096 tokens at 16 heads: log-sigmoid of a biased projection, kept in 32 bits
        dict(name="linear gate f32", op="linear", M=4096, N=2048, K=2048, io="bf16", out="f32", act="logsigmoid",
             bias=True, residual=False, extra=0),
        # a projection in prefill at the headline's 32768 tokens
        dict(name="linear prefill", op="linear", M=32768, N=4096, K=4096, io="bf16", out="bf16", act="silu", bias=True,
             residual=False, extra=0),
        # the output projection in prefill from 8-bit operands, ragged token count, the residual added
        dict(name="linear prefill f8", op="linear", M=16361, N=4096, K=4096, io="f8", out="bf16", act="none",
             bias=True, residual=True, extra=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("step", "norm", "linear"))
    if op == "step":
        K, V = rng.choice((64, 128)), rng.choice((64, 128))
        qk_heads = rng.choice((1, 2, 3, 8, 16, 32))
        heads = qk_heads * rng.choice((1, 2)) if qk_heads <= 16 else qk_heads
        tokens = rng.choice((1, 1, 2, 3, 5, 8))
        reqs = _log(rng, 1, max(1, 512 // tokens))
        return dict(op="step", reqs=reqs, pad=rng.randint(0, reqs // 4), slots=reqs + rng.randint(0, 9), tokens=tokens,
                    packed=tokens > 1 and rng.random() < 0.6, heads=heads, qk_heads=qk_heads, K=K, V=V,
                    io=rng.choice(("bf16", "bf16", "f16")), state=rng.choice(("f32", "f32", "bf16")),
                    logits=rng.random() < 0.3)
    if op == "norm":
        dim = rng.choice((64, 128, 256, 2048, 4096, _log(rng, 8, 16384), 8 * _log(rng, 1, 2048)))
        rows = _log(rng, 1, max(1, (32768 * 4096) // max(dim, 128)))
        io = rng.choice(("bf16", "f16"))
        return dict(op="norm", rows=rows, dim=dim, io=io, out=rng.choice((io, "f8", "f32")),
                    residual=rng.random() < 0.5, weight=rng.random() < 0.8, extra=rng.choice((0, 0, 8, 24)))
    io = rng.choice(("bf16", "f16", "f8"))
    N = rng.choice((32, 16 * _log(rng, 1, 512), _log(rng, 1, 8192), 4096))
    K = rng.choice((64, 2048, 4096, 16 * _log(rng, 2, 512), _log(rng, 16, 8192)))
    M = _log(rng, 1, max(1, min(32768, (32768 * 4096 * 4096) // (max(N, 256) * max(K, 256)))))
    act = rng.choice(("none", "none", "silu", "gelu", "sigmoid", "logsigmoid"))
    return dict(op="linear", M=M, N=N, K=K, io=io, out=rng.choice(("bf16", "bf16", "f16", "f32")), act=act,
                bias=rng.random() < 0.5, residual=rng.random() < 0.4, extra=rng.choice((0, 0, 16, 48)))


# ------------------------------------------------------------------ inputs
def _rows(x, stride):
    """x [M, D] as the first D columns of rows `stride` elements apart."""
    buf = torch.zeros((x.shape[0], stride), dtype=x.dtype, device=x.device)
    buf[:, : x.shape[1]] = x
    return buf[:, : x.shape[1]]


def _quantised(x):
    amax = x.abs().amax(dim=-1).clamp_min(AMAX_FLOOR)
    return (x * (F8_MAX / amax)[:, None]).to(torch.float8_e4m3fn), amax / F8_MAX


def _lengths(case, seed):
    """Tokens of each request: fixed, or (packed) 0 .. tokens in turn, in an order of the seed's."""
    live, most = case["reqs"], case["tokens"]
    if not case["packed"]:
        return [most] * live
    order = torch.randperm(live, generator=torch.Generator().manual_seed(1000003 * seed + 17)).tolist()
    return [(most + i) % (most + 1) for i in order]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    s = dict(case=dict(case))
    io = DTYPES[case["io"]]
    if case["op"] == "step":
        H, Hq, K, V, N = case["heads"], case["qk_heads"], case["K"], case["V"], case["reqs"]
        lens = _lengths(case, seed)
        B, T = (1, sum(lens)) if case["packed"] else (N, case["tokens"])

        def unit(x):
            return (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-12)).to(io)

        beta = randn(B, T, H)
        order = torch.randperm(case["slots"], generator=gen, device="cuda")[:N].to(torch.int32)
        if case["pad"]:
            order[N - case["pad"]:] = -1  # padding of the batch: no state, o is zero
        s.update(q=unit(randn(B, T, Hq, K)), k=unit(randn(B, T, Hq, K)), v=randn(B, T, H, V).to(io),
                 g=torch.nn.functional.logsigmoid(randn(B, T, H, K) + 3.0),
                 beta=(beta if case["logits"] else torch.sigmoid(beta)).to(io),
                 state=(0.1 * randn(case["slots"], H, K, V)).to(DTYPES[case["state"]]), slots=order,
                 cu=None, live=N - case["pad"])
        if case["packed"]:
            s["cu"] = torch.tensor([0] + lens).cumsum(0).to(device="cuda", dtype=torch.int32)
    elif case["op"] == "norm":
        M, D = case["rows"], case["dim"]
        stride = D + case["extra"]
        s["x"] = _rows(randn(M, D).to(io), stride) if case["extra"] else randn(M, D).to(io)
        s["residual"] = (2.0 * randn(M, D)).to(io) if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * randn(D)).to(io) if case["weight"] else None
    else:
        M, N, K = case["M"], case["N"], case["K"]
        x, w = randn(M, K), randn(N, K) / math.sqrt(K)
        s.update(xs=None, ws=None)
        if case["io"] == "f8":
            x, s["xs"] = _quantised(x)
            w, s["ws"] = _quantised(w)
        else:
            x, w = x.to(io), w.to(io)
        even = -(-K // 16) * 16  # rows start on 16 bytes
        s["x"] = x if K == even and not case["extra"] else _rows(x, even + case["extra"])
        s["w"] = w if K == even else _rows(w, even)
        s["bias"] = 0.5 * randn(N) if case["bias"] else None
        s["residual"] = randn(M, N).to(DTYPES[case["out"]]) if case["residual"] else None
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if op == "step":
        return _own_step(s) if own else _plain_step(s)
    if op == "norm":
        return _own_norm(s) if own else _plain_norm(s)
    return _own_linear(s) if own else _plain_linear(s)


def _own_step(s):
    import chunked_gated_delta_gb300 as kda
    c = s["case"]
    o = kda.step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"], cu_seqlens=s["cu"],
                 beta_logits=c["logits"])
    return {"o": o, "state": s["state"]}


def _plain_step(s):
    c = s["case"]
    H, live, T, device = c["heads"], s["live"], c["tokens"], s["q"].device
    group = H // c["qk_heads"]
    slots = s["slots"][:live].long()
    S = s["state"].index_select(0, slots).float()
    if s["cu"] is None:
        first = torch.arange(live, device=device) * T
        count = torch.full((live,), T, device=device)
    else:
        first = s["cu"][:live].long()
        count = s["cu"][1: live + 1].long() - first
    q, k, v, g, beta = (s[n].flatten(0, 1) for n in ("q", "k", "v", "g", "beta"))
    o = torch.zeros((q.shape[0] + 1, H, c["V"]), device=device)  # the last row takes what no request has
    for t in range(T):
        has = t < count
        row = (first + t).clamp_max(q.shape[0] - 1)
        qt = q[row].float().repeat_interleave(group, 1)
        kt = k[row].float().repeat_interleave(group, 1)
        bt = beta[row].float()
        bt = torch.sigmoid(bt) if c["logits"] else bt
        new = S * torch.exp(g[row])[..., None]
        delta = bt[..., None] * (v[row].float() - (new * kt[..., None]).sum(-2))
        new = new + kt[..., None] * delta[..., None, :]
        S = torch.where(has[:, None, None, None], new, S) if c["packed"] else new
        ot = (S * qt[..., None]).sum(-2) * c["K"] ** -0.5
        o[torch.where(has, row, q.shape[0])] = ot
    s["state"].index_copy_(0, slots, S.to(s["state"].dtype))
    return {"o": o[:-1].view(s["v"].shape).to(s["v"].dtype), "state": s["state"]}


def _own_norm(s):
    import chunked_gated_delta_gb300 as kda
    y, scale, summed = kda.rms_norm(s["x"], s["weight"], residual=s["residual"], out_dtype=DTYPES[s["case"]["out"]])
    return {"y": y, "scale": scale, "sum": summed}


def _plain_norm(s):
    x = s["x"].float()
    summed = None
    if s["residual"] is not None:
        x = x + s["residual"].float()
        summed = x.to(s["x"].dtype)
    y = x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6))
    if s["weight"] is not None:
        y = y * s["weight"].float()
    scale = None
    if s["case"]["out"] == "f8":
        y, scale = _quantised(y)
    return {"y": y.to(DTYPES[s["case"]["out"]]), "scale": scale, "sum": summed}


def _own_linear(s):
    import chunked_gated_delta_gb300 as kda
    c = s["case"]
    return kda.linear(s["x"], s["w"], bias=s["bias"], act=c["act"], residual=s["residual"], x_scale=s["xs"],
                      w_scale=s["ws"], out_dtype=DTYPES[c["out"]])


def _plain_linear(s):
    c = s["case"]
    y = s["x"].float() @ s["w"].float().t()
    if s["xs"] is not None:
        y = y * s["xs"][:, None] * s["ws"]
    if s["bias"] is not None:
        y = y + s["bias"]
    if c["act"] == "silu":
        y = y / (1.0 + torch.exp(-y))
    elif c["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    elif c["act"] == "sigmoid":
        y = 1.0 / (1.0 + torch.exp(-y))
    elif c["act"] == "logsigmoid":
        y = y.clamp_max(0.0) - torch.log1p(torch.exp(-y.abs()))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DTYPES[c["out"]])


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4, "f8": 1}
    b = size[case["io"]]
    if case["op"] == "step":
        live, H = case["reqs"] - case["pad"], case["heads"]
        per = case["tokens"] * (0.5 if case["packed"] else 1.0)
        token = 2 * case["qk_heads"] * case["K"] * b + H * (2 * case["V"] * b + 4 * case["K"] + b)
        state = 2 * H * case["K"] * case["V"] * size[case["state"]]
        return {"bytes": live * (state + per * token), "flops": live * per * H * case["K"] * case["V"] * 7.0}
    if case["op"] == "norm":
        n = case["rows"] * case["dim"]
        moved = n * (b + size[case["out"]] + (2 * b if case["residual"] else 0))
        return {"bytes": moved + (4 * case["rows"] if case["out"] == "f8" else 0) + case["dim"] * b * case["weight"],
                "flops": 5.0 * n}
    M, N, K = case["M"], case["N"], case["K"]
    moved = (M + N) * K * b + M * N * size[case["out"]] * (2 if case["residual"] else 1) + 4 * N * case["bias"]
    if case["io"] == "f8":
        moved += 4 * (M + N)
    return {"bytes": moved, "flops": 2.0 * M * N * K}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "step":
        return _exact_step(case, s)
    if case["op"] == "norm":
        x = s["x"].double()
        if s["residual"] is not None:
            x = x + s["residual"].double()
        y = x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + 1e-6)
        y = y * s["weight"].double() if s["weight"] is not None else y
        scale = None
        if case["out"] == "f8":
            amax = y.abs().amax(-1, keepdim=True).clamp(min=AMAX_FLOOR)
            scale = amax[:, 0] / F8_MAX
            y = _e4m3(y * (F8_MAX / amax))
        return {"y": y, "scale": scale, "sum": x if s["residual"] is not None else None}
    x, w = s["x"].double(), s["w"].double()
    if s["xs"] is not None:
        x, w = x * s["xs"].double()[:, None], w * s["ws"].double()[:, None]
    y = torch.mm(x, w.T)
    y = y + s["bias"].double() if s["bias"] is not None else y
    y = {"none": lambda t: t, "silu": lambda t: t * torch.sigmoid(t), "gelu": torch.nn.functional.gelu,
         "sigmoid": torch.sigmoid, "logsigmoid": torch.nn.functional.logsigmoid}[case["act"]](y)
    return y + s["residual"].double() if s["residual"] is not None else y


def _e4m3(y):
    """Nearest e4m3 value of each y (|y| <= 448), ties to the even mantissa, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _exact_step(case, s):
    live, H, K, V = s["live"], case["heads"], case["K"], case["V"]
    lens = [case["tokens"]] * live if s["cu"] is None else s["cu"].diff().tolist()
    starts = [n * case["tokens"] for n in range(live)] if s["cu"] is None else s["cu"][:live].tolist()
    rows = s["v"].shape[0] * s["v"].shape[1]
    head = torch.arange(H, device="cuda") // (H // case["qk_heads"])
    q, k = (s[n].reshape(rows, -1, K)[:, head].double() for n in ("q", "k"))
    v, g, beta = s["v"].reshape(rows, H, V).double(), s["g"].reshape(rows, H, K).double(), s["beta"].reshape(rows, H)
    beta = torch.sigmoid(beta.double()) if case["logits"] else beta.double()
    state, o = s["state"].double(), torch.zeros((rows, H, V), dtype=torch.float64, device="cuda")
    slots = s["slots"].long()
    for t in range(case["tokens"]):
        which = [n for n in range(live) if t < lens[n]]
        if not which:
            break
        at = torch.tensor([starts[n] + t for n in which], device="cuda")
        into = slots[torch.tensor(which, device="cuda")]
        S = g[at].exp().unsqueeze(-1) * state[into]
        seen = torch.matmul(k[at].unsqueeze(-2), S).squeeze(-2)
        S = S + torch.matmul(k[at].unsqueeze(-1), (beta[at].unsqueeze(-1) * (v[at] - seen)).unsqueeze(-2))
        state[into] = S
        o[at] = torch.matmul(q[at].unsqueeze(-2), S).squeeze(-2) / math.sqrt(K)
    return {"o": o.reshape(s["v"].shape), "state": state}
