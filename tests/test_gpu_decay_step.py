"""decay_step against the recurrence in 64 bits, and against decay_fwd: a prompt and then tokens.

Tolerances: the output's rounding, plus the worst case of fp32: per token the decay and the update
(4 roundings of the state's largest value), and K + 4 roundings of a sum of K products."""
from __future__ import annotations

import pytest
import torch

import chunked_gated_delta_gb300 as kda
from chunked_gated_delta_gb300 import binding
from decay_util import make, offsets, spans
from ops_util import EPS32, HALF_ULP, TINY, Guarded, assert_close

pytestmark = pytest.mark.gpu


def reference(x, state, slots, bounds, scale):
    H, K = state.shape[1:3]
    q, k, v = (x[n].flatten(0, 1).double() for n in ("q", "k", "v"))
    group = H // q.shape[1]
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    g = x["g"].double().flatten(0, 1) if x["g"].dim() == 3 else x["g"].double().expand(q.shape[0], H)
    out, o = state.double().clone(), torch.zeros_like(v)
    bound_o, bound_s = torch.zeros_like(v), torch.zeros_like(out)
    for n, (a, b) in enumerate(bounds):
        if slots[n] < 0:
            continue
        S, W = out[slots[n]], out[slots[n]].abs()  # W: the largest that S's terms can add up to
        for i, t in enumerate(range(a, b)):
            e = torch.exp(g[t])[:, None, None]
            S = e * S + k[t][:, :, None] * v[t][:, None, :]
            W = e * W + k[t].abs()[:, :, None] * v[t].abs()[:, None, :]
            o[t] = scale * torch.einsum("hkv,hk->hv", S, q[t])
            per = EPS32 * (4 * (i + 1) + K + 4)
            bound_o[t] = per * abs(scale) * torch.einsum("hkv,hk->hv", W, q[t].abs())
        out[slots[n]], bound_s[slots[n]] = S, EPS32 * 4 * (b - a + 1) * W
    return o, out, bound_o, bound_s


def check(x, state, slots, bounds, cu=None, scale=None, status=None):
    io = x["q"].dtype
    where = list(range(len(bounds))) if slots is None else slots
    o_ref, s_ref, bo, bs = reference(x, state, where, bounds, x["q"].shape[-1] ** -0.5 if scale is None else scale)
    got = state.clone()
    sl = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    o = kda.decay_step(x["q"], x["k"], x["v"], x["g"], got, slots=sl, scale=scale, cu_seqlens=cu, status=status)
    torch.cuda.synchronize()
    assert_close(o.flatten(0, 1), o_ref, HALF_ULP[io] * 1.01, bo + TINY[io], "o")
    used = {s for s, (a, b) in zip(where, bounds) if s >= 0 and b > a}
    for s in range(state.shape[0]):
        if s in used:
            assert_close(got[s], s_ref[s], HALF_ULP[state.dtype] * 1.01, bs[s], f"state {s}")
        else:
            assert torch.equal(got[s].view(torch.uint8), state[s].view(torch.uint8)), f"slot {s} was touched"
    return o, got


def cache(S, H, K, V, dtype=torch.float32, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + 99)
    return (0.3 * torch.randn((S, H, K, V), generator=gen, device="cuda")).to(dtype)


def rows(B, T):
    return [(b * T, (b + 1) * T) for b in range(B)]


@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("io,st", [(torch.bfloat16, torch.float32), (torch.float16, torch.bfloat16),
                                   (torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32)])
@pytest.mark.parametrize("B,T", [(1, 1), (3, 1), (2, 3), (200, 1)])
def test_types_and_dims(K, V, io, st, B, T):
    x = make(B, T, 4, K, V, hq=2, io=io, h0=False, do=False, seed=K + V + T)
    check(x, cache(B, 4, K, V, st), None, rows(B, T))


@pytest.mark.parametrize("H,hq", [(1, 1), (5, 5), (6, 2), (32, 32), (64, 8)])
@pytest.mark.parametrize("gate", ["token", "head"])
def test_heads(H, hq, gate):
    x = make(7, 1, H, 128, 128, hq=hq, gate=gate, h0=False, do=False, seed=H)
    check(x, cache(9, H, 128, 128), [8, 0, 3, 1, 7, 2, 5], rows(7, 1), scale=1.0)


@pytest.mark.parametrize("T", [2, 3, 4, 5, 7, 8, 9, 16, 33])
@pytest.mark.parametrize("B", [1, 40])
def test_several_tokens(T, B):
    x = make(B, T, 8, 128, 64, h0=False, do=False, seed=T)
    check(x, cache(B, 8, 128, 64), None, rows(B, T))


@pytest.mark.parametrize("reps", [1, 40])
def test_packed_and_padded(reps):
    lens = [0, 1, 5, 0, 3, 4, 2, 9] * reps
    x = make(1, sum(lens), 4, 128, 128, hq=2, h0=False, do=False)
    slots = [-1 if i % 5 == 4 else len(lens) + 2 - i for i in range(len(lens))]
    o, _ = check(x, cache(len(lens) + 3, 4, 128, 128), slots, spans(lens), cu=offsets(lens))
    for (a, b), s in zip(spans(lens), slots):
        if s < 0:
            assert bool((o[0, a:b] == 0).all())


@pytest.mark.parametrize("N", [4, 300])
def test_bad_slots(N):
    """A slot outside the cache, or given before, has zeros and leaves the cache alone."""
    x = make(N, 1, 2, 64, 64, h0=False, do=False)
    state = cache(N + 1, 2, 64, 64)
    slots = list(range(N))
    slots[1], slots[3] = N + 5, 2
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = state.clone()
    o = kda.decay_step(x["q"], x["k"], x["v"], x["g"], got, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"), status=word)
    assert binding.status(word) == 8
    assert bool((o[[1, 3]] == 0).all())
    fine = [n for n in range(N) if n not in (1, 3)]
    y = {n: x[n][fine] for n in ("q", "k", "v", "g")}
    want = state.clone()
    o2 = kda.decay_step(*y.values(), want, slots=torch.tensor(fine, dtype=torch.int32, device="cuda"))
    assert torch.equal(o[fine], o2) and torch.equal(got, want)


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements, its far end used."""
    S = 2 ** 31 // (32 * 128 * 128) + 2
    state = torch.zeros((S, 32, 128, 128), dtype=torch.bfloat16, device="cuda")
    x = make(2, 1, 32, 128, 128, h0=False, do=False)
    state[-1] = 0.25
    small = state[[0, S - 1]].clone()
    o = kda.decay_step(x["q"], x["k"], x["v"], x["g"], state, slots=torch.tensor([0, S - 1], dtype=torch.int32, device="cuda"))
    want = kda.decay_step(x["q"], x["k"], x["v"], x["g"], small)
    assert torch.equal(o, want) and torch.equal(state[[0, S - 1]], small) and bool((state[1:-1] == 0).all())


def test_rows_of_a_wider_projection_and_guards():
    x = make(5, 2, 4, 64, 128, hq=2, h0=False, do=False)
    wide = torch.randn(5, 2, 2 * 128 + 512 + 3, device="cuda").to(torch.bfloat16)
    y = dict(x)
    for n, a, w, h in (("q", 1, 128, 2), ("k", 129, 128, 2), ("v", 257, 512, 4)):
        y[n] = wide[..., a:a + w].unflatten(-1, (h, -1))
        y[n].copy_(x[n])
    state = Guarded((6, 4, 64, 128), torch.float32, cache(6, 4, 64, 128))
    out = Guarded((5, 2, 4, 128), torch.bfloat16)
    want_state = state.t.clone()
    want = kda.decay_step(x["q"], x["k"], x["v"], x["g"], want_state)
    kda.decay_step(y["q"], y["k"], y["v"], x["g"], state.t, out=out.t)
    torch.cuda.synchronize()
    assert torch.equal(out.t, want) and torch.equal(state.t, want_state) and out.intact() and state.intact()


def test_prompt_then_tokens():
    """A prompt by decay_fwd and tokens by decay_step agree with the whole by decay_fwd (fp32 states)."""
    x = make(2, 300, 4, 128, 128, h0=False, do=False)
    o, ht = kda.decay_fwd(x["q"], x["k"], x["v"], x["g"])
    first = {n: x[n][:, :290].contiguous() for n in ("q", "k", "v", "g")}
    rest = {n: x[n][:, 290:] for n in ("q", "k", "v", "g")}
    rest = {n: t.contiguous() for n, t in rest.items()}
    _, state = kda.decay_fwd(*first.values())
    tail = kda.decay_step(*rest.values(), state)
    off = (state - ht).norm() / ht.norm()
    assert off.item() <= 2e-5
    d = (tail.float() - o[:, 290:].float()).norm() / o[:, 290:].float().norm()
    assert d.item() <= 4 * HALF_ULP[torch.bfloat16]


def test_graph():
    x = make(6, 1, 4, 128, 128, h0=False, do=False)
    start = cache(6, 4, 128, 128)
    eager = start.clone()
    want = [kda.decay_step(x["q"], x["k"], x["v"], x["g"], eager) for _ in range(3)]
    state, out = start.clone(), torch.empty_like(x["v"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.decay_step(x["q"], x["k"], x["v"], x["g"], state, out=out)
    state.copy_(start)
    for w in want:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
    assert torch.equal(state, eager)


def test_refusals():
    x = make(2, 1, 2, 64, 64, h0=False, do=False)
    state = cache(2, 2, 64, 64)
    a = (x["q"], x["k"], x["v"], x["g"])
    for bad in (state.half(), state[:, :1], state.cpu(), state[:1]):
        with pytest.raises((TypeError, kda.KdaError)):
            kda.decay_step(*a, bad)
    with pytest.raises(TypeError):
        kda.decay_step(*a, state, slots=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        kda.decay_step(*a, state, slots=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError):
        kda.decay_step(x["q"], x["k"], x["v"].half(), x["g"], state)
    with pytest.raises(TypeError):
        kda.decay_step(*a, state, out=torch.empty(2, 1, 2, 64, device="cuda"))
