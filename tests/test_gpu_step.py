"""kda.step against the recurrence in 64 bits: types, head layouts, packed and
padded batches, strides, slots, long offsets, and what it refuses.

Tolerances: one rounding of each output to its type, plus the worst case of the
fp32 arithmetic per token (step_reference).
"""
from __future__ import annotations

import ctypes

import pytest
import torch

import chunked_gated_delta_gb300 as kda
from chunked_gated_delta_gb300 import binding
from ops_util import HALF_ULP, TINY, Guarded, assert_close, step_reference

pytestmark = pytest.mark.gpu


def inputs(B, T, H, K, V, hq=None, io=torch.bfloat16, logits=False, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + 7)

    def randn(*s):
        return torch.randn(s, generator=gen, device="cuda")

    def unit(x):
        return (x / x.norm(dim=-1, keepdim=True)).to(io)

    hq = hq or H
    beta = randn(B, T, H)
    return dict(q=unit(randn(B, T, hq, K)), k=unit(randn(B, T, hq, K)), v=randn(B, T, H, V).to(io),
                g=torch.nn.functional.logsigmoid(randn(B, T, H, K) + 2.0),
                beta=(beta if logits else torch.sigmoid(beta)).to(io))


def cache(S, H, K, V, dtype=torch.float32, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + 99)
    return (0.3 * torch.randn((S, H, K, V), generator=gen, device="cuda")).to(dtype)


def check(x, state, slots, bounds, cu=None, logits=False, scale=None, status=None):
    """Runs step on a copy of the cache and compares o, the named states and the untouched ones."""
    K = x["q"].shape[-1]
    scale_v = K ** -0.5 if scale is None else scale
    where = list(range(len(bounds))) if slots is None else slots
    o_ref, s_ref, (eo, es) = step_reference(x["q"], x["k"], x["v"], x["g"], x["beta"], state, where, bounds, scale_v,
                                            logits)
    got = state.clone()
    sl = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    o = kda.step(x["q"], x["k"], x["v"], x["g"], x["beta"], got, slots=sl, scale=scale, cu_seqlens=cu,
                 beta_logits=logits, status=status)
    torch.cuda.synchronize()
    io = x["q"].dtype
    assert_close(o.reshape(o_ref.shape), o_ref, HALF_ULP[io] * 1.01, eo + TINY[io], "o")
    used = {s for s, (a, b) in zip(where, bounds) if s >= 0 and b > a}
    for s in range(state.shape[0]):
        if s in used:
            assert_close(got[s], s_ref[s], HALF_ULP[state.dtype] * 1.01, es, f"state {s}")
        else:
            assert torch.equal(got[s].view(torch.uint8), state[s].view(torch.uint8)), f"slot {s} was touched"
    return o, got


@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("io,st,logits", [(torch.bfloat16, torch.float32, False), (torch.float16, torch.bfloat16, True),
                                          (torch.bfloat16, torch.bfloat16, False),
                                          (torch.float16, torch.float32, False)])
@pytest.mark.parametrize("B,T", [(1, 1), (3, 1), (2, 3)])
def test_types_and_dims(K, V, io, st, logits, B, T):
    x = inputs(B, T, 4, K, V, hq=2, io=io, logits=logits, seed=K + V + T)
    check(x, cache(B, 4, K, V, st), None, [(b * T, (b + 1) * T) for b in range(B)], logits=logits)


@pytest.mark.parametrize("H,hq", [(1, 1), (5, 5), (6, 2), (32, 32), (64, 8)])
def test_heads(H, hq):
    check(inputs(7, 1, H, 128, 128, hq=hq, seed=H), cache(9, H, 128, 128), [8, 0, 3, 1, 7, 2, 5],
          [(i, i + 1) for i in range(7)], scale=1.0)


def test_many_sequences_every_rule():
    """Enough sequences that each way of cutting the columns is taken (1 to 700 of them)."""
    for B in (1, 2, 5, 20, 80, 700):
        check(inputs(B, 1, 2, 128, 128, seed=B), cache(B, 2, 128, 128), None, [(i, i + 1) for i in range(B)])
        check(inputs(B, 1, 2, 64, 64, seed=B), cache(B, 2, 64, 64), None, [(i, i + 1) for i in range(B)])


@pytest.mark.parametrize("B,H,K,V,st", [(420, 32, 128, 128, torch.float32), (1400, 8, 64, 64, torch.float32),
                                        (900, 16, 128, 64, torch.bfloat16)])
def test_long_streams_repeat(B, H, K, V, st):
    """More states per SM than any ring or table of the kernel holds, again and again: every call gives what the
    same call gives on small parts of the batch (which take the other kernel), to a rounding."""
    x = inputs(B, 1, H, K, V, seed=B)
    state = cache(B, H, K, V, st)
    parts = state.clone()
    o_parts = torch.cat([kda.step(*(x[n][i:i + 2] for n in ("q", "k", "v", "g", "beta")), parts[i:i + 2])
                         for i in range(0, B, 2)])
    for _ in range(12):
        got = state.clone()
        o = kda.step(x["q"], x["k"], x["v"], x["g"], x["beta"], got)
        assert_close(o, o_parts.double(), 2 * HALF_ULP[torch.bfloat16], 1e-3)
        assert_close(got, parts.double(), 2 * HALF_ULP[st], 1e-3)


@pytest.mark.parametrize("lens", [[0], [1], [5], [0, 1, 5, 0, 2, 9, 0], [0, 0, 0], [70, 1, 3]])
def test_packed_lengths(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    x = inputs(1, cu[-1], 3, 128, 64, seed=len(lens))
    slots = [(5 * i + 2) % (len(lens) + 4) for i in range(len(lens))]
    assert len(set(slots)) == len(slots)
    check(x, cache(len(lens) + 4, 3, 128, 64), slots, list(zip(cu, cu[1:])),
          cu=torch.tensor(cu, dtype=torch.int32, device="cuda"))


def test_padding_takes_no_state_and_its_inputs_do_not_matter():
    x = inputs(6, 2, 2, 128, 128)
    bad = [1, 4]
    for n in ("q", "k", "v", "g", "beta"):
        x[n][bad] = float("nan")
    state = cache(5, 2, 128, 128)
    state[4] = float("inf")  # a slot nobody names
    clean = {n: torch.nan_to_num(t) for n, t in x.items()}
    slots = [3, -1, 0, 2, -7, 1]
    o_ref, s_ref, (eo, es) = step_reference(*(clean[n] for n in ("q", "k", "v", "g", "beta")), state, slots,
                                            [(2 * i, 2 * i + 2) for i in range(6)], 128 ** -0.5)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = state.clone()
    o = kda.step(x["q"], x["k"], x["v"], x["g"], x["beta"], got, status=word,
                 slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    assert binding.status(word) == 0
    assert (o[bad] == 0).all()
    assert_close(o.reshape(o_ref.shape), o_ref, HALF_ULP[torch.bfloat16] * 1.01, eo)
    assert torch.equal(got[4], state[4])
    assert_close(got[:4], s_ref[:4], HALF_ULP[torch.float32], es)


def test_extreme_inputs():
    """beta 0 leaves the decayed state; g = -inf forgets it; g = 0 and beta 1 with a unit key writes v exactly back."""
    x = inputs(3, 1, 2, 64, 64)
    state = cache(3, 2, 64, 64)
    x["beta"][0] = 0.0
    x["g"][1] = float("-inf")
    x["g"][2] = 0.0
    x["beta"][2] = 1.0
    x["k"][2] = 0.0
    x["k"][2, ..., 5] = 1.0
    _, got = check(x, state, None, [(i, i + 1) for i in range(3)])
    assert_close(got[2][:, 5], x["v"][2, 0].double(), 1e-6, 1e-6)


def test_strided_token_rows():
    """q, k, v, g, beta as parts of wider projections' outputs."""
    B, T, H, K, V = 4, 3, 2, 128, 64
    x = inputs(B, T, H, K, V)
    wide = torch.full((B, T, 2 * H * K + H * V + H + 3), float("nan"), dtype=torch.bfloat16, device="cuda")
    parts, at = {}, 1
    for n in ("q", "k", "v", "beta"):
        w = x[n][0, 0].numel()
        wide[..., at:at + w] = x[n].reshape(B, T, w)
        parts[n] = wide[..., at:at + w].unflatten(-1, tuple(x[n].shape[2:]))
        at += w
    gw = torch.full((B, T, H * K + 5), float("nan"), device="cuda")
    gw[..., 2:2 + H * K] = x["g"].reshape(B, T, H * K)
    parts["g"] = gw[..., 2:2 + H * K].unflatten(-1, (H, K))
    assert not parts["q"].is_contiguous() and not parts["g"].is_contiguous()
    state = cache(B, H, K, V)
    s1, s2 = state.clone(), state.clone()
    o1 = kda.step(x["q"], x["k"], x["v"], x["g"], x["beta"], s1)
    o2 = kda.step(parts["q"], parts["k"], parts["v"], parts["g"], parts["beta"], s2)
    assert torch.equal(o1, o2) and torch.equal(s1, s2)
    one = {n: t[:, 1:2] for n, t in parts.items()}  # one token out of three
    s3, s4 = state.clone(), state.clone()
    o3 = kda.step(*(one[n] for n in ("q", "k", "v", "g", "beta")), s3)
    o4 = kda.step(*(one[n].contiguous() for n in ("q", "k", "v", "g", "beta")), s4)
    assert torch.equal(o3, o4) and torch.equal(s3, s4)


def test_continues_the_forward():
    """Prefill with kda.fwd, then tokens one by one and several at once: o and the state of one longer forward,
    to the forward's own tolerance (its operands are rounded to bf16, the step's are not)."""
    from parity_util import REL_HT, REL_O
    B, T, n, H = 2, 150, 7, 3
    x = inputs(B, T + n, H, 128, 128, seed=5)
    names = ("q", "k", "v", "g", "beta")
    o_all, h_all = kda.fwd(*(x[m] for m in names))
    _, state = kda.fwd(*(x[m][:, :T].contiguous() for m in names))
    other = state.clone()
    outs = [kda.step(*(x[m][:, T + i:T + i + 1] for m in names), state) for i in range(n)]
    once = kda.step(*(x[m][:, T:].contiguous() for m in names), other)
    o = torch.cat(outs, 1)
    assert torch.equal(o, once) and torch.equal(state, other)
    ref = o_all[:, T:].double()
    assert (o.double() - ref).norm() <= 2 * REL_O * ref.norm()
    assert (state.double() - h_all.double()).norm() <= 2 * REL_HT * h_all.double().norm()


def test_slots_outside_or_twice_are_refused():
    x = inputs(5, 2, 2, 128, 128)
    state = cache(4, 2, 128, 128)
    slots = [2, 4, 2, 0, 1 << 30]  # 4 and 2^30 lie outside, 2 is given twice
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = Guarded(state.shape, torch.float32, state)
    out = Guarded(x["v"].shape, torch.bfloat16)
    kda.step(x["q"], x["k"], x["v"], x["g"], x["beta"], got.t, status=word, out=out.t,
             slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    assert binding.status(word) == 8
    assert got.intact() and out.intact()
    o_ref, s_ref, (eo, es) = step_reference(x["q"], x["k"], x["v"], x["g"], x["beta"], state, [2, -1, -1, 0, -1],
                                            [(2 * i, 2 * i + 2) for i in range(5)], 128 ** -0.5)
    assert_close(out.t.reshape(o_ref.shape), o_ref, HALF_ULP[torch.bfloat16] * 1.01, eo)
    assert_close(got.t, s_ref, HALF_ULP[torch.float32], es)
    with pytest.raises(kda.KdaError):  # sequences beyond the cache, where slot n is sequence n
        kda.step(x["q"], x["k"], x["v"], x["g"], x["beta"], got.t)


@pytest.mark.parametrize("cu,bad", [([0, 4, 3, 6], [1]), ([1, 2, 3, 6], [0]), ([0, 2, 3, 5], [2]),
                                    ([0, 2, 900, 6], [1, 2]), ([0, -5, 3, 6], [0, 1])])
def test_bad_offsets_are_skipped(cu, bad):
    x = inputs(1, 6, 2, 64, 64)
    state = cache(3, 2, 64, 64)
    got, out = Guarded(state.shape, torch.float32, state), Guarded(x["v"].shape, torch.bfloat16)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.step(x["q"], x["k"], x["v"], x["g"], x["beta"], got.t, status=word, out=out.t,
             cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    assert binding.status(word) == 7
    assert got.intact() and out.intact()
    for n in range(3):
        assert torch.equal(got.t[n], state[n]) == (n in bad)


def test_offsets_beyond_32_bits():
    """A cache of more than 2^31 elements."""
    S, H = 4200, 32
    state = torch.zeros((S, H, 128, 128), dtype=torch.bfloat16, device="cuda")
    assert state.numel() > 1 << 31
    x = inputs(2, 1, H, 128, 128)
    some = cache(2, H, 128, 128, torch.bfloat16)
    state[S - 1], state[3] = some[0], some[1]
    o = kda.step(x["q"], x["k"], x["v"], x["g"], x["beta"], state,
                 slots=torch.tensor([S - 1, 3], dtype=torch.int32, device="cuda"))
    small = some.clone()
    assert torch.equal(o, kda.step(x["q"], x["k"], x["v"], x["g"], x["beta"], small))
    assert torch.equal(state[S - 1], small[0]) and torch.equal(state[3], small[1])
    assert int(torch.count_nonzero(state[4:S - 1].view(torch.int16).flatten(1).any(1))) == 0


def test_stream_graph_and_repeat():
    x = inputs(9, 2, 4, 128, 128)
    state = cache(9, 4, 128, 128)
    ref_s = state.clone()
    ref = kda.step(x["q"], x["k"], x["v"], x["g"], x["beta"], ref_s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s1, s2 = state.clone(), state.clone()
    side.wait_stream(torch.cuda.current_stream())
    o1 = kda.step(x["q"], x["k"], x["v"], x["g"], x["beta"], s1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o1, ref) and torch.equal(s1, ref_s)
    out = torch.empty_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.step(x["q"], x["k"], x["v"], x["g"], x["beta"], s2, out=out)
    s2.copy_(state)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(s2, ref_s)


def test_python_refusals():
    x = inputs(2, 1, 2, 128, 128)
    state = cache(2, 2, 128, 128)

    def call(**kw):
        a = dict(x, state=state)
        a.update(kw)
        return kda.step(a["q"], a["k"], a["v"], a["g"], a["beta"], a["state"], slots=a.get("slots"))

    for bad in (dict(q=x["q"].float()), dict(k=x["k"].half()), dict(g=x["g"].bfloat16()), dict(state=state.half()),
                dict(state=state[:, :1]), dict(state=state.transpose(2, 3)), dict(beta=x["beta"][:, :, :1]),
                dict(k=x["k"][:, :, :1]), dict(q=x["q"].cpu()), dict(v=x["v"].transpose(2, 3)),
                dict(q=x["q"][:1].expand(2, 1, 2, 128)), dict(slots=torch.zeros(2, dtype=torch.int64, device="cuda")),
                dict(slots=torch.zeros(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(TypeError):
            call(**bad)
    with pytest.raises(kda.KdaError):  # K = 32
        kda.step(x["q"][..., :32].contiguous(), x["k"][..., :32].contiguous(), x["v"], x["g"][..., :32].contiguous(),
                 x["beta"], cache(2, 2, 32, 128))
    assert ctypes.sizeof(binding.StepOpts) == 64
