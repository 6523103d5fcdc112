"""kda.step where the sequences and heads are many enough for its streaming kernel
(at least two per SM): types, packed lengths in every order, padding, refusals,
strides and alignments, against the recurrence in 64 bits (as test_gpu_step.py)."""
from __future__ import annotations

import random

import pytest
import torch

import chunked_gated_delta_gb300 as kda
from chunked_gated_delta_gb300 import binding
from ops_util import HALF_ULP, Guarded, assert_close, step_reference
from test_gpu_step import cache, check, inputs

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("io,st,logits", [(BF16, F32, False), (F16, BF16, True), (BF16, BF16, False), (F16, F32, False)])
@pytest.mark.parametrize("T", [1, 2, 7])
def test_types_and_dims(K, V, io, st, logits, T):
    B, H = 5, 64
    x = inputs(B, T, H, K, V, hq=32, io=io, logits=logits, seed=K + V + T)
    check(x, cache(B, H, K, V, st), None, [(b * T, (b + 1) * T) for b in range(B)], logits=logits)


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("K,V,st", [(128, 128, F32), (128, 64, BF16), (64, 128, F32)])
def test_packed_in_any_order(seed, K, V, st):
    rng = random.Random(seed)
    n, H = rng.choice(((30, 16), (77, 5), (200, 2), (520, 1), (700, 1))), None
    n, H = n
    lens = [rng.choice((0, 0, 1, 1, 2, 5, rng.randint(0, 20))) for _ in range(n)]
    if seed == 5:
        lens[n // 2] = 300  # one long among short ones
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    slots = rng.sample(range(n + 3), n)
    for i in rng.sample(range(n), n // 7):
        slots[i] = -1
    x = inputs(1, cu[-1], H, K, V, seed=seed)
    check(x, cache(n + 3, H, K, V, st, seed=seed), slots, list(zip(cu, cu[1:])),
          cu=torch.tensor(cu, dtype=torch.int32, device="cuda"))


def test_all_empty_and_all_padding():
    H = 128
    state = cache(4, H, 64, 64)
    got = state.clone()
    empty = inputs(1, 0, H, 64, 64)
    kda.step(*(empty[n] for n in ("q", "k", "v", "g", "beta")), got,
             cu_seqlens=torch.zeros(5, dtype=torch.int32, device="cuda"))
    x = inputs(4, 2, H, 64, 64)
    o = kda.step(*(x[n] for n in ("q", "k", "v", "g", "beta")), got,
                 slots=torch.full((4,), -1, dtype=torch.int32, device="cuda"))
    assert (o == 0).all() and torch.equal(got, state)


def test_slots_outside_or_twice_are_refused():
    H = 64
    x = inputs(7, 2, H, 128, 128)
    state = cache(4, H, 128, 128)
    slots = [2, 4, 2, 0, 1 << 30, -1, 2]
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, out = Guarded(state.shape, F32, state), Guarded(x["v"].shape, BF16)
    kda.step(x["q"], x["k"], x["v"], x["g"], x["beta"], got.t, status=word, out=out.t,
             slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    assert binding.status(word) == 8 and got.intact() and out.intact()
    o_ref, s_ref, (eo, es) = step_reference(x["q"], x["k"], x["v"], x["g"], x["beta"], state, [2, -1, -1, 0, -1, -1, -1],
                                            [(2 * i, 2 * i + 2) for i in range(7)], 128 ** -0.5)
    assert_close(out.t.reshape(o_ref.shape), o_ref, HALF_ULP[BF16] * 1.01, eo)
    assert_close(got.t, s_ref, HALF_ULP[F32], es)


@pytest.mark.parametrize("cu,bad", [([0, 4, 3, 6], [1]), ([1, 2, 3, 6], [0]), ([0, 2, 3, 5], [2]),
                                    ([0, 2, 900, 6], [1, 2]), ([0, -5, 3, 6], [0, 1])])
def test_bad_offsets_are_skipped(cu, bad):
    H = 128
    x = inputs(1, 6, H, 64, 64)
    state = cache(3, H, 64, 64)
    got, out = Guarded(state.shape, F32, state), Guarded(x["v"].shape, BF16)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.step(x["q"], x["k"], x["v"], x["g"], x["beta"], got.t, status=word, out=out.t,
             cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    assert binding.status(word) == 7 and got.intact() and out.intact()
    for n in range(3):
        assert torch.equal(got.t[n], state[n]) == (n in bad)


@pytest.mark.parametrize("lead", [0, 1, 2, 4])
@pytest.mark.parametrize("K,V", [(128, 128), (64, 64)])
def test_strided_token_rows(lead, K, V):
    """Parts of wider rows, on and off the boundaries that wide loads need."""
    B, T, H = 5, 3, 64
    x = inputs(B, T, H, K, V)
    wide = torch.full((B, T, 2 * H * K + H * V + H + 9), float("nan"), dtype=BF16, device="cuda")
    gw = torch.full((B, T, H * K + 7), float("nan"), device="cuda")
    parts, at = {}, lead
    for n in ("q", "k", "v", "beta"):
        w = x[n][0, 0].numel()
        wide[..., at:at + w] = x[n].reshape(B, T, w)
        parts[n] = wide[..., at:at + w].unflatten(-1, tuple(x[n].shape[2:]))
        at += w
    gw[..., lead:lead + H * K] = x["g"].reshape(B, T, H * K)
    parts["g"] = gw[..., lead:lead + H * K].unflatten(-1, (H, K))
    state = cache(B, H, K, V)
    s1, s2 = state.clone(), state.clone()
    names = ("q", "k", "v", "g", "beta")
    o1 = kda.step(*(x[n] for n in names), s1)
    o2 = kda.step(*(parts[n] for n in names), s2)
    assert torch.equal(o1, o2) and torch.equal(s1, s2)


def test_graph_and_repeat():
    x = inputs(40, 2, 16, 128, 64)
    names = ("q", "k", "v", "g", "beta")
    state = cache(40, 16, 128, 64)
    ref_s = state.clone()
    ref = kda.step(*(x[n] for n in names), ref_s)
    s2, out = state.clone(), torch.empty_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.step(*(x[n] for n in names), s2, out=out)
    for _ in range(10):
        s2.copy_(state)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(s2, ref_s)
