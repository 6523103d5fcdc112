"""cu_seqlens out of order, beyond the rows or short of them: decay_bwd and decay_step report it and write nothing,
whichever kernels a head layout and a form of the decay bring in."""
from __future__ import annotations

import ctypes

import pytest
import torch

import chunked_gated_delta_gb300 as kda
from chunked_gated_delta_gb300 import binding
from decay_util import make

pytestmark = pytest.mark.gpu

P = ctypes.c_void_p
BAD = ([0, 100, 50, 300], [0, 200, 100, 300], [0, 100, 200, 299], [1, 100, 200, 300], [0, 100, 400, 300], [0, -5, 200, 300])
GRADS = ("dq", "dk", "dv", "dg", "dh0")


def backward(x, cu, word):
    """kda_decay_bwd into tensors of sevens, with a workspace of 3.0s (its contents on entry do not matter)."""
    B, T, H, V = x["v"].shape
    hq, K = x["q"].shape[2:]
    dims, head = kda.make_dims(B, T, H, K, V, cu.numel() - 1), x["g"].dim() == 1
    opts = binding.DecayOpts(qk_heads=0 if hq == H else hq, head_gate=int(head))
    ws = torch.full((kda.decay_workspace_size(dims, True, hq, head) // 4,), 3.0, device="cuda")
    out = {n: torch.full_like(x[s], 7.0) for n, s in zip(GRADS, ("q", "k", "v", "g", "h0"))}
    p = lambda t: P(t.data_ptr())  # noqa: E731
    rc = kda.load_library().kda_decay_bwd(p(x["q"]), p(x["k"]), p(x["v"]), p(x["g"]), p(x["do"]), K ** -0.5, p(x["h0"]),
                                          p(x["dht"]), p(cu), *(p(out[n]) for n in GRADS), ctypes.byref(dims),
                                          ctypes.byref(opts), p(word) if word is not None else None, p(ws), ws.numel() * 4,
                                          P(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("H,hq", [(4, 4), (4, 2), (4, 1), (6, 2)])
@pytest.mark.parametrize("gate", ["token", "head"])
def test_no_gradient_is_written(H, hq, gate):
    x = make(1, 300, H, 64, 64, hq=hq, gate=gate, N=3)
    for cu in BAD:
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
        for w in (word, None):
            for n, t in backward(x, bad, w).items():
                assert bool((t == 7.0).all()), (n, cu)
        assert binding.status(word) == 7
    good = torch.tensor([0, 100, 100, 300], dtype=torch.int32, device="cuda")
    want = kda.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], h0=x["h0"], dht=x["dht"], cu_seqlens=good)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = backward(x, good, word)
    assert binding.status(word) == 0 and all(torch.equal(got[n], w) for n, w in zip(GRADS, want))


def test_no_gradient_of_many_sequences_is_written():
    """More sequences than a block has threads, one of them out of order."""
    lens = [(5 * i) % 7 for i in range(700)]
    x = make(1, sum(lens), 3, 64, 64, hq=1, gate="head", N=len(lens))
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    for i in (1, 350, 699):
        bad = cu.clone()
        bad[i] = sum(lens) + 1
        for n, t in backward(x, bad.cuda(), None).items():
            assert bool((t == 7.0).all()), (n, i)


def step(x, state, cu, slots, word):
    out = torch.full_like(x["v"], 7.0)
    kda.decay_step(x["q"], x["k"], x["v"], x["g"], state, slots=slots, cu_seqlens=cu, out=out, status=word)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("with_slots", [True, False])
@pytest.mark.parametrize("K,V,st", [(128, 128, torch.float32), (64, 64, torch.bfloat16), (64, 128, torch.float32)])
def test_no_state_and_no_output_is_written(K, V, st, with_slots):
    """0, 3, 1, 4 among them: by their own bounds alone the first and the last sequence would both have rows 1 and 2."""
    x = make(1, 4, 4, K, V, hq=2, h0=False, do=False)
    start = torch.randn((5, 4, K, V), generator=torch.Generator(device="cuda").manual_seed(K), device="cuda").to(st)
    slots = torch.tensor([4, 1, 2], dtype=torch.int32, device="cuda") if with_slots else None
    for cu in ([0, 3, 1, 4], [0, 1, 2, 3], [1, 2, 3, 4], [0, 1, 2, 5], [0, -1, 2, 4], [0, 0, 5, 4], [0, 4, 4, 3]):
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        state, bad = start.clone(), torch.tensor(cu, dtype=torch.int32, device="cuda")
        out = step(x, state, bad, slots, word)
        assert binding.status(word) == 7, cu
        assert torch.equal(state, start) and bool((out == 7.0).all()), cu
        assert bool((step(x, state, bad, slots, None) == 7.0).all()) and torch.equal(state, start)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    state, good = start.clone(), torch.tensor([0, 1, 3, 4], dtype=torch.int32, device="cuda")
    out = step(x, state, good, slots, word)
    assert binding.status(word) == 0 and bool((out != 7.0).any()) and not torch.equal(state, start)


def test_one_of_many_sequences_is_out_of_order():
    """More sequences than a block has threads; a slot given twice and one outside the cache do not hide it."""
    N = 300
    x = make(1, 2 * N, 2, 64, 64, h0=False, do=False)
    start = torch.randn((N + 1, 2, 64, 64), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    slots = torch.arange(N, dtype=torch.int32, device="cuda")
    slots[7], slots[9] = 6, N + 5
    cu = torch.arange(0, 2 * N + 1, 2, dtype=torch.int32)
    for i in (1, 2, 3, 4, 150, N - 3, N - 2, N - 1):
        bad = cu.clone()
        bad[i] = 2 * N + 1
        state, word = start.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
        out = step(x, state, bad.cuda(), slots, word)
        assert word.item() != 0 and torch.equal(state, start) and bool((out == 7.0).all()), i


@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 127, 128, 129, 515])
def test_each_of_so_many_sequences_out_of_order(N):
    """The offset that is wrong: any of them, the first and the last among them; and none."""
    x = make(1, 3 * N, 1, 64, 64, h0=False, do=False)
    start = torch.zeros((N, 1, 64, 64), device="cuda")
    cu = torch.arange(0, 3 * N + 1, 3, dtype=torch.int32, device="cuda")
    for i in sorted({*range(min(N, 9) + 1), N // 2, N - 1, N}):
        bad = cu.clone()
        bad[i] = 2 if i == 0 else int(cu[i - 1]) - 1 if i < N else 3 * N - 1
        state, word = start.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
        out = step(x, state, bad, None, word)
        assert binding.status(word) == 7 and bool((state == 0.0).all()) and bool((out == 7.0).all()), i
    state, word = start.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    step(x, state, cu, None, word)
    assert binding.status(word) == 0 and bool((state != 0.0).any(-1).any(-1).all())
