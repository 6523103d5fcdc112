"""cu_seqlens out of order, beyond the rows or short of them: decay_bwd reports it and writes nothing, whichever kernels
a head layout and a form of the decay bring in."""
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
