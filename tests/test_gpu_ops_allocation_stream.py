"""Outputs of step, rms_norm and linear belong to the stream that the call runs on:
memory that the current stream may still use, or soon gives away, is not theirs."""
from __future__ import annotations

from types import SimpleNamespace

import pytest
import torch

import chunked_gated_delta_gb300 as kda

pytestmark = pytest.mark.gpu

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn
M, D = 512, 1024


def randn(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def calls():
    """name -> a function of the stream that returns the allocated outputs."""
    x, r = randn(M, D, seed=1).to(BF16), randn(M, D, seed=2).to(BF16)
    w = (randn(D, D, seed=3) / 32).to(BF16)
    q, k = (torch.nn.functional.normalize(randn(M, 1, 4, 64, seed=s), dim=-1).to(BF16) for s in (4, 5))
    v, g = randn(M, 1, 4, 64, seed=6).to(BF16), -torch.rand((M, 1, 4, 64), device="cuda")
    beta, state = torch.rand((M, 1, 4), device="cuda").to(BF16), 0.1 * randn(M, 4, 64, 64, seed=7)
    return {"step": lambda s: (kda.step(q, k, v, g, beta, state.clone() if s is None else state, stream=s),),
            "rms_norm": lambda s: kda.rms_norm(x, residual=r, out_dtype=F8, stream=s),
            "linear": lambda s: (kda.linear(x, w, residual=r, act="silu", stream=s),)}


def stream_of_block(t):
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in the allocator's segments")


@pytest.mark.parametrize("op", ["step", "rms_norm", "linear"])
def test_outputs_are_allocated_for_the_given_stream(op):
    call = calls()[op]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    before = torch.cuda.current_stream()
    outs = call(side)
    assert torch.cuda.current_stream() == before
    side.synchronize()
    assert all(stream_of_block(t) == side.cuda_stream for t in outs)
    with torch.cuda.stream(side):
        assert all(stream_of_block(t) == side.cuda_stream for t in call(None))
    side.synchronize()
    assert all(stream_of_block(t) == before.cuda_stream for t in call(None))
    assert all(stream_of_block(t) == before.cuda_stream for t in call(torch.cuda.default_stream()))
    torch.cuda.synchronize()


@pytest.mark.parametrize("op", ["step", "rms_norm", "linear"])
def test_memory_with_work_pending_is_not_taken(op):
    """Blocks of the outputs' sizes are freed while the current stream still has to write them."""
    call = calls()[op]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    held = [torch.empty_like(t) for t in want]
    torch.cuda._sleep(20_000_000)  # about 10 ms
    for t in held:
        t.view(torch.uint8).fill_(0xFF)
    pending = {t.data_ptr() for t in held}
    del held, t
    outs = call(side)
    torch.cuda.synchronize()
    assert not pending & {t.data_ptr() for t in outs}
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(outs, want))


@pytest.mark.parametrize("op", ["step", "rms_norm", "linear"])
def test_another_librarys_stream(op):
    """An object with a handle and no more."""
    call = calls()[op]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = call(SimpleNamespace(cuda_stream=side.cuda_stream))
    torch.cuda.synchronize()
    assert all(stream_of_block(t) == side.cuda_stream for t in outs)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(outs, want))
