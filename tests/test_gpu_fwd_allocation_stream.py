"""What fwd, state_map, chain_states and bwd_dh allocate belongs to the stream that
they run on, and what they fill for their kernels is filled there."""
from __future__ import annotations

from types import SimpleNamespace

import pytest
import torch

import chunked_gated_delta_gb300 as kda
from chunked_gated_delta_gb300 import dist as kdist
from chunked_gated_delta_gb300 import synth
from parity_util import make, to_dev

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "g", "beta")


def stream_of_block(t):
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in the allocator's segments")


def calls():
    """name -> a function of the stream that returns the allocated tensors."""
    x = synth.make_inputs(make(B=2, T=300, H=3, seed=31))
    d = to_dev(x)
    a = [d[n] for n in NAMES]
    dims = kda.make_dims(2, 300, 3, 128, 128)
    ws = kda.new_workspace(dims, "cuda")
    kda.fwd(*a, h0=d["h0"], workspace=ws)
    pq = torch.stack([kda.state_map(*a)[0], kda.state_map(*a)[0]])
    maps, _, _ = kda.state_map(*a, workspace=ws)
    shard = kdist.plan_shard(2, 300, 3, 1, 2, None)
    do = d["v"].clone()

    def bwd(s):
        return kda.bwd_dh(x["scale"], do, d["v"], None, dims, ws, stream=s)

    def finish(s):
        return kdist.context_parallel_finish(pq, 1, ws, dims, x["scale"], h0=d["h0"], stream=s)

    return {"fwd": lambda s: kda.fwd(*a, h0=d["h0"], stream=s),
            "state_map": lambda s: kda.state_map(*a, stream=s)[:1],
            "chain_states": lambda s: (kda.chain_states(pq, d["h0"], stream=s),),
            "bwd_dh": bwd, "context_parallel_finish": finish,
            "fwd_shard": lambda s: kdist.fwd_shard(shard, *a, h0=d["h0"], stream=s)}


@pytest.mark.parametrize("op", ["fwd", "state_map", "chain_states", "bwd_dh", "context_parallel_finish", "fwd_shard"])
def test_allocations_on_another_stream(op):
    """The current stream is kept busy (about 10 ms) when the call is made on the other one, and then writes
    blocks of the outputs' sizes that were freed: the call takes none of them."""
    call = calls()[op]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    before = torch.cuda.current_stream()
    held = [torch.empty_like(t) for t in want]
    torch.cuda._sleep(20_000_000)
    for t in held:
        t.view(torch.uint8).fill_(0xFF)
    pending = {t.data_ptr() for t in held}
    del held, t
    outs = call(side)
    assert torch.cuda.current_stream() == before
    side.synchronize()
    got = [t.clone() for t in outs]
    torch.cuda.synchronize()
    assert not pending & {t.data_ptr() for t in outs}
    assert all(stream_of_block(t) == side.cuda_stream for t in outs)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


@pytest.mark.parametrize("op", ["fwd", "chain_states", "bwd_dh"])
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
