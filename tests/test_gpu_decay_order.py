"""Order and place of decay_fwd, decay_bwd, decay_step and rotary: inputs written by the kernel right
before, outputs read and inputs overwritten right after, two streams at once with workspaces of their
own, outputs of another stream's memory, and tensors of more than 2^31 elements."""
from __future__ import annotations

import pytest
import torch

import chunked_gated_delta_gb300 as kda
from decay_util import make, offsets

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "g", "do", "h0", "dht")


def both(x, stream=None):
    o, ht = kda.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], stream=stream)
    return (o, ht, *kda.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], h0=x["h0"], dht=x["dht"], stream=stream))


@pytest.mark.parametrize("T,H,hq", [(300, 8, 8), (2600, 2, 1)])
def test_inputs_written_right_before_and_overwritten_right_after(T, H, hq):
    src = [make(1, T, H, 128, 128, hq=hq, seed=i) for i in range(3)]
    want = []
    for x in src:
        torch.cuda.synchronize()
        want.append([t.clone() for t in both(x)])
        torch.cuda.synchronize()
    buf = {n: torch.empty_like(src[0][n]) for n in NAMES}
    for _ in range(5):
        got = []
        for x in src:
            for n in NAMES:
                buf[n].copy_(x[n])
            got.append(both(buf))
            for n in NAMES:
                buf[n].fill_(float("nan"))
        for a, b in zip(got, want):
            for t, u in zip(a, b):
                assert torch.equal(t, u)


def test_a_chain_of_operators():
    """norm -> rotary in place -> prompt -> step on its state, again and again without a wait."""
    x = [make(2, 140, 4, 64, 64, h0=False, do=False, seed=i) for i in range(4)]
    freqs, _ = kda.rotary_freqs(64)
    pos = torch.arange(140, device="cuda").expand(2, 140).contiguous()

    def run(y):
        q, k = (kda.rms_norm(y[n])[0] for n in ("q", "k"))
        kda.rotary(q, k, pos, freqs, q_out=q, k_out=k)
        o, s = kda.decay_fwd(q, k, y["v"], y["g"])
        tail = [kda.decay_step(*(t[:, i:i + 1].contiguous() for t in (q, k, y["v"], y["g"])), s) for i in range(4)]
        return (o, s, *tail)

    want = []
    for y in x:
        want.append([t.clone() for t in run(y)])
        torch.cuda.synchronize()
    got = [run(y) for _ in range(6) for y in x]
    for i, a in enumerate(got):
        for t, u in zip(a, want[i % 4]):
            assert torch.equal(t, u)


def test_two_streams_at_once():
    xs = [make(1, 3000, 3, 128, 128, seed=i) for i in range(2)]
    want = [[t.clone() for t in both(x)] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [both(x, stream=s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for t, u in zip(a, b):
                assert torch.equal(t, u)


def test_pairs_on_two_streams_at_once():
    """Clusters of two calls on the same SMs, with more of them than fit at once."""
    xs = [make(2, 2100, 16, 128, 64, hq=8, seed=i) for i in range(2)]
    want = [[t.clone() for t in both(x)] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [both(x, stream=s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for t, u in zip(a, b):
                assert torch.equal(t, u)


def test_outputs_belong_to_the_stream():
    """What a call on another stream allocates is that stream's: memory freed there with work pending is not handed
    to this one (the workspace is freed as the call returns)."""
    x = make(1, 2600, 2, 128, 128)
    want = both(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = both(x, stream=side)
        noise = [torch.full((1 << 22,), float("nan"), device="cuda") for _ in range(8)]  # on the current stream
        torch.cuda.synchronize()
        for t, u in zip(got, want):
            assert torch.equal(t, u)
        del noise


def test_packed_sequences_of_one_graph_with_other_lengths():
    """A captured call takes the lengths that cu_seqlens holds when it is replayed."""
    lens = [[100, 0, 300, 29], [1, 400, 20, 8]]
    x = make(1, 429, 2, 128, 128, N=4, do=False)
    want = [kda.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], cu_seqlens=offsets(n)) for n in lens]
    cu, o, ht = offsets(lens[0]), torch.empty_like(x["v"]), torch.empty_like(x["h0"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], cu_seqlens=cu, out=o, final_state=ht)
    for i in (0, 1, 0):
        cu.copy_(offsets(lens[i]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[i][0]) and torch.equal(ht, want[i][1])


def test_more_than_31_bits_of_elements():
    B, T, H, K = 9, 16500, 128, 128
    assert B * T * H * K > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(0)
    q, k, v, do = (torch.randn((B, T, H, K), generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    g = -0.05 * torch.rand((B, T, H), generator=gen, device="cuda")
    o, ht = kda.decay_fwd(q, k, v, g, scale=1e-3)
    tail = [t[-1:].contiguous() for t in (q, k, v, g)]
    o1, ht1 = kda.decay_fwd(*tail, scale=1e-3)
    assert (o[-1:].float() - o1.float()).norm() <= 1e-2 * o1.float().norm() and (ht[-1:] - ht1).norm() <= 1e-5 * ht1.norm()
    del o, o1
    dq, dk, dv, dg, dh0 = kda.decay_bwd(q, k, v, g, do, scale=1e-3)
    want = kda.decay_bwd(*tail, do[-1:].contiguous(), scale=1e-3)
    for name, a, b in zip(("dq", "dk", "dv", "dg", "dh0"), (dq, dk, dv, dg, dh0), want):
        assert (a[-1:].float() - b.float()).norm() <= (1e-5 if name in ("dg", "dh0") else 1e-2) * b.float().norm(), name
