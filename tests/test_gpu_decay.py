"""decay_fwd and decay_bwd against 64 bits (decay_util): types, head layouts, lengths around the
chunk's and a warp's ends, packed rows with empty sequences, decays from none to all, states, strides,
sequences cut into pieces, and what they refuse."""
from __future__ import annotations

import pytest
import torch

import chunked_gated_delta_gb300 as kda
from chunked_gated_delta_gb300 import binding
from decay_util import compare, make, offsets, spans
from ops_util import Guarded

pytestmark = pytest.mark.gpu


def run(x, cu=None, grads=True, **kw):
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, ht = kda.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], cu_seqlens=cu, status=word, **kw)
    got = {"o": o, "ht": ht}
    if grads:
        names = ("dq", "dk", "dv", "dg", "dh0")
        got.update(zip(names, kda.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], h0=x["h0"], dht=x["dht"],
                                            cu_seqlens=cu, status=word, **kw)))
    torch.cuda.synchronize()
    assert word.item() == 0
    return got


def rows(B, T):
    return [(b * T, (b + 1) * T) for b in range(B)]


@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16])
def test_forward_types_and_dims(K, V, io):
    x = make(2, 300, 2, K, V, io=io, seed=K + V, do=False)
    compare(run(x, grads=False), x, rows(2, 300))


@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16])
def test_gradients_types_and_dims(K, V, io):
    x = make(2, 300, 2, K, V, io=io, seed=K + V)
    compare(run(x), x, rows(2, 300))


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 255, 256, 257, 384, 511])
def test_lengths(T):
    x = make(1, T, 3, 128, 128, seed=T)
    compare(run(x), x, rows(1, T))


@pytest.mark.parametrize("H,hq", [(1, 1), (5, 5), (6, 2), (8, 1), (12, 4)])
@pytest.mark.parametrize("gate", ["token", "head"])
def test_heads(H, hq, gate):
    x = make(2, 200, H, 128, 64, hq=hq, gate=gate, seed=H)
    compare(run(x), x, rows(2, 200))


@pytest.mark.parametrize("H,hq", [(2, 1), (6, 3), (12, 3), (16, 2), (16, 1), (7, 1)])
@pytest.mark.parametrize("K,V,io", [(128, 128, torch.bfloat16), (64, 128, torch.float16), (128, 64, torch.float16)])
def test_groups(H, hq, K, V, io):
    """Value heads that share q and k, by twos, fours, eights and others: their gradients are summed, rows behind a
    sequence's end left out, with the same bits each time."""
    lens = [1, 0, 129, 300, 127]
    x = make(1, sum(lens), H, K, V, hq=hq, io=io, N=len(lens), seed=H + hq)
    a, b = run(x, cu=offsets(lens)), run(x, cu=offsets(lens))
    compare(a, x, spans(lens))
    for name in ("dq", "dk", "dv", "dg", "dh0"):
        assert torch.equal(a[name], b[name])


@pytest.mark.parametrize("lens", [[5], [0, 7, 0, 130, 128, 1, 0], [300, 1, 2, 299], [0, 0]])
@pytest.mark.parametrize("K,V,io", [(128, 128, torch.bfloat16), (64, 64, torch.float16)])
def test_packed(lens, K, V, io):
    x = make(1, sum(lens), 4, K, V, hq=2, io=io, N=len(lens), seed=len(lens))
    compare(run(x, cu=offsets(lens)), x, spans(lens))


def test_many_packed():
    lens = [(7 * i) % 23 for i in range(700)]
    x = make(1, sum(lens), 2, 64, 64, N=len(lens))
    compare(run(x, cu=offsets(lens)), x, spans(lens))


@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("h0", [True, False])
def test_states(state, h0):
    x = make(2, 130, 2, 128, 128, state=state, h0=h0)
    got = run(x, grads=False, state_dtype=state)
    assert got["ht"].dtype == state
    compare(got, x, rows(2, 130))
    if h0 or state == torch.float32:
        if not h0:
            x["dht"] = None
        compare(run(x), x, rows(2, 130))
    o, none = kda.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], output_final_state=False)
    assert none is None and torch.equal(o, got["o"])
    assert kda.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], h0=x["h0"], want_dh0=False)[4] is None


@pytest.mark.parametrize("mean", [-3.0, 0.0, 8.0, 15.0])
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16])
def test_decays(mean, io):
    x = make(1, 400, 2, 128, 128, mean=mean, io=io, seed=int(mean) + 9)
    compare(run(x), x, rows(1, 400))


def test_no_decay_and_total_decay():
    """g = 0 keeps everything; g = -1000 (or any below, -inf among them) at a token wipes the state there: what is before
    it does not reach what is behind, and the tokens behind it keep their decays to fp32."""
    x = make(1, 400, 3, 128, 128, mean=6.0)
    x["g"][:, :, 0] = 0.0
    x["g"][:, 57::61, 1] = -1000.0
    x["g"][:, 130, 2] = -1000.0
    compare(run(x), x, rows(1, 400))
    a = run(x)
    for low in (-1e30, -torch.inf):
        x["g"][:, 130, 2] = low
        b = run(x)
        for n in ("o", "ht", "dq", "dk", "dv", "dg", "dh0"):
            assert torch.equal(a[n], b[n]) and torch.isfinite(b[n].float()).all(), n


def test_scale():
    x = make(1, 150, 2, 64, 128)
    o, ht = kda.decay_fwd(x["q"], x["k"], x["v"], x["g"], scale=0.7, h0=x["h0"])
    grads = kda.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], scale=0.7, h0=x["h0"], dht=x["dht"])
    compare(dict(o=o, ht=ht, **dict(zip(("dq", "dk", "dv", "dg", "dh0"), grads))), x, rows(1, 150), scale=0.7)


def test_large_states_in_fp16():
    """States far above fp16's range stay finite and exact: they are products' operands by a power of two."""
    x = make(1, 300, 2, 128, 128, io=torch.float16, mean=9.0)
    x["h0"] *= 1e6
    x["dht"] *= 1e5
    x["q"] *= 2.0 ** -8
    x["do"] *= 2.0 ** -10
    compare(run(x, grads=False), x, rows(1, 300))
    got = run(x)
    got = {n: got[n] for n in ("dq", "dg", "dh0")}  # (dk and dv are beyond fp16)
    compare(got, x, rows(1, 300))


@pytest.mark.parametrize("T,H", [(4096, 1), (3001, 2), (6000, 3)])
def test_cut_sequences(T, H):
    """Few heads over long sequences run in pieces."""
    d = kda.make_dims(1, T, H, 64, 64)
    assert kda.decay_workspace_size(d, False) > 0
    x = make(1, T, H, 64, 64, mean=5.0, seed=T)
    compare(run(x), x, rows(1, T))


def test_cut_packed():
    lens = [2500, 0, 1, 2049, 130, 640]
    x = make(1, sum(lens), 2, 128, 128, N=len(lens), mean=6.0, gate="head")
    assert kda.decay_workspace_size(kda.make_dims(1, sum(lens), 2, 128, 128, len(lens)), False) > 0
    compare(run(x, cu=offsets(lens)), x, spans(lens))


def test_differences():
    """dg and dq against differences of the forward's own sum, in 64 bits of the reference's forward."""
    from decay_util import reference
    x = make(1, 200, 1, 64, 64, mean=2.0)
    dq, _, _, dg, _ = kda.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], h0=x["h0"], dht=x["dht"])

    def total(y):
        r, _ = reference(y, rows(1, 200))
        return (r["o"] * x["do"].double().flatten(0, 1)).sum() + (r["ht"] * x["dht"].double()).sum()

    for t in (0, 77, 128, 199):
        step = 1e-4
        up, down = ({**x, "g": x["g"].double().clone()} for _ in range(2))
        up["g"][0, t, 0] += step
        down["g"][0, t, 0] -= step
        slope = ((total(up) - total(down)) / (2 * step)).item()
        assert abs(dg[0, t, 0].item() - slope) <= 1e-4 * max(1.0, abs(slope)), t
        up, down = ({**x, "q": x["q"].double().clone()} for _ in range(2))
        up["q"][0, t, 0, 5] += step
        down["q"][0, t, 0, 5] -= step
        slope = ((total(up) - total(down)) / (2 * step)).item()
        assert abs(dq[0, t, 0, 5].item() - slope) <= 2.0 ** -6 * max(1.0, abs(slope)), t


def test_rows_of_a_wider_projection():
    B, T, H, K, V = 2, 140, 2, 64, 128
    x = make(B, T, H, K, V)
    wide = torch.randn(B, T, 2 * H * K + 2 * H * V + 8, device="cuda").to(torch.bfloat16)
    y, at = dict(x), 0
    for n, w in (("q", H * K), ("k", H * K), ("v", H * V), ("do", H * V)):
        part = wide[..., at:at + w].unflatten(-1, (H, -1))
        part.copy_(x[n])
        y[n], at = part, at + w
    gates = torch.randn(B, T, H + 3, device="cuda")
    gates[..., 1:H + 1] = x["g"]
    y["g"] = gates[..., 1:H + 1]
    a, b = run(x), run(y)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_neighbours_do_not_reach_a_sequence():
    """NaN in the rows of the next sequence, and behind the last, changes nothing; nothing else is written."""
    lens = [70, 200, 33]
    x = make(1, sum(lens), 2, 128, 128, N=3)
    want = run(x, cu=offsets(lens))
    bad = {n: (t.clone() if torch.is_tensor(t) else t) for n, t in x.items()}
    for n in ("q", "k", "v", "do"):
        bad[n][:, 70:270] = torch.nan
    got = run(bad, cu=offsets(lens))
    for n in ("o", "dq", "dk", "dv", "dg"):
        for a, b in ((0, 70), (270, 303)):
            assert torch.equal(got[n][:, a:b], want[n][:, a:b]), n
    for n in ("ht", "dh0"):
        assert torch.equal(got[n][[0, 2]], want[n][[0, 2]]), n
    o, ht = Guarded((1, 303, 2, 128), torch.bfloat16), Guarded((3, 2, 128, 128), torch.float32)
    kda.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], cu_seqlens=offsets(lens), out=o.t, final_state=ht.t)
    torch.cuda.synchronize()
    assert o.intact() and ht.intact() and torch.equal(o.t, want["o"]) and torch.equal(ht.t, want["ht"])


def test_same_bits_twice_and_in_a_graph():
    x = make(1, 2100, 2, 128, 128, hq=1, gate="head")
    d = kda.make_dims(1, 2100, 2, 128, 128)
    ws = [torch.empty(kda.decay_workspace_size(d, back, 1, True), dtype=torch.uint8, device="cuda") for back in (False, True)]
    want = run(x)
    o, ht = torch.empty_like(want["o"]), torch.empty_like(want["ht"])
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kda.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], h0=x["h0"], dht=x["dht"])
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kda.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], workspace=ws[0], out=o, final_state=ht)
        grads = kda.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], h0=x["h0"], dht=x["dht"], workspace=ws[1])
    for w in ws:
        w.fill_(0xFF)  # (its contents on entry do not matter: NaN here)
    for _ in range(2):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want["o"]) and torch.equal(ht, want["ht"])
        for n, y in zip(("dq", "dk", "dv", "dg", "dh0"), grads):
            assert torch.equal(y, want[n]), n


def test_bad_offsets_are_reported():
    x = make(1, 300, 2, 64, 64, N=3)
    for cu in ([0, 100, 50, 300], [0, 100, 200, 299], [1, 100, 200, 300], [0, 100, 400, 300], [0, -5, 200, 300]):
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
        o = torch.full((1, 300, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        kda.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], cu_seqlens=bad, status=word, out=o)
        assert binding.status(word) == 7 and bool((o == 7.0).all())
        word.zero_()
        kda.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], h0=x["h0"], cu_seqlens=bad, status=word)
        assert binding.status(word) == 7
    run(x, cu=offsets([100, 100, 100]))


def test_bad_offsets_of_pairs_are_reported():
    """A pair's two CTAs leave together, and what comes after is as always."""
    x = make(1, 300, 4, 64, 64, hq=2, N=3)
    for cu in ([0, 100, 50, 300], [0, 100, 200, 299], [0, 100, 400, 300]):
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
        kda.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], h0=x["h0"], dht=x["dht"], cu_seqlens=bad, status=word)
        torch.cuda.synchronize()
        assert word.item() != 0
    compare(run(x, cu=offsets([100, 150, 50])), x, spans([100, 150, 50]))


def test_no_tokens():
    for shape in ((2, 0), (1, 0)):
        x = make(*shape, 2, 64, 64)
        got = run(x)
        assert torch.equal(got["ht"], x["h0"]) and torch.equal(got["dh0"], x["dht"]) and got["o"].numel() == 0
    x = make(1, 0, 2, 64, 64, gate="head")
    assert torch.equal(run(x)["dg"], torch.zeros(2, device="cuda"))


def test_on_another_stream():
    x = make(1, 700, 4, 128, 128)
    want = run(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, ht = kda.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], stream=side)
    grads = kda.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], h0=x["h0"], dht=x["dht"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for n, y in zip(("o", "ht", "dq", "dk", "dv", "dg", "dh0"), (o, ht, *grads)):
        assert torch.equal(y, want[n]), n


def test_refusals():
    x = make(1, 20, 2, 64, 64)
    ok = (x["q"], x["k"], x["v"], x["g"])

    def no(error, *a, **kw):
        with pytest.raises(error):
            kda.decay_fwd(*a, **kw)

    no(TypeError, x["q"].float(), *ok[1:])
    no(TypeError, x["q"], x["k"].half(), *ok[2:])
    no(TypeError, x["q"][:, :10], *ok[1:])
    no(TypeError, *ok[:3], x["g"].half())
    no(TypeError, *ok[:3], x["g"][..., :1])
    no(TypeError, *ok, h0=x["h0"].half())
    no(TypeError, *ok, h0=x["h0"], state_dtype=torch.bfloat16)
    no(TypeError, *ok, h0=x["h0"][:, :1])
    no(TypeError, *ok, cu_seqlens=torch.tensor([0, 20]))
    no(TypeError, x["q"].cpu(), *ok[1:])
    no(TypeError, *ok, workspace=torch.empty(8, device="cuda"))
    no(TypeError, *ok, out=torch.empty(1, 20, 2, 64, device="cuda"))
    no(kda.KdaError, *ok, h0=x["h0"], final_state=x["h0"])          # (one memory)
    no(kda.KdaError, x["q"][..., :32].contiguous(), x["k"][..., :32].contiguous(), *ok[2:])
    odd = torch.empty(1, 20, 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")[..., :128].unflatten(-1, (2, 64))
    no(kda.KdaError, odd, *ok[1:])                                   # (rows off 16 bytes)
    with pytest.raises(TypeError):
        kda.decay_bwd(*ok, x["do"].float())
    with pytest.raises(TypeError):
        kda.decay_bwd(*ok, x["do"], h0=x["h0"], dht=x["dht"].to(torch.bfloat16))
    with pytest.raises(kda.KdaError):
        kda.decay_bwd(*ok, x["do"], workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
