"""decay_fwd and decay_bwd in fp16 with scores far below and above fp16's range: scale (q_i . k_j) and
scale (do_i . v_j) are operands of products, and keep their bits whatever their size.

Bounds, u = 2^-11: o, dq, dk, dv are held to u |ref| (the output's rounding; 2^-25 below fp16's normal range) and
(u + 2^-15) W, W the same sum over absolute values, as in decay_util. A score is rounded next to a power of two that
brings the largest that it can be, scale K max|q| max|k|, to 2^13 or more, so it is off by u of itself or by 2^-25 / 2^13 of
that one: over the up to 128 terms of a sum 2^-31 of it times the largest other factor. States, dh0 and dg as in
decay_util (2^-15 W, and for dg 2^-20 of a chunk's pairs), without its allowance for small numbers."""
from __future__ import annotations

import pytest
import torch

import chunked_gated_delta_gb300 as kda
from decay_util import make, offsets, reference, spans
from ops_util import HALF_ULP, TINY, assert_close

pytestmark = pytest.mark.gpu

F16 = torch.float16
U = HALF_ULP[F16]


def largest(x, a, b, scale):
    return scale * x[a].shape[-1] * x[a].abs().max().item() * x[b].abs().max().item()


def compare(got, x, bounds):
    scale = x["q"].shape[-1] ** -0.5
    ref, W = reference(x, bounds, scale, "dq" in got)
    score = largest(x, "q", "k", scale)
    dscore = largest(x, "do", "v", scale) if "do" in x else 0.0
    top = {n: x[n].abs().max().item() for n in ("q", "k", "v", "do") if n in x}
    for name, y in got.items():
        r, w = ref[name], W[name]
        y = y.reshape(r.shape)
        assert torch.isfinite(y).all(), name
        if name in ("o", "dv", "dq", "dk"):
            most = score * top["v" if name == "o" else "do"] if name in ("o", "dv") else dscore * top["k" if name == "dq" else "q"]
            if name in ("dq", "dk"):
                most *= x["v"].shape[2] // x["q"].shape[2]
            assert_close(y, r, U * 1.01, (U + 2.0 ** -15) * w + 2.0 ** -31 * most + TINY[F16], name)
            normal = r.abs() >= 2.0 ** -13  # (below, the output's own steps are wider than 2^-11)
            assert normal.double().mean() > 0.25  # (of the reference: enough of it is looked at)
            off = ((y.double() - r)[normal].norm() / r[normal].norm()).item()
            assert off <= 2 * U, (name, off)
        elif name == "dg":
            pairs = (x["q"].double().abs().flatten(0, 1) * W["dq"]).sum(-1)
            pairs = pairs.repeat_interleave(x["v"].shape[2] // pairs.shape[1], 1)
            most = torch.stack([pairs[a:b].sum(0) for a, b in bounds if b > a]).amax(0)
            assert_close(y, r, 2.0 ** -23, 2.0 ** -15 * w + 2.0 ** -20 * most, name)
        else:
            assert_close(y, r, 2.0 ** -23, 2.0 ** -15 * w, name)


def run(x, cu=None, grads=True):
    o, ht = kda.decay_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], cu_seqlens=cu)
    got = {"o": o, "ht": ht}
    if grads:
        got.update(zip(("dq", "dk", "dv", "dg", "dh0"), kda.decay_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], h0=x["h0"],
                                                                      dht=x["dht"], cu_seqlens=cu)))
    torch.cuda.synchronize()
    return got


def sized(x, **powers):
    """Tensors times powers of two (what leaves fp16's normal range is rounded here, before all)."""
    for n, p in powers.items():
        if x.get(n) is not None:
            x[n] = (x[n].float() * 2.0 ** p).to(x[n].dtype)
    return x


@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("powers", [dict(q=-8, k=-8, v=10), dict(q=-13, k=-2, v=12), dict(q=2, k=-13, v=10), dict(q=12, k=12, v=-14, h0=-4)])
@pytest.mark.parametrize("h0", [False, True])
def test_forward(K, V, powers, h0):
    x = sized(make(2, 300, 2, K, V, io=F16, mean=6.0, seed=K + V, do=False, h0=h0), **powers)
    compare(run(x, grads=False), x, spans([300, 300]))


@pytest.mark.parametrize("powers", [dict(q=-8, k=-8, v=10), dict(q=12, k=12, v=-14, h0=-4)])
def test_forward_packed_and_cut(powers):
    lens = [2500, 0, 1, 33, 130, 640]
    x = sized(make(1, sum(lens), 2, 64, 64, io=F16, hq=1, N=len(lens), mean=4.0, do=False), **powers)
    compare(run(x, offsets(lens), False), x, spans(lens))


def test_forward_tokens_of_very_different_size():
    """Tokens of 2^-12 of others' size among them: their scores keep their bits, as do others of other 32 tokens."""
    x = sized(make(1, 256, 2, 128, 64, io=F16, mean=8.0, h0=False, do=False), v=9, k=-4)
    x["q"] *= torch.exp2(-2.0 * (torch.arange(256, device="cuda") % 7)).to(F16)[None, :, None, None]
    compare(run(x, grads=False), x, spans([256]))


def test_forward_rows_behind_the_end():
    """What lies behind a sequence's end does not choose its scores' power of two (whole rows of other sequences, and NaN)."""
    lens = [70, 57, 33]
    x = sized(make(1, sum(lens), 2, 64, 64, io=F16, N=3, mean=4.0, do=False), q=-7, k=-7, v=9)
    want = run(x, offsets(lens), False)
    for value in (60000.0, torch.nan):
        y = {n: (t.clone() if torch.is_tensor(t) else t) for n, t in x.items()}
        for n in ("q", "k"):
            y[n][:, 70:127] = value
        got = run(y, offsets(lens), False)
        for a, b in ((0, 70), (127, 160)):
            assert torch.equal(got["o"][:, a:b], want["o"][:, a:b]), value
        assert torch.equal(got["ht"][[0, 2]], want["ht"][[0, 2]])
    compare(want, x, spans(lens))


def test_forward_that_grows():
    """g above zero (not what a decay is for) multiplies scores by up to 2^11 over a chunk."""
    x = make(1, 128, 2, 64, 64, io=F16, h0=False, do=False)
    x["g"] = torch.rand(x["g"].shape, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda") * 0.12
    compare(run(x, grads=False), x, spans([128]))


SMALL, LARGE = dict(q=-7, k=-7, v=8, do=8, dht=-8), dict(q=8, k=8, v=-9, do=-9, h0=-9)


@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("powers", [SMALL, LARGE], ids=["small scores", "small gradients of scores"])
@pytest.mark.parametrize("H,hq", [(2, 2), (4, 2), (4, 1)])
def test_gradients(K, V, powers, H, hq):
    x = sized(make(1, 300, H, K, V, hq=hq, io=F16, mean=3.0, seed=K + V), **powers)
    compare(run(x), x, spans([300]))


@pytest.mark.parametrize("hq", [2, 1])
def test_gradients_of_scores_above_fp16s_range(hq):
    x = sized(make(2, 200, 2, 64, 64, hq=hq, io=F16, mean=3.0), q=11, k=11, v=-12, do=-9, h0=-12)
    q, k = (t.double().transpose(1, 2) for t in (x["q"], x["k"]))
    assert 64 ** -0.5 * (q @ k.transpose(-1, -2)).tril().abs().max().item() > 2 * 65504
    compare(run(x), x, spans([200, 200]))


@pytest.mark.parametrize("gate", ["token", "head"])
def test_gradients_packed(gate):
    lens = [1, 0, 129, 300, 127]
    x = sized(make(1, sum(lens), 4, 64, 128, hq=2, io=F16, gate=gate, N=len(lens), mean=3.0), **SMALL)
    compare({n: t for n, t in run(x, offsets(lens)).items() if gate == "token" or n != "dg"}, x, spans(lens))
