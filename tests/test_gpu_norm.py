"""kda.rms_norm against the formula in 64 bits.

Tolerances: one rounding of each output to its type, plus the fp32 arithmetic:
a sum of squares of positive terms joins at most 32 + 10 terms in a row (45
roundings, halved by the root), a division, a root and three products: 32
roundings of 2^-24.  An 8-bit code stands for a value within half a step (and
those 32 roundings) of y * 448 / a.
"""
from __future__ import annotations

import pytest
import torch

import chunked_gated_delta_gb300 as kda
from ops_util import EPS32, HALF_ULP, TINY, Guarded, assert_close

pytestmark = pytest.mark.gpu

F32_REL = 32 * EPS32
F8 = torch.float8_e4m3fn


def randn(*shape, seed=0, dtype=torch.float32):
    gen = torch.Generator(device="cuda").manual_seed(seed + 3)
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def reference(x, w, r, eps):
    s = x.double() + (r.double() if r is not None else 0.0)
    y = s / torch.sqrt(s.square().mean(-1, keepdim=True) + eps)
    return (y * w.double() if w is not None else y), s


def check(x, w=None, r=None, out=None, eps=1e-6):
    out = x.dtype if out is None else out
    y_ref, s_ref = reference(x, w, r, eps)
    y, scale, s = kda.rms_norm(x, w, residual=r, eps=eps, out_dtype=out)
    torch.cuda.synchronize()
    assert y.dtype == out and y.shape == x.shape and (scale is None) == (out != F8) and (s is None) == (r is None)
    if r is not None:
        assert_close(s, s_ref, HALF_ULP[x.dtype] * 1.01, TINY[x.dtype], "sum")
    if out != F8:
        rel = F32_REL + (HALF_ULP[out] * 1.01 if out != torch.float32 else 0.0)
        assert_close(y, y_ref, rel, TINY[out], "y")
        return
    a = y_ref.abs().amax(-1).clamp_min(1e-30)
    assert_close(scale, a / 448, F32_REL, 0.0, "scale")
    want = y_ref * (448 / a)[..., None]
    half_step = torch.exp2(torch.floor(torch.log2(want.abs().clamp_min(2.0 ** -6))) - 4)
    assert_close(y.float(), want, 2 * F32_REL, half_step * (1 + 1e-9), "codes")


DIMS = [1, 2, 7, 8, 24, 64, 100, 128, 129, 250, 256, 264, 500, 512, 1000, 1024, 1032, 2048, 3333, 4096, 4104, 5003,
        8192, 9001, 16384, 20000, 32761, 32768]


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16, torch.float32])
def test_dims_and_types(dim, io):
    for rows, residual, weight, out in ((1, True, True, F8), (3, False, True, io), (37, True, False, torch.float32),
                                        (2, False, False, F8), (9, True, True, io)):
        x = randn(rows, dim, seed=dim, dtype=io)
        r = 2 * randn(rows, dim, seed=dim + 1, dtype=io) if residual else None
        w = (1 + 0.3 * randn(dim, seed=dim + 2)).to(io) if weight else None
        check(x, w, r, out)


def test_weight_in_32_bits_and_shapes():
    x = randn(2, 3, 5, 128, dtype=torch.bfloat16)
    check(x, 1 + randn(128, seed=4), None)
    check(x, 1 + randn(128, seed=4), x.flip(0), F8)
    check(x.float(), 1 + randn(128, seed=4), None, F8, eps=0.0)
    check(x[0, 0, 0], None, None)  # one row as a vector
    y, s, r = kda.rms_norm(x[:0], None)
    assert y.shape == x[:0].shape and s is None and r is None


@pytest.mark.parametrize("out", [None, F8, torch.float32])
def test_strides_and_alignment(out):
    """Rows apart from one another, and rows that start off 16 bytes."""
    wide = randn(11, 1000, dtype=torch.bfloat16)
    for a, b in ((0, 512), (8, 520), (1, 513), (3, 900)):
        check(wide[:, a:b], None, None, out)
        check(wide[:, a:b], (1 + randn(1000, dtype=torch.bfloat16))[a:b].clone(), wide.flip(0)[:, a:b], out)
    check(wide[::2, :128], None, None, out)
    check(wide[:, :600].unflatten(0, (11, 1)), None, None, out)


@pytest.mark.parametrize("dim", [31, 33, 127, 250, 513, 1001, 4095, 5003, 16383, 32761])
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16, torch.float32])
def test_rows_off_16_bytes(dim, io):
    """Every distance of a row's start from 16 bytes; x, residual and sum alike or not; nothing outside is written."""
    flat = randn(40 * dim + 64, seed=dim, dtype=io)
    for lead in (0, 1, 3, 7):
        x = flat[lead:lead + 17 * dim].view(17, dim)
        for rlead in (lead, lead + 1):
            r = flat.flip(0)[rlead:rlead + 17 * dim].view(17, dim)
            for out in (io, F8, torch.float32):
                check(x, 1 + 0.3 * randn(dim, seed=2).to(io), r, out)
                check(x, None, None, out)
        raw = torch.full((17 * dim + 32,), 7.0, dtype=io, device="cuda")
        part = raw[lead:lead + 17 * dim].view(17, dim)
        y, _, s = kda.rms_norm(x, None, residual=x, residual_out=part)
        torch.cuda.synchronize()
        assert torch.equal(part, (x.float() + x.float()).to(io))
        assert (raw[:lead] == 7).all() and (raw[lead + 17 * dim:] == 7).all()


@pytest.mark.parametrize("dim", [1032, 2048, 2056, 4096, 5000, 8192])
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16, torch.float32])
def test_many_long_rows_with_residual(dim, io):
    """Enough rows for the kernel that streams them, contiguous and apart, in place, and rows with NaN."""
    for rows in (2432, 2500, 7001):
        wide = 2 * randn(rows, dim + 16, seed=rows, dtype=io)
        for x, r in ((randn(rows, dim, seed=dim, dtype=io), wide[:, :dim].contiguous()),
                     (wide[:, 8:dim + 8], wide.flip(0)[:, :dim])):
            for out in (io, F8, torch.float32):
                check(x, (1 + 0.3 * randn(dim, seed=2)).to(io), r, out)
        x, r, w = randn(rows, dim, seed=1, dtype=io), randn(rows, dim, seed=2, dtype=io), 1 + randn(dim, seed=3)
        x[17, 5], x[rows - 1, dim - 1] = float("nan"), float("nan")
        y0, q0, s0 = kda.rms_norm(x, w, residual=r, out_dtype=F8)
        y, q, s = kda.rms_norm(x, w, residual=r, out_dtype=F8, residual_out=r)
        torch.cuda.synchronize()
        assert s is r
        for a, b in ((y0, y), (q0, q), (s0, s)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        bad = torch.isnan(q)
        assert bad[[17, rows - 1]].all() and int(bad.sum()) == 2 and torch.isnan(y.float()[bad]).all()


def test_sum_in_place():
    for dim in (128, 4096, 5003):
        x, r = randn(13, dim, dtype=torch.bfloat16), randn(13, dim, seed=1, dtype=torch.bfloat16)
        w = randn(dim, seed=2)
        y0, _, s0 = kda.rms_norm(x, w, residual=r)
        for into in ("r", "x"):
            xx, rr = x.clone(), r.clone()
            dst = rr if into == "r" else xx
            y, _, s = kda.rms_norm(xx, w, residual=rr, residual_out=dst)
            assert s is dst and torch.equal(y, y0) and torch.equal(s, s0)
        apart = torch.zeros(13, dim + 8, dtype=torch.bfloat16, device="cuda")
        kda.rms_norm(x, w, residual=r, residual_out=apart[:, :dim])
        assert torch.equal(apart[:, :dim], s0) and (apart[:, dim:] == 0).all()


@pytest.mark.parametrize("dim", [8, 128, 1000, 1001, 4096, 32768])
def test_nothing_outside_the_outputs(dim):
    for rows in (1, 5, 31):
        x = randn(rows, dim, dtype=torch.bfloat16)
        for out in (torch.bfloat16, F8, torch.float32):
            y = Guarded((rows, dim), out)
            s = Guarded((rows, dim), torch.bfloat16)
            kda.rms_norm(x, None, residual=x, out_dtype=out, out=y.t, residual_out=s.t)
            torch.cuda.synchronize()
            assert y.intact() and s.intact()


@pytest.mark.parametrize("dim", [100, 128, 4096])
@pytest.mark.parametrize("out", [torch.bfloat16, F8])
def test_zero_nan_and_infinite_rows(dim, out):
    """A row of zeros gives zeros; one with a NaN or an infinity is NaN where the formula is; the others are not."""
    x = randn(6, dim, dtype=torch.bfloat16)
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, dim - 1] = float("inf")
    y, scale, _ = kda.rms_norm(x, None, out_dtype=out)
    y = y.float()
    assert (y[1] == 0).all() and torch.isfinite(y[[0, 4, 5]]).all()
    assert torch.isnan(y[2]).all()
    assert torch.isnan(y[3, dim - 1])
    if out == F8:
        assert torch.isnan(y[3]).all() and torch.isnan(scale[2:4]).all()
        assert torch.allclose(scale[1], torch.tensor(1e-30 / 448, device="cuda"), rtol=1e-5, atol=0)
    else:
        assert (y[3, : dim - 1] == 0).all()
    z = torch.full((2, dim), 1e-4, dtype=torch.bfloat16, device="cuda")  # small rows: eps counts
    check(z, None, None, out)


def test_more_than_2_to_31_elements():
    rows, dim = 70000, 32768
    x = torch.empty((rows, dim), dtype=torch.bfloat16, device="cuda")
    x.fill_(2.0)
    x[:, ::2] = -1.0
    x[rows - 1] = randn(dim, dtype=torch.bfloat16)
    y, scale, _ = kda.rms_norm(x, None, out_dtype=F8)
    y_ref, _ = reference(x[rows - 2:], None, None, 1e-6)
    got = y[rows - 2:].double() * scale[rows - 2:, None].double()
    assert ((got - y_ref).norm(dim=1) <= 0.04 * y_ref.norm(dim=1)).all()  # e4m3: at most half of 2^-3 each
    assert torch.equal(y[:rows - 1].view(torch.uint8)[::997], y[:1].view(torch.uint8).expand(rows - 1, dim)[::997])


def test_stream_graph_and_repeat():
    x, r = randn(64, 4096, dtype=torch.bfloat16), randn(64, 4096, seed=1, dtype=torch.bfloat16)
    ref = kda.rms_norm(x, None, residual=r, out_dtype=F8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kda.rms_norm(x, None, residual=r, out_dtype=F8, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = kda.rms_norm(x, None, residual=r, out_dtype=F8)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(out, ref))


def test_python_refusals():
    x = randn(4, 128, dtype=torch.bfloat16)
    for kw in (dict(x=x.cpu()), dict(x=x.to(torch.float64)), dict(x=x.t()), dict(out_dtype=torch.float16),
               dict(residual=x.float()), dict(residual=x[:2]), dict(weight=x[0, :64]), dict(weight=x[0].half()),
               dict(x=x[:1].expand(4, 128)), dict(residual_out=x.float()), dict(out=x.float())):
        a = dict(x=x)
        a.update(kw)
        with pytest.raises(TypeError):
            kda.rms_norm(**a)
    with pytest.raises(kda.KdaError):
        kda.rms_norm(x, eps=-1.0)
    with pytest.raises(kda.KdaError):
        kda.rms_norm(torch.zeros(1, 32769, dtype=torch.bfloat16, device="cuda"))
