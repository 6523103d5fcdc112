"""kda.linear against the formula in 64 bits.

Tolerances: the products are exact in fp32 and the tensor cores add them with at
worst one truncation (2^-23) of the running sum per group of eight k, so the
accumulator is within (K / 8 + 8) 2^-23 sum_k |x w| of the sum; the activations
stretch an error by at most 1.2; the epilogue's own arithmetic is 16 roundings
of its terms; and the output is rounded once to its type.
"""
from __future__ import annotations

import math

import pytest
import torch

import chunked_gated_delta_gb300 as kda
from ops_util import EPS32, HALF_ULP, TINY, Guarded, assert_close

pytestmark = pytest.mark.gpu

BF16, F16, F32, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
ACTS = {None: lambda t: t, "silu": lambda t: t * torch.sigmoid(t), "gelu": torch.nn.functional.gelu,
        "sigmoid": torch.sigmoid, "logsigmoid": torch.nn.functional.logsigmoid}


def randn(*shape, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + 11)
    return torch.randn(shape, generator=gen, device="cuda")


def padded(x, extra=0, fill=float("nan")):
    """x as the first columns of rows that start on 16 bytes; what lies between the rows is `fill`."""
    wide = -(-x.shape[1] // 16) * 16 + extra
    buf = torch.full((x.shape[0] + 1, wide), fill, device="cuda").to(x.dtype)
    buf[: x.shape[0], : x.shape[1]] = x
    return buf[: x.shape[0], : x.shape[1]]


def operands(M, N, K, io, extra=0, seed=0):
    x, w = randn(M, K, seed=seed), randn(N, K, seed=seed + 1) / math.sqrt(K)
    xs = ws = None
    if io == F8:
        xs, ws = x.abs().amax(1).clamp_min(1e-20) / 448, w.abs().amax(1).clamp_min(1e-20) / 448
        x, w = x / xs[:, None], w / ws[:, None]
    return padded(x.to(io), extra), padded(w.to(io), extra), xs, ws


def check(M, N, K, io=BF16, out=None, act=None, bias=True, residual=False, extra=0, seed=0, got=None):
    x, w, xs, ws = operands(M, N, K, io, extra, seed)
    out_t = out or (BF16 if io == F8 else io)
    b = 0.5 * randn(N, seed=seed + 2) if bias else None
    r = randn(M, N, seed=seed + 3).to(out_t) if residual else None
    y = kda.linear(x, w, bias=b, act=act, residual=r, x_scale=xs, w_scale=ws, out_dtype=out, out=got)
    torch.cuda.synchronize()
    assert y.dtype == out_t and y.shape == (M, N)
    xd, wd = x.double(), w.double()
    if io == F8:
        xd, wd = xd * xs.double()[:, None], wd * ws.double()[:, None]
    pre, size = xd @ wd.T, xd.abs() @ wd.abs().T
    if b is not None:
        pre, size = pre + b.double(), size + b.double().abs()
    ref = ACTS[act](pre)
    arith = 1.2 * (K / 8 + 8) * 2.0 ** -23 * size + 16 * EPS32 * (size + ref.abs() + 1.0)
    if r is not None:
        ref = ref + r.double()
        arith = arith + 16 * EPS32 * r.double().abs()
    assert_close(y, ref, HALF_ULP[out_t] * 1.01, arith * (1 + HALF_ULP[out_t]) + TINY[out_t], (M, N, K, io, out, act))
    if out_t == F32:
        assert (y.double() - ref).norm() <= 1e-5 * ref.norm()
    return y


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 100, 128, 129, 200, 257, 511, 700])
@pytest.mark.parametrize("N,K", [(1, 1), (7, 64), (32, 2048), (127, 100), (128, 513), (129, 65), (500, 1000),
                                 (640, 4096)])
def test_sizes(M, N, K):
    check(M, N, K, seed=M + N + K)
    check(M, N, K, io=F8, act="silu", seed=M + N + K)


@pytest.mark.parametrize("io", [BF16, F16, F8])
@pytest.mark.parametrize("out", [BF16, F16, F32])
@pytest.mark.parametrize("act", list(ACTS))
def test_types_and_activations(io, out, act):
    check(5, 200, 320, io, out, act, bias=True, residual=False)
    check(130, 256, 512, io, out, act, bias=False, residual=True)
    check(300, 264, 192, io, out, act, bias=True, residual=True)


@pytest.mark.parametrize("M", [1, 40, 300, 2500, 5000])
@pytest.mark.parametrize("N", [32, 2048, 2056, 4096, 4100])
def test_larger(M, N):
    check(M, N, 2048, act="silu", residual=True, seed=M)
    check(M, N, 1040, io=F8, out=F32, act="logsigmoid", seed=M)


@pytest.mark.parametrize("K", [1, 3, 8, 15, 17, 63, 129, 255, 4097])
@pytest.mark.parametrize("io", [BF16, F8])
def test_odd_k_reads_nothing_past_its_rows(K, io):
    """NaN lies between the rows and after the last one."""
    for M in (3, 70, 600):
        check(M, 136, K, io, seed=K)
        check(M, 136, K, io, extra=32, seed=K)


def test_deep_k():
    for M in (1, 150, 3000):
        check(M, 256, 20000, out=F32)
        check(M, 256, 33008, io=F8, out=F32)


def test_in_place_strided_and_batched():
    for M in (3, 90, 1000):
        x, w, _, _ = operands(M, 384, 256, BF16)
        r = randn(M, 384, seed=5).to(BF16)
        ref = kda.linear(x, w, residual=r)
        z = r.clone()
        assert kda.linear(x, w, residual=z, out=z) is z and torch.equal(z, ref)
        for lead in (0, 1, 8):  # a part of wider rows, on and off 16 bytes
            wide = torch.full((M, 400), 7.0, dtype=BF16, device="cuda")
            wide[:, lead:lead + 384] = r
            part = wide[:, lead:lead + 384]
            kda.linear(x, w, residual=part, out=part)
            assert torch.equal(part, ref)
            assert (wide[:, :lead] == 7).all() and (wide[:, lead + 384:] == 7).all()
    x, w, _, _ = operands(24, 100, 64, BF16)
    x = x.contiguous()
    assert torch.equal(kda.linear(x.view(2, 3, 4, 64), w).view(24, 100), kda.linear(x, w))
    assert torch.equal(kda.linear(x[5], w), kda.linear(x[5:6], w)[0])
    assert kda.linear(x[:0], w).shape == (0, 100)


@pytest.mark.parametrize("M,N", [(1, 1), (5, 129), (17, 250), (129, 130), (257, 520), (1000, 1032)])
@pytest.mark.parametrize("out", [BF16, F32])
def test_nothing_outside_the_output(M, N, out):
    g = Guarded((M, N), out)
    check(M, N, 192, out=out, got=g.t, residual=True)
    assert g.intact()


@pytest.mark.parametrize("M,N", [(70, 2049), (300, 4095), (1000, 999), (4097, 1023)])
@pytest.mark.parametrize("io,out", [(BF16, BF16), (F16, F32), (F8, BF16), (F8, F32)])
def test_rows_off_16_bytes(M, N, io, out):
    """y and the residual as columns of wider tensors, no row of them on a set place; what lies around y stays."""
    x, w, xs, ws = operands(M, N, 320, io, seed=N)
    kw = dict(act="silu", x_scale=xs, w_scale=ws, out_dtype=out)
    wide = randn(M, N + 6, seed=7).to(out)
    buf = wide.clone()
    y = buf[:, 3 : N + 3]
    kda.linear(x, w, residual=wide[:, 1 : N + 1], out=y, **kw)
    xd, wd = x.double(), w.double()
    if io == F8:
        xd, wd = xd * xs.double()[:, None], wd * ws.double()[:, None]
    pre, size, r = xd @ wd.T, xd.abs() @ wd.abs().T, wide[:, 1 : N + 1].double()
    ref = ACTS["silu"](pre)
    arith = 1.2 * (320 / 8 + 8) * 2.0 ** -23 * size + 16 * EPS32 * (size + ref.abs() + 1.0 + r.abs())
    assert_close(y, ref + r, HALF_ULP[out] * 1.01, arith * (1 + HALF_ULP[out]) + TINY[out], (M, N, io, out))
    assert torch.equal(buf[:, :3], wide[:, :3]) and torch.equal(buf[:, N + 3 :], wide[:, N + 3 :])
    z = wide.clone()
    kda.linear(x, w, residual=z[:, 1 : N + 1], out=z[:, 1 : N + 1], **kw)
    assert torch.equal(z[:, 1 : N + 1], y)


def test_bad_rows_stay_by_themselves():
    """An infinity or NaN in a row of x reaches that row of y alone; one in a row of w, that column."""
    for M in (20, 400):
        x, w, _, _ = operands(M, 300, 256, BF16)
        ref = kda.linear(x, w, act="silu")
        x[7, 3], x[11, 255], w[200, 9] = float("nan"), float("inf"), float("nan")
        y = kda.linear(x, w, act="silu")
        assert torch.isnan(y[7]).all() and not torch.isfinite(y[11, :200]).all() and torch.isnan(y[:, 200]).all()
        rows = [i for i in range(M) if i not in (7, 11)]
        cols = [j for j in range(300) if j != 200]
        assert torch.equal(y[rows][:, cols], ref[rows][:, cols])


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("out", [BF16, F32])
def test_activations_of_extreme_values(act, out):
    """Through the bias: NaN stays NaN, infinities and large values give the functions' limits."""
    vals = [float("nan"), float("inf"), 1e30, 200.0, 89.0, 20.0, 1e-6, 0.0, -1e-6, -20.0, -89.0, -104.0, -200.0, -1e30]
    b = torch.tensor(vals * 20, device="cuda")
    want = ACTS[act](b.double())
    for M in (1, 20, 300, 4096):
        x, w = torch.zeros((M, 64), device="cuda").to(BF16), torch.zeros((280, 64), device="cuda").to(BF16)
        y = kda.linear(x, w, bias=b, act=act, out_dtype=out).double()
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(y), nan.expand(M, -1))
        ok = ~nan & torch.isfinite(want.to(out))
        assert torch.equal(y[:, ~nan & ~ok], want[~nan & ~ok].expand(M, -1))
        assert_close(y[:, ok], want[ok].expand(M, -1), HALF_ULP[out] + 2.0 ** -20, 1e-30)


def test_output_beyond_32_bits():
    M, N, K = 70000, 32768, 64
    x, w, _, _ = operands(M, N, K, BF16)
    y = kda.linear(x, w)
    assert y.numel() > 1 << 31
    for rows in (slice(0, 3), slice(M - 300, M)):
        ref = x[rows].double() @ w.double().T
        size = x[rows].double().abs() @ w.double().abs().T
        assert_close(y[rows], ref, HALF_ULP[BF16] * 1.01, 2 * (K / 8 + 8) * 2.0 ** -23 * size)


def test_stream_graph_repeat_and_status():
    for M in (4, 200, 3000):
        x, w, _, _ = operands(M, 1024, 1024, BF16)
        ref = kda.linear(x, w, act="gelu")
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        assert torch.equal(kda.linear(x, w, act="gelu", status=word), ref)
        assert kda.status(word) == 0
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = kda.linear(x, w, act="gelu", stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, ref)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = kda.linear(x, w, act="gelu")
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, ref)


def test_python_refusals():
    x, w, xs, ws = operands(4, 64, 64, BF16)
    x, w = x.contiguous(), w.contiguous()
    for kw in (dict(x=x.float()), dict(w=w.half()), dict(x=x.cpu()), dict(w=w[:, :32]), dict(bias=x[0]),
               dict(x_scale=torch.ones(4, device="cuda")), dict(residual=torch.zeros(4, 64, device="cuda")),
               dict(out_dtype=F8), dict(w=w.t().contiguous().t()), dict(x=x[:1].expand(4, 64)),
               dict(out=torch.zeros(4, 64, device="cuda"))):
        a = dict(x=x, w=w)
        a.update(kw)
        with pytest.raises(TypeError):
            kda.linear(**a)
    with pytest.raises(ValueError):
        kda.linear(x, w, act="relu")
    with pytest.raises(TypeError):
        kda.linear(x.to(F8), w.to(F8))  # no scales
    for bad in (randn(4, 63).to(BF16), randn(4, 65).to(BF16).view(-1)[1:].view(-1)[:256].view(4, 64)):
        with pytest.raises(kda.KdaError):  # rows that do not start on 16 bytes
            kda.linear(bad, randn(64, bad.shape[1]).to(BF16))
