"""rotary against the rotation in 64 bits: types, both layouts, parts of heads, odd sizes, far and
negative positions, strides, in place, back again.

Tolerance: the output's rounding; the cosines and sines are right to 2^-22 (the angle to 2^-25 of half a turn,
sincospif, the amplitude's product), and two products and their sum round in fp32: 2^-21 (|x| + |y|) amplitude."""
from __future__ import annotations

import pytest
import torch

import chunked_gated_delta_gb300 as kda
from ops_util import HALF_ULP, TINY, Guarded, assert_close

pytestmark = pytest.mark.gpu


def reference(x, pos, freqs, amplitude, interleaved, inverse):
    half = freqs.numel()
    angle = pos.double()[..., None, None] * freqs
    angle = -angle if inverse else angle
    c, s = amplitude * torch.cos(angle), amplitude * torch.sin(angle)
    y, W = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    i = torch.arange(half, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    u, v = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = u * c - v * s, u * s + v * c
    W[..., a] = W[..., b] = amplitude * (u.abs() + v.abs())
    return y, W


def check(q, k, pos, freqs, amplitude=1.0, interleaved=False, inverse=False, **kw):
    got = kda.rotary(q, k, pos, freqs, amplitude, interleaved, inverse, **kw)
    torch.cuda.synchronize()
    for x, y in zip((q, k), got):
        if x is None:
            assert y is None
            continue
        ref, W = reference(x, pos, freqs, amplitude, interleaved, inverse)
        assert_close(y, ref, HALF_ULP[x.dtype] * 1.01, 2.0 ** -21 * W + TINY[x.dtype])
        assert torch.equal(y[..., 2 * freqs.numel():], x[..., 2 * freqs.numel():])
    return got


def randn(*s, dtype=torch.bfloat16, seed=0):
    return torch.randn(s, generator=torch.Generator(device="cuda").manual_seed(seed + sum(s)), device="cuda").to(dtype)


def positions(B, T, first=0, dtype=torch.int64):
    return (first + torch.arange(B * T, device="cuda").view(B, T) % max(T, 1) + 17 * torch.arange(B, device="cuda")[:, None]).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(128, 128), (128, 64), (64, 64), (96, 48), (256, 32), (72, 72), (2, 2), (7, 6), (130, 66), (36, 20)])
def test_types_layouts_parts(dtype, interleaved, D, R):
    freqs, _ = kda.rotary_freqs(R)
    for inverse in (False, True):
        check(randn(2, 9, 5, D, dtype=dtype), randn(2, 9, 2, D, dtype=dtype), positions(2, 9), freqs, interleaved=interleaved, inverse=inverse)


@pytest.mark.parametrize("B,T,H,Hk", [(1, 1, 1, 1), (1, 1, 32, 8), (59, 1, 32, 8), (3, 700, 4, 4), (1, 5000, 3, 1), (2, 40, 64, 64)])
def test_shapes(B, T, H, Hk):
    freqs, _ = kda.rotary_freqs(128, base=1e6)
    check(randn(B, T, H, 128), randn(B, T, Hk, 128), positions(B, T), freqs)
    check(randn(B, T, H, 128), None, positions(B, T, dtype=torch.int32), freqs)


@pytest.mark.parametrize("first", [0, 4095, 10 ** 6, 2 ** 31 - 40, -10 ** 6, 2 ** 40])
@pytest.mark.parametrize("scaling,factor", [(None, 1.0), ("linear", 8.0), ("ntk", 4.0), ("yarn", 32.0)])
def test_far_positions(first, scaling, factor):
    """The angle keeps its bits at any position (fp64's own product is off by 2^-53 of the angle: beyond 10^9 that
    shows, and the reference takes the angle from whole numbers)."""
    freqs, amplitude = kda.rotary_freqs(64, base=5e5, scaling=scaling, factor=factor)
    q = randn(1, 30, 2, 64, dtype=torch.float32)
    pos = positions(1, 30, first)
    if abs(first) < 2 ** 32:
        check(q, None, pos, freqs, amplitude)
        return
    got, _ = kda.rotary(q, None, pos, freqs, amplitude)
    # position p = p0 + r: the angle of p0 in whole turns of freqs / (2 pi) to 2^-64, as the kernel has it
    turns = [int((f * 0.15915494309189535 % 1.0) * 2.0 ** 64) for f in freqs.cpu().tolist()]
    frac = torch.tensor([[((p * t) % 2 ** 64) / 2 ** 64 for t in turns] for p in pos[0].tolist()], dtype=torch.float64, device="cuda")
    angle = frac[None, :, None, :] * 2 * torch.pi
    x, y = q.double()[..., :32], q.double()[..., 32:]
    c, s = amplitude * torch.cos(angle), amplitude * torch.sin(angle)
    W = amplitude * (x.abs() + y.abs())
    assert_close(got[..., :32], x * c - y * s, HALF_ULP[torch.float32], 2.0 ** -21 * W)
    assert_close(got[..., 32:], x * s + y * c, HALF_ULP[torch.float32], 2.0 ** -21 * W)


def test_any_frequency():
    freqs = torch.tensor([0.0, 1.0, 3.5, -2.0, 7.0, 100.0, 1e-12, 2 * torch.pi], dtype=torch.float64, device="cuda")
    check(randn(1, 50, 2, 16, dtype=torch.float32), None, positions(1, 50), freqs, 0.5)


@pytest.mark.parametrize("D,extra", [(64, 8), (64, 3), (48, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_strides_and_in_place(D, extra, interleaved):
    freqs, _ = kda.rotary_freqs(32)
    wide = randn(2, 11, 5 * D + extra)
    q, k = wide[..., :3 * D].unflatten(-1, (3, D)), wide[..., 3 * D:5 * D].unflatten(-1, (2, D))
    pos = positions(2, 11)
    a, b = check(q, k, pos, freqs, interleaved=interleaved)
    tail = wide[..., 5 * D:].clone()
    c, d = kda.rotary(q, k, pos, freqs, interleaved=interleaved, q_out=q, k_out=k)
    assert c is q and d is k and torch.equal(q, a) and torch.equal(k, b) and torch.equal(wide[..., 5 * D:], tail)
    out = Guarded((2, 11, 3, D), torch.bfloat16)
    kda.rotary(a, None, pos, freqs, interleaved=interleaved, inverse=True, q_out=out.t)
    torch.cuda.synchronize()
    assert out.intact()


def test_inverse_is_the_gradient():
    """The rotation's gradient is the rotation back (times amplitude): <R x, y> = <x, R^T y>."""
    freqs, amplitude = kda.rotary_freqs(64, scaling="yarn", factor=8.0)
    x, y = randn(1, 40, 2, 64, dtype=torch.float32), randn(1, 40, 2, 64, dtype=torch.float32, seed=5)
    pos = positions(1, 40, 1000)
    a, _ = kda.rotary(x, None, pos, freqs, amplitude)
    b, _ = kda.rotary(y, None, pos, freqs, amplitude, inverse=True)
    left, right = (a.double() * y.double()).sum(-1), (x.double() * b.double()).sum(-1)
    bound = 2.0 ** -19 * amplitude * x.double().norm(dim=-1) * y.double().norm(dim=-1)
    assert bool(((left - right).abs() <= bound).all())


def test_graph_and_stream():
    freqs, _ = kda.rotary_freqs(128)
    q, k, pos = randn(4, 3, 8, 128), randn(4, 3, 2, 128), positions(4, 3)
    want = kda.rotary(q, k, pos, freqs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kda.rotary(q, k, pos, freqs, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    out = [torch.zeros_like(x) for x in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.rotary(q, k, pos, freqs, q_out=out[0], k_out=out[1])
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, out):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_no_tokens_and_refusals():
    freqs, _ = kda.rotary_freqs(64)
    q, k, pos = randn(2, 3, 2, 64), randn(2, 3, 2, 64), positions(2, 3)
    a, b = kda.rotary(q[:, :0], k[:, :0], pos[:, :0].contiguous(), freqs)
    assert a.numel() == 0 and b.numel() == 0
    for args in ((q.double(), None, pos, freqs), (q, k.half(), pos, freqs), (q, k[:1], pos, freqs), (q, k, pos.float(), freqs),
                 (q, k, pos[:1], freqs), (q, k, pos, freqs.float()), (q[..., :62], None, pos, freqs), (q.cpu(), None, pos, freqs)):
        with pytest.raises(TypeError):
            kda.rotary(*args)
    with pytest.raises(TypeError):
        kda.rotary(q, k, pos, freqs, q_out=torch.empty_like(q).half())
    wide = torch.empty(2, 3, 2 * 64 + 8, dtype=torch.bfloat16, device="cuda")[..., :128].unflatten(-1, (2, 64))
    wide.copy_(q)
    with pytest.raises(kda.KdaError):  # the same memory with another stride
        kda.rotary(wide, None, pos, freqs, q_out=wide.as_strided((2, 3, 2, 64), (3 * 128, 128, 64, 1)))


@pytest.mark.parametrize("T,H,Hk,D,R", [(1823, 1, 0, 16, 16), (1825, 1, 0, 16, 16), (30011, 1, 0, 16, 8), (20011, 1, 1, 24, 16), (40000, 1, 0, 2, 2),
                                        (9001, 8, 1, 256, 256), (4001, 2, 1, 7, 6), (5555, 32, 8, 128, 64), (3001, 2, 0, 1024, 1024)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_tokens_taken_together(T, H, Hk, D, R, interleaved):
    """Tokens of few heads share a CTA's pass: every size of such a group, a last one that is cut short, in place."""
    freqs, _ = kda.rotary_freqs(R)
    pos = torch.randperm(T, generator=torch.Generator().manual_seed(T)).cuda()[None]
    for dtype in (torch.bfloat16, torch.float32):
        q, k = randn(1, T, H, D, dtype=dtype), randn(1, T, Hk, D, dtype=dtype) if Hk else None
        a, b = check(q, k, pos, freqs, interleaved=interleaved)
        kda.rotary(q, k, pos, freqs, interleaved=interleaved, q_out=q, k_out=k)
        assert torch.equal(q, a) and (b is None or torch.equal(k, b))
