"""Order on one stream around step, rms_norm and linear, whose kernels start while
the kernel before them ends (programmatic dependent launch): inputs written by
the kernel right before, outputs read and inputs overwritten right after, the
operators right after one another, and a state updated in place by many steps."""
from __future__ import annotations

import pytest
import torch

import chunked_gated_delta_gb300 as kda

pytestmark = pytest.mark.gpu

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.mark.parametrize("M", [1, 37, 300, 4096])
def test_a_chain_of_operators(M):
    """norm -> linear -> norm -> linear + residual, with a filling kernel before and after each input's use."""
    gen = torch.Generator(device="cuda").manual_seed(M)
    D = 1024
    src = [torch.randn((M, D), generator=gen, device="cuda").to(BF16) for _ in range(4)]
    w1 = (torch.randn((D, D), generator=gen, device="cuda") / 32).to(BF16)
    w1s = w1.float().abs().amax(1) / 448
    w1q = (w1.float() / w1s[:, None]).to(F8)
    w2 = (torch.randn((D, D), generator=gen, device="cuda") / 32).to(BF16)

    def layer(x):
        q, scale, s = kda.rms_norm(x, None, residual=x, out_dtype=F8)
        h = kda.linear(q, w1q, act="silu", x_scale=scale, w_scale=w1s)
        n, _, _ = kda.rms_norm(h)
        return kda.linear(n, w2, residual=s)

    want = []
    for x in src:
        torch.cuda.synchronize()
        want.append(layer(x).clone())
        torch.cuda.synchronize()
    x = torch.empty_like(src[0])
    for _ in range(20):
        got = []
        for i in range(4):
            x.copy_(src[i])          # written right before
            got.append(layer(x))
            x.fill_(float("nan"))    # overwritten right after
        for g, e in zip(got, want):
            assert torch.equal(g, e)


@pytest.mark.parametrize("B,H", [(3, 4), (40, 32)])
def test_many_steps_in_place(B, H):
    """Fifty steps enqueued without a wait give what they give with one after each."""
    gen = torch.Generator(device="cuda").manual_seed(B)

    def randn(*s):
        return torch.randn(s, generator=gen, device="cuda")

    def unit(x):
        return (x / x.norm(dim=-1, keepdim=True)).to(BF16)

    n = 50
    x = [(unit(randn(B, 1, H, 128)), unit(randn(B, 1, H, 128)), randn(B, 1, H, 128).to(BF16), -torch.rand(
        (B, 1, H, 128), generator=gen, device="cuda"), torch.sigmoid(randn(B, 1, H)).to(BF16)) for _ in range(n)]
    start = 0.1 * randn(B, H, 128, 128)
    a, b = start.clone(), start.clone()
    waited, buf = [], tuple(torch.empty_like(t) for t in x[0])
    for t in x:
        waited.append(kda.step(*t, a))
        torch.cuda.synchronize()
    got = []
    for t in x:
        for d, s in zip(buf, t):
            d.copy_(s)
        got.append(kda.step(*buf, b))
        buf[2].fill_(float("nan"))
    torch.cuda.synchronize()
    assert torch.equal(a, b) and all(torch.equal(p, q) for p, q in zip(waited, got))
