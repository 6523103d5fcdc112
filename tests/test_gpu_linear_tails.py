"""kda.linear's activations far out, where exp(-|v|) leaves fp32's normal range."""
from __future__ import annotations

import pytest
import torch

import chunked_gated_delta_gb300 as kda
from ops_util import HALF_ULP

pytestmark = pytest.mark.gpu

ACTS = {"silu": lambda t: t * torch.sigmoid(t), "sigmoid": torch.sigmoid, "logsigmoid": torch.nn.functional.logsigmoid}


@pytest.mark.parametrize("M", [1, 20, 300, 4096])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", list(ACTS))
def test_activations_at_the_end_of_the_range(act, out, M):
    """Through the bias, |v| from 40 to 140.  fp32: within 2^-20 of every result that is a normal number, and the
    others within 2^-126; 16 bits: 2^-15 beside the rounding (the approximate exponential at |v| = 87 is within 104
    units of 2^-23), and SiLU may be zero below v = -87 (1.2e-36 in size)."""
    v = torch.cat([torch.linspace(40, 140, 401), torch.tensor([87.25, 87.3125, 88.5, 88.75, 1e4, 1e30, 3e38])])
    v = torch.cat([v, -v]).float().cuda()
    x = torch.zeros((M, 64), device="cuda", dtype=torch.bfloat16)
    w = torch.zeros((v.numel(), 64), device="cuda", dtype=torch.bfloat16)
    y = kda.linear(x, w, bias=v, act=act, out_dtype=out).double()
    want = ACTS[act](v.double())
    small = 1.2e-36 if act == "silu" and out != torch.float32 else 2.0 ** -126
    lim = (2.0 ** -20 if out == torch.float32 else 2.0 ** -15 + HALF_ULP[out]) * want.abs() + torch.where(
        want.abs() < small, small, 0.0)
    assert ((y - want).abs() <= lim).all(), ((y - want).abs() - lim).max().item()
