"""The served layer's output projection behind the head norm: with e4m3 operands
the same formula as with 16-bit ones, for norm weights far from one and small o."""
from __future__ import annotations

import pytest
import torch

from chunked_gated_delta_gb300 import layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [(1, 1), (2, 150)])
@pytest.mark.parametrize("size", [1.0, 3e-4])
@pytest.mark.parametrize("head_norm", [0.3, 1.0, 2.0])
@pytest.mark.parametrize("eight_bit", [False, True])
def test_output_of_scaled_head_norms(eight_bit, head_norm, size, tokens):
    """Tolerances, of the norm of the whole: 16 bits: the operand's rounding and y's, 2^-8 each at most, 1 percent;
    8 bits: an e4m3 rounding moves an element by at most 2^-4 of itself, 2^-4 / sqrt(3) rms (3.6 percent), 5 percent."""
    D, H, V = 512, 8, 128
    m = layer.KdaLayer.random(D, H, 128, V, eight_bit=eight_bit, seed=1)
    m.head_norm = head_norm * m.head_norm
    gen = torch.Generator(device="cuda").manual_seed(2)
    o = (size * torch.randn((*tokens, H, V), generator=gen, device="cuda")).bfloat16()
    total = torch.zeros((*tokens, D), dtype=torch.bfloat16, device="cuda")
    y = m._output(o, total).double()
    od = o.double()
    n = od / torch.sqrt(od.square().mean(-1, keepdim=True) + m.eps) * m.head_norm.double()
    w = m.out.w.double()
    w = w * m.out.scale.double()[:, None] if eight_bit else w
    ref = n.reshape(*tokens, H * V) @ w.T
    assert (y - ref).norm() <= (0.05 if eight_bit else 0.01) * ref.norm()


def test_rows_to_eight_bits_are_not_normed():
    """Codes and scales are those of the rows themselves: scale = max |n| / 448, codes its nearest multiples."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    n = torch.randn((300, 1024), generator=gen, device="cuda") * torch.logspace(-12, 6, 300, device="cuda")[:, None]
    n[7] = 0
    for io in (torch.bfloat16, torch.float32):
        x = n.to(io)
        weight = torch.full((1024,), layer._NO_NORM_WEIGHT, device="cuda")
        codes, scale, _ = layer.kda.rms_norm(x, weight, eps=layer._NO_NORM_EPS, out_dtype=torch.float8_e4m3fn)
        a = x.double().abs().amax(1).clamp_min(1e-30)
        assert ((scale.double() - a / 448).abs() <= 2.0 ** -22 * a / 448).all()
        want = x.double() * (448 / a)[:, None]
        half_step = torch.exp2(torch.floor(torch.log2(want.abs().clamp_min(2.0 ** -6))) - 4)
        assert ((codes.double() - want).abs() <= half_step + 2.0 ** -21 * want.abs()).all()
