"""How right rotary's angles are, seen where a sine or a cosine is small: there it is the angle's error that shows.

Bound: the angle to 2^-31 of a turn, 2^-65 of a turn per position (a position's share of a turn has 64 bits) and 2^-52
of position * freq (the frequency's own rounding and the reference's product); the sine and cosine themselves 2^-23 (one unit
in the last place) and two more roundings, 2^-22 of the value in all."""
from __future__ import annotations

import math

import pytest
import torch

import chunked_gated_delta_gb300 as kda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,first", [(128, 0), (128, 1000000), (6, -70000)])
def test_angles(dim, first, interleaved):
    half, T = dim // 2, 20000
    gen = torch.Generator().manual_seed(dim + first)
    freqs = torch.rand(half, generator=gen, dtype=torch.float64).cuda()
    q = torch.zeros((1, T, 1, dim), device="cuda")
    x, y = (slice(0, dim, 2), slice(1, dim, 2)) if interleaved else (slice(0, half), slice(half, dim))
    q[..., x] = 1.0
    pos = first + torch.arange(T, device="cuda")[None]
    got, _ = kda.rotary(q, None, pos, freqs, interleaved=interleaved)
    angle = pos.double()[..., None] * freqs
    near = 0
    for part, want in ((x, torch.cos(angle)), (y, torch.sin(angle))):
        off = (got[0, :, 0, part].double() - want[0]).abs()
        bound = 2 * math.pi * (2.0 ** -31 + pos[0].abs().double()[:, None] * 2.0 ** -65) + 2.0 ** -52 * angle[0].abs() + 2.0 ** -22 * want[0].abs()
        assert bool((off <= bound).all()), (off / bound).max().item()
        near += int((want.abs() < 2.0 ** -7).sum())
    assert near > 100  # small ones were among them
