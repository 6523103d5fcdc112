"""CPU checks of rotary_freqs beside test_decay_host.py's: what the amplitude is at factors up to one."""
from __future__ import annotations

import math

import pytest

import chunked_gated_delta_gb300 as kda


@pytest.mark.parametrize("factor", [0.25, 0.5, 0.999, 1.0])
def test_yarns_amplitude_is_not_below_one(factor):
    """0.1 ln(factor) + 1 belongs to contexts that are longer; those that are not keep cosines and sines as they are."""
    freqs, amplitude = kda.rotary_freqs(64, scaling="yarn", factor=factor, device="cpu")
    assert amplitude == 1.0
    plain, _ = kda.rotary_freqs(64, device="cpu")
    assert bool((freqs >= plain * (1.0 - 1e-15)).all()) and freqs[0] == 1.0


@pytest.mark.parametrize("factor", [1.5, 4.0, 32.0])
def test_yarns_amplitude_above_one(factor):
    _, amplitude = kda.rotary_freqs(64, scaling="yarn", factor=factor, device="cpu")
    assert abs(amplitude - (0.1 * math.log(factor) + 1.0)) < 1e-15


def test_other_scalings_have_none():
    for scaling in (None, "linear", "ntk"):
        for factor in (0.5, 4.0):
            assert kda.rotary_freqs(64, scaling=scaling, factor=factor, device="cpu")[1] == 1.0
