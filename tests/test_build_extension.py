"""The Python extension is taken only with the torch that it was built against."""
from __future__ import annotations

import pytest

from chunked_gated_delta_gb300 import binding, build


@pytest.fixture
def other_torch(monkeypatch):
    """The extension as built; torch replaced by another version since."""
    binding.load_library()
    if not build.up_to_date():
        build.build()
    import torch
    monkeypatch.setattr(binding, "_calls", None)
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")


def test_it_is_built_again(other_torch):
    assert not build.up_to_date()


def test_it_is_not_loaded(other_torch):
    with pytest.raises(RuntimeError, match="another torch"):
        binding._layer_calls()
