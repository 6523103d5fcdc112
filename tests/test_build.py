"""The in-tree build: what is left when the Python extension cannot be built."""
from __future__ import annotations

import os
import sys

import pytest

from chunked_gated_delta_gb300 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """build.py on a tree of one small source."""
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(build, "sources", lambda: [str(src)])
    monkeypatch.setattr(build, "_inputs", lambda: [str(src)])
    for name, path in (("LIB", "libone.so"), ("EXTENSION", "_one.so"), ("OBJDIR", "obj")):
        monkeypatch.setattr(build, name, str(tmp_path / path))
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    try:
        build._nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")
    return tmp_path


def test_a_failing_extension_leaves_the_library(tree, monkeypatch):
    def fail():
        raise RuntimeError("compiling layer_calls.cpp failed")

    monkeypatch.setattr(build, "_compile_extension", fail)
    with pytest.raises(RuntimeError, match="layer_calls"):
        build.build(force=True)
    assert os.path.exists(build.LIB) and not os.path.exists(build.EXTENSION)
    assert not build.up_to_date()


def test_without_torch_the_library_alone_is_built(tree, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # (importing it raises ImportError)
    assert build.build(force=True) == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.EXTENSION)
    assert build.up_to_date()
