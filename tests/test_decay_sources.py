"""Orders in the kernels of linear attention with a decay per head that no run would show to be wrong, read in their
sources on the CPU."""
from __future__ import annotations

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "chunked_gated_delta_gb300", "csrc")


def source(name):
    """Without comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", ["decay_scan.cuh", "decay_grads.cu"])
def test_dependents_are_let_in_when_tmem_is_had(name):
    """The launch of dependents counts for a block as soon as one of its threads has asked for it. It is asked for behind a
    barrier of the whole block that the allocating warp reaches with its TMEM: a dependent on the same SM that took it first
    would wait for this grid, and this grid for the TMEM."""
    text = source(name)
    alloc = text.index("ptx::tmem_alloc(")
    sync = text.index("__syncthreads();", alloc)
    launch = text.index("ptx::grid_dep_launch();", alloc)
    assert sync < launch
    assert "grid_dep_launch" not in text[text.rindex("__global__", 0, alloc):alloc]


def test_barriers_of_a_pair_are_waited_for_in_the_clusters_scope():
    """The other CTA arrives on may_give, and its copies complete given: an acquire at the CTA's own scope would not order
    what it did before them."""
    text = source("decay_grads.cu")
    for bar in ("may_give", "given"):
        waits = re.findall(r"(\w+)\(sm\.%s, " % bar, text)
        assert waits and all(w == "wait_cluster" for w in waits), (bar, waits)
    assert re.search(r"auto wait_cluster = [^;]*;\s*wait_or_note<true>\(", text) or \
        re.search(r"auto wait_cluster = \[&\][^{]*\{\s*wait_or_note<true>\(", text)
    wait = source("decay.cuh")
    wait = wait[wait.index("template <bool CLUSTER = false>"):]
    assert "try_wait<CLUSTER>(bar, parity)" in wait[:wait.index("\n}")]
    assert "mbarrier.try_wait.parity.acquire.cluster" in source("waits.cuh")


@pytest.mark.parametrize("name", sorted(n for n in os.listdir(CSRC) if n.startswith(("decay", "rotary"))))
def test_nothing_is_loaded_past_the_coherent_caches(name):
    """These kernels may be resident before the one in front of them has written (the states of a cache, the totals that a
    join rewrites in place): its memory is not read-only for their lifetime, as non-coherent loads require."""
    assert not re.search(r"__ldg\(|ld\.global\.nc|__restrict__", source(name))
