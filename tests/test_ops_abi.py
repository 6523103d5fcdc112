"""CPU checks of the C entries of the served layer's operators: bad arguments
are refused before any driver call (here, without a GPU, a launch would fail
with KDA_ERR_CUDA = 5), and calls without work return at once."""
import ctypes

import pytest

import chunked_gated_delta_gb300 as kda
from chunked_gated_delta_gb300 import binding

FAKE = 1 << 20  # a 16-byte-aligned non-null address; never dereferenced on these paths
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    return kda.load_library()


def call_step(lib, dims=(2, 1, 4, 128, 128, 0), opts=None, q=FAKE, state=FAKE, slots=None, cu=None, o=FAKE, g=FAKE,
              word=None, **kw):
    o_ = binding.StepOpts(**{"num_slots": 8, **kw}) if opts is None else opts
    d = kda.make_dims(*dims) if dims else None
    return lib.kda_step(P(q), P(FAKE), P(FAKE), P(g), P(FAKE), 0.1, P(state), P(slots), P(cu), P(o),
                        ctypes.byref(d) if d else None, ctypes.byref(o_) if o_ else None, P(word), None)


def test_step_refusals(lib):
    assert call_step(lib, dims=None) == 1 and call_step(lib, opts=False) == 1
    assert call_step(lib, dims=(2, 1, 4, 96, 128, 0)) == 2 and call_step(lib, dims=(2, 1, 4, 128, 32, 0)) == 2
    for dims in ((0, 1, 4, 128, 128, 0), (2, -1, 4, 128, 128, 0), (2, 1, 0, 128, 128, 0), (2, 1, 4, 128, 128, -1)):
        assert call_step(lib, dims=dims) == 1
    assert call_step(lib, cu=FAKE) == 1                                       # cu_seqlens without num_seqs
    assert call_step(lib, dims=(1, 4, 4, 128, 128, 3)) == 1                   # num_seqs without cu_seqlens
    assert call_step(lib, dims=(2, 4, 4, 128, 128, 3), cu=FAKE) == 1          # packed needs B = 1
    for kw in (dict(io_dtype=2), dict(state_dtype=2), dict(beta_logits=2), dict(reserved=1), dict(num_slots=0),
               dict(num_slots=1), dict(qk_heads=3), dict(qk_heads=-1), dict(qk_heads=8), dict(q_stride=511),
               dict(v_stride=1), dict(g_stride=-512), dict(beta_stride=3)):
        assert call_step(lib, **kw) == 1, kw
    assert call_step(lib, q=0) == 1 and call_step(lib, state=0) == 1 and call_step(lib, o=0) == 1
    assert call_step(lib, q=FAKE + 1) == 3 and call_step(lib, g=FAKE + 2) == 3
    assert call_step(lib, state=FAKE + 8) == 3 and call_step(lib, o=FAKE + 8) == 3
    assert call_step(lib, slots=FAKE + 2) == 3 and call_step(lib, word=FAKE + 1) == 3
    assert call_step(lib, dims=(1, 1 << 30, 4, 128, 128, 0)) == 2             # rows beyond 32-bit coordinates
    assert call_step(lib, dims=(2, 0, 4, 128, 128, 0), q=0, state=0, o=0) == 0  # no tokens: nothing to do


def call_norm(lib, rows=4, dim=128, x=FAKE, r=None, w=None, y=FAKE, scale=None, s=None, opts=None, **kw):
    o = binding.NormOpts(**{"eps": 1e-6, **kw}) if opts is None else opts
    return lib.kda_rms_norm(P(x), P(r), P(w), P(y), P(scale), P(s), rows, dim, ctypes.byref(o) if o else None, None)


def test_norm_refusals(lib):
    assert call_norm(lib, opts=False) == 1
    assert call_norm(lib, rows=-1) == 1 and call_norm(lib, dim=0) == 1
    assert call_norm(lib, dim=32769) == 2 and call_norm(lib, rows=1 << 31) == 2
    for kw in (dict(io_dtype=3), dict(io_dtype=-1), dict(out_dtype=1), dict(out_dtype=4), dict(weight_f32=2),
               dict(eps=-1.0), dict(eps=float("nan")), dict(x_stride=127), dict(residual_stride=-1),
               dict(sum_stride=1), dict(out_dtype=3), dict(scale=FAKE)):
        assert call_norm(lib, **kw) == 1, kw
    assert call_norm(lib, x=0) == 1 and call_norm(lib, y=0) == 1
    assert call_norm(lib, x=FAKE + 1) == 3 and call_norm(lib, r=FAKE + 1) == 3
    assert call_norm(lib, w=FAKE + 2, weight_f32=1) == 3 and call_norm(lib, scale=FAKE + 2, out_dtype=3) == 3
    assert call_norm(lib, rows=0, x=0, y=0) == 0                              # nothing to do


def call_linear(lib, M=4, N=128, K=64, x=FAKE, w=FAKE, b=None, r=None, xs=None, ws=None, y=FAKE, word=None, opts=None,
                **kw):
    o = binding.LinearOpts(**kw) if opts is None else opts
    return lib.kda_linear(P(x), P(w), P(b), P(r), P(xs), P(ws), P(y), M, N, K, ctypes.byref(o) if o else None, P(word),
                          None)


def test_linear_refusals(lib):
    assert call_linear(lib, opts=False) == 1
    assert call_linear(lib, M=-1) == 1 and call_linear(lib, N=0) == 1 and call_linear(lib, K=0) == 1
    for kw in (dict(io_dtype=2), dict(io_dtype=4), dict(out_dtype=3), dict(act=5), dict(act=-1), dict(reserved=1),
               dict(io_dtype=3), dict(io_dtype=3, xs=FAKE), dict(xs=FAKE), dict(ws=FAKE), dict(x_stride=63),
               dict(w_stride=8), dict(residual_stride=127), dict(y_stride=-128)):
        assert call_linear(lib, **kw) == 1, kw
    assert call_linear(lib, x=0) == 1 and call_linear(lib, w=0) == 1 and call_linear(lib, y=0) == 1
    assert call_linear(lib, x=FAKE + 8) == 3 and call_linear(lib, w=FAKE + 2) == 3 and call_linear(lib, K=63) == 3
    assert call_linear(lib, x_stride=68) == 3 and call_linear(lib, w_stride=65) == 3
    assert call_linear(lib, y=FAKE + 1) == 3 and call_linear(lib, r=FAKE + 1) == 3 and call_linear(lib, b=FAKE + 2) == 3
    assert call_linear(lib, word=FAKE + 2) == 3
    assert call_linear(lib, M=1 << 31) == 2 and call_linear(lib, N=1 << 31) == 2
    assert call_linear(lib, M=0, x=0, y=0) == 0                               # nothing to do


def test_bad_slots_has_a_name():
    assert "slot" in kda.status_string(8) and binding.STATUS_NAMES[8] == "KDA_ERR_BAD_SLOTS"
