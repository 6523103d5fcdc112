"""CPU checks of linear attention with a decay per head and of rotary positions: what the C entries
refuse before any driver call, workspace sizes, frequencies against their formulas, devices, and
which calls the served layer makes."""
from __future__ import annotations

import ctypes
import math
from types import SimpleNamespace

import pytest
import torch

import chunked_gated_delta_gb300 as kda
from chunked_gated_delta_gb300 import binding, layer
from test_layer_host import Operators
from test_ops_devices import Named

FAKE = 1 << 20  # an aligned non-null address; never dereferenced on these paths
P = ctypes.c_void_p
BF16, F32, F64, I32, I64 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.int64


@pytest.fixture(scope="module")
def lib():
    return kda.load_library()


def refs(dims, opts, kw):
    o = binding.DecayOpts(**kw) if opts is None else opts
    d = kda.make_dims(*dims) if dims else None
    return (ctypes.byref(d) if d else None), (ctypes.byref(o) if o else None)


def call_fwd(lib, dims=(2, 4, 4, 128, 128, 0), opts=None, q=FAKE, k=FAKE, v=FAKE, g=FAKE, h0=None, cu=None, o=FAKE, ht=None,
             word=None, ws=FAKE, size=1 << 40, **kw):
    d, p = refs(dims, opts, kw)
    return lib.kda_decay_fwd(P(q), P(k), P(v), P(g), 0.1, P(h0), P(cu), P(o), P(ht), d, p, P(word), P(ws), size, None)


def call_bwd(lib, dims=(2, 4, 4, 128, 128, 0), opts=None, q=FAKE, do=FAKE, h0=None, dht=None, cu=None, dq=FAKE, dg=FAKE,
             dh0=None, word=None, ws=FAKE, size=1 << 40, **kw):
    d, p = refs(dims, opts, kw)
    return lib.kda_decay_bwd(P(q), P(FAKE), P(FAKE), P(FAKE), P(do), 0.1, P(h0), P(dht), P(cu), P(dq), P(FAKE), P(FAKE),
                             P(dg), P(dh0), d, p, P(word), P(ws), size, None)


def call_step(lib, dims=(2, 1, 4, 128, 128, 0), opts=None, q=FAKE, state=FAKE, slots=None, cu=None, o=FAKE, g=FAKE,
              word=None, **kw):
    d, p = refs(dims, opts, {"num_slots": 8, **kw})
    return lib.kda_decay_step(P(q), P(FAKE), P(FAKE), P(g), 0.1, P(state), P(slots), P(cu), P(o), d, p, P(word), None)


BAD_DIMS = (((0, 1, 4, 128, 128, 0), 1), ((2, -1, 4, 128, 128, 0), 1), ((2, 1, 0, 128, 128, 0), 1),
            ((2, 1, 4, 128, 128, -1), 1), ((2, 4, 4, 128, 128, 3), 1), ((2, 1, 4, 96, 128, 0), 2),
            ((2, 1, 4, 128, 32, 0), 2), ((1, 1 << 30, 4, 128, 128, 0), 2))
BAD_OPTS = (dict(io_dtype=2), dict(state_dtype=2), dict(head_gate=2), dict(reserved=1), dict(qk_heads=3),
            dict(qk_heads=-1), dict(qk_heads=8), dict(q_stride=504), dict(v_stride=8), dict(g_stride=3),
            dict(head_gate=1, g_stride=4))


@pytest.mark.parametrize("call", [call_fwd, call_bwd, call_step])
def test_refusals_that_they_share(lib, call):
    assert call(lib, dims=None) == 1 and call(lib, opts=False) == 1
    for dims, code in BAD_DIMS:
        assert call(lib, dims=dims, cu=FAKE if dims[5] > 0 else None) == code, dims
    for kw in BAD_OPTS:
        assert call(lib, **kw) == 1, kw
    assert call(lib, cu=FAKE) == 1 and call(lib, dims=(1, 4, 4, 128, 128, 3)) == 1
    assert call(lib, q=0) == 1 and call(lib, q=FAKE + 1) == 3 and call(lib, word=FAKE + 2) == 3


def test_forward_refusals(lib):
    assert call_fwd(lib, o=0) == 1 and call_fwd(lib, num_slots=1) == 1 and call_fwd(lib, do_stride=512) == 1
    assert call_fwd(lib, h0=FAKE, ht=FAKE) == 1                       # one memory for both
    for kw in (dict(q=FAKE + 8), dict(v=FAKE + 2), dict(o=FAKE + 8), dict(ht=FAKE + 8), dict(g=FAKE + 2),
               dict(q_stride=516), dict(k_stride=513)):
        assert call_fwd(lib, **kw) == 3, kw
    long = (1, 40000, 1, 128, 128, 0)                                 # cut into pieces: needs a workspace
    assert call_fwd(lib, dims=long, ws=0) == 4 and call_fwd(lib, dims=long, size=1000) == 4
    assert call_fwd(lib, dims=long, ws=FAKE + 128) == 4
    assert call_fwd(lib, dims=(2, 0, 4, 128, 128, 0), q=0, k=0, v=0, g=0, o=0) == 0  # nothing to do


def test_backward_refusals(lib):
    assert call_bwd(lib, do=0) == 1 and call_bwd(lib, dq=0) == 1 and call_bwd(lib, dg=0) == 1 and call_bwd(lib, num_slots=1) == 1
    assert call_bwd(lib, h0=FAKE, dh0=FAKE) == 1 and call_bwd(lib, dht=FAKE, dh0=FAKE) == 1
    for kw in (dict(do=FAKE + 8), dict(dq=FAKE + 8), dict(dh0=FAKE + 4), dict(dg=FAKE + 1), dict(do_stride=516)):
        assert call_bwd(lib, **kw) == 3, kw
    assert call_bwd(lib, ws=0) == 4 and call_bwd(lib, size=100) == 4 and call_bwd(lib, ws=FAKE + 64) == 4


def test_step_refusals(lib):
    assert call_step(lib, num_slots=0) == 1 and call_step(lib, num_slots=1) == 1 and call_step(lib, do_stride=512) == 1
    assert call_step(lib, state=0) == 1 and call_step(lib, o=0) == 1
    assert call_step(lib, state=FAKE + 8) == 3 and call_step(lib, o=FAKE + 8) == 3 and call_step(lib, slots=FAKE + 2) == 3
    assert call_step(lib, dims=(2, 0, 4, 128, 128, 0), q=0, state=0, o=0) == 0


def test_rotary_refusals(lib):
    def call(tokens=4, hq=2, hk=1, dim=64, q=FAKE, k=FAKE * 3, pos=FAKE, freqs=FAKE, qo=FAKE * 2, ko=FAKE * 4, opts=None, **kw):
        o = binding.RotaryOpts(**{"pairs": 32, "amplitude": 1.0, **kw}) if opts is None else opts
        return lib.kda_rotary(P(q), P(k), P(pos), P(freqs), P(qo), P(ko), tokens, hq, hk, dim, ctypes.byref(o) if o else None, None)

    assert call(opts=False) == 1
    for kw in (dict(tokens=-1), dict(hq=0), dict(hk=-1), dict(dim=0), dict(pairs=0), dict(pairs=33), dict(io_dtype=3),
               dict(positions_i64=2), dict(interleaved=2), dict(inverse=-1), dict(reserved=1), dict(q_stride=127),
               dict(k_out_stride=8), dict(q=0), dict(k=0), dict(pos=0), dict(freqs=0), dict(qo=0), dict(ko=0),
               dict(qo=FAKE, q_stride=136), dict(ko=FAKE * 3, k_out_stride=72), dict(ko=FAKE * 2), dict(qo=FAKE * 3),
               dict(ko=FAKE)):
        assert call(**kw) == 1, kw
    assert call(dim=2048, pairs=513) == 2
    for kw in (dict(q=FAKE + 1), dict(ko=FAKE + 1), dict(pos=FAKE + 2), dict(positions_i64=1, pos=FAKE + 4), dict(freqs=FAKE + 4)):
        assert call(**kw) == 3, kw
    assert call(tokens=0, q=0, k=0, qo=0, ko=0, pos=0, freqs=0) == 0


def test_workspace_sizes():
    many, one = kda.make_dims(4, 8192, 32, 128, 128), kda.make_dims(1, 65536, 2, 128, 128)
    assert kda.decay_workspace_size(many, False) == 0       # as many sequences x heads as SMs: nothing is cut
    assert kda.decay_workspace_size(one, False) > 0
    states = 2 * 4 * 64 * 32 * 4 * 128 * 128                # before each of 64 chunks, and its gradient, in 4 bytes
    back = kda.decay_workspace_size(many, True)
    assert states <= back <= states + (1 << 20)
    grouped = kda.decay_workspace_size(many, True, qk_heads=8)
    assert grouped - back >= 2 * 4 * 8192 * 32 * 128 * 4    # fp32 dq and dk per value head, but of groups of two
    assert kda.decay_workspace_size(many, True, qk_heads=16) == back
    assert kda.decay_workspace_size(many, True, qk_heads=32) == back
    assert kda.decay_workspace_size(many, True, head_gate=True) - back >= 4 * 8192 * 32 * 4
    with pytest.raises(kda.KdaError):
        kda.decay_workspace_size(kda.make_dims(1, 5, 3, 128, 96), False)
    with pytest.raises(kda.KdaError):
        kda.decay_workspace_size(many, False, qk_heads=5)


@pytest.mark.parametrize("dim,base", [(64, 1e4), (128, 5e5), (2, 1e4), (96, 1e6)])
def test_frequencies(dim, base):
    plain, one = kda.rotary_freqs(dim, base=base, device="cpu")
    want = torch.tensor([base ** (-2.0 * i / dim) for i in range(dim // 2)], dtype=torch.float64)
    assert plain.dtype == F64 and one == 1.0 and torch.allclose(plain, want, rtol=1e-14, atol=0)
    linear, _ = kda.rotary_freqs(dim, base=base, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(linear, want / 4.0, rtol=1e-14, atol=0)
    ntk, _ = kda.rotary_freqs(dim, base=base, scaling="ntk", factor=4.0, device="cpu")
    assert ntk[0] == 1.0 and (dim == 2 or abs(ntk[-1] / (want[-1] / 4.0) - 1.0) < 1e-12)  # the fastest kept, the slowest divided
    yarn, amplitude = kda.rotary_freqs(dim, base=base, scaling="yarn", factor=16.0, original_length=8192, device="cpu")
    assert abs(amplitude - (0.1 * math.log(16.0) + 1.0)) < 1e-15
    share = (want / yarn - 1.0) / 15.0                       # 0 where kept, 1 where divided
    turns = want * 8192 / (2 * math.pi)
    assert bool((share >= -1e-12).all()) and bool((share <= 1.0 + 1e-12).all()) and bool((share.diff() >= -1e-12).all())
    if dim > 2:
        assert bool((share[turns > 64.0] == 0).all()) and bool(((1.0 - share[turns < 0.5]).abs() < 1e-9).all())


def test_frequencies_refused():
    for bad in (dict(dim=63), dict(dim=0), dict(dim=64, base=0.0), dict(dim=64, factor=0.0), dict(dim=64, scaling="other")):
        with pytest.raises(ValueError):
            kda.rotary_freqs(**bad, device="cpu")


IN = {"q": ((2, 3, 2, 64), BF16), "k": ((2, 3, 2, 64), BF16), "v": ((2, 3, 4, 64), BF16), "g": ((2, 3, 4), F32)}
PACKED = {n: ((1, 6, *s[2:]), t) for n, (s, t) in IN.items()}
STATE, WORD = ((2, 4, 64, 64), F32), ((1,), I32)
CALLS = {
    "fwd": (kda.decay_fwd, {**IN, "h0": STATE, "final_state": STATE, "out": IN["v"], "status": WORD, "workspace": ((4096,), torch.uint8)}),
    "packed fwd": (kda.decay_fwd, {**PACKED, "cu_seqlens": ((3,), I32)}),
    "bwd": (kda.decay_bwd, {**IN, "do": IN["v"], "h0": STATE, "dht": STATE, "status": WORD, "workspace": ((4096,), torch.uint8)}),
    "step": (kda.decay_step, {**IN, "state": STATE, "slots": ((2,), I32), "out": IN["v"], "status": WORD}),
    "rotary": (kda.rotary, {"q": IN["q"], "k": IN["k"], "positions": ((2, 3), I64), "freqs": ((16,), F64),
                            "q_out": IN["q"], "k_out": IN["k"]}),
}


@pytest.mark.parametrize("call,other", [(c, n) for c, (_, a) in CALLS.items() for n in a])
def test_one_tensor_on_another_gpu(call, other):
    fn, args = CALLS[call]
    given = {n: Named(shape, dtype, "cuda:1" if n == other else "cuda:0") for n, (shape, dtype) in args.items()}
    with pytest.raises(TypeError, match="on one device"):
        fn(**given)


@pytest.mark.parametrize("call", list(CALLS))
def test_a_stream_of_another_gpu(call):
    fn, args = CALLS[call]
    given = {n: Named(shape, dtype) for n, (shape, dtype) in args.items()}
    with pytest.raises(TypeError, match="stream must be of the tensors' device"):
        fn(**given, stream=SimpleNamespace(cuda_stream=0, device_index=1))


class DecayOperators(Operators):
    def rotary_freqs(self, dim, device="cpu", **kw):
        return kda.rotary_freqs(dim, device=device, **kw)

    def rotary(self, q, k, positions, freqs, amplitude, interleaved, q_out=None, k_out=None):
        self.calls.append(("rotary", positions))
        assert q_out is q and k_out is k

    def decay_step(self, q, k, v, g, state, slots=None, cu_seqlens=None, status=None):
        self.calls.append(("decay_step", status))
        self.g = g
        return v.clone()

    def decay_fwd(self, q, k, v, g, h0=None, cu_seqlens=None, workspace=None, status=None):
        self.calls.append(("decay_fwd", status))
        self.g = g
        return v.clone(), torch.zeros((v.shape[0], v.shape[2], q.shape[-1], v.shape[-1]))


@pytest.mark.parametrize("constant", [False, True])
@pytest.mark.parametrize("path", ["prefill", "decode"])
def test_the_layers_calls(monkeypatch, path, constant):
    ops = DecayOperators()
    monkeypatch.setattr(layer, "kda", ops)
    m = layer.DecayLayer.random(128, 4, 2, 64, 64, constant_decay=constant, seed=1, device="cpu")
    x = torch.randn((2, 3, 128), generator=torch.Generator().manual_seed(4)).bfloat16()
    word = torch.zeros(1, dtype=torch.int32)
    pos = torch.tensor([[5, 6, 7], [0, 1, 2]])
    if path == "prefill":
        m.prefill(x, status=word)
        assert [p.tolist() for n, p in ops.calls if n == "rotary"] == [[[0, 1, 2]] * 2]
    else:
        m.decode(x, torch.zeros((2, 4, 64, 64)), pos, status=word)
        assert [p for n, p in ops.calls if n == "rotary"] == [pos]
    takes = [(n, s) for n, s in ops.calls if n in ("linear", "decay_step", "decay_fwd")]
    assert [n for n, _ in takes].count("linear") == (4 if constant else 5) and all(s is word for _, s in takes)
    assert tuple(ops.g.shape) == ((4,) if constant else (2, 3, 4)) and ops.g.dtype == F32
