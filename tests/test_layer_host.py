"""The served layer's composition (layer.KdaLayer) on the CPU: the three operators
are replaced by their formulas, so what is tested is which calls the layer makes."""
from __future__ import annotations

import pytest
import torch

from chunked_gated_delta_gb300 import layer

F8 = torch.float8_e4m3fn


class Operators:
    """rms_norm, linear, step and fwd by their formulas on CPU tensors."""

    def __init__(self):
        self.calls = []

    def rms_norm(self, x, weight=None, residual=None, eps=1e-6, out_dtype=None):
        self.calls.append(("rms_norm", None))
        s = x.float() + (residual.float() if residual is not None else 0.0)
        y = s / torch.sqrt(s.square().mean(-1, keepdim=True) + eps)
        y = y * weight.float() if weight is not None else y
        total = s.to(x.dtype) if residual is not None else None
        if out_dtype != F8:
            return y.to(out_dtype or x.dtype), None, total
        a = y.abs().amax(-1).clamp_min(1e-30)
        return (y * (448.0 / a)[..., None]).to(F8), a / 448.0, total

    def linear(self, x, w, bias=None, act=None, residual=None, x_scale=None, w_scale=None, out_dtype=None, status=None):
        self.calls.append(("linear", status))
        y = x.float() @ w.float().T
        if x_scale is not None:
            y = y * x_scale[..., None] * w_scale
        y = y + bias if bias is not None else y
        y = {None: lambda t: t, "silu": torch.nn.functional.silu, "sigmoid": torch.sigmoid,
             "logsigmoid": torch.nn.functional.logsigmoid}[act](y)
        y = y + residual.float() if residual is not None else y
        return y.to(out_dtype or x.dtype)

    def step(self, q, k, v, g, beta, state, slots=None, cu_seqlens=None, status=None):
        self.calls.append(("step", status))
        return v.clone()

    def fwd(self, q, k, v, g, beta, h0=None, cu_seqlens=None, workspace=None):
        self.calls.append(("fwd", None))
        B, _, H, V = v.shape
        return v.clone(), torch.zeros((B, H, q.shape[-1], V))


@pytest.fixture
def ops(monkeypatch):
    fake = Operators()
    monkeypatch.setattr(layer, "kda", fake)
    return fake


@pytest.mark.parametrize("size", [1.0, 3e-4])
@pytest.mark.parametrize("head_norm", [0.3, 1.0, 2.0])
def test_eight_bit_output_is_the_sixteen_bit_formula(ops, head_norm, size):
    """The output projection's operand in 8 bits stands for the head-normed rows themselves, whatever the norm's
    weight and however small o is.  An e4m3 rounding moves an element by at most 2^-4 of itself, 2^-4 / sqrt(3) rms
    (3.6 percent); the projection of random weights keeps that share of its norm, and 5 percent bounds it."""
    D, H, V = 192, 4, 64
    m = layer.KdaLayer.random(D, H, 64, V, eight_bit=True, seed=1, device="cpu")
    m.head_norm = head_norm * m.head_norm
    gen = torch.Generator().manual_seed(2)
    o = (size * torch.randn((3, 5, H, V), generator=gen)).bfloat16()
    total = torch.zeros((3, 5, D), dtype=torch.bfloat16)
    y = m._output(o, total).double()
    od = o.double()
    n = od / torch.sqrt(od.square().mean(-1, keepdim=True) + m.eps) * m.head_norm.double()
    ref = n.reshape(3, 5, H * V) @ (m.out.w.double() * m.out.scale.double()[:, None]).T
    assert (y - ref).norm() <= 0.05 * ref.norm()


@pytest.mark.parametrize("eight_bit", [False, True])
@pytest.mark.parametrize("path", ["prefill", "decode"])
def test_every_projection_reports_to_the_status_word(ops, path, eight_bit):
    m = layer.KdaLayer.random(128, 2, 64, 64, eight_bit=eight_bit, seed=1, device="cpu")
    x = torch.randn((2, 3, 128), generator=torch.Generator().manual_seed(4)).bfloat16()
    word = torch.zeros(1, dtype=torch.int32)
    if path == "prefill":
        m.prefill(x, status=word)
    else:
        m.decode(x, torch.zeros((2, 2, 64, 64)), status=word)
    takes = [(name, status) for name, status in ops.calls if name in ("linear", "step")]
    assert [name for name, _ in takes].count("linear") == 6
    assert all(status is word for _, status in takes)
