"""A served KDA layer from the library's operators: the path from a layer's
input to its output, for a prompt (kda.fwd) and for new tokens (kda.step).

    x, residual -> rms_norm (the sum, 8 bits or 16)
                -> linear x 5: q, k, v (silu), g (log-sigmoid, fp32, biased), beta (sigmoid)
                -> rms_norm of the heads of q and k (unit length)
                -> fwd | step
                -> rms_norm of the heads of o (with e4m3 operands then to 8 bits, a scale a token)
                -> linear, the residual added

Shapes: x [B, T, D] (or one packed row [1, total, D] with cu_seqlens), hidden
size D, H heads of K (q, k, g) and V (v, o).  The weights are those of a model
that serves with this layer; ``random`` makes seeded ones for tests and timing.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import binding as kda

_F8 = torch.float8_e4m3fn
# rms_norm with these two only turns rows into 8 bits: beside 2^100 the mean square of a row is below the last bit
# (as long as its elements are below 2^37), so the division is by 2^50, and the weight's 2^50 takes it back, both exactly.
_NO_NORM_EPS, _NO_NORM_WEIGHT = 2.0 ** 100, 2.0 ** 50


def quantise_rows(w):
    """w [N, K] as e4m3 codes and one fp32 scale per row (w ~ codes * scale[:, None]), once, when a model is loaded."""
    scale = w.float().abs().amax(1).clamp_min(1e-30) / 448.0
    return (w.float() / scale[:, None]).to(_F8), scale


@dataclass
class Projection:
    """A linear layer's weight [N, K] (16 bits, or e4m3 with row scales) and fp32 bias."""
    w: torch.Tensor
    scale: torch.Tensor | None = None
    bias: torch.Tensor | None = None

    def __call__(self, x, x_scale, act=None, residual=None, out_dtype=None, status=None):
        return kda.linear(x, self.w, bias=self.bias, act=act, residual=residual, x_scale=x_scale, w_scale=self.scale,
                          out_dtype=out_dtype, status=status)


class KdaLayer:
    def __init__(self, heads, K, V, q, k, v, g, beta, out, norm, head_norm, eps=1e-6):
        """q, k, g: [H K, D], v: [H V, D], beta: [H, D], out: [D, H V] (Projection, all
        of one operand type); norm [D], head_norm [V]: weights of the norms."""
        self.heads, self.K, self.V, self.eps = heads, K, V, eps
        self.q, self.k, self.v, self.g, self.beta, self.out = q, k, v, g, beta, out
        self.norm, self.head_norm = norm, head_norm
        self.eight_bit = q.w.dtype == _F8
        # rms_norm over a head times K^-1/2 is division by the head's length
        self.unit = torch.full((K,), K ** -0.5, dtype=torch.float32, device=norm.device)
        self.no_norm = torch.full((heads * V,), _NO_NORM_WEIGHT, dtype=torch.float32, device=norm.device)

    @classmethod
    def random(cls, D, heads, K, V, eight_bit=False, seed=0, device="cuda", dtype=torch.bfloat16):
        gen = torch.Generator(device=device).manual_seed(seed)

        def projection(n, k, bias=None):
            w = torch.randn((n, k), generator=gen, device=device) / k ** 0.5
            w, scale = quantise_rows(w) if eight_bit else (w.to(dtype), None)
            return Projection(w, scale, bias)

        gate_bias = torch.full((heads * K,), 3.0, device=device)  # decays near 1, as synth.py draws them
        return cls(heads, K, V, projection(heads * K, D), projection(heads * K, D), projection(heads * V, D),
                   projection(heads * K, D, gate_bias), projection(heads, D), projection(D, heads * V),
                   1.0 + 0.1 * torch.randn(D, generator=gen, device=device),
                   1.0 + 0.1 * torch.randn(V, generator=gen, device=device))

    def _norm(self, x, weight, residual=None):
        """The rows as the projections take them: (codes, scales) or (16 bits, None), and the residual's sum."""
        return kda.rms_norm(x, weight, residual=residual, eps=self.eps, out_dtype=_F8 if self.eight_bit else None)

    def _inputs(self, x, residual, status):
        B, T, _ = x.shape
        H, io = self.heads, x.dtype
        n, scale, total = self._norm(x, self.norm, residual)
        q, k, v = (p(n, scale, act="silu", out_dtype=io, status=status).view(B, T, H, -1)
                   for p in (self.q, self.k, self.v))
        g = self.g(n, scale, act="logsigmoid", out_dtype=torch.float32, status=status).view(B, T, H, self.K)
        beta = self.beta(n, scale, act="sigmoid", out_dtype=io, status=status)
        q, k = (kda.rms_norm(t, self.unit, eps=self.eps)[0] for t in (q, k))
        return (q, k, v, g, beta), x if total is None else total

    def _output(self, o, total, status=None):
        B, T, H, V = o.shape
        n, _, _ = kda.rms_norm(o, self.head_norm, eps=self.eps)
        n, scale = n.view(B, T, H * V), None
        if self.eight_bit:  # one scale per token for the projection's operand, which is not normed again
            n, scale, _ = kda.rms_norm(n, self.no_norm, eps=_NO_NORM_EPS, out_dtype=_F8)
        return self.out(n, scale, residual=total, out_dtype=total.dtype, status=status)

    def prefill(self, x, residual=None, h0=None, cu_seqlens=None, workspace=None, status=None):
        """Prompts: (y [B, T, D], the states [N, H, K, V] after them).  y holds x + residual + the layer's output.
        ``status`` takes the projections' errors (see kda.step); the forward's are in ``workspace`` (kda.status)."""
        inputs, total = self._inputs(x, residual, status)
        o, state = kda.fwd(*inputs, h0=h0, cu_seqlens=cu_seqlens, workspace=workspace)
        return self._output(o, total, status), state

    def decode(self, x, state, slots=None, residual=None, cu_seqlens=None, status=None):
        """New tokens: y [B, T, D]; the cache of states [slots, H, K, V] is updated in place (see kda.step).
        ``status`` takes the errors of the step and of the projections."""
        inputs, total = self._inputs(x, residual, status)
        o = kda.step(*inputs, state, slots=slots, cu_seqlens=cu_seqlens, status=status)
        return self._output(o, total, status)
