"""Shared helpers of the tests of the served layer's operators (decode step,
RMS norm, projection): 64-bit references and rounding bounds."""
from __future__ import annotations

import torch

# relative half-ulp of a rounding to each type (elementwise bound of one rounding): 2^-8 for bf16's 8-bit significand
HALF_ULP = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32)}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}  # half the least subnormal
EPS32 = 2.0 ** -24

GUARD = 1 << 12


class Guarded:
    """A tensor inside a pattern-filled allocation: what lies before and after it must not change."""

    def __init__(self, shape, dtype, fill=None):
        n = 1
        for s in shape:
            n *= s
        self.nbytes = n * torch.empty((), dtype=dtype).element_size()
        self.raw = torch.full((self.nbytes + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.t = self.raw[GUARD:GUARD + self.nbytes].view(dtype).view(shape)
        if fill is not None:
            self.t.copy_(fill)

    def intact(self):
        return bool((self.raw[:GUARD] == 0xA5).all()) and bool((self.raw[GUARD + self.nbytes:] == 0xA5).all())


def assert_close(got, ref, rel, abs_, what=""):
    """|got - ref| <= rel |ref| + abs_ in every element (abs_ a number or a tensor)."""
    err = (got.double() - ref).abs()
    lim = rel * ref.abs() + abs_
    assert not torch.isnan(err).any(), (what, "NaN")
    worst = (err / lim.clamp_min(1e-300)).max().item() if err.numel() else 0.0
    assert worst <= 1.0, (what, worst)


def step_reference(q, k, v, g, beta, state, slots, bounds, scale, logits=False):
    """The recurrence in 64 bits, sequence by sequence.  bounds: [(first row, end row)] over the flattened
    token rows.  Returns (o, state, bound) with bound a worst-case fp32 error of o and of the state: per
    token, the decay (3 roundings), S^T k and S^T q (K + 3 roundings of at most sqrt(K) max|S|), and the update."""
    H, K, V = state.shape[1:]
    group = H // q.shape[-2]
    rows = q.shape[0] * q.shape[1]
    q, k = (x.reshape(rows, x.shape[2], K).double().repeat_interleave(group, 1) for x in (q, k))
    v, g, beta = v.reshape(rows, H, V).double(), g.reshape(rows, H, K).double(), beta.reshape(rows, H).double()
    beta = torch.sigmoid(beta) if logits else beta
    out = state.double().clone()
    o = torch.zeros((rows, H, V), dtype=torch.float64, device=q.device)
    worst_o = worst_s = 0.0
    per = EPS32 * (8 + (K + 4) * K ** 0.5)
    for n, (a, b) in enumerate(bounds):
        if slots[n] < 0:
            continue
        S = out[slots[n]]
        top = max(1.0, S.abs().max().item()) if S.numel() else 1.0
        for i, t in enumerate(range(a, b)):
            S = torch.exp(g[t])[..., None] * S
            d = beta[t][..., None] * (v[t] - torch.einsum("hkv,hk->hv", S, k[t]))
            S = S + k[t][..., None] * d[:, None, :]
            top = max(top, S.abs().max().item(), d.abs().max().item())
            o[t] = scale * torch.einsum("hkv,hk->hv", S, q[t])
            worst_s = max(worst_s, (i + 1) * per * top)
            worst_o = max(worst_o, (i + 2) * per * top * abs(scale) * K ** 0.5)
        out[slots[n]] = S
    return o, out, (worst_o, worst_s)
