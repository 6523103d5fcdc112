"""Linear attention with a decay per head in 64 bits, and the bounds that its tests hold the kernels to.

The reference is the whole sequence's quadratic form, with autograd for the gradients; it knows no chunks:
    o = scale ((q k^T * D) v + exp(G) q S0),  S_T = exp(G_T) S0 + (k exp(G_T - G))^T v,  D_ij = exp(G_i - G_j), j <= i.

Bounds. Every output is a sum of products that each round at most one factor to 16 bits (a score, or a
state as an operand) beside fp32's own work. With W the same sum over the absolute values of the inputs
(all terms positive), u half a unit of the 16-bit type:
    o, dq, dk, dv: u |ref| (the output's rounding) + (u + 2^-15) W
    ht, dh0, dg:   2^-15 W   (keys in two parts, 2^-17 each; exponentials 2^-21; sums of up to 128 terms 2^-17; a
                   chunk's decay 2^-23 per chunk), and the states' own rounding where they are bf16.
fp16 parts below its normal range round to 2^-25 instead, which counts times what they are multiplied by.
dg is also a difference of sums over a chunk's pairs (2^-20 of those)."""
from __future__ import annotations

import torch

from ops_util import HALF_ULP, TINY, assert_close


def make(B, T, H, K, V, hq=None, io=torch.bfloat16, mean=3.0, gate="token", state=torch.float32, h0=True, N=None, seed=0,
         do=True):
    gen = torch.Generator(device="cuda").manual_seed(seed + 11)

    def randn(*s):
        return torch.randn(s, generator=gen, device="cuda")

    hq = hq or H
    N = N or B
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(io)  # noqa: E731
    x = dict(q=unit(randn(B, T, hq, K)), k=unit(randn(B, T, hq, K)), v=randn(B, T, H, V).to(io),
             g=torch.nn.functional.logsigmoid((randn(H) if gate == "head" else randn(B, T, H)) + mean))
    x["h0"] = (0.3 * randn(N, H, K, V)).to(state) if h0 else None
    if do:
        x["do"] = randn(B, T, H, V).to(io)
        x["dht"] = (0.3 * randn(N, H, K, V)).to(state)
    return x


def _run(x, bounds, scale, grads, absolute):
    """(o, ht, and with grads dq, dk, dv, dg, dh0) over flattened rows in 64 bits."""
    H = x["v"].shape[2]
    take = (lambda t: t.double().abs()) if absolute else (lambda t: t.double())
    q, k, v = (take(x[n]).flatten(0, 1) for n in ("q", "k", "v"))
    group = H // q.shape[1]
    g = x["g"].double()
    S0 = x.get("h0")
    N, K, V = len(bounds), q.shape[-1], v.shape[-1]
    S0 = torch.zeros((N, H, K, V), dtype=torch.float64, device=q.device) if S0 is None else take(S0)
    leaves = [t.requires_grad_(grads) for t in (q, k, v, g, S0)]
    rows = g.flatten(0, 1) if g.dim() == 3 else g.expand(q.shape[0], H)
    o, ht = [torch.zeros((0, H, V), dtype=torch.float64, device=q.device)], []
    for n, (a, b) in enumerate(bounds):
        qs, ks = (t[a:b].repeat_interleave(group, 1).transpose(0, 1) for t in (q, k))
        vs, G = v[a:b].transpose(0, 1), rows[a:b].t().cumsum(-1)
        i = torch.arange(b - a, device=q.device)
        low = i[:, None] >= i
        D = torch.exp((G[:, :, None] - G[:, None, :]).masked_fill(~low, 0.0)) * low
        out = scale * ((qs @ ks.transpose(-1, -2) * D) @ vs + torch.exp(G)[..., None] * (qs @ S0[n]))
        o.append(out.transpose(0, 1))
        end = G[:, -1:] if b > a else torch.zeros((H, 1), dtype=torch.float64, device=q.device)
        ht.append(torch.exp(end)[..., None] * S0[n] + (ks * torch.exp(end - G)[..., None]).transpose(-1, -2) @ vs)
    o, ht = torch.cat(o), torch.stack(ht)
    if not grads:
        return {"o": o, "ht": ht}
    dht = torch.zeros_like(ht) if x.get("dht") is None else take(x["dht"])
    got = torch.autograd.grad((o, ht), leaves, (take(x["do"]).flatten(0, 1), dht))
    return dict(zip(("dq", "dk", "dv", "dg", "dh0"), got), o=o.detach(), ht=ht.detach())


def reference(x, bounds, scale=None, grads=False):
    """The outputs and, for each, the sum over absolute values."""
    scale = x["q"].shape[-1] ** -0.5 if scale is None else scale
    return _run(x, bounds, scale, grads, False), _run(x, bounds, scale, grads, True)


def compare(got, x, bounds, scale=None, rows=None):
    """got: {name: tensor}; every output against the reference, element by element and as a whole."""
    grads = "dq" in got
    ref, W = reference(x, bounds, scale, grads)
    io = x["q"].dtype
    u = HALF_ULP[io]
    small = 2.0 ** -24 if io == torch.float16 else 0.0
    for name, y in got.items():
        if y is None:
            continue
        r, w = ref[name], W[name]
        y = y.reshape(r.shape)
        if name in ("o", "dq", "dk", "dv"):
            # (fp16 scores and outputs below its normal range round to 2^-25)
            lim = (u + 2.0 ** -15) * w + TINY[io] + small * (128 * 8 if io == torch.float16 else 0)
            assert_close(y, r, u * 1.01, lim, name)
            whole = 2 * u
        elif name == "dg":
            pairs = (x["q"].double().abs().flatten(0, 1) * W["dq"]).sum(-1)  # [rows, Hqk]
            H = x["v"].shape[2]
            pairs = pairs.repeat_interleave(H // pairs.shape[1], 1)
            most = torch.stack([pairs[a:b].sum(0) if b > a else pairs.new_zeros(H) for a, b in bounds]).amax(0)
            assert_close(y, r, 2.0 ** -23, 2.0 ** -15 * w + 2.0 ** -20 * most + small, name)
            # The sum over all tokens (g [H]) has its terms' errors, 1e-5 of each at most, while the terms themselves
            # may cancel to anything: as a whole it is held to 1e-5 of the sum of their absolute values.
            whole = 1e-5 if x["g"].dim() == 3 else 1e-5 * (w.norm() / r.norm()).item()
        else:
            half = HALF_ULP[y.dtype]
            assert_close(y, r, half * 1.01, 2.0 ** -15 * w + small * 64 + TINY[y.dtype], name)
            whole = 1e-5 if y.dtype == torch.float32 else 2 * half
        norm = r.norm()
        if norm > 0:
            off = ((y.double() - r).norm() / norm).item()
            assert off <= whole, (name, off, whole)


def spans(lens):
    out, at = [], 0
    for n in lens:
        out.append((at, at + n))
        at += n
    return out


def offsets(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(device="cuda", dtype=torch.int32)
