"""The served layer (layer.KdaLayer): its wiring against the formulas in 64 bits
on the same weights, and decoding after a prompt against one longer prompt."""
from __future__ import annotations

import pytest
import torch

from chunked_gated_delta_gb300 import layer

pytestmark = pytest.mark.gpu


def weight(p):
    w = p.w.double()
    return w * p.scale.double()[:, None] if p.scale is not None else w


def reference(m, x, residual, state):
    """The layer in 64 bits, token by token; returns (y, state)."""
    B, T, D = x.shape
    H, K, V = m.heads, m.K, m.V
    total = x.double() + residual.double()

    def rms(t, w):
        return t / torch.sqrt(t.square().mean(-1, keepdim=True) + m.eps) * w.double()

    n = rms(total, m.norm)
    silu = torch.nn.functional.silu
    q, k, v = (silu(n @ weight(p).T).view(B, T, H, -1) for p in (m.q, m.k, m.v))
    g = torch.nn.functional.logsigmoid(n @ weight(m.g).T + m.g.bias.double()).view(B, T, H, K)
    beta = torch.sigmoid(n @ weight(m.beta).T)
    q, k = (t / t.norm(dim=-1, keepdim=True) for t in (q, k))
    S, os = state.double(), []
    for t in range(T):
        S = S * g[:, t].exp()[..., None]
        d = beta[:, t][..., None] * (v[:, t] - torch.einsum("bhkv,bhk->bhv", S, k[:, t]))
        S = S + k[:, t][..., None] * d[:, :, None]
        os.append(torch.einsum("bhkv,bhk->bhv", S, q[:, t]) * K ** -0.5)
    o = rms(torch.stack(os, 1), m.head_norm).reshape(B, T, H * V)
    if m.eight_bit:
        o = rms(o, torch.ones(H * V, device=x.device))
    return total + o @ weight(m.out).T, S


@pytest.mark.parametrize("eight_bit", [False, True])
@pytest.mark.parametrize("T", [1, 3])
def test_decode_matches_the_formulas(eight_bit, T):
    """Tolerances: with 16-bit operands every tensor between the operators is rounded to bf16 (2^-9 rms): the
    layer's output, behind five of them in a row, is held to 2 percent; with e4m3 operands (2^-5 rms a rounding,
    two on the way) to 10."""
    D, H, K, V, B = 256, 4, 64, 64, 5
    m = layer.KdaLayer.random(D, H, K, V, eight_bit=eight_bit, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((B, T, D), generator=gen, device="cuda").bfloat16()
    r = torch.randn((B, T, D), generator=gen, device="cuda").bfloat16()
    state = 0.3 * torch.randn((B, H, K, V), generator=gen, device="cuda")
    y_ref, s_ref = reference(m, x, r, state)
    y = m.decode(x, state, residual=r)
    tol = 0.10 if eight_bit else 0.02
    part, part_ref = y.double() - (x.double() + r.double()), y_ref - (x.double() + r.double())
    assert (part - part_ref).norm() <= tol * part_ref.norm() + 2.0 ** -8 * (x.double() + r.double()).norm()
    assert (state.double() - s_ref).norm() <= tol * s_ref.norm()


@pytest.mark.parametrize("eight_bit", [False, True])
def test_prompt_then_tokens(eight_bit):
    """Prompt of 130 tokens, then 6 tokens (one by one, and several at once), is close to a prompt of 136: the same
    projections of the same rows, so the difference is the forward's own rounding of its operands."""
    D, H, K, V, B, T, n = 512, 4, 128, 128, 2, 130, 6
    m = layer.KdaLayer.random(D, H, K, V, eight_bit=eight_bit, seed=5)
    gen = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn((B, T + n, D), generator=gen, device="cuda").bfloat16()
    y_all, s_all = m.prefill(x)
    _, s = m.prefill(x[:, :T].contiguous())
    cache = torch.full((5, H, K, V), float("nan"), device="cuda")
    slots = torch.tensor([4, 1], dtype=torch.int32, device="cuda")
    cache[4], cache[1] = s[0], s[1]
    ys = [m.decode(x[:, T + i:T + i + 1].contiguous(), cache, slots=slots) for i in range(3)]
    ys.append(m.decode(x[:, T + 3:].contiguous(), cache, slots=slots))
    y = torch.cat(ys, 1).double()
    ref = y_all[:, T:].double()
    assert (y - ref).norm() <= 0.02 * ref.norm()
    assert (torch.stack([cache[4], cache[1]]).double() - s_all.double()).norm() <= 0.02 * s_all.double().norm()
    assert torch.isnan(cache[[0, 2, 3]]).all()


def test_packed_prompts_and_packed_tokens():
    D, H, K, V = 256, 2, 64, 128
    m = layer.KdaLayer.random(D, H, K, V, seed=7)
    lens = [70, 1, 129]
    cu = torch.tensor([0, 70, 71, 200], dtype=torch.int32, device="cuda")
    x = torch.randn((1, 200, D), device="cuda").bfloat16()
    y, s = m.prefill(x, cu_seqlens=cu)
    for i, L in enumerate(lens):
        a = int(cu[i])
        yi, si = m.prefill(x[:, a:a + L].contiguous())
        assert (yi.double() - y[:, a:a + L].double()).norm() <= 0.01 * yi.double().norm()
        assert (si[0].double() - s[i].double()).norm() <= 0.01 * si.double().norm()
    new = torch.randn((1, 4, D), device="cuda").bfloat16()
    cu2 = torch.tensor([0, 3, 3, 4], dtype=torch.int32, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = s.clone()
    y2 = m.decode(new, s, cu_seqlens=cu2, status=word)
    assert y2.shape == (1, 4, D) and int(word) == 0 and torch.equal(s[1], before[1])
    one = before[2:3].clone()
    y3 = m.decode(new[:, 3:].contiguous(), one)
    assert (y3.double() - y2[:, 3:].double()).norm() <= 0.01 * y3.double().norm()


def test_decode_in_a_graph():
    D, H, K, V, B = 512, 4, 128, 128, 3
    m = layer.KdaLayer.random(D, H, K, V, eight_bit=True, seed=11)
    x = torch.randn((B, 1, D), device="cuda").bfloat16()
    start = 0.1 * torch.randn((B, H, K, V), device="cuda")
    a, b = start.clone(), start.clone()
    want = [m.decode(x, a).clone() for _ in range(3)]
    m.decode(x, b.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = m.decode(x, b)
    b.copy_(start)
    for w in want:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, w)
    assert torch.equal(a, b)
