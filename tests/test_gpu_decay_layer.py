"""The served layer with a decay per head (layer.DecayLayer): its wiring against the formulas in 64
bits on the same weights, decoding after a prompt against one longer prompt, and a training step of
its core (rotary, decay_fwd, and back) against autograd in 64 bits."""
from __future__ import annotations

import pytest
import torch

import chunked_gated_delta_gb300 as kda
from chunked_gated_delta_gb300 import layer
from test_gpu_layer import weight

pytestmark = pytest.mark.gpu


def turned(x, pos, m):
    half = m.freqs.numel()
    angle = pos.double()[..., None, None] * m.freqs
    c, s = m.amplitude * torch.cos(angle), m.amplitude * torch.sin(angle)
    i = torch.arange(half, device=x.device)
    a, b = (2 * i, 2 * i + 1) if m.interleaved else (i, i + half)
    y = x.clone()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return y


def reference(m, x, residual, state, pos):
    """The layer in 64 bits, token by token; returns (y, state)."""
    B, T, D = x.shape
    H, K, V = m.heads, m.K, m.V
    total = x.double() + residual.double()

    def rms(t, w):
        return t / torch.sqrt(t.square().mean(-1, keepdim=True) + m.eps) * w.double()

    n = rms(total, m.norm)
    silu = torch.nn.functional.silu
    q, k, v = (silu(n @ weight(p).T).view(B, T, h, -1) for p, h in ((m.q, m.qk_heads), (m.k, m.qk_heads), (m.v, H)))
    g = m.g.double().expand(B, T, H) if torch.is_tensor(m.g) else \
        torch.nn.functional.logsigmoid(n @ weight(m.g).T + m.g.bias.double())
    q, k = (turned(t / t.norm(dim=-1, keepdim=True), pos, m).repeat_interleave(H // m.qk_heads, 2) for t in (q, k))
    S, os = state.double(), []
    for t in range(T):
        S = S * g[:, t].exp()[..., None, None] + k[:, t][..., None] * v[:, t][:, :, None]
        os.append(torch.einsum("bhkv,bhk->bhv", S, q[:, t]) * K ** -0.5)
    o = rms(torch.stack(os, 1), m.head_norm).reshape(B, T, H * V)
    if m.eight_bit:
        o = rms(o, torch.ones(H * V, device=x.device))
    return total + o @ weight(m.out).T, S


@pytest.mark.parametrize("eight_bit", [False, True])
@pytest.mark.parametrize("T", [1, 3, 150])
@pytest.mark.parametrize("kw", [dict(), dict(constant_decay=True, part=32, interleaved=True, scaling="yarn", factor=8.0)])
def test_the_formulas(eight_bit, T, kw):
    """Tolerances as of KdaLayer's test: five roundings to bf16 in a row within 2 percent, two to e4m3 within 10."""
    D, H, Hq, K, V, B = 256, 4, 2, 64, 64, 3
    m = layer.DecayLayer.random(D, H, Hq, K, V, eight_bit=eight_bit, seed=3, **kw)
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((B, T, D), generator=gen, device="cuda").bfloat16()
    r = torch.randn((B, T, D), generator=gen, device="cuda").bfloat16()
    state = 0.3 * torch.randn((B, H, K, V), generator=gen, device="cuda")
    pos = 5000 + m.prompt_positions(B, T)
    y_ref, s_ref = reference(m, x, r, state, pos)
    if T > 100:
        y, state = m.prefill(x, residual=r, h0=state, positions=pos)
    else:
        y = m.decode(x, state, pos, residual=r)
    tol = 0.10 if eight_bit else 0.02
    part, part_ref = y.double() - (x.double() + r.double()), y_ref - (x.double() + r.double())
    assert (part - part_ref).norm() <= tol * part_ref.norm() + 2.0 ** -8 * (x.double() + r.double()).norm()
    assert (state.double() - s_ref).norm() <= tol * s_ref.norm()


def test_prompt_then_tokens():
    D, H, Hq, K, V, B, T, n = 512, 4, 4, 128, 128, 2, 130, 6
    m = layer.DecayLayer.random(D, H, Hq, K, V, seed=5, part=64)
    x = torch.randn((B, T + n, D), generator=torch.Generator(device="cuda").manual_seed(9), device="cuda").bfloat16()
    y_all, s_all = m.prefill(x)
    _, s = m.prefill(x[:, :T].contiguous())
    cache = torch.full((5, H, K, V), float("nan"), device="cuda")
    slots = torch.tensor([4, 1], dtype=torch.int32, device="cuda")
    cache[4], cache[1] = s[0], s[1]
    pos = m.prompt_positions(B, T + n)
    ys = [m.decode(x[:, t:t + 1].contiguous(), cache, pos[:, t:t + 1].contiguous(), slots=slots) for t in range(T, T + 3)]
    ys.append(m.decode(x[:, T + 3:].contiguous(), cache, pos[:, T + 3:].contiguous(), slots=slots))
    y, ref = torch.cat(ys, 1).double(), y_all[:, T:].double()
    assert (y - ref).norm() <= 0.02 * ref.norm()
    assert (torch.stack([cache[4], cache[1]]).double() - s_all.double()).norm() <= 0.02 * s_all.double().norm()
    assert torch.isnan(cache[[0, 2, 3]]).all()


def test_packed_prompts():
    D, H, K, V = 256, 2, 64, 128
    m = layer.DecayLayer.random(D, H, 1, K, V, seed=7)
    lens, cu = [70, 0, 1, 129], torch.tensor([0, 70, 70, 71, 200], dtype=torch.int32, device="cuda")
    assert m.prompt_positions(1, 200, cu)[0].tolist() == [i for n in lens for i in range(n)]
    x = torch.randn((1, 200, D), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16()
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, s = m.prefill(x, cu_seqlens=cu, status=word)
    assert int(word) == 0
    for i, L in enumerate(lens):
        if L == 0:
            assert bool((s[i] == 0).all())
            continue
        a = int(cu[i])
        yi, si = m.prefill(x[:, a:a + L].contiguous())
        assert (yi.double() - y[:, a:a + L].double()).norm() <= 0.01 * yi.double().norm()
        assert (si[0].double() - s[i].double()).norm() <= 0.01 * si.double().norm()


def test_decode_in_a_graph():
    D, H, K, V, B = 512, 4, 128, 128, 3
    m = layer.DecayLayer.random(D, H, 2, K, V, eight_bit=True, seed=11)
    x = torch.randn((B, 1, D), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    pos = torch.tensor([[7], [1000], [0]], device="cuda")
    start = 0.1 * torch.randn((B, H, K, V), device="cuda")
    a, b = start.clone(), start.clone()
    want = []
    for i in range(3):
        want.append(m.decode(x, a, pos + i).clone())
    at = pos.clone()
    m.decode(x, b.clone(), at)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = m.decode(x, b, at)
    b.copy_(start)
    for i, w in enumerate(want):
        at.copy_(pos + i)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, w)
    assert torch.equal(a, b)


@pytest.mark.parametrize("hq", [4, 2])
def test_a_training_step_of_the_core(hq):
    """rotary -> decay_fwd, and decay_bwd -> rotary back, for q, k, v, g and h0. Tolerance: the 16-bit roundings of
    the turned q and k, of the scores and of the gradients, four of 2^-9 rms in a row: 1 percent."""
    B, T, H, K, V = 2, 300, 4, 64, 128
    gen = torch.Generator(device="cuda").manual_seed(1)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    unit = lambda t: (t / t.norm(dim=-1, keepdim=True)).bfloat16()  # noqa: E731
    q, k, v = unit(randn(B, T, hq, K)), unit(randn(B, T, hq, K)), randn(B, T, H, V).bfloat16()
    g, h0 = torch.nn.functional.logsigmoid(randn(B, T, H) + 2.0), 0.3 * randn(B, H, K, V)
    do, dht = randn(B, T, H, V).bfloat16(), 0.3 * randn(B, H, K, V)
    freqs, amplitude = kda.rotary_freqs(K, scaling="yarn", factor=4.0)
    pos = layer.DecayLayer.prompt_positions(B, T)
    tq, tk = kda.rotary(q, k, pos, freqs, amplitude)
    kda.decay_fwd(tq, tk, v, g, h0=h0)
    dq, dk, dv, dg, dh0 = kda.decay_bwd(tq, tk, v, g, do, h0=h0, dht=dht)
    dq, dk = kda.rotary(dq, dk, pos, freqs, amplitude, inverse=True)

    class M:
        pass
    m = M()
    m.freqs, m.amplitude, m.interleaved = freqs, amplitude, False
    leaves = [t.double().requires_grad_() for t in (q, k, v, g, h0)]
    a, b = (turned(t, pos, m).repeat_interleave(H // hq, 2) for t in leaves[:2])
    S, loss = leaves[4], 0.0
    for t in range(T):
        S = S * leaves[3][:, t].exp()[..., None, None] + b[:, t][..., None] * leaves[2][:, t][:, :, None]
        loss = loss + (torch.einsum("bhkv,bhk->bhv", S, a[:, t]) * K ** -0.5 * do[:, t].double()).sum()
    loss = loss + (S * dht.double()).sum()
    for name, got, want in zip(("dq", "dk", "dv", "dg", "dh0"), (dq, dk, dv, dg, dh0), torch.autograd.grad(loss, leaves)):
        assert (got.double() - want).norm() <= 0.01 * want.norm(), name
