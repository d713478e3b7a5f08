"""The operators of a conditioned block together, as workloads/block_step.py runs them."""
from __future__ import annotations

import math

import pytest

from tests.parity import say

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    assert _t.cuda.is_available(), "GPU tests need a ROCm device"
    import bit_post_quantization_amd  # noqa: F401  (fails loudly if the library is missing)
    return _t


def _attend(t, half, qkv, kv_text, gammas, lens):
    """The attention half's middle in 64 bits: from the linears' rows to [B, L, hidden]."""
    B, L = qkv.shape[:2]
    H, D = half.heads, half.dim
    norm = lambda x, g: x / t.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * g  # noqa: E731
    q, k, v = qkv.view(B, L, 3 * H, D).split(H, 2)
    kt, vt = kv_text.view(B, -1, 2 * H, D).split(H, 2)
    axis = D // 4 * 2
    freq = 10000.0 ** (-2.0 * t.arange(axis // 2, device="cuda", dtype=t.float64) / axis)
    angle = t.cat([half.pos[:, a:a + 1].double() * freq for a in range(2)], 1)[:, None]

    def turn(x):
        a, b = x[..., 0:2 * axis:2], x[..., 1:2 * axis:2]
        pair = t.stack([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1)
        return t.cat([pair.flatten(-2), x[..., 2 * axis:]], -1)

    q, k = turn(norm(q, gammas[0])), turn(norm(k, gammas[1]))
    k, v = t.cat([k, norm(kt, gammas[2])], 1), t.cat([v, vt], 1)
    q, k, v = (x.transpose(1, 2) for x in (q, k, v))
    s = q @ k.transpose(2, 3) * D ** -0.5
    keys = t.arange(s.shape[-1], device="cuda")
    s = s.masked_fill((keys >= lens[:, None])[:, None, None], -math.inf)
    return (t.softmax(s, -1) @ v).transpose(1, 2).reshape(B, L, H * D)


def test_block_step_against_64_bits(torch):
    """In fp32 through the whole chain: attention's output from the linears' rows, and the
    gains' gradients by differentiation of the formula. Stages: norm, turn, scores,
    weights, sum, and back; each adds at most (16 + 4 sqrt(n)) EPS of the largest value
    of its kind, n the longest sum; a factor 4 for what one stage's error grows to in
    the next."""
    from workloads.block_step import AttentionHalf, inputs
    t = torch
    half = AttentionHalf(heads=4, dim=72, grid=(6, 9), text_hidden=288, y_dtype="f32")
    half.gamma_q.copy_(t.linspace(0.5, 1.5, 72))
    half.gamma_text.fill_(1.3)
    x, c, text, lens = inputs(half, 3, 20)
    y, saved = half.forward(x, c, text, lens, save=True)
    gate, qkv, kv_text, o = saved[0], saved[1], saved[2], saved[6]
    gammas = [p.double().requires_grad_() for p in half.parameters()]
    ref = _attend(t, half, qkv.double(), kv_text.double(), gammas, lens + 54)
    tol = 6 * 4 * (16 + 4 * math.sqrt(74)) * EPS  # 74 keys are the longest sum
    mid = ref.detach()
    err = float((o.view(ref.shape).double() - mid).abs().max() / mid.abs().max())
    say(f"[block step] attention off by {err:.2e} of its largest value, allowed {tol:.2e}")
    assert err <= tol
    dy = t.randn(y.shape, generator=t.Generator(device="cuda").manual_seed(0), device="cuda")
    grads = half.backward(dy, saved)
    do = (dy.double() * gate.double()).view(-1, half.hidden) @ half.proj_deq.double()
    want = t.autograd.grad(ref, gammas, do.view(ref.shape))
    for g, w, name in zip(grads, want, ("gamma_q", "gamma_k", "gamma_text")):
        # a sum over all rows and keys of products of either sign, each off by tol of itself
        size = float(do.abs().mean()) * math.sqrt(3 * 54 * 4 * 74)
        err = float((g.double() - w).abs().max())
        say(f"  d{name} off by {err:.2e}, allowed {tol * size:.2e}, largest {float(w.abs().max()):.2e}")
        assert err <= tol * size


def test_block_step_serves_and_trains(torch):
    from workloads.block_step import serve, train
    y = serve(batch=2)
    assert y.shape == (2, 256, 1152) and bool(torch.isfinite(y).all())
    losses = train(steps=3, batch=2)
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses)


def test_block_step_text_past_its_length_does_not_count(torch):
    from workloads.block_step import AttentionHalf, inputs
    half = AttentionHalf(heads=2, dim=64, grid=(4, 4), text_hidden=128)
    x, c, text, lens = inputs(half, 3, 20)
    lens[1] = 0
    # what the quantizer's scale sees stays the same: the padding is copied from within
    a = half.forward(x, c, text, lens)
    for b in range(3):
        n = int(lens[b])
        if n < 20:
            text[b, n:] = text[b, n:].flip(0)
    assert torch.equal(half.forward(x, c, text, lens), a)
