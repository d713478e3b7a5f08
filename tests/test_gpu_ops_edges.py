"""The operators beside the layer where they can go wrong: sums that cancel,
values that are not finite, the forms that only large calls take, lifetimes.

Bounds as in test_gpu_ops: (16 + 4 sqrt(n)) EPS times the sum of the products'
magnitudes for a sum of n products, 2^-8 of itself for a result rounded to bf16.
"""
from __future__ import annotations

import math

import pytest

from tests.parity import say
from tests.test_gpu_ops import EPS, _dt, _round, _within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    assert _t.cuda.is_available(), "GPU tests need a ROCm device"
    import bit_post_quantization_amd  # noqa: F401  (fails loudly if the library is missing)
    return _t


# ---------------------------------------------------------------- adapters ----

@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("rank", [4, 16, 31, 64, 128])
def test_lora_gradient_sums_that_cancel(torch, x, rank):
    # Three rows a request whose products cancel up to their roundings: what is
    # left shows how many bits of dS, S and dY the sums saw. 16 bits of an operand
    # would miss the bound, which is relative to the products and not to the sum.
    from bit_post_quantization_amd import LoraAdapters
    say(f"[lora grad cancel] x {x} rank {rank}")
    g = torch.Generator(device="cuda")
    g.manual_seed(rank)
    n, N, K = 24, 1, 48

    def normal(*s):
        return torch.empty(s, device="cuda").normal_(generator=g)

    def cancelling(*s):  # [n, 3, ...]: the third row is minus the sum of the others
        v = normal(n, 2, *s)
        return torch.cat([v, -v.sum(1, keepdim=True)], 1).reshape(3 * n, *s)

    off = torch.arange(n + 1, dtype=torch.int32, device="cuda") * 3
    ids = torch.arange(n, dtype=torch.int32, device="cuda")
    A, B = normal(n, rank, K).bfloat16(), normal(n, N, rank).bfloat16()
    L = LoraAdapters(A, B, x_dtype=x)
    same = lambda *s: normal(n, 1, *s).expand(n, 3, *s).reshape(3 * n, *s)  # noqa: E731
    # dA = sum of dS^T X with dS = dY B: n = N + 3 products
    X, dY, S = same(K).to(_dt(torch, x)), cancelling(N), normal(3 * n, rank)
    _, dA, _ = L.grad(X, off, ids, S, dY)
    v = lambda t: t.double().view(n, 3, -1)  # noqa: E731
    ref = ((v(dY) @ B.double()).transpose(1, 2) @ v(X))
    mag = ((v(dY).abs() @ B.double().abs()).transpose(1, 2) @ v(X).abs())
    _within(dA, ref, (16 + 4 * math.sqrt(N + 3)) * EPS * mag + _round(torch, ref, dA.dtype), "dA")
    # dB = sum of dY^T S: n = 3 products
    N = 70
    L = LoraAdapters(A, normal(n, N, rank).bfloat16(), x_dtype=x)
    dY, S = same(N), cancelling(rank)
    _, _, dB = L.grad(X, off, ids, S, dY)
    ref = v(dY).transpose(1, 2) @ v(S)
    mag = v(dY).abs().transpose(1, 2) @ v(S).abs()
    _within(dB, ref, (16 + 4 * math.sqrt(3)) * EPS * mag + _round(torch, ref, dB.dtype), "dB")


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("rank", [3, 33, 66])
def test_lora_gradient_ranks_that_cancel(torch, x, rank):
    # dX = dS A where the ranks cancel in threes: B's third column is minus the
    # sum of the other two (exactly: their values are small whole numbers) and
    # A's three rows are one. n = N + 3 products.
    from bit_post_quantization_amd import LoraAdapters
    say(f"[lora grad cancel] dX x {x} rank {rank}")
    g = torch.Generator(device="cuda")
    g.manual_seed(rank)
    M, N, K, t = 200, 1, 48, rank // 3
    b = torch.randint(1, 60, (1, N, t, 2), generator=g, device="cuda").float()
    B = torch.cat([b, -b.sum(-1, keepdim=True)], -1).reshape(1, N, rank).bfloat16()
    A = torch.empty((1, t, 1, K), device="cuda").normal_(generator=g).expand(1, t, 3, K)
    A = A.reshape(1, rank, K).bfloat16()
    keep = torch.zeros(t, 3, dtype=torch.bool, device="cuda")
    keep[0] = True  # one triple at a time: the others' storage holds zeros
    X = torch.empty((M, K), device="cuda").normal_(generator=g).to(_dt(torch, x))
    dY = torch.empty((M, N), device="cuda").normal_(generator=g)
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    ids = torch.zeros(1, dtype=torch.int32, device="cuda")
    for k in {0, t // 2, t - 1}:
        keep.zero_()
        keep[k] = True
        Bk = B * keep.view(1, 1, rank)
        L = LoraAdapters(A, Bk, x_dtype=x)
        dX, _, _ = L.grad(X, off, ids, torch.zeros(M, rank, device="cuda"), dY)
        dS = dY.double() @ Bk[0].double()
        ref, mag = dS @ A[0].double(), dS.abs() @ A[0].double().abs()
        _within(dX, ref, (16 + 4 * math.sqrt(N + 3)) * EPS * mag + _round(torch, ref, dX.dtype),
                f"dX, ranks {3 * k}..")
