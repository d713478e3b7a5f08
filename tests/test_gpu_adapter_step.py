"""The operators together around one quantized linear (workloads/adapter_step.py)."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    assert _t.cuda.is_available(), "GPU tests need a ROCm device"
    import bit_post_quantization_amd  # noqa: F401  (fails loudly if the library is missing)
    return _t


def test_step_gradients_match_differentiation(torch):
    # The step's gradients against differentiating, in 64 bits, the norm, the
    # frozen linear as its dequantized weights, and the adapter. fp32 roundings of
    # sums over 256 rows and 160 or 96 columns: 1e-5 of a gradient's size.
    from workloads.adapter_step import AdapterLayer
    N, K, G, M = 160, 96, 8, 256
    layer = AdapterLayer(N, K, groups=G, adapters=2, rank=8)
    torch.manual_seed(0)
    layer.B.normal_(0, 0.1)
    layer.gamma.normal_(1, 0.2)
    layer.beta.normal_(0, 0.2)
    image = torch.randn(2, M // 2, K, device="cuda")
    off = torch.tensor([0, 100, 256], dtype=torch.int32, device="cuda")
    ids = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    Y, saved = layer.forward(image, off, ids, save=True)
    dY = torch.randn_like(Y)
    got = layer.backward(dY, saved, off, ids)
    p = [t.double().requires_grad_() for t in layer.parameters()]
    A, B, gamma, beta = p
    xg = image.double().view(2, M // 2, G, K // G)
    m = xg.mean((1, 3), keepdim=True)
    r = 1 / ((xg - m).square().mean((1, 3), keepdim=True) + 1e-5).sqrt()
    z = ((xg - m) * r).reshape(M, K) * gamma + beta
    x = z * torch.sigmoid(z)
    out = x @ layer.W_deq.double().t()
    parts = [2.0 * (x[:100] @ A[1].t()) @ B[1].t(), 2.0 * (x[100:] @ A[0].t()) @ B[0].t()]
    ref = torch.autograd.grad(out + torch.cat(parts), p, dY.double())
    for name, a, b in zip(("A", "B", "gamma", "beta"), got, ref):
        err = float((a.double() - b).abs().max() / b.abs().max())
        print(name, err, flush=True)
        assert err <= 1e-5, name


def test_training_lowers_the_loss(torch):
    from workloads.adapter_step import train
    losses = train(steps=12, batch=2, positions=64, N=256, K=256)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses


def test_served_requests_are_those_alone(torch):
    # rows of one request in the batch equal the request run by itself with its
    # adapter's weights added to nothing else; the bare one is the frozen layer
    from workloads.adapter_step import AdapterLayer
    layer = AdapterLayer(192, 128, groups=8, adapters=3, rank=4)
    torch.manual_seed(1)
    layer.B.normal_(0, 0.05)
    x = torch.randn(3 * 40, 128, device="cuda")
    off = torch.tensor([0, 40, 80, 120], dtype=torch.int32, device="cuda")
    base = torch.randn(120, 192, device="cuda")
    both = layer.lora.apply(x, off, torch.tensor([2, -1, 0], dtype=torch.int32, device="cuda"), base)
    assert torch.equal(both[40:80], base[40:80])
    one = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    for lo, a in ((0, 2), (80, 0)):
        alone = layer.lora.apply(x[lo:lo + 40], one, torch.tensor([a], dtype=torch.int32, device="cuda"),
                                 base[lo:lo + 40])
        assert torch.equal(alone, both[lo:lo + 40])
