"""Adapters trained and served beside one frozen quantized linear.

    python -m workloads.adapter_step [--steps N] [--rank R]

A layer of a denoiser whose weights are 8-bit codes: the channels-last image is
group-normalised (with SiLU), its positions go through the quantized linear, and
low-rank adapters add what the frozen codes cannot learn (HQ-DM explainer 2.2).

  train   one adapter on a batch: norm -> quantize -> GEMM + adapter -> loss ->
          the adapter's and the norm's gradients -> clipping by their global norm
          -> update. The frozen linear passes its gradient on through its
          dequantized weights (straight through the activation quantizer).
  serve   a guided step for several requests, each with an adapter of its own or
          none: norm -> quantize -> GEMM with the CFG combine -> their adapters.

Synthetic, seeded inputs. All operators run in the library's kernels; torch holds
the tensors, forms the loss and its dY, applies the update, and multiplies dY with
the dequantized weights.
"""
from __future__ import annotations

import argparse

import torch

from bit_post_quantization_amd import GradSet, GroupNormAct, LoraAdapters, QuantLinear

from . import device


class AdapterLayer:
    """Norm, quantized linear [K -> N] and its adapters (n of them, one stored rank)."""

    def __init__(self, N: int, K: int, groups: int = 32, adapters: int = 1, rank: int = 16,
                 seed: int = 0):
        W = device.weight_normal(torch, seed, "adapter_step/W", N, K)
        self.linear = QuantLinear(W)
        codes, scales = self.linear.weights()
        self.W_deq = codes.float() * scales[:, None]
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.A = torch.empty((adapters, rank, K), device="cuda").normal_(0, K ** -0.5, generator=g)
        self.B = torch.zeros((adapters, N, rank), device="cuda")
        self.gamma = torch.ones(K, device="cuda")
        self.beta = torch.zeros(K, device="cuda")
        self.scales = torch.full((adapters,), 2.0, device="cuda")
        self.norm = GroupNormAct(self.gamma, self.beta, groups, act="silu")
        self.lora = LoraAdapters(self.A, self.B, scales=self.scales)
        # The parameters' gradients stay where they are, so that their clipping is
        # set up once.
        self.grads = [torch.empty_like(p) for p in self.parameters()]
        self.clipping = GradSet(self.grads)

    def parameters(self):
        return [self.A, self.B, self.gamma, self.beta]

    def forward(self, image, row_offsets, adapter, cfg: int = 0, w: float = 1.0, save: bool = False):
        """image [B, L, K] -> [B * L, N] (half the rows with cfg); with ``save`` also
        what :meth:`backward` needs."""
        x, mean, rstd = self.norm.forward(image, stats=True)
        rows = x.view(-1, x.shape[-1])
        codes, s = self.linear.quantize(rows)
        base = self.linear.gemm(codes, s, cfg=cfg, w=w)
        out = self.lora.apply(rows, row_offsets, adapter, base, out=base, cfg=cfg, w=w, save=save)
        return (out[0], (image, rows, mean, rstd, out[1])) if save else out

    def backward(self, dY, saved, row_offsets, adapter):
        """Gradients of :meth:`parameters`: ``self.grads``, written anew."""
        image, rows, mean, rstd, S = saved
        dx, _, _ = self.lora.grad(rows, row_offsets, adapter, S, dY, out=self.grads[:2])
        dx.addmm_(dY, self.W_deq)  # through the frozen linear
        self.norm.grad(dx.view_as(image), image, mean, rstd, out=self.grads[2:])
        return self.grads


def train(steps: int = 20, batch: int = 4, positions: int = 256, N: int = 1152, K: int = 1152,
          rank: int = 16, lr: float = 0.1, max_norm: float = 1.0, seed: int = 0):
    """[loss of every step]: an adapter learns what another one adds to the layer."""
    layer = AdapterLayer(N, K, rank=rank, seed=seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    image = torch.empty((batch, positions, K), device="cuda").normal_(generator=g)
    off = torch.tensor([0, batch * positions], dtype=torch.int32, device="cuda")
    ids = torch.zeros(1, dtype=torch.int32, device="cuda")
    layer.B.normal_(0, 0.02, generator=g)
    target = layer.forward(image, off, ids)
    layer.B.zero_()
    losses = []
    for _ in range(steps):
        Y, saved = layer.forward(image, off, ids, save=True)
        diff = Y - target
        losses.append(float(diff.square().mean()))
        grads = layer.backward(diff * (2.0 / diff.shape[0]), saved, off, ids)
        layer.clipping.clip(max_norm)
        for p, d in zip(layer.parameters(), grads):
            p.sub_(d, alpha=lr)
    return losses


def serve(requests: int = 4, positions: int = 256, N: int = 1152, K: int = 1152, rank: int = 16,
          w: float = 4.0, seed: int = 0):
    """Guided output [requests * positions, N]; the last request runs no adapter."""
    layer = AdapterLayer(N, K, adapters=requests, rank=rank, seed=seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 2)
    layer.B.normal_(0, 0.02, generator=g)
    image = torch.empty((2 * requests, positions, K), device="cuda").normal_(generator=g)
    off = torch.arange(requests + 1, dtype=torch.int32, device="cuda") * positions
    ids = torch.arange(requests, dtype=torch.int32, device="cuda")
    ids[-1] = -1
    return layer.forward(image, off, ids, cfg=1, w=w)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--rank", type=int, default=16)
    a = ap.parse_args()
    for i, loss in enumerate(train(a.steps, rank=a.rank)):
        print(f"step {i:3d}  loss {loss:.6f}", flush=True)
    y = serve(rank=a.rank)
    print(f"guided step for 4 requests: {tuple(y.shape)}, mean square {float(y.square().mean()):.4f}")


if __name__ == "__main__":
    main()
