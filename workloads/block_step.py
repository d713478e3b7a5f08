"""The attention half of a conditioned block between its frozen quantized linears.

    python -m workloads.block_step [--steps N]

A block of a text-conditioned denoiser whose linears are codes: the conditioning vector
of each image modulates the normed tokens through a 4-bit linear, the quantized qkv
linear's rows become normed, rotated queries and keys and values in one pass, the
prompt's keys and values are written behind the image's, the image's queries look at
both, and the quantized output linear's result is gated and added.

  serve   one call for a batch of images with padded prompts of unlike lengths.
  train   the gains of the head norms (what is left to learn where linears are frozen):
          forward -> loss -> gradients through attention and the head norms -> clipping by
          their global norm -> update. The frozen linears pass gradients on through
          their dequantized weights (straight through the activation quantizer).

Synthetic, seeded inputs. torch holds the tensors, norms and modulates the tokens, forms
the loss and multiplies with the dequantized weights; the rest runs in the library's
kernels.
"""
from __future__ import annotations

import argparse

import torch

from bit_post_quantization_amd import (CrossAttention, GradSet, GroupLinear4, HeadNormRope,
                                       QuantLinear)

from . import device


class AttentionHalf:
    """hidden = heads * dim channels; positions on a grid of two axes; prompts of
    ``text_hidden`` channels."""

    def __init__(self, heads: int = 16, dim: int = 72, grid=(16, 16), text_hidden: int = 1152,
                 y_dtype: str = "bf16", seed: int = 0):
        self.heads, self.dim, self.y = heads, dim, y_dtype
        n = heads * dim
        self.hidden = n

        def weight(name, rows, cols):
            return device.weight_normal(torch, seed, f"block_step/{name}", rows, cols)

        self.modulation = GroupLinear4(weight("modulation", 3 * n, n), group=128, act="silu")
        self.qkv = QuantLinear(weight("qkv", 3 * n, n))
        self.text_kv = QuantLinear(weight("text_kv", 2 * n, text_hidden))
        self.proj = QuantLinear(weight("proj", n, n), x_dtype=y_dtype)
        codes, scales = self.proj.weights()
        self.proj_deq = codes.float() * scales[:, None]
        self.gamma_q, self.gamma_k = (torch.ones(dim, device="cuda") for _ in range(2))
        self.gamma_text = torch.ones(dim, device="cuda")
        axis = dim // 4 * 2
        self.image_heads = HeadNormRope((heads, heads, heads), dim, self.gamma_q, self.gamma_k,
                                        axes=(axis, axis), y_dtype=y_dtype)
        self.text_heads = HeadNormRope((0, heads, heads), dim, gamma_k=self.gamma_text,
                                       y_dtype=y_dtype)
        self.attention = CrossAttention(heads, dim)
        h, w = grid
        self.pos = torch.stack(torch.meshgrid(torch.arange(h), torch.arange(w), indexing="ij"),
                               -1).reshape(-1, 2).to(torch.int32).cuda()
        # The gradients stay where they are, so that their clipping is set up once.
        self.grads = [torch.empty_like(p) for p in self.parameters()]
        self.clipping = GradSet(self.grads)

    def parameters(self):
        return [self.gamma_q, self.gamma_k, self.gamma_text]

    def forward(self, x, c, text, text_lens, save: bool = False):
        """x [B, L, hidden], c [B, hidden], text [B, T, text_hidden], text_lens int32 [B] ->
        [B, L, hidden]; with ``save`` also what :meth:`backward` needs."""
        B, L, n = x.shape
        T = text.shape[1]
        shift, scale, gate = self.modulation.apply(c).view(B, 1, 3 * n).split(n, 2)
        mean = x.mean(-1, keepdim=True)
        var = (x - mean).square().mean(-1, keepdim=True)
        rows = ((x - mean) * torch.rsqrt(var + 1e-6) * (1 + scale) + shift).view(B * L, n)
        qkv = self.qkv.forward(rows).view(B, L, 3 * n)
        kv_text = self.text_kv.forward(text.reshape(B * T, -1)).view(B, T, 2 * n)
        dt = {"f32": torch.float32, "bf16": torch.bfloat16}[self.y]
        q = torch.empty((B, L, self.heads, self.dim), dtype=dt, device="cuda")
        k, v = torch.empty((2, B, L + T, self.heads, self.dim), dtype=dt, device="cuda")
        self.image_heads.forward(qkv, self.pos, out=(q, k[:, :L], v[:, :L]))
        self.text_heads.forward(kv_text, out=(None, k[:, L:], v[:, L:]))
        lens = text_lens + L
        o, lse = self.attention.forward(q, k, v, lens=lens, save=True)
        y = x + gate * self.proj.forward(o.view(B * L, n)).view(B, L, n)
        return (y, (gate, qkv, kv_text, q, k, v, o, lse, lens)) if save else y

    def backward(self, dy, saved):
        """Gradients of :meth:`parameters`: ``self.grads``, written anew."""
        gate, qkv, kv_text, q, k, v, o, lse, lens = saved
        B, L, n = qkv.shape[0], qkv.shape[1], self.hidden
        do = ((dy * gate).reshape(B * L, n) @ self.proj_deq).to(o.dtype).view(o.shape)
        dq, dk, dv = self.attention.grad(do, q, k, v, o, lse, lens=lens)
        self.image_heads.grad((dq, dk[:, :L], dv[:, :L]), qkv, self.pos, out=self.grads[:2])
        self.text_heads.grad((None, dk[:, L:], dv[:, L:]), kv_text, out=(None, self.grads[2]))
        return self.grads


def inputs(half: AttentionHalf, batch: int, text_len: int, seed: int = 0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    L = half.pos.shape[0]
    x, c, text = (torch.empty(s, device="cuda").normal_(generator=g) for s in (
        (batch, L, half.hidden), (batch, half.hidden), (batch, text_len, half.text_kv.K)))
    lens = torch.tensor([text_len - (5 * b) % text_len for b in range(batch)], dtype=torch.int32,
                        device="cuda")
    return x, c, text, lens


def serve(batch: int = 8, text_len: int = 77, seed: int = 0):
    half = AttentionHalf(seed=seed)
    return half.forward(*inputs(half, batch, text_len, seed))


def train(steps: int = 10, batch: int = 4, text_len: int = 77, lr: float = 0.5,
          max_norm: float = 1.0, seed: int = 0):
    """[loss of every step]: the gains learn those of another block."""
    half = AttentionHalf(seed=seed)
    data = inputs(half, batch, text_len, seed)
    half.gamma_q.fill_(1.5)
    half.gamma_text.fill_(0.5)
    target = half.forward(*data)
    for p in half.parameters():
        p.fill_(1.0)
    losses = []
    for _ in range(steps):
        y, saved = half.forward(*data, save=True)
        diff = y - target
        losses.append(float(diff.square().sum(-1).mean()))
        grads = half.backward(diff * (2.0 / diff[..., 0].numel()), saved)
        half.clipping.clip(max_norm)
        for p, d in zip(half.parameters(), grads):
            p.sub_(d, alpha=lr)
    return losses


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    for i, loss in enumerate(train(a.steps)):
        print(f"step {i:3d}  loss {loss:.8f}", flush=True)
    y = serve()
    print(f"8 images with prompts: {tuple(y.shape)}, mean square {float(y.square().mean()):.4f}")


if __name__ == "__main__":
    main()
