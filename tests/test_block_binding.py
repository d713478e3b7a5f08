"""What the binding of a conditioned block's operators does around its C calls, on the CPU."""
from __future__ import annotations

import pytest
import torch

from bit_post_quantization_amd import QLError, _lib, block


@pytest.fixture
def on_cpu(monkeypatch):
    """CPU tensors pass for device 0's; the C calls do nothing."""
    monkeypatch.setattr(block, "_device", lambda: -1)
    monkeypatch.setattr(block, "_stream", lambda dev: 7)
    for name in ("qlinear_attention", "qlinear_attention_grad", "qlinear_rows4", "qlinear_heads",
                 "qlinear_heads_grad"):
        monkeypatch.setattr(block, name, lambda *a: None)


def _rows():
    d = object.__new__(block.GroupLinear4)
    d.N, d.K, d.group, d.s_dtype, d.bias = 64, 128, 64, torch.float32, None
    d.desc = _lib.QlRows4(N=64, K=128, group=64, x_dtype=0, s_dtype=0, act=0, packed=0x1000)
    d.packed, d._made_on, d._sizes = torch.empty(0), 7, {}
    return d


def test_sizes_remembered_are_bounded(on_cpu):
    # a server's batches differ from call to call: what is remembered does not grow without end
    rows, attn = _rows(), block.CrossAttention(2, 64)
    for m in range(1, 5000):
        attn.forward(torch.empty(1, m, 2, 64), torch.empty(1, 3, 2, 64), torch.empty(1, 3, 2, 64))
        if m < 4200:
            rows.apply(torch.empty(m, 128))
    assert len(attn._sizes) <= 4096 and len(rows._sizes) <= 4096


def test_attention_shapes(on_cpu):
    a = block.CrossAttention(4, 64, kv_heads=2)
    q, k = torch.zeros(2, 3, 4, 64), torch.zeros(2, 6, 2, 64)
    assert a.forward(q, k, k).shape == q.shape
    out, lse = a.forward(q, k, k, save=True)
    assert lse.shape == (2, 4, 3) and lse.dtype == torch.float32
    assert [t.shape for t in a.grad(q, q, k, k, out, lse)] == [q.shape, k.shape, k.shape]
    # [B, heads, L, dim] storage as it lies, and one batch entry of keys for all
    assert a.forward(q.transpose(1, 2).contiguous().transpose(1, 2), k, k).shape == q.shape
    a.forward(q, k[:1].expand(2, -1, -1, -1), k)
    for bad in (lambda: a.forward(q, k, k[:, :5]), lambda: a.forward(q, k, k.bfloat16()),
                lambda: a.forward(q[0], k[0], k[0]), lambda: a.forward(q, k[:1], k[:1]),
                lambda: a.forward(q.double(), k.double(), k.double()),
                lambda: a.forward(q, k, k, lens=torch.zeros(2)),
                lambda: a.forward(q, k, k, mask=torch.zeros(2, 6)),
                lambda: a.forward(q, k, k, mask=torch.zeros(1, 6, dtype=torch.bool).expand(2, -1)),
                lambda: a.forward(q.transpose(2, 3).contiguous().transpose(2, 3), k, k),
                lambda: a.grad(q, q, k, k, out, lse[:, :3])):
        with pytest.raises(QLError):
            bad()


def test_rows4_shapes(on_cpu):
    r = _rows()
    assert r.apply(torch.zeros(3, 128)).shape == (3, 64)
    assert r.apply(torch.zeros(0, 128)).shape == (0, 64)
    for bad in (lambda: r.apply(torch.zeros(3, 127)), lambda: r.apply(torch.zeros(3, 128).half()),
                lambda: r.apply(torch.zeros(3, 256)[:, ::2]),
                lambda: r.apply(torch.zeros(3, 128), out=torch.zeros(3, 63))):
        with pytest.raises(QLError):
            bad()
