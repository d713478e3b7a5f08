"""What the binding of the operators beside the layer does around its C calls, on the CPU."""
from __future__ import annotations

import pytest
import torch

from bit_post_quantization_amd import _lib, ops


class _Table:
    """Stands for the device table: remembers which streams it was lent to."""

    def __init__(self):
        self.lent = []

    def data_ptr(self):
        return 0x10000

    def record_stream(self, s):
        self.lent.append(s)


@pytest.fixture
def grad_set(monkeypatch):
    """A set made on stream 7 whose C calls do nothing, and the handle of the current stream."""
    now = [7]
    monkeypatch.setattr(ops, "_device", lambda: 0)
    monkeypatch.setattr(ops, "_stream", lambda dev: now[0])
    monkeypatch.setattr(ops, "_flat", lambda t, *a: 0)
    monkeypatch.setattr(ops, "qlinear_grad_norm", lambda *a: None)
    monkeypatch.setattr(ops, "qlinear_grad_clip", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: now[0])
    s = object.__new__(ops.GradSet)
    s.grads = s.out = []
    s.units, s.device, s._made_on, s.table = 0, torch.device("cpu", 0), 7, _Table()
    return s, now


def test_grad_table_is_lent_to_the_stream_that_reads_it(grad_set):
    # else the set's end gives its memory to the stream it was made on, under a
    # kernel of another one that still reads addresses from it
    s, now = grad_set
    s.clip(1.0)
    assert s.table.lent == []
    now[0] = 9
    s.partials()
    assert s.table.lent == [9]
    now[0] = 11
    s.clip(1.0, partials=torch.zeros(_lib.QL_GRAD_PARTIALS, dtype=torch.float64))
    assert s.table.lent == [9, 11]


def test_sizes_remembered_are_bounded(monkeypatch):
    # a server's batches differ in rows and requests from call to call: what is
    # remembered of them does not grow without end
    lora = object.__new__(ops.LoraAdapters)
    lora.desc = _lib.QlLora(N=64, K=32, rank=8, n_adapters=2, x_dtype=0, w_dtype=0, A=0x1000,
                            B=0x1000)
    lora._bytes = {}
    norm = object.__new__(ops.GroupNormAct)
    norm.C = 16
    norm.desc = _lib.QlNorm(batch=0, positions=0, channels=16, groups=4, x_dtype=0, w_dtype=0, act=0,
                            eps=1e-5)
    norm._sizes = {}
    for m in range(1, 6000):
        n = lora._workspace_bytes(m, 1, 0, 1)
        assert n == lora._workspace_bytes(m, 1, 0, 1) == ops.qlinear_lora_workspace(lora.desc, m, 1, 0, 1)
        d, nb = norm._of(torch.float32, 2, m, 16, 1)
        assert d.positions == m and nb == ops.qlinear_group_norm_workspace(d, 1)
    assert len(lora._bytes) <= 4096 and len(norm._sizes) <= 4096
