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
