"""What a conditioned block's operators refuse or keep alive in corners of their calls, on the
CPU."""
from __future__ import annotations

import ctypes

import pytest
import torch

from bit_post_quantization_amd import QLError, _lib, block
from tests.test_block_abi import A, ARG, OK, U, _attn, _heads, _heads_calls, _msg
from tests.test_block_binding import _rows, on_cpu  # noqa: F401


def test_heads_empty_batch_keeps_its_parameters():
    """Gradients of a batch without positions are written too (zeros): over the gammas they are
    refused as in any other call."""
    d = _heads(positions=0, gamma_q=A, gamma_k=A + 512)
    none = dict(x=U, pos=U, q=None, k=None, v=None, dx=U, ws=U, nb=0)
    for gq, gk in ((A, U), (U, A + 512), (A + 512, U), (A + 1024, A + 1024)):
        _, b, _, msg = _heads_calls(d, gq=gq, gk=gk, **none)
        assert b == ARG and "must differ" in msg, (gq, gk, msg)


def test_attention_scale_past_its_base_two_form():
    """scale log2(e) is what the kernels multiply with: it has to be finite too."""
    n, L = ctypes.c_int64(), _lib.load()
    for scale, status in ((3e38, ARG), (2.4e38, ARG), (2.3e38, OK), (1e-30, OK)):
        assert L.qlinear_attention_workspace(ctypes.byref(_attn(scale=scale)), 0,
                                             ctypes.byref(n)) == status, scale
        assert status == OK or "scale" in _msg()


HUGE = (1 << 32) + 5  # as an int32: 5


def test_sizes_past_32_bits_are_refused(on_cpu):  # noqa: F811
    """Sizes reach the C ABI as 32-bit numbers: what does not fit is refused, not cut off."""
    far = lambda *s: torch.zeros(1).expand(*s)  # noqa: E731
    a = block.CrossAttention(1, 8)
    h = block.HeadNormRope((1, 0, 0), 8, norm="none")
    r = _rows()
    small = torch.zeros(1, 3, 1, 8)
    for call in (lambda: r.apply(far(HUGE, 128)),
                 lambda: h.forward(far(1, HUGE, 8)),
                 lambda: h.forward(far(HUGE, 1, 8)),
                 lambda: a.forward(far(1, HUGE, 1, 8), small, small),
                 lambda: a.forward(small, far(1, HUGE, 1, 8), far(1, HUGE, 1, 8)),
                 lambda: a.forward(far(HUGE, 1, 1, 8), far(HUGE, 1, 1, 8), far(HUGE, 1, 1, 8)),
                 lambda: block.CrossAttention(HUGE, 8),
                 lambda: block.CrossAttention(1, (1 << 32) + 8),
                 lambda: block.HeadNormRope((HUGE, 0, 0), 8),
                 lambda: block.HeadNormRope((1, 0, 0), (1 << 32) + 8),
                 lambda: block.HeadNormRope((1, 0, 0), 8, axes=((1 << 32) + 2,)),
                 lambda: block.GroupLinear4(far(HUGE, 32)),
                 lambda: block.GroupLinear4.from_codes(far(HUGE, 32), small, 32),
                 lambda: block.CrossAttention(4 - (1 << 32), 8)):
        with pytest.raises(QLError) as e:
            call()
        assert "2^31" in str(e.value), e.value


class _Kept:
    """A tensor's place: which streams were told of it."""

    def __init__(self):
        self.on = []

    def record_stream(self, stream):
        self.on.append(stream)

    def get_device(self):
        return -1

    def data_ptr(self):
        return 0x1000


def test_what_a_layer_holds_outlives_it_on_other_streams(on_cpu, monkeypatch):  # noqa: F811
    """Kernels on another stream than the layer's read its packed weights and bias, or its
    frequencies and gammas: all of them are recorded there, and nothing on its own stream."""
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: "side")
    r = _rows()
    r.packed, r.bias = _Kept(), _Kept()
    r.apply(torch.zeros(2, 128))
    assert r.packed.on == [] and r.bias.on == []
    r._made_on = 8
    r.apply(torch.zeros(2, 128))
    assert r.packed.on == ["side"] and r.bias.on == ["side"]
    h = block.HeadNormRope((1, 1, 0), 8)
    h.gamma_q, h.gamma_k = _Kept(), _Kept()
    x = torch.zeros(1, 2, 16)
    h.forward(x)
    assert h.gamma_q.on == [] and h.gamma_k.on == []
    h._made_on = 8
    h.forward(x)
    assert h.gamma_q.on == ["side"] and h.gamma_k.on == ["side"]
    h.gamma_q = None  # 1
    h.forward(x)
    assert h.gamma_k.on == ["side", "side"]


def test_missing_arguments_are_refused(on_cpu, monkeypatch):  # noqa: F811
    """A tensor that is not there, or a size of 0, raises what other arguments that do not fit
    raise."""
    a, x = block.CrossAttention(2, 64), torch.zeros(1, 3, 2, 64)
    h, rows = block.HeadNormRope((1, 1, 0), 8, norm="none"), torch.zeros(1, 2, 16)
    lse, part = torch.zeros(1, 2, 3), torch.zeros(1, 2, 1, 8, dtype=torch.bfloat16)
    codes = torch.zeros(4, 32, dtype=torch.int8)
    for call in (lambda: a.forward(x, x, None), lambda: a.forward(x, None, x),
                 lambda: a.forward(None, x, x), lambda: a.grad(None, x, x, x, x, lse),
                 lambda: a.grad(x, x, x, x, x, None),
                 lambda: a.grad(x, x, x, x, x, lse, into=(x, None, x)),
                 lambda: a.forward(x, x, x, lens=3), lambda: a.forward(x, x, x, mask=[True] * 3),
                 lambda: h.forward(None), lambda: h.forward(rows, out=(part, None, None)),
                 lambda: h.grad((part, None, None), rows), lambda: _rows().apply(None),
                 lambda: block.CrossAttention(2, 0), lambda: block.CrossAttention(2, -8),
                 lambda: block.GroupLinear4.from_codes(codes, None, 32)):
        with pytest.raises(QLError):
            call()
