"""More host-side argument checks of the operators beside the layer, on the CPU: as in
test_ops_abi, every refusal is decided before anything is enqueued. (No call here may
be one that is accepted: its addresses lead nowhere.)"""
import ctypes

import pytest

from bit_post_quantization_amd import _lib
from tests.test_ops_abi import A, U, _lora, _msg, _norm, _req


def _overlap(batch, positions, channels, yb, yr):
    at = [b * yb + r * yr + c for b in range(batch) for r in range(positions)
          for c in range(channels)]
    return len(set(at)) < len(at)


@pytest.mark.parametrize("batch,positions,channels,yb,yr", [
    (2, 9, 4, 0, 4),     # an expanded tensor
    (2, 1, 4, 3, 4),     # one position an image
    (3, 9, 4, 35, 4),    # the last position of an image is the next one's first
    (2, 5, 4, 7, 8),     # a row of one image reaches into a row of the other
    (5, 4, 4, 6, 25),    # an image's rows leave room for four others, not for five
    (4, 7, 2, 3, 8),     # only the fourth image meets the first one's next row but one
])
def test_norm_refuses_overlapping_images_of_an_output(batch, positions, channels, yb, yr):
    assert _overlap(batch, positions, channels, yb, yr)
    L = _lib.load()
    d = ctypes.byref(_norm(batch=batch, positions=positions, channels=channels, groups=1))
    xb = positions * channels
    st = L.qlinear_group_norm(d, A, xb, channels, 2 * A, yb, yr, U, U, A, 1 << 30, U)
    assert st == _lib.QL_ERR_ARG and "y: images overlap" in _msg()
    st = L.qlinear_group_norm_grad(d, A, xb, channels, A, xb, channels, A, A, 2 * A, yb, yr, A, A,
                                   A, 1 << 30, U)
    assert st == _lib.QL_ERR_ARG and "dx: images overlap" in _msg()


@pytest.mark.parametrize("N", [(1 << 31) - 1, (1 << 31) - 600, (1 << 31) - 65792])
def test_lora_gradient_counts_the_chunks_of_n(N):
    # a grid (and, at the end, 32-bit column numbers) that wide outputs alone pass
    L = _lib.load()
    n = ctypes.c_int64()
    d = ctypes.byref(_lora(N=N, rank=1))
    assert L.qlinear_lora_workspace(d, 1, 1, 0, 1, ctypes.byref(n)) == _lib.QL_ERR_UNSUPPORTED
    assert "one launch" in _msg()
    assert L.qlinear_lora_grad(d, A, 64, 1, ctypes.byref(_req()), A, A, N, A, 64, A, A, A, 1 << 62,
                               U) == _lib.QL_ERR_UNSUPPORTED
    # the largest that stays below it
    d = ctypes.byref(_lora(N=(1 << 31) - 66560, rank=1))
    assert L.qlinear_lora_workspace(d, 1, 1, 0, 1, ctypes.byref(n)) == _lib.QL_OK


def test_lora_requests_may_be_none_without_rows():
    L = _lib.load()
    n = ctypes.c_int64()
    d = ctypes.byref(_lora())
    for grad in (0, 1):
        assert L.qlinear_lora_workspace(d, 0, 0, 0, grad, ctypes.byref(n)) == _lib.QL_OK
        assert L.qlinear_lora_workspace(d, 1, 0, 0, grad, ctypes.byref(n)) == _lib.QL_ERR_ARG
        assert L.qlinear_lora_workspace(d, 0, -1, 0, grad, ctypes.byref(n)) == _lib.QL_ERR_ARG
    q = ctypes.byref(_req(n_requests=0, row_offsets=U, adapter=U))
    assert L.qlinear_lora(d, U, 64, 0, q, 0, 1.0, U, 100, U, 100, U, U, 0, U) == _lib.QL_OK
    assert L.qlinear_lora(d, A, 64, 1, ctypes.byref(_req(n_requests=0)), 0, 1.0, A, 100, A + 64, 100,
                          U, A, 1 << 30, U) == _lib.QL_ERR_ARG


def test_gradients_of_parameters_must_differ():
    # given tensors: one for both, or the parameter itself, would be a silent race
    L = _lib.load()
    q = ctypes.byref(_req())
    for dX, dA, dB in ((A, 2 * A, 2 * A), (A, A, 2 * A), (A, 2 * A, A), (U, A, A)):
        assert L.qlinear_lora_grad(ctypes.byref(_lora()), 4 * A, 64, 16, q, A, A, 100, dX, 64, dA, dB, A,
                                   1 << 30, U) == _lib.QL_ERR_ARG
        assert "must differ" in _msg()
    for dg, db in ((3 * A, 3 * A), (A, 3 * A), (3 * A, 2 * A), (U, A), (2 * A, U)):
        d = ctypes.byref(_norm(gamma=A, beta=2 * A))
        assert L.qlinear_group_norm_grad(d, 5 * A, 216, 24, 6 * A, 216, 24, A, A, 7 * A, 216, 24, dg, db,
                                         A, 1 << 30, U) == _lib.QL_ERR_ARG
        assert "must differ" in _msg()
