"""Host-side argument checks of the operators beside the layer: every refusal
is decided before anything is enqueued, so these run on the CPU."""
import ctypes

import pytest

from bit_post_quantization_amd import _lib

A, U = 0x10000, None  # an address that is never followed; NULL


def _lora(**kw):
    base = dict(N=100, K=64, rank=8, n_adapters=2, x_dtype=0, w_dtype=0, A=A, B=A, scales=U,
                ranks=U)
    base.update(kw)
    return _lib.QlLora(**base)


def _req(**kw):
    base = dict(n_requests=3, row_offsets=A, adapter=A)
    base.update(kw)
    return _lib.QlRequests(**base)


def _msg():
    return _lib.load().qlinear_last_error().decode()


@pytest.mark.parametrize("kw,status,frag", [
    (dict(N=0), _lib.QL_ERR_ARG, "N = 0"),
    (dict(K=8), _lib.QL_ERR_ARG, "K = 8"),
    (dict(K=72), _lib.QL_ERR_ARG, "K = 72"),
    (dict(K=65552), _lib.QL_ERR_ARG, "K = 65552"),
    (dict(rank=0), _lib.QL_ERR_ARG, "rank = 0"),
    (dict(rank=129), _lib.QL_ERR_UNSUPPORTED, "rank = 129"),
    (dict(n_adapters=0), _lib.QL_ERR_ARG, "n_adapters"),
    (dict(n_adapters=65536), _lib.QL_ERR_UNSUPPORTED, "n_adapters"),
    (dict(N=1 << 28), _lib.QL_ERR_UNSUPPORTED, "2^31"),
    (dict(x_dtype=2), _lib.QL_ERR_ARG, "x_dtype"),
    (dict(w_dtype=-1), _lib.QL_ERR_ARG, "w_dtype"),
])
def test_lora_descriptor(kw, status, frag):
    L = _lib.load()
    n = ctypes.c_int64()
    d = _lora(**kw)
    assert L.qlinear_lora_workspace(ctypes.byref(d), 16, 1, 0, 0, ctypes.byref(n)) == status
    assert frag in _msg()
    assert L.qlinear_lora(ctypes.byref(d), A, 64, 16, ctypes.byref(_req()), 0, 1.0, A, 100, A, 100,
                          U, A, 1 << 30, U) == status
    assert L.qlinear_lora_grad(ctypes.byref(d), A, 64, 16, ctypes.byref(_req()), A, A, 100, A, 64,
                               A, A, A, 1 << 30, U) == status


def test_lora_workspace_query():
    L = _lib.load()
    n = ctypes.c_int64()
    d = _lora()
    query = L.qlinear_lora_workspace
    assert query(U, 16, 1, 0, 0, ctypes.byref(n)) == _lib.QL_ERR_ARG
    assert query(ctypes.byref(d), -1, 1, 0, 0, ctypes.byref(n)) == _lib.QL_ERR_ARG
    assert query(ctypes.byref(d), 16, 0, 0, 0, ctypes.byref(n)) == _lib.QL_ERR_ARG
    assert query(ctypes.byref(d), 16, 1, 2, 0, ctypes.byref(n)) == _lib.QL_ERR_ARG
    assert query(ctypes.byref(d), 16, 1, 0, 2, ctypes.byref(n)) == _lib.QL_ERR_ARG
    assert query(ctypes.byref(d), 16, 1, 0, 0, U) == _lib.QL_ERR_ARG
    assert query(ctypes.byref(d), (1 << 23) + 1, 1, 0, 0, ctypes.byref(n)) == \
        _lib.QL_ERR_UNSUPPORTED
    for M, reqs, N, grad in ((1 << 23, 1 << 23, 100, 0), (1 << 23, 1 << 23, 100, 1),
                             (1 << 23, 1 << 16, 1 << 20, 0)):  # past the grid's limit
        assert query(ctypes.byref(_lora(N=N)), M, reqs, 0, grad, ctypes.byref(n)) == \
            _lib.QL_ERR_UNSUPPORTED
        assert "one launch" in _msg()
    for M, grad, least in ((16, 0, 0), (16, 1, 16 * 8 * 4), (1 << 20, 0, (1 << 20) * 8 * 4)):
        assert query(ctypes.byref(d), M, 1, 0, grad, ctypes.byref(n)) == _lib.QL_OK
        assert n.value >= least


def _apply(d=None, X=A, ldx=64, M=16, q="ok", cfg=0, base=A, ldb=100, Y=A + 64, ldy=100, S=U, ws=A,
           nb=1 << 30):
    d = _lora() if d is None else d
    q = _req() if q == "ok" else q
    return _lib.load().qlinear_lora(ctypes.byref(d), X, ldx, M, ctypes.byref(q) if q else U, cfg,
                                    1.0, base, ldb, Y, ldy, S, ws, nb, U)


@pytest.mark.parametrize("kw,frag", [
    (dict(q=None), "requests"),
    (dict(q=_req(row_offsets=U)), "row_offsets"),
    (dict(q=_req(adapter=U)), "row_offsets or adapter"),
    (dict(q=_req(adapter=A + 2)), "4-byte"),
    (dict(M=-1), "M = -1"),
    (dict(cfg=2), "cfg = 2"),
    (dict(cfg=1, M=15), "even"),
    (dict(X=U), "X or Y"),
    (dict(Y=U), "X or Y"),
    (dict(X=A + 2), "X is not"),
    (dict(Y=A + 2), "4-byte"),
    (dict(S=A + 1), "4-byte"),
    (dict(ldx=63), "ldx = 63"),
    (dict(ldy=99), "ldy = 99"),
    (dict(ldb=99), "ldb = 99"),
    (dict(base=A, Y=A, ldb=100, ldy=101), "another row stride"),
    (dict(M=1 << 20, ws=U), "workspace is NULL"),
    (dict(ws=A + 8), "16-byte"),
    (dict(M=1 << 20, nb=1 << 20), "workspace holds"),
    (dict(d=_lora(A=U)), "A or B"),
    (dict(d=_lora(B=U)), "A or B"),
    (dict(d=_lora(A=A + 4)), "A must be"),
    (dict(d=_lora(B=A + 2)), "B is not"),
    (dict(d=_lora(ranks=A + 1)), "4-byte"),
])
def test_lora_refusals(kw, frag):
    assert _apply(**kw) == _lib.QL_ERR_ARG
    assert frag in _msg()


def test_lora_empty_is_a_no_op():
    assert _apply(M=0, X=U, Y=U, base=U) == _lib.QL_OK


@pytest.mark.parametrize("kw,frag", [
    (dict(X=U), "X, S or dY"),
    (dict(S=U), "X, S or dY"),
    (dict(dY=U), "X, S or dY"),
    (dict(dY=A + 2), "element-aligned"),
    (dict(dX=A + 2), "element-aligned"),
    (dict(dA=A + 1), "element-aligned"),
    (dict(ldx=63), "ldx = 63"),
    (dict(lddy=99), "lddy = 99"),
    (dict(lddx=60), "lddx = 60"),
    (dict(ws=U), "workspace is NULL"),
    (dict(ws=A + 8), "16-byte"),
    (dict(nb=64), "workspace holds"),
])
def test_lora_grad_refusals(kw, frag):
    a = dict(X=A, ldx=64, M=16, S=A, dY=A, lddy=100, dX=A, lddx=64, dA=A, dB=A, ws=A, nb=1 << 30)
    a.update(kw)
    st = _lib.load().qlinear_lora_grad(
        ctypes.byref(_lora()), a["X"], a["ldx"], a["M"], ctypes.byref(_req()), a["S"], a["dY"],
        a["lddy"], a["dX"], a["lddx"], a["dA"], a["dB"], a["ws"], a["nb"], U)
    assert st == _lib.QL_ERR_ARG
    assert frag in _msg()


def _norm(**kw):
    base = dict(batch=2, positions=9, channels=24, groups=8, x_dtype=0, w_dtype=0, act=1, eps=1e-5,
                gamma=A, beta=A)
    base.update(kw)
    return _lib.QlNorm(**base)


@pytest.mark.parametrize("kw,status,frag", [
    (dict(batch=-1), _lib.QL_ERR_ARG, "batch"),
    (dict(positions=-1), _lib.QL_ERR_ARG, "positions"),
    (dict(channels=0), _lib.QL_ERR_ARG, "channels"),
    (dict(groups=7), _lib.QL_ERR_ARG, "multiple of groups"),
    (dict(batch=65536), _lib.QL_ERR_UNSUPPORTED, "batch"),
    (dict(channels=8200), _lib.QL_ERR_UNSUPPORTED, "8192"),
    (dict(channels=4098, groups=2049), _lib.QL_ERR_UNSUPPORTED, "2048"),
    (dict(positions=(1 << 30) + 1), _lib.QL_ERR_UNSUPPORTED, "positions"),
    (dict(batch=2049, channels=2048, groups=2048), _lib.QL_ERR_UNSUPPORTED, "4194304"),
    (dict(x_dtype=3), _lib.QL_ERR_ARG, "x_dtype"),
    (dict(w_dtype=3), _lib.QL_ERR_ARG, "w_dtype"),
    (dict(act=2), _lib.QL_ERR_ARG, "act"),
    (dict(eps=0.0), _lib.QL_ERR_ARG, "eps"),
    (dict(eps=float("nan")), _lib.QL_ERR_ARG, "eps"),
    (dict(gamma=A + 2), _lib.QL_ERR_ARG, "gamma"),
])
def test_norm_descriptor(kw, status, frag):
    L = _lib.load()
    n = ctypes.c_int64()
    d = ctypes.byref(_norm(**kw))
    assert L.qlinear_group_norm_workspace(d, 0, ctypes.byref(n)) == status
    assert frag in _msg()
    assert L.qlinear_group_norm(d, A, 216, 24, A, 216, 24, U, U, A, 1 << 30, U) == status
    assert L.qlinear_group_norm_grad(d, A, 216, 24, A, 216, 24, A, A, A, 216, 24, A, A, A, 1 << 30,
                                     U) == status


@pytest.mark.parametrize("kw,frag", [
    (dict(x=U), "x is NULL"),
    (dict(y=U), "y is NULL"),
    (dict(x=A + 2), "x is not"),
    (dict(xr=23), "x: row stride 23"),
    (dict(yr=23), "y: row stride 23"),
    (dict(yb=-1), "negative"),
    (dict(y=A, yr=25), "other strides"),
    (dict(mean=A + 2), "mean"),
    (dict(ws=U), "workspace is NULL"),
    (dict(nb=1), "workspace holds"),
])
def test_norm_refusals(kw, frag):
    a = dict(x=A, xb=216, xr=24, y=A + 4096, yb=216, yr=24, mean=U, rstd=U, ws=A, nb=1 << 30)
    a.update(kw)
    # positions enough that the call takes a workspace
    st = _lib.load().qlinear_group_norm(ctypes.byref(_norm(positions=100000)), a["x"], a["xb"], a["xr"], a["y"],
                                        a["yb"], a["yr"], a["mean"], a["rstd"], a["ws"], a["nb"], U)
    assert st == _lib.QL_ERR_ARG
    assert frag in _msg()


@pytest.mark.parametrize("kw,frag", [
    (dict(dy=U), "dy is NULL"),
    (dict(x=U), "x is NULL"),
    (dict(dx=U), "dx is NULL"),
    (dict(mean=U), "mean or rstd"),
    (dict(dxr=23), "dx: row stride"),
    (dict(dx=A, dxr=30), "other strides"),
    (dict(dgamma=A + 2), "dgamma"),
    (dict(nb=1), "workspace holds"),
])
def test_norm_grad_refusals(kw, frag):
    a = dict(dy=A, x=A, dx=A + 8192, dxr=24, mean=A, rstd=A, dgamma=A, dbeta=A, ws=A, nb=1 << 30)
    a.update(kw)
    st = _lib.load().qlinear_group_norm_grad(
        ctypes.byref(_norm()), a["dy"], 216, 24, a["x"], 216, 24, a["mean"], a["rstd"], a["dx"],
        216, a["dxr"], a["dgamma"], a["dbeta"], a["ws"], a["nb"], U)
    assert st == _lib.QL_ERR_ARG
    assert frag in _msg()


def test_norm_empty_is_a_no_op():
    d = _norm(positions=0)
    assert _lib.load().qlinear_group_norm(ctypes.byref(d), U, 0, 24, U, 0, 24, U, U, U, 0, U) == \
        _lib.QL_OK


def test_grad_clip_refusals():
    L = _lib.load()
    for st in (L.qlinear_grad_norm(U, 1, 1, A, U), L.qlinear_grad_norm(A, -1, 1, A, U),
               L.qlinear_grad_norm(A, 0, 1, A, U), L.qlinear_grad_norm(A, 1, -1, A, U),
               L.qlinear_grad_norm(A, 1, 1, U, U), L.qlinear_grad_norm(A + 4, 1, 1, A, U),
               L.qlinear_grad_clip(U, 1, 1, A, 1.0, A, U), L.qlinear_grad_clip(A, 1, 1, U, 1.0, A, U),
               L.qlinear_grad_clip(A, 1, 1, A, -1.0, A, U),
               L.qlinear_grad_clip(A, 1, 1, A, float("nan"), A, U),
               L.qlinear_grad_clip(A, 1, 1, A, 1.0, U, U),
               L.qlinear_grad_clip(A, 1, 1, A, 1.0, A + 2, U)):
        assert st == _lib.QL_ERR_ARG
