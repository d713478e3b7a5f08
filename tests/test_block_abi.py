"""Host-side argument checks of a conditioned block's operators: every refusal is decided
before anything is enqueued, so these run on the CPU."""
import ctypes

import pytest

from bit_post_quantization_amd import _lib

A, U = 0x10000, None  # an address that is never followed; NULL
ARG, UNSUP, OK = _lib.QL_ERR_ARG, _lib.QL_ERR_UNSUPPORTED, _lib.QL_OK
ref = ctypes.byref


def _msg():
    return _lib.load().qlinear_last_error().decode()


def _rows4(**kw):
    base = dict(N=100, K=64, group=32, x_dtype=0, s_dtype=0, act=0, packed=A, bias=U)
    base.update(kw)
    return _lib.QlRows4(**base)


def _view(p=A, batch=1 << 20, row=1 << 12, head=96):
    return _lib.QlHeadsView(p, batch, row, head)


@pytest.mark.parametrize("kw,status,frag", [
    (dict(N=0), ARG, "N = 0"),
    (dict(N=(1 << 22) + 1), UNSUP, "N = "),
    (dict(K=8), ARG, "K = 8"),
    (dict(K=72), ARG, "K = 72"),
    (dict(K=65552), ARG, "K = 65552"),
    (dict(group=48), ARG, "group"),
    (dict(x_dtype=2), ARG, "x_dtype"),
    (dict(s_dtype=-1), ARG, "s_dtype"),
    (dict(act=2), ARG, "act"),
    (dict(N=1 << 22, K=4096), UNSUP, "2^34"),
])
def test_rows4_descriptor(kw, status, frag):
    L, n, d = _lib.load(), ctypes.c_int64(), _rows4(**kw)
    assert L.qlinear_rows4_bytes(ref(d), ref(n)) == status
    assert frag in _msg()
    assert L.qlinear_rows4_workspace(ref(d), 1, ref(n)) == status
    assert L.qlinear_rows4_pack(ref(d), A, A, A, U) == status
    assert L.qlinear_rows4_quantize(ref(d), A, 0, A, U) == status
    assert L.qlinear_rows4_unpack(ref(d), A, A, U) == status
    assert L.qlinear_rows4(ref(d), A, 1 << 20, 1, A + 64, 1 << 23, A, 1 << 40, U) == status


def test_rows4_calls():
    L, n, d = _lib.load(), ctypes.c_int64(), _rows4()
    assert L.qlinear_rows4_bytes(U, ref(n)) == ARG
    assert L.qlinear_rows4_bytes(ref(d), U) == ARG
    assert L.qlinear_rows4_bytes(ref(d), ref(n)) == OK
    # 7 tiles of 16 channels by one unit of 128 inputs, 4 scales of 32 a channel
    assert n.value == 7 * 1024 + 7 * 16 * 4 * 4
    assert L.qlinear_rows4_workspace(ref(d), -1, ref(n)) == ARG
    assert L.qlinear_rows4_workspace(ref(d), (1 << 20) + 1, ref(n)) == UNSUP
    assert L.qlinear_rows4_workspace(ref(d), 4, U) == ARG
    assert L.qlinear_rows4_pack(ref(d), U, A, A, U) == ARG
    assert L.qlinear_rows4_pack(ref(d), A, U, A, U) == ARG
    assert L.qlinear_rows4_pack(ref(d), A, A, U, U) == ARG
    assert L.qlinear_rows4_pack(ref(d), A, A, A + 8, U) == ARG
    assert L.qlinear_rows4_pack(ref(d), A, A + 2, A, U) == ARG
    assert L.qlinear_rows4_quantize(ref(d), U, 0, A, U) == ARG
    assert L.qlinear_rows4_quantize(ref(d), A, 3, A, U) == ARG
    assert L.qlinear_rows4_unpack(ref(_rows4(packed=U)), A, A, U) == ARG
    assert L.qlinear_rows4_unpack(ref(d), U, U, U) == OK

    def call(d=d, X=A, ldx=64, M=3, Y=A + 64, ldy=100, ws=A, nb=1 << 30):
        return L.qlinear_rows4(ref(d), X, ldx, M, Y, ldy, ws, nb, U)

    for kw, frag in ((dict(X=U), "NULL"), (dict(Y=U), "NULL"), (dict(X=A + 2), "aligned"),
                     (dict(Y=A + 2), "aligned"), (dict(ldx=63), "ldx"), (dict(ldy=99), "ldy"),
                     (dict(M=-1), "M ="), (dict(Y=A), "Y is X"),
                     (dict(d=_rows4(packed=U)), "packed"), (dict(d=_rows4(packed=A + 4)), "packed"),
                     (dict(d=_rows4(bias=A + 1)), "bias"), (dict(ws=A + 8), "workspace")):
        assert call(**kw) == ARG, kw
        assert frag in _msg(), (kw, _msg())
    big = _rows4(N=64, K=8192)
    assert L.qlinear_rows4_workspace(ref(big), 4, ref(n)) == OK and n.value > 0
    assert call(d=big, ldx=8192, M=4, nb=n.value - 1) == ARG and "needs" in _msg()
    assert call(d=big, ldx=8192, M=4, ws=U) == ARG and "NULL" in _msg()
    assert call(M=0, X=U, Y=U) == OK


def _heads(axis_dims=(36, 36), **kw):
    base = dict(batch=2, positions=5, q_heads=2, k_heads=1, v_heads=1, dim=72, x_dtype=0, y_dtype=1,
                w_dtype=0, norm=1, eps=1e-6, gamma_q=A, gamma_k=U, n_axes=len(axis_dims), pairs=0,
                freqs=A, pos_dtype=0)
    base.update(kw)
    d = _lib.QlHeads(**base)
    for i, v in enumerate(axis_dims[:4]):
        d.axis_dims[i] = v
    return d


def _heads_calls(d, **kw):
    """Status of the forward and the backward call."""
    L = _lib.load()
    a = dict(x=A, xb=1440, xr=288, pos=A, pb=0, q=_view(A + 4096), k=_view(A + 8192),
             v=_view(A + 12288), dx=A + 64, db=1440, dr=288, gq=A + 128, gk=A + 256, ws=A, nb=1 << 30)
    a.update(kw)
    y = [None if a[n] is None else ref(a[n]) for n in "qkv"]
    f = L.qlinear_heads(ref(d), a["x"], a["xb"], a["xr"], a["pos"], a["pb"], *y, U)
    msg = _msg()
    b = L.qlinear_heads_grad(ref(d), *y, a["x"], a["xb"], a["xr"], a["pos"], a["pb"], a["dx"],
                             a["db"], a["dr"], a["gq"], a["gk"], a["ws"], a["nb"], U)
    return f, b, msg, _msg()


@pytest.mark.parametrize("kw,status,frag", [
    (dict(batch=-1), ARG, "batch"),
    (dict(positions=-1), ARG, "positions"),
    (dict(batch=1 << 12, positions=1 << 12), UNSUP, "2^24"),
    (dict(q_heads=-1), ARG, "heads"),
    (dict(q_heads=0, k_heads=0, v_heads=0), ARG, "no heads"),
    (dict(q_heads=4096), UNSUP, "4096"),
    (dict(dim=76), ARG, "dim"),
    (dict(dim=0), ARG, "dim"),
    (dict(dim=168), UNSUP, "dim"),
    (dict(x_dtype=7), ARG, "x_dtype"),
    (dict(y_dtype=7), ARG, "y_dtype"),
    (dict(w_dtype=7), ARG, "w_dtype"),
    (dict(norm=2), ARG, "norm"),
    (dict(norm=0), ARG, "without a norm"),
    (dict(eps=0.0), ARG, "eps"),
    (dict(eps=float("nan")), ARG, "eps"),
    (dict(gamma_q=A + 2), ARG, "aligned"),
    (dict(n_axes=5), ARG, "n_axes"),
    (dict(axis_dims=(36, 35)), ARG, "even"),
    (dict(axis_dims=(36, 0)), ARG, ">= 2"),
    (dict(axis_dims=(36, 38)), ARG, "add up"),
    (dict(pairs=2), ARG, "pairs"),
    (dict(pos_dtype=2), ARG, "pos_dtype"),
])
def test_heads_descriptor(kw, status, frag):
    d, n = _heads(**kw), ctypes.c_int64()
    assert _lib.load().qlinear_heads_workspace(ref(d), ref(n)) == status
    assert frag in _msg()
    assert _heads_calls(d)[:2] == (status, status)


@pytest.mark.parametrize("kw,frag", [
    (dict(x=U), "x is NULL"), (dict(x=A + 2), "x does not start"), (dict(xr=287), "x: row stride"),
    (dict(xb=-1), "negative"), (dict(pos=U), "pos"), (dict(pos=A + 2), "pos"),
    (dict(pb=-1), "pos: batch"), (dict(q=None), "q is NULL"), (dict(q=_view(U)), "q is NULL"),
    (dict(k=_view(A + 1)), "k does not start"), (dict(v=_view(row=-64)), "negative"),
])
def test_heads_arguments(kw, frag):
    f, b, mf, mb = _heads_calls(_heads(), **kw)
    assert (f, b) == (ARG, ARG) and frag in mf and frag in mb


def test_heads_outputs():
    d = _heads()
    for kw, frag in ((dict(q=_view(A + 4096, batch=0)), "rows overlap"),
                     (dict(q=_view(A + 4096, head=64)), "rows overlap"),  # 72 channels
                     (dict(q=_view(A)), "must differ"), (dict(k=_view(A + 4096)), "must differ")):
        f, _, msg, _ = _heads_calls(d, **kw)
        assert f == ARG and frag in msg, (kw, msg)
    for kw, frag in ((dict(dx=U), "dx is NULL"), (dict(dx=A), "dx must differ"),
                     (dict(dx=A + 4096), "dx must differ"), (dict(db=0), "rows overlap"),
                     (dict(dr=287), "row stride"), (dict(gq=A + 2), "aligned"),
                     (dict(gq=A + 256), "must differ"), (dict(gk=A), "must differ"),
                     (dict(ws=U), "workspace"), (dict(ws=A + 8), "workspace"),
                     (dict(nb=16), "workspace")):
        f, b, _, msg = _heads_calls(d, **kw)
        assert b == ARG and frag in msg, (kw, msg)
    none = _heads(norm=0, gamma_q=U)
    _, b, _, msg = _heads_calls(none)
    assert b == ARG and "without a norm" in msg


def test_heads_empty_batch():
    assert _heads_calls(_heads(positions=0), x=U, pos=U, q=None, k=None, v=None, gq=U, gk=U,
                        dx=U, ws=U, nb=0)[:2] == (OK, OK)


def _attn(**kw):
    base = dict(batch=2, q_len=5, k_len=7, heads=4, kv_heads=2, dim=64, dtype=1, scale=0.125,
                k_lens=U, k_mask=U, mask_batch=7)
    base.update(kw)
    return _lib.QlAttn(**base)


def _attn_calls(d, **kw):
    L = _lib.load()
    a = dict(q=_view(A), k=_view(2 * A), v=_view(3 * A), out=_view(4 * A), lse=A, dout=_view(5 * A),
             dq=_view(6 * A), dk=_view(7 * A), dv=_view(8 * A), ws=A, nb=1 << 40)
    a.update(kw)
    r = {n: None if v is None else ref(v) for n, v in a.items()
         if isinstance(v, _lib.QlHeadsView) or v is None}
    f = L.qlinear_attention(ref(d), r["q"], r["k"], r["v"], r["out"], a["lse"], a["ws"], a["nb"], U)
    msg = _msg()
    b = L.qlinear_attention_grad(ref(d), r["dout"], r["q"], r["k"], r["v"], r["out"], a["lse"],
                                 r["dq"], r["dk"], r["dv"], a["ws"], a["nb"], U)
    return f, b, msg, _msg()


@pytest.mark.parametrize("kw,status,frag", [
    (dict(batch=-1), ARG, "batch"),
    (dict(q_len=-1), ARG, "q_len"),
    (dict(k_len=-1), ARG, "k_len"),
    (dict(heads=0), ARG, "heads"),
    (dict(heads=5), ARG, "multiple"),
    (dict(kv_heads=0), ARG, "kv_heads"),
    (dict(dim=60), ARG, "dim"),
    (dict(dim=168), UNSUP, "dim"),
    (dict(dtype=2), ARG, "dtype"),
    (dict(scale=0.0), ARG, "scale"),
    (dict(scale=-1.0), ARG, "scale"),
    (dict(scale=float("inf")), ARG, "scale"),
    (dict(scale=float("nan")), ARG, "scale"),
    (dict(batch=1 << 16, q_len=1 << 16), UNSUP, "2^31"),
    (dict(batch=1 << 16, k_len=1 << 16), UNSUP, "2^31"),
    (dict(batch=1 << 23, q_len=1), UNSUP, "one launch"),
    (dict(k_lens=A + 2), ARG, "k_lens"),
    (dict(k_mask=A, mask_batch=-1), ARG, "mask_batch"),
])
def test_attention_descriptor(kw, status, frag):
    L, d, n = _lib.load(), _attn(**kw), ctypes.c_int64()
    for grad in (0, 1):
        assert L.qlinear_attention_workspace(ref(d), grad, ref(n)) == status
        assert frag in _msg()
    assert _attn_calls(d)[:2] == (status, status)


def test_attention_arguments():
    d = _attn()
    for name in ("q", "k", "v", "out"):
        for v in (None, _view(U), _view(A + 8), _view(A, row=(1 << 12) + 4), _view(A, head=-64)):
            f, b, mf, mb = _attn_calls(d, **{name: v})
            assert (f, b) == (ARG, ARG) and name in mf and name in mb
    for name in ("dout", "dq", "dk", "dv"):
        for v in (None, _view(U), _view(A + 8), _view(A, row=(1 << 12) + 4), _view(A, head=-64)):
            f, b, _, mb = _attn_calls(d, **{name: v}, nb=0, ws=U)
            assert b == ARG and name in mb
    for name in ("out", "dq", "dk", "dv"):  # rows of an output that share elements
        for v in (_view(9 * A, batch=0), _view(9 * A, row=64), _view(9 * A, head=32),
                  _view(9 * A, batch=4 << 12)):
            f, b, mf, mb = _attn_calls(d, **{name: v})
            assert "overlap" in (mf if name == "out" else mb), (name, mf, mb)
    assert _attn_calls(d, out=_view(A))[0] == ARG
    assert _attn_calls(d, out=_view(2 * A))[0] == ARG
    for kw in (dict(dq=_view(A)), dict(dk=_view(2 * A)), dict(dv=_view(4 * A)),
               dict(dk=_view(8 * A)), dict(dq=_view(7 * A)), dict(lse=U), dict(lse=A + 2),
               dict(ws=U), dict(ws=A + 8), dict(nb=0)):
        assert _attn_calls(d, **kw)[1] == ARG, kw


def test_attention_workspace():
    L, n = _lib.load(), ctypes.c_int64()
    query = L.qlinear_attention_workspace
    assert query(U, 0, ref(n)) == ARG
    assert query(ref(_attn()), 0, U) == ARG
    assert query(ref(_attn()), 2, ref(n)) == ARG
    assert query(ref(_attn()), 0, ref(n)) == OK and n.value == 0
    assert query(ref(_attn()), 1, ref(n)) == OK and n.value >= 2 * 4 * 5 * 4
    long = _attn(q_len=1, k_len=1 << 20)  # one token over a long cache: the keys are shared out
    assert query(ref(long), 0, ref(n)) == OK and n.value >= 2 * 2 * 4 * 65 * 4
    assert _attn_calls(long, nb=n.value - 1)[0] == ARG
    wide = _attn(q_len=1 << 16, k_len=64)  # few keys, many rows: so are the rows
    assert query(ref(wide), 1, ref(n)) == OK
    assert n.value >= 2 * 4 * (1 << 16) * 4 + 2 * 2 * 2 * 64 * 2 * 64 * 4


def test_attention_empty():
    nothing = dict(q=None, out=None, dout=None, dq=None, lse=U, ws=U, nb=0)
    assert _attn_calls(_attn(batch=0), k=None, v=None, dk=None, dv=None, **nothing)[:2] == (OK, OK)
    f, b, _, _ = _attn_calls(_attn(q_len=0, k_len=0), k=None, v=None, dk=None, dv=None, **nothing)
    assert (f, b) == (OK, OK)
