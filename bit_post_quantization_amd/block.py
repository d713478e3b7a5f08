"""Operators of a conditioned transformer block: the C ABI function for function
(same names), and a small class for each that checks tensors and allocates outputs.

  GroupLinear4    few rows against 4-bit weights with a scale for each group of inputs
  HeadNormRope    norms of queries and keys for each head and their rotation by
                  positions of several axes, in one pass
  CrossAttention  attention to the states of another sequence

The rules of the operators beside the layer (ops.py) hold for these too: tensors are on
the current device, calls are asynchronous on the current stream or on ``stream``,
arguments that do not fit raise QLError before anything is enqueued, and autograd sees
none of the calls: gradients are the classes' ``grad`` methods.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence

import torch

from . import _lib
from ._lib import QL_ERR_ARG, QlAttn, QLError, QlHeads, QlHeadsView, QlRows4, check
from .ops import (_ACTS, _DT, _F32, _F64, _I32, _L, _NAMES, _byref, _device, _flat, _need, _on,
                  _ptr, _refuse, _remember, _rows, _stream)

_NORMS = {"none": _lib.QL_HEADS_NONE, "rms": _lib.QL_HEADS_RMS}
_PAIRS = {"adjacent": _lib.QL_PAIRS_ADJACENT, "halves": _lib.QL_PAIRS_HALVES}
_POS = {torch.int32: _lib.QL_POS_I32, torch.float32: _lib.QL_POS_F32}


# ------------------------------------------------------- C ABI, same names ----
# Pointers are addresses (int or None); views are QlHeadsView or None; stream is
# a raw handle.

def qlinear_rows4_bytes(desc: QlRows4) -> int:
    n = ctypes.c_int64()
    check(_L.qlinear_rows4_bytes(_byref(desc), _byref(n)))
    return n.value


def qlinear_rows4_pack(desc: QlRows4, codes, scales, packed, stream) -> None:
    check(_L.qlinear_rows4_pack(_byref(desc), codes, scales, packed, stream))


def qlinear_rows4_quantize(desc: QlRows4, W, w_dtype: int, packed, stream) -> None:
    check(_L.qlinear_rows4_quantize(_byref(desc), W, w_dtype, packed, stream))


def qlinear_rows4_unpack(desc: QlRows4, codes, scales, stream) -> None:
    check(_L.qlinear_rows4_unpack(_byref(desc), codes, scales, stream))


def qlinear_rows4_workspace(desc: QlRows4, M: int) -> int:
    n = ctypes.c_int64()
    check(_L.qlinear_rows4_workspace(_byref(desc), M, _byref(n)))
    return n.value


def qlinear_rows4(desc: QlRows4, X, ldx, M, Y, ldy, workspace, workspace_bytes, stream) -> None:
    check(_L.qlinear_rows4(_byref(desc), X, ldx, M, Y, ldy, workspace, workspace_bytes, stream))


def qlinear_heads_workspace(desc: QlHeads) -> int:
    n = ctypes.c_int64()
    check(_L.qlinear_heads_workspace(_byref(desc), _byref(n)))
    return n.value


def _ref(view: Optional[QlHeadsView]):
    return None if view is None else _byref(view)


def qlinear_heads(desc: QlHeads, x, x_batch, x_row, pos, pos_batch, q, k, v, stream) -> None:
    check(_L.qlinear_heads(_byref(desc), x, x_batch, x_row, pos, pos_batch, _ref(q), _ref(k),
                           _ref(v), stream))


def qlinear_heads_grad(desc: QlHeads, dq, dk, dv, x, x_batch, x_row, pos, pos_batch, dx, dx_batch,
                       dx_row, dgamma_q, dgamma_k, workspace, workspace_bytes, stream) -> None:
    check(_L.qlinear_heads_grad(_byref(desc), _ref(dq), _ref(dk), _ref(dv), x, x_batch, x_row, pos,
                                pos_batch, dx, dx_batch, dx_row, dgamma_q, dgamma_k, workspace,
                                workspace_bytes, stream))


def qlinear_attention_workspace(desc: QlAttn, grad: int = 0) -> int:
    n = ctypes.c_int64()
    check(_L.qlinear_attention_workspace(_byref(desc), grad, _byref(n)))
    return n.value


def qlinear_attention(desc: QlAttn, q, k, v, out, lse, workspace, workspace_bytes, stream) -> None:
    check(_L.qlinear_attention(_byref(desc), _byref(q), _byref(k), _byref(v), _byref(out), lse,
                               workspace, workspace_bytes, stream))


def qlinear_attention_grad(desc: QlAttn, dout, q, k, v, out, lse, dq, dk, dv, workspace,
                           workspace_bytes, stream) -> None:
    check(_L.qlinear_attention_grad(_byref(desc), _byref(dout), _byref(q), _byref(k), _byref(v),
                                    _byref(out), lse, _byref(dq), _byref(dk), _byref(dv),
                                    workspace, workspace_bytes, stream))


def _keep(dev: int, *tensors) -> None:
    """Memory of tensors (None: no matter) goes to no other use before the current stream is
    done with it."""
    stream = torch.cuda.current_stream(dev)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _fit(*sizes: int) -> None:
    """Sizes go to the C ABI as 32-bit numbers, which ctypes would cut off."""
    for n in sizes:
        if not -(1 << 31) <= n < 1 << 31:
            raise QLError(QL_ERR_ARG, f"size {n}: less than 2^31")


def _there(t, name: str) -> None:
    if not isinstance(t, torch.Tensor):
        raise QLError(QL_ERR_ARG, f"{name} is not a tensor")


# ----------------------------------------------------------------- 4-bit rows ----

class GroupLinear4:
    """A linear [K -> N] with 4-bit weight codes and a scale for each ``group`` (32, 64 or
    128) of input channels, meant for few rows: the modulation of a block by one
    conditioning vector an image. ``act`` ("none" or "silu") is applied to the input;
    ``bias`` f32 [N] is used where it is.

    From weights W [N, K] (f32 or bf16) by the groups' largest values (scales of
    ``s_dtype``), or from codes that are there (:meth:`from_codes`). The packed weights are
    made once, on the current stream, which the constructor waits for; keep the layer
    while a captured graph with its calls is replayed."""

    def __init__(self, W, group: int = 128, bias=None, act: str = "none", s_dtype: str = "f32",
                 stream=None):
        _need(isinstance(W, torch.Tensor) and W.dim() == 2, "W must be [N, K]")
        _fit(*W.shape, group)
        _need(W.dtype in _DT, f"W is {W.dtype}: f32 or bf16 only")
        _need(s_dtype in _NAMES, f"s_dtype {s_dtype!r} is not one of {sorted(_NAMES)}")
        w = _flat(W, "W", _device(), W.dtype, W.shape)
        self._make(W.shape, group, bias, act, _NAMES[s_dtype], stream, W.device,
                   lambda s: qlinear_rows4_quantize(self.desc, w, _DT[W.dtype], self.desc.packed, s))

    @classmethod
    def from_codes(cls, codes, scales, group: int, bias=None, act: str = "none", stream=None):
        """From codes int8 [N, K] in [-8, 7] and scales [N, ceil(K / group)], f32 or bf16."""
        self = cls.__new__(cls)
        _need(isinstance(codes, torch.Tensor) and codes.dim() == 2, "codes must be [N, K]")
        _fit(*codes.shape)
        _need(group in (32, 64, 128), f"group = {group} must be 32, 64 or 128")
        _there(scales, "scales")
        _need(scales.dtype in _DT, f"scales is {scales.dtype}: f32 or bf16 only")
        dev, (N, K) = _device(), codes.shape
        c = _flat(codes, "codes", dev, torch.int8, codes.shape)
        s = _flat(scales, "scales", dev, scales.dtype, (N, -(-K // group)))
        self._make(codes.shape, group, bias, act, scales.dtype, stream, codes.device,
                   lambda stream: qlinear_rows4_pack(self.desc, c, s, self.desc.packed, stream))
        return self

    def _make(self, shape, group, bias, act, s_dtype, stream, device, fill):
        if stream is not None:
            with _on(stream):
                return self._make(shape, group, bias, act, s_dtype, None, device, fill)
        _need(act in _ACTS, f"act {act!r} is not one of {sorted(_ACTS)}")
        self.N, self.K = shape
        self.group, self.s_dtype, self.bias = group, s_dtype, bias
        if bias is not None:
            _flat(bias, "bias", _device(), _F32, (self.N,))
        self.desc = QlRows4(N=self.N, K=self.K, group=group, x_dtype=_lib.QL_F32,
                            s_dtype=_DT[s_dtype], act=_ACTS[act], packed=None, bias=_ptr(bias))
        self.packed = torch.empty(qlinear_rows4_bytes(self.desc), dtype=torch.uint8, device=device)
        self.desc.packed = self.packed.data_ptr()
        self._made_on = _stream(_device())
        fill(self._made_on)
        torch.cuda.current_stream().synchronize()  # other streams may use the layer at once
        self._sizes = {}  # descriptor and workspace bytes by type and rows of a call

    def _ready(self, dev: int) -> int:
        """The current stream's handle, on which the packed weights and the bias may be read from
        now on."""
        _need(dev == self.packed.get_device(), "the layer's weights are not on the current device")
        s = _stream(dev)
        if s != self._made_on:  # their memory outlives the layer until this stream is done
            _keep(dev, self.packed, self.bias)
        return s

    def apply(self, X, out=None, stream=None):
        """act(X) W^T + bias, f32 [M, N], from X [M, K] (f32 or bf16)."""
        if stream is not None:
            with _on(stream):
                return self.apply(X, out)
        _there(X, "X")
        _need(X.dim() == 2, f"X must be [M, {self.K}]")
        dev, M, dt = _device(), X.shape[0], X.dtype
        size = self._sizes.get((dt, M))
        if size is None:
            _need(dt in _DT, f"X is {dt}: f32 or bf16 only")
            _fit(M)
            d = QlRows4.from_buffer_copy(self.desc)
            d.x_dtype = _DT[dt]
            size = _remember(self._sizes, (dt, M), (d, qlinear_rows4_workspace(d, M)))
        d, nb = size
        ldx = _rows(X, "X", dev, dt, (M, self.K))
        s = self._ready(dev)
        if out is None:
            out, ldy = torch.empty((M, self.N), dtype=_F32, device=X.device), self.N
        else:
            ldy = _rows(out, "out", dev, _F32, (M, self.N))
        ws = torch.empty(nb, dtype=torch.uint8, device=X.device) if nb else None
        qlinear_rows4(d, X.data_ptr(), ldx, M, out.data_ptr(), ldy, _ptr(ws), nb, s)
        return out

    def weights(self, stream=None):
        """(codes int8 [N, K], scales [N, ceil(K / group)])."""
        if stream is not None:
            with _on(stream):
                return self.weights()
        s = self._ready(_device())
        codes = torch.empty((self.N, self.K), dtype=torch.int8, device=self.packed.device)
        scales = torch.empty((self.N, -(-self.K // self.group)), dtype=self.s_dtype,
                             device=self.packed.device)
        qlinear_rows4_unpack(self.desc, codes.data_ptr(), scales.data_ptr(), s)
        return codes, scales


# --------------------------------------------------------------- norms, turns ----

def _view(t, name: str, dev: int, dtype, shape, dense) -> QlHeadsView:
    """A [B, L, H, D] tensor, whose channels are contiguous, as the C ABI takes it; `dense`
    are the strides of a packed one."""
    _there(t, name)
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape:
        _refuse(t, name, dev, dtype, shape)
    if t.is_contiguous():
        return QlHeadsView(t.data_ptr(), *dense)
    sb, sl, sh, sd = t.stride()
    _need(sd == 1, f"{name}: channels are not contiguous")
    return QlHeadsView(t.data_ptr(), sb, sl, sh)


class HeadNormRope:
    """What stands between a qkv linear and attention: queries and keys normed for
    each head and rotated by their positions, values converted, in one pass.

    ``heads`` = (query, key, value heads) of ``dim`` channels side by side in a row of the
    input (any may be 0: queries alone, or an encoder's keys and values). ``norm`` "rms"
    (x / sqrt(mean of squares + eps) * gamma; gammas [dim], f32 or bf16, may be None for 1)
    or "none". ``axes``: channels of a head that turn with each axis of the positions, in
    order; the rest do not turn. Pair i of an axis of d channels turns by position *
    theta ** (-2 i / d), or by ``freqs`` (a sequence, radians for one unit of position,
    all axes' pairs in order); its members are ``pairs`` "adjacent" (2 i, 2 i + 1) or
    "halves" (i, d / 2 + i). Outputs are of ``y_dtype``. Keep the layer while a captured
    graph with its calls is replayed (it holds the table of frequencies)."""

    def __init__(self, heads: Sequence[int], dim: int, gamma_q=None, gamma_k=None,
                 norm: str = "rms", axes: Sequence[int] = (), pairs: str = "adjacent",
                 theta: float = 10000.0, freqs: Optional[Sequence[float]] = None,
                 eps: float = 1e-6, y_dtype: str = "bf16"):
        _need(norm in _NORMS, f"norm {norm!r} is not one of {sorted(_NORMS)}")
        _need(pairs in _PAIRS, f"pairs {pairs!r} is not one of {sorted(_PAIRS)}")
        _need(y_dtype in _NAMES, f"y_dtype {y_dtype!r} is not one of {sorted(_NAMES)}")
        _need(len(heads) == 3, "heads must be (query, key, value heads)")
        _need(len(axes) <= _lib.QL_MAX_AXES, f"at most {_lib.QL_MAX_AXES} axes")
        _fit(dim, *heads, *axes)
        given = [t for t in (gamma_q, gamma_k) if t is not None]
        w = given[0].dtype if given else _F32
        _need(w in _DT, f"gamma_q is {w}: f32 or bf16 only")
        dev = _device()
        for t, name in ((gamma_q, "gamma_q"), (gamma_k, "gamma_k")):
            if t is not None:
                _flat(t, name, dev, w, (dim,))
        self.heads, self.dim, self.axes = tuple(int(h) for h in heads), dim, tuple(axes)
        self.gamma_q, self.gamma_k, self.y_dtype = gamma_q, gamma_k, _NAMES[y_dtype]
        self.desc = QlHeads(batch=0, positions=0, q_heads=self.heads[0], k_heads=self.heads[1],
                            v_heads=self.heads[2], dim=dim, x_dtype=_lib.QL_F32,
                            y_dtype=_DT[self.y_dtype], w_dtype=_DT[w], norm=_NORMS[norm], eps=eps,
                            gamma_q=_ptr(gamma_q), gamma_k=_ptr(gamma_k), n_axes=len(axes),
                            pairs=_PAIRS[pairs], freqs=None, pos_dtype=_lib.QL_POS_I32)
        for i, d in enumerate(axes):
            self.desc.axis_dims[i] = d
        qlinear_heads_workspace(self.desc)  # its checks
        if freqs is None:
            freqs = [theta ** (-2.0 * i / d) for d in axes for i in range(d // 2)]
        _need(len(freqs) == sum(axes) // 2, "freqs must list one value for each pair that turns")
        self.freqs = torch.tensor([f / (2.0 * math.pi) for f in freqs], dtype=_F64,
                                  device=torch.device("cuda", dev)) if axes else None
        self.desc.freqs = _ptr(self.freqs)
        self._dev, self._made_on = dev, _stream(dev)
        self._alike = self.heads[0] == self.heads[1] == self.heads[2]
        self._sizes = {}  # what :meth:`_size` makes, by size of call

    def _call(self, x, pos):
        """(device, stream, size, x's batch and row stride, positions' address and batch
        stride) of a call; a size is (descriptor, workspace bytes, shapes of q, k and v,
        their dense strides)."""
        _there(x, "x")
        dev, dt, shape = _device(), x.dtype, x.shape
        if x.get_device() != dev or dev != self._dev:
            _need(dev == self._dev, "the layer was made on another device")
            _refuse(x, "x", dev, dt, shape)
        kind, own = None, False
        if self.axes:
            _need(isinstance(pos, torch.Tensor) and pos.dtype in _POS,
                  "pos must be an int32 or f32 tensor")
            kind, own = pos.dtype, pos.dim() == 3
        size = self._sizes.get((dt, shape, kind))
        if size is None:
            size = self._size(dt, shape, kind)
        n = shape[2]
        if x.is_contiguous():
            xb, xr = shape[1] * n, n
        else:
            xb, xr, xc = x.stride()
            _need(xc == 1 or n == 1, "x: channels are not contiguous")
        at, pb = None, 0
        if kind is not None:
            want = (shape[1], len(self.axes))
            at = _flat(pos, "pos", dev, kind, (shape[0], *want) if own else want)
            pb = want[0] * want[1] if own else 0
        s = _stream(dev)
        if s != self._made_on:  # what the layer holds outlives it until this stream is done
            _keep(dev, self.freqs, self.gamma_q, self.gamma_k)
        return dev, s, size, xb, xr, at, pb

    def _size(self, dt, shape, kind):
        _need(dt in _DT, f"x is {dt}: f32 or bf16 only")
        n = sum(self.heads) * self.dim
        _need(len(shape) == 3 and shape[2] == n, f"x is {tuple(shape)}, not [B, L, {n}]")
        _fit(*shape)
        d = QlHeads.from_buffer_copy(self.desc)
        d.batch, d.positions, d.x_dtype = shape[0], shape[1], _DT[dt]
        d.pos_dtype = _lib.QL_POS_I32 if kind is None else _POS[kind]
        parts = [(shape[0], shape[1], h, self.dim) if h else None for h in self.heads]
        dense = [(shape[1] * h * self.dim, h * self.dim, self.dim) for h in self.heads]
        return _remember(self._sizes, (dt, shape, kind),
                         (d, qlinear_heads_workspace(d), parts, dense))

    def _views(self, tensors, names, dev, size):
        """Views of a triple as the C ABI takes them, None for a part without heads."""
        return [None if shape is None else _view(t, name, dev, self.y_dtype, shape, strides)
                for t, name, shape, strides in zip(tensors, names, size[2], size[3])]

    def forward(self, x, pos=None, out=None, stream=None):
        """(q, k, v) from x [B, L, heads * dim] (f32 or bf16): [B, L, heads, dim] each, None
        for a part without heads; written into the triple ``out`` where it is given
        (any strides with contiguous channels, so a longer sequence's slice will do).
        ``pos`` int32 or f32 [L, axes], or [B, L, axes]."""
        if stream is not None:
            with _on(stream):
                return self.forward(x, pos, out)
        dev, s, size, xb, xr, at, pb = self._call(x, pos)
        if out is None:
            if self._alike:  # one allocation for all three: an allocation takes the host 1 us
                out = torch.empty((3, *size[2][0]), dtype=self.y_dtype, device=x.device).unbind(0)
            else:
                out = [None if shape is None else
                       torch.empty(shape, dtype=self.y_dtype, device=x.device) for shape in size[2]]
            views = [None if t is None else QlHeadsView(t.data_ptr(), *dense)
                     for t, dense in zip(out, size[3])]
        else:
            out = [None if shape is None else t for t, shape in zip(out, size[2])]
            views = self._views(out, ("q", "k", "v"), dev, size)
        qlinear_heads(size[0], x.data_ptr(), xb, xr, at, pb, *views, s)
        return tuple(out)

    def grad(self, dy, x, pos=None, out=None, stream=None):
        """(dx, dgamma_q, dgamma_k) for dy = (dq, dk, dv) of :meth:`forward` (None for a
        part without heads); the last two in the gammas' type, None where the gamma is,
        written into the pair ``out`` where it is given."""
        if stream is not None:
            with _on(stream):
                return self.grad(dy, x, pos, out)
        dev, s, size, xb, xr, at, pb = self._call(x, pos)
        d, nb = size[:2]
        _, L, n = x.shape
        views = self._views(dy, ("dq", "dk", "dv"), dev, size)
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        gammas = (self.gamma_q, self.gamma_k)
        if out is None:
            out = [None if g is None else torch.empty_like(g) for g in gammas]
        else:
            for t, g, name in zip(out, gammas, ("dgamma_q", "dgamma_k")):
                _need((t is None) == (g is None), f"{name} is given without its parameter, or not")
                if t is not None:
                    _flat(t, name, dev, g.dtype, g.shape)
        ws = torch.empty(nb, dtype=torch.uint8, device=x.device) if nb else None
        qlinear_heads_grad(d, *views, x.data_ptr(), xb, xr, at, pb, dx.data_ptr(), L * n, n,
                           _ptr(out[0]), _ptr(out[1]), _ptr(ws), nb, s)
        return dx, out[0], out[1]


# ------------------------------------------------------------------ attention ----

class CrossAttention:
    """Attention of ``heads`` query heads of ``dim`` channels to the states of another
    sequence (or of the same one), whose ``kv_heads`` heads are shared by neighbouring
    query heads. Tensors are [B, L, heads, dim], f32 or bf16, with any strides that are
    multiples of 16 bytes (so [B, heads, L, dim] is taken transposed) and contiguous
    channels; ``scale`` defaults to dim ** -0.5.

    ``lens`` int32 [B] says how many keys of each batch entry count, ``mask`` bool (or
    uint8) [B, k_len] which ones; with both, those that both name. Others take no
    part, whatever they hold. A query without any key that counts gets 0, one whose keys
    count and all score -infinity NaN."""

    def __init__(self, heads: int, dim: int, kv_heads: Optional[int] = None,
                 scale: Optional[float] = None):
        self.heads, self.dim = heads, dim
        self.kv_heads = heads if kv_heads is None else kv_heads
        _fit(heads, dim, self.kv_heads)
        self.desc = QlAttn(batch=0, q_len=0, k_len=0, heads=heads, kv_heads=self.kv_heads, dim=dim,
                           dtype=_lib.QL_F32, scale=max(dim, 1) ** -0.5 if scale is None else scale)
        qlinear_attention_workspace(self.desc)  # its checks
        self._sizes = {}  # descriptor and workspace bytes by size of call

    def _call(self, dev, q, k, lens, mask, grad):
        """(descriptor, workspace bytes, shapes of queries and keys, their dense strides)
        of a call."""
        _there(k, "k")
        key = (q.dtype, q.shape, k.shape, grad)
        size = self._sizes.get(key)
        if size is None:
            size = self._size(key, q, k, grad)
        if lens is None and mask is None:
            return size
        d = QlAttn.from_buffer_copy(size[0])
        if lens is not None:
            _there(lens, "lens")
            d.k_lens = _flat(lens, "lens", dev, _I32, (d.batch,))
        if mask is not None:
            _there(mask, "mask")
            _need(mask.dtype in (torch.bool, torch.uint8), f"mask is {mask.dtype}, not bool")
            d.mask_batch = _rows(mask, "mask", dev, mask.dtype, (d.batch, d.k_len))
            d.k_mask = mask.data_ptr()
        return (d, *size[1:])

    def _size(self, key, q, k, grad):
        _need(q.dim() == 4 and k.dim() == 4, "q and k must be [B, L, heads, dim]")
        _need(q.dtype in _DT, f"q is {q.dtype}: f32 or bf16 only")
        _fit(*q.shape, *k.shape)
        d = QlAttn.from_buffer_copy(self.desc)
        d.batch, d.q_len, d.k_len, d.dtype = q.shape[0], q.shape[1], k.shape[1], _DT[q.dtype]
        D, shapes, dense = self.dim, [], []
        for L, h in ((d.q_len, self.heads), (d.k_len, self.kv_heads)):
            shapes.append((d.batch, L, h, D))
            dense.append((L * h * D, h * D, D))
        return _remember(self._sizes, key,
                         (d, qlinear_attention_workspace(d, grad), *shapes, *dense))

    def forward(self, q, k, v, lens=None, mask=None, out=None, save: bool = False, stream=None):
        """softmax(scale q k^T) v in q's type and shape; with ``save`` returns (out, lse),
        lse f32 [B, heads, q_len], for :meth:`grad`."""
        if stream is not None:
            with _on(stream):
                return self.forward(q, k, v, lens, mask, out, save)
        _there(q, "q")
        dev, dt = _device(), q.dtype
        d, nb, qs, ks, qd, kd = self._call(dev, q, k, lens, mask, 0)
        vq, vk = _view(q, "q", dev, dt, qs, qd), _view(k, "k", dev, dt, ks, kd)
        vv = _view(v, "v", dev, dt, ks, kd)
        if out is None:
            out = torch.empty(qs, dtype=dt, device=q.device)
            vo = QlHeadsView(out.data_ptr(), *qd)
        else:
            vo = _view(out, "out", dev, dt, qs, qd)
        lse = torch.empty((qs[0], qs[2], qs[1]), dtype=_F32, device=q.device) if save else None
        ws = torch.empty(nb, dtype=torch.uint8, device=q.device) if nb else None
        qlinear_attention(d, vq, vk, vv, vo, _ptr(lse), _ptr(ws), nb, _stream(dev))
        return (out, lse) if save else out

    def grad(self, dout, q, k, v, out, lse, lens=None, mask=None, into=None, stream=None):
        """(dq, dk, dv) of :meth:`forward`, from the out and lse that it gave, for the same
        lens and mask; written into the triple ``into`` where it is given. The
        gradient of a key head is summed over the query heads that share it."""
        if stream is not None:
            with _on(stream):
                return self.grad(dout, q, k, v, out, lse, lens, mask, into)
        _there(q, "q")
        dev, dt = _device(), q.dtype
        d, nb, qs, ks, qd, kd = self._call(dev, q, k, lens, mask, 1)
        vq, vk = _view(q, "q", dev, dt, qs, qd), _view(k, "k", dev, dt, ks, kd)
        vv, vd = _view(v, "v", dev, dt, ks, kd), _view(dout, "dout", dev, dt, qs, qd)
        vo = _view(out, "out", dev, dt, qs, qd)
        _there(lse, "lse")
        at = _flat(lse, "lse", dev, _F32, (qs[0], qs[2], qs[1]))
        if into is None:
            into = [torch.empty(s, dtype=dt, device=q.device) for s in (qs, ks, ks)]
        views = [_view(t, name, dev, dt, s, n) for t, name, s, n in
                 zip(into, ("dq", "dk", "dv"), (qs, ks, ks), (qd, kd, kd))]
        ws = torch.empty(nb, dtype=torch.uint8, device=q.device) if nb else None
        qlinear_attention_grad(d, vd, vq, vk, vv, vo, at, *views, _ptr(ws), nb, _stream(dev))
        return tuple(into)
