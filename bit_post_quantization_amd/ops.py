"""Operators beside the quantized linear: the C ABI function for function (same
names), and a small class for each that checks tensors and allocates outputs.

  LoraAdapters  low-rank adapters of many requests beside one projection
  GroupNormAct  group normalisation with an activation, channels last
  GradSet       global norm and clipping of many gradients

Tensors must be on the current device. Every call is asynchronous on the
current stream, or on ``stream``; what a call allocates belongs to the stream
that it runs on. Arguments that do not fit raise QLError before anything is
enqueued.

As with the layer itself, autograd sees none of the calls: results carry no
graph, also where an argument requires grad, and the gradients are the classes'
``grad`` methods.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import _lib
from ._lib import QL_ERR_ARG, QLError, QlLora, QlNorm, QlRequests, check

_L = _lib.load()
_DT = {torch.float32: _lib.QL_F32, torch.bfloat16: _lib.QL_BF16}
_NAMES = {"f32": torch.float32, "bf16": torch.bfloat16}
_ACTS = {"none": _lib.QL_ACT_NONE, "silu": _lib.QL_ACT_SILU}
_F32, _I32, _F64 = torch.float32, torch.int32, torch.float64
_byref = ctypes.byref
_device = torch.cuda.current_device
# Raw handle of a device's current stream. torch's Stream object costs 3 us to
# make, as much as a kernel launch.
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)

# The checks below run on every call, before a launch that takes the host 4 us:
# they look at a tensor as few times as they can.


def _need(ok: bool, msg: str) -> None:
    if not ok:
        raise QLError(QL_ERR_ARG, msg)


def _refuse(t, name: str, dev: int, dtype, shape) -> None:
    _need(isinstance(t, torch.Tensor) and t.get_device() == dev,
          f"{name} must be a tensor on the current device")
    _need(t.dtype == dtype, f"{name} is {t.dtype}, not {dtype}")
    raise QLError(QL_ERR_ARG, f"{name} is {tuple(t.shape)}, not {tuple(shape)}")


def _flat(t, name: str, dev: int, dtype, shape) -> int:
    """Address of a contiguous tensor of this type and shape."""
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape:
        _refuse(t, name, dev, dtype, shape)
    if not t.is_contiguous():
        raise QLError(QL_ERR_ARG, f"{name} is not contiguous")
    return t.data_ptr()


def _rows(t, name: str, dev: int, dtype, shape) -> int:
    """Row stride of a matrix whose rows are contiguous."""
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape:
        _refuse(t, name, dev, dtype, shape)
    rows, cols = shape
    if t.is_contiguous() or rows == 0:
        return cols
    _need(cols == 1 or t.stride(1) == 1, f"{name}: rows are not contiguous")
    if rows == 1:
        return cols
    _need(t.stride(0) >= cols, f"{name}: rows overlap")
    return t.stride(0)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


_MOST_SIZES = 4096  # sizes of calls whose workspace a layer remembers


def _remember(sizes: dict, key, value):
    if len(sizes) >= _MOST_SIZES:
        sizes.clear()
    sizes[key] = value
    return value


def _on(stream):
    """Context in which `stream` (a torch stream or a raw handle) is current."""
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int)
                             else stream)


# ------------------------------------------------------- C ABI, same names ----
# Pointers are addresses (int or None); stream is a raw handle.

def qlinear_lora_workspace(desc: QlLora, M: int, n_requests: int, cfg: int = 0,
                           grad: int = 0) -> int:
    n = ctypes.c_int64()
    check(_L.qlinear_lora_workspace(_byref(desc), M, n_requests, cfg, grad, _byref(n)))
    return n.value


def qlinear_lora(desc: QlLora, X, ldx, M, requests: QlRequests, cfg, w, base, ldb, Y, ldy, S,
                 workspace, workspace_bytes, stream) -> None:
    check(_L.qlinear_lora(_byref(desc), X, ldx, M, _byref(requests), cfg, w, base, ldb, Y, ldy, S,
                          workspace, workspace_bytes, stream))


def qlinear_lora_grad(desc: QlLora, X, ldx, M, requests: QlRequests, S, dY, lddy, dX, lddx, dA, dB,
                      workspace, workspace_bytes, stream) -> None:
    check(_L.qlinear_lora_grad(_byref(desc), X, ldx, M, _byref(requests), S, dY, lddy, dX, lddx, dA,
                               dB, workspace, workspace_bytes, stream))


def qlinear_group_norm_workspace(desc: QlNorm, grad: int = 0) -> int:
    n = ctypes.c_int64()
    check(_L.qlinear_group_norm_workspace(_byref(desc), grad, _byref(n)))
    return n.value


def qlinear_group_norm(desc: QlNorm, x, x_batch, x_row, y, y_batch, y_row, mean, rstd, workspace,
                       workspace_bytes, stream) -> None:
    check(_L.qlinear_group_norm(_byref(desc), x, x_batch, x_row, y, y_batch, y_row, mean, rstd,
                                workspace, workspace_bytes, stream))


def qlinear_group_norm_grad(desc: QlNorm, dy, dy_batch, dy_row, x, x_batch, x_row, mean, rstd, dx,
                            dx_batch, dx_row, dgamma, dbeta, workspace, workspace_bytes,
                            stream) -> None:
    check(_L.qlinear_group_norm_grad(_byref(desc), dy, dy_batch, dy_row, x, x_batch, x_row, mean,
                                     rstd, dx, dx_batch, dx_row, dgamma, dbeta, workspace,
                                     workspace_bytes, stream))


def qlinear_grad_norm(table, n: int, units: int, partials, stream) -> None:
    check(_L.qlinear_grad_norm(table, n, units, partials, stream))


def qlinear_grad_clip(table, n: int, units: int, partials, max_norm: float, norm, stream) -> None:
    check(_L.qlinear_grad_clip(table, n, units, partials, max_norm, norm, stream))


# ---------------------------------------------------------------- adapters ----

class LoraAdapters:
    """Adapters A [n, rank, K], B [n, N, rank] (f32 or bf16) of one projection.

    ``scales`` f32 [n] (None: 1) and ``ranks`` int32 [n] (None: all of the
    stored rank) are device tensors. All of them are used where they are: update
    them in place. The rows of a call belong to requests:
    request i owns rows [row_offsets[i], row_offsets[i+1]) and runs adapter
    ``adapter[i]`` (-1: none); both are int32 device tensors."""

    def __init__(self, A, B, scales=None, ranks=None, x_dtype: str = "f32"):
        _need(x_dtype in _NAMES, f"x_dtype {x_dtype!r} is not one of {sorted(_NAMES)}")
        _need(A.dim() == 3 and B.dim() == 3 and A.shape[0] == B.shape[0]
              and A.shape[1] == B.shape[2], "A and B must be [n, rank, K] and [n, N, rank]")
        _need(A.dtype in _DT, f"A is {A.dtype}: f32 or bf16 only")
        dev = _device()
        _flat(A, "A", dev, A.dtype, A.shape)
        _flat(B, "B", dev, A.dtype, B.shape)
        n, self.rank, self.K = A.shape
        self.N = B.shape[1]
        if scales is not None:
            _flat(scales, "scales", dev, _F32, (n,))
        if ranks is not None:
            _flat(ranks, "ranks", dev, _I32, (n,))
        self.A, self.B, self.scales, self.ranks = A, B, scales, ranks
        self.x_dtype = _NAMES[x_dtype]
        self.desc = QlLora(N=self.N, K=self.K, rank=self.rank, n_adapters=n,
                           x_dtype=_DT[self.x_dtype], w_dtype=_DT[A.dtype], A=_ptr(A), B=_ptr(B),
                           scales=_ptr(scales), ranks=_ptr(ranks))
        self._bytes = {}  # workspace bytes by size of call
        self._workspace_bytes(0, 1, 0, 0)  # its checks

    def _workspace_bytes(self, *size) -> int:
        n = self._bytes.get(size)
        if n is None:
            n = _remember(self._bytes, size, qlinear_lora_workspace(self.desc, *size))
        return n

    @staticmethod
    def _requests(dev, row_offsets, adapter) -> QlRequests:
        n = adapter.numel()
        return QlRequests(n, _flat(row_offsets, "row_offsets", dev, _I32, (n + 1,)),
                          _flat(adapter, "adapter", dev, _I32, (n,)))

    def apply(self, X, row_offsets, adapter, base=None, out=None, cfg: int = 0, w: float = 1.0,
              save: bool = False, stream=None):
        """base + scale_a (X A_a^T) B_a^T, f32 [M, N] ([M/2, N] with cfg = 1, whose
        offsets partition M/2 rows). ``out`` may be ``base``; None allocates. With
        ``save`` returns (out, S), S f32 [M, rank] for :meth:`grad`."""
        if stream is not None:
            with _on(stream):
                return self.apply(X, row_offsets, adapter, base, out, cfg, w, save)
        dev, M = _device(), X.shape[0]
        shape = (M // 2 if cfg else M, self.N)
        ldx = _rows(X, "X", dev, self.x_dtype, (M, self.K))
        ldb = 0 if base is None else _rows(base, "base", dev, _F32, shape)
        q = self._requests(dev, row_offsets, adapter)
        if out is None:
            out, ldy = torch.empty(shape, dtype=_F32, device=X.device), self.N
        else:
            ldy = _rows(out, "out", dev, _F32, shape)
        S = torch.empty((M, self.rank), dtype=_F32, device=X.device) if save else None
        nb = self._workspace_bytes(M, q.n_requests, cfg, 0)
        ws = torch.empty(nb, dtype=torch.uint8, device=X.device) if nb else None
        qlinear_lora(self.desc, X.data_ptr(), ldx, M, q, cfg, w, _ptr(base), ldb, out.data_ptr(),
                     ldy, _ptr(S), _ptr(ws), nb, _stream(dev))
        return (out, S) if save else out

    def grad(self, X, row_offsets, adapter, S, dY, need_dx: bool = True, stream=None, out=None):
        """(dX, dA, dB) of :meth:`apply` (cfg = 0): dX is the adapters' part only
        (None without ``need_dx``); dA, dB in the adapters' type, written into the
        pair ``out`` where it is given (every element, so that one :class:`GradSet`
        serves all steps)."""
        if stream is not None:
            with _on(stream):
                return self.grad(X, row_offsets, adapter, S, dY, need_dx, out=out)
        dev, M = _device(), X.shape[0]
        ldx = _rows(X, "X", dev, self.x_dtype, (M, self.K))
        lddy = _rows(dY, "dY", dev, _F32, (M, self.N))
        s_ptr = _flat(S, "S", dev, _F32, (M, self.rank))
        q = self._requests(dev, row_offsets, adapter)
        dX = torch.empty((M, self.K), dtype=self.x_dtype, device=X.device) if need_dx else None
        if out is None:
            dA, dB = torch.empty_like(self.A), torch.empty_like(self.B)
        else:
            dA, dB = out
            _flat(dA, "dA", dev, self.A.dtype, self.A.shape)
            _flat(dB, "dB", dev, self.B.dtype, self.B.shape)
        nb = self._workspace_bytes(M, q.n_requests, 0, 1)
        ws = torch.empty(nb, dtype=torch.uint8, device=X.device)
        qlinear_lora_grad(self.desc, X.data_ptr(), ldx, M, q, s_ptr, dY.data_ptr(), lddy, _ptr(dX),
                          self.K, dA.data_ptr(), dB.data_ptr(), ws.data_ptr(), nb, _stream(dev))
        return dX, dA, dB


# -------------------------------------------------------------- group norm ----

def _image(t, name: str, dev: int, dtype, shape):
    """(batch, positions, channels, batch stride, row stride) of [B, L, C], or of
    [B, C, H, W] in channels-last order."""
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape:
        _refuse(t, name, dev, dtype, shape)
    if len(shape) == 3:
        B, L, C = shape
        if t.is_contiguous():
            return B, L, C, L * C, C
        sb, row, sc = t.stride()
    else:
        _need(len(shape) == 4, f"{name} must be [B, L, C] or channels-last [B, C, H, W]")
        B, C, H, W = shape
        sb, sc, sh, sw = t.stride()
        _need(H == 1 or W == 1 or sh == W * sw, f"{name}: positions are not evenly spaced")
        L, row = H * W, sw if W > 1 else sh
    _need(C == 1 or sc == 1, f"{name}: channels are not contiguous")
    return B, L, C, sb if B > 1 else 0, row if L > 1 else C


def _like(t):
    """An uninitialised tensor of t's shape, packed, channels last."""
    if t.dim() == 4:
        return torch.empty(t.shape, dtype=t.dtype, device=t.device,
                           memory_format=torch.channels_last)
    return torch.empty(t.shape, dtype=t.dtype, device=t.device)


class GroupNormAct:
    """Group normalisation and an activation ("none" or "silu") of channels-last
    images: [B, L, C], or [B, C, H, W] in torch's channels_last order, f32 or
    bf16. gamma and beta [C] (f32 or bf16, both alike) may be None."""

    def __init__(self, gamma, beta, groups: int, eps: float = 1e-5, act: str = "silu",
                 channels: Optional[int] = None):
        _need(act in _ACTS, f"act {act!r} is not one of {sorted(_ACTS)}")
        given = [t for t in (gamma, beta) if t is not None]
        _need(bool(given) or channels is not None, "channels is needed without gamma and beta")
        self.C = given[0].numel() if given else int(channels)
        w = given[0].dtype if given else _F32
        _need(w in _DT, f"gamma is {w}: f32 or bf16 only")
        for t, name in ((gamma, "gamma"), (beta, "beta")):
            if t is not None:
                _flat(t, name, _device(), w, (self.C,))
        self.gamma, self.beta, self.groups = gamma, beta, groups
        self.desc = QlNorm(batch=0, positions=0, channels=self.C, groups=groups,
                           x_dtype=_lib.QL_F32, w_dtype=_DT[w], act=_ACTS[act], eps=eps,
                           gamma=_ptr(gamma), beta=_ptr(beta))
        qlinear_group_norm_workspace(self.desc)  # its checks
        self._sizes = {}  # descriptor and workspace bytes by size of call

    def _of(self, dtype, B, L, C, grad):
        d = self._sizes.get((dtype, B, L, grad))
        if d is None:
            d = QlNorm.from_buffer_copy(self.desc)
            d.batch, d.positions, d.x_dtype = B, L, _DT[dtype]
            d = _remember(self._sizes, (dtype, B, L, grad),
                          (d, qlinear_group_norm_workspace(d, grad)))
        _need(C == self.C, f"x has {C} channels, not {self.C}")
        return d

    def forward(self, x, out=None, stats: bool = False, stream=None):
        """act(norm(x)); ``out`` may be ``x``. With ``stats`` returns (out, mean,
        rstd), f32 [B, groups] each, for :meth:`grad`."""
        if stream is not None:
            with _on(stream):
                return self.forward(x, out, stats)
        dev, dt, shape = _device(), x.dtype, x.shape
        _need(dt in _DT, f"x is {dt}: f32 or bf16 only")
        B, L, C, xb, xr = _image(x, "x", dev, dt, shape)
        d, nb = self._of(dt, B, L, C, 0)
        if out is None:
            out = _like(x)
            yb, yr = L * C, C
        else:
            _, _, _, yb, yr = _image(out, "out", dev, dt, shape)
        mean = rstd = None
        if stats:
            mean, rstd = torch.empty((2, B, self.groups), dtype=_F32, device=x.device)
        ws = torch.empty(nb, dtype=torch.uint8, device=x.device) if nb else None
        qlinear_group_norm(d, x.data_ptr(), xb, xr, out.data_ptr(), yb, yr, _ptr(mean), _ptr(rstd),
                           _ptr(ws), nb, _stream(dev))
        return (out, mean, rstd) if stats else out

    def grad(self, dy, x, mean, rstd, stream=None, out=None):
        """(dx, dgamma, dbeta); the last two in gamma's type, None where the
        parameter is, written into the pair ``out`` where it is given."""
        if stream is not None:
            with _on(stream):
                return self.grad(dy, x, mean, rstd, out=out)
        dev, dt, shape = _device(), x.dtype, x.shape
        _need(dt in _DT, f"x is {dt}: f32 or bf16 only")
        B, L, C, xb, xr = _image(x, "x", dev, dt, shape)
        _, _, _, db, dr = _image(dy, "dy", dev, dt, shape)
        d, nb = self._of(dt, B, L, C, 1)
        m = _flat(mean, "mean", dev, _F32, (B, self.groups))
        r = _flat(rstd, "rstd", dev, _F32, (B, self.groups))
        dx = _like(x)
        if out is None:
            dgamma = None if self.gamma is None else torch.empty_like(self.gamma)
            dbeta = None if self.beta is None else torch.empty_like(self.beta)
        else:
            dgamma, dbeta = out
            for t, p, name in ((dgamma, self.gamma, "dgamma"), (dbeta, self.beta, "dbeta")):
                _need((t is None) == (p is None), f"{name} is given without its parameter, or not")
                if t is not None:
                    _flat(t, name, dev, p.dtype, p.shape)
        ws = torch.empty(nb, dtype=torch.uint8, device=x.device) if nb else None
        qlinear_group_norm_grad(d, dy.data_ptr(), db, dr, x.data_ptr(), xb, xr, m, r, dx.data_ptr(),
                                L * C, C, _ptr(dgamma), _ptr(dbeta), _ptr(ws), nb, _stream(dev))
        return dx, dgamma, dbeta


# ---------------------------------------------------------------- clipping ----

def _order(t):
    """The strides of a tensor that fills its storage's span without gaps or
    repeats (channels last, transposed, ...), None for any other."""
    n = 1
    for stride, size in sorted((s, k) for s, k in zip(t.stride(), t.shape) if k != 1):
        if stride != n:
            return None
        n *= size
    return [s for s, k in zip(t.stride(), t.shape) if k != 1]


class GradSet:
    """Gradients to be clipped by their global norm, in place or into ``out``
    (tensors of the same sizes, f32 or bf16 each). They may lie in any dense order
    (channels last, transposed); an ``out`` lies in its gradient's order. What is
    written overlaps nothing else that is listed: a gradient that two parameters
    share is listed once.

    Made once for gradients that stay where they are (the set holds the tensors
    and a device table of their addresses); make a new one when a tensor is
    replaced, and keep the set while a captured graph with its calls is replayed."""

    def __init__(self, grads: Sequence, out: Optional[Sequence] = None):
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        _need(len(self.grads) == len(self.out), "out must list one tensor for each gradient")
        dev, rows, unit, spans = _device(), [], 0, []
        for g, o in zip(self.grads, self.out):
            n, plain = g.numel(), True
            for t, name in ((g, "gradient"), (o, "out")):
                _need(t.dtype in _DT, f"{name} is {t.dtype}: f32 or bf16 only")
                if t.get_device() != dev:
                    _refuse(t, name, dev, t.dtype, t.shape)
                if not t.is_contiguous():
                    plain = False
                    _need(_order(t) is not None, f"{name} is not dense")
            _need(o.numel() == n, "out and its gradient differ in size")
            _need(plain or o is g or (o.shape == g.shape and _order(o) == _order(g)),
                  "out lies in another order than its gradient")
            _need(_ptr(g) != _ptr(o) or g.dtype == o.dtype or n == 0,
                  "out is its gradient with another type")
            at, to = _ptr(g), _ptr(o)
            rows.append((at, to, n, unit, _DT[g.dtype] | _DT[o.dtype] << 32))
            if n:
                spans.append((to, to + n * o.element_size(), True))
                if at != to:
                    spans.append((at, at + n * g.element_size(), False))
            unit += -(-n // _lib.QL_GRAD_UNIT)
        # Different workgroups write what they write and read what they read.
        read = written = 0  # ends of what lies before
        for lo, hi, out in sorted(spans):
            _need(lo >= (max(read, written) if out else written),
                  "an out overlaps another one or another gradient (or a gradient is listed twice)")
            read, written = (read, max(written, hi)) if out else (max(read, hi), written)
        self.units = unit
        self.device = torch.device("cuda", dev)
        self._made_on = _stream(dev)
        self.table = torch.tensor(rows, dtype=torch.int64).reshape(-1, 5).to(self.device)

    def _ready(self) -> int:
        """The current stream's handle, on which the table may be read from now on."""
        dev = _device()
        _need(dev == self.device.index, "the set's tensors are not on the current device")
        s = _stream(dev)
        if s != self._made_on:  # the table's memory outlives the set until this stream is done
            self.table.record_stream(torch.cuda.current_stream(dev))
        return s

    def partials(self, stream=None):
        """f64 [QL_GRAD_PARTIALS], adding up to the squared norm. Gradients sharded
        over processes: all-reduce them and hand them to :meth:`clip`."""
        if stream is not None:
            with _on(stream):
                return self.partials()
        s = self._ready()
        p = torch.empty(_lib.QL_GRAD_PARTIALS, dtype=_F64, device=self.device)
        qlinear_grad_norm(self.table.data_ptr(), len(self.grads), self.units, p.data_ptr(), s)
        return p

    def clip(self, max_norm: float, partials=None, stream=None):
        """out = gradient * min(1, max_norm / (norm + 1e-6)); the norm before, f32 []."""
        if stream is not None:
            with _on(stream):
                return self.clip(max_norm, partials)
        s = self._ready()
        p = self.partials() if partials is None else partials
        at = _flat(p, "partials", self.device.index, _F64, (_lib.QL_GRAD_PARTIALS,))
        norm = torch.empty((), dtype=_F32, device=self.device)
        qlinear_grad_clip(self.table.data_ptr(), len(self.grads), self.units, at, max_norm,
                          norm.data_ptr(), s)
        return norm
