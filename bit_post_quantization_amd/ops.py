"""Operators beside the quantized linear: the C ABI function for function (same
names), and a small class for each that checks tensors and allocates outputs.

  LoraAdapters  low-rank adapters of many requests beside one projection
  GroupNormAct  group normalisation with an activation, channels last
  GradSet       global norm and clipping of many gradients

Tensors must be on the current device. Every call is asynchronous on the
current stream, or on ``stream``; what a call allocates belongs to the stream
that it runs on. Arguments that do not fit raise QLError before anything is
enqueued.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional, Sequence

import torch

from . import _lib
from ._lib import QL_ERR_ARG, QLError, QlLora, QlNorm, QlRequests, check

_DT = {torch.float32: _lib.QL_F32, torch.bfloat16: _lib.QL_BF16}
_NAMES = {"f32": torch.float32, "bf16": torch.bfloat16}
_ACTS = {"none": _lib.QL_ACT_NONE, "silu": _lib.QL_ACT_SILU}
_byref = ctypes.byref


def _need(ok: bool, msg: str) -> None:
    if not ok:
        raise QLError(QL_ERR_ARG, msg)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check(t, name: str, dtype, shape=None) -> None:
    if not (isinstance(t, torch.Tensor) and t.is_cuda and
            t.get_device() == torch.cuda.current_device()):
        raise QLError(QL_ERR_ARG, f"{name} must be a tensor on the current device")
    if t.dtype != dtype:
        raise QLError(QL_ERR_ARG, f"{name} is {t.dtype}, not {dtype}")
    if shape is not None and t.shape != shape:
        raise QLError(QL_ERR_ARG, f"{name} is {tuple(t.shape)}, not {tuple(shape)}")


def _flat(t, name: str, dtype, shape=None) -> None:
    _check(t, name, dtype, shape)
    if not t.is_contiguous():
        raise QLError(QL_ERR_ARG, f"{name} is not contiguous")


def _rows(t, name: str, dtype, shape) -> int:
    """Row stride of a matrix whose rows are contiguous."""
    _check(t, name, dtype, shape)
    rows, cols = shape
    if t.is_contiguous() or rows == 0:
        return cols
    _need(cols == 1 or t.stride(1) == 1, f"{name}: rows are not contiguous")
    if rows == 1:
        return cols
    _need(t.stride(0) >= cols, f"{name}: rows overlap")
    return t.stride(0)


# Raw handle of the current stream. torch's Stream object costs 3 us to make,
# a third of a small call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)
_HERE = contextlib.nullcontext()


def _on(stream):
    """(context under which to allocate, raw stream) of a call."""
    if stream is None:
        return _HERE, _raw_stream(torch.cuda.current_device())
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    return torch.cuda.stream(stream), stream.cuda_stream


def _workspace(nbytes: int):
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda") if nbytes else None


def _nbytes(workspace) -> int:
    return 0 if workspace is None else workspace.numel()


# ------------------------------------------------------- C ABI, same names ----

def qlinear_lora_workspace(desc: QlLora, M: int, n_requests: int, cfg: int = 0,
                           grad: int = 0) -> int:
    n = ctypes.c_int64()
    check(_lib.load().qlinear_lora_workspace(_byref(desc), M, n_requests, cfg, grad, _byref(n)))
    return n.value


def qlinear_lora(desc: QlLora, X, ldx, M, requests: QlRequests, cfg, w, base, ldb, Y, ldy, S,
                 workspace, stream) -> None:
    check(_lib.load().qlinear_lora(_byref(desc), _ptr(X), ldx, M, _byref(requests), cfg, w,
                                   _ptr(base), ldb, _ptr(Y), ldy, _ptr(S), _ptr(workspace),
                                   _nbytes(workspace), stream))


def qlinear_lora_grad(desc: QlLora, X, ldx, M, requests: QlRequests, S, dY, lddy, dX, lddx, dA, dB,
                      workspace, stream) -> None:
    check(_lib.load().qlinear_lora_grad(_byref(desc), _ptr(X), ldx, M, _byref(requests), _ptr(S),
                                        _ptr(dY), lddy, _ptr(dX), lddx, _ptr(dA), _ptr(dB),
                                        _ptr(workspace), _nbytes(workspace), stream))


def qlinear_group_norm_workspace(desc: QlNorm, grad: int = 0) -> int:
    n = ctypes.c_int64()
    check(_lib.load().qlinear_group_norm_workspace(_byref(desc), grad, _byref(n)))
    return n.value


def qlinear_group_norm(desc: QlNorm, x, x_strides, y, y_strides, mean, rstd, workspace,
                       stream) -> None:
    check(_lib.load().qlinear_group_norm(_byref(desc), _ptr(x), *x_strides, _ptr(y), *y_strides,
                                         _ptr(mean), _ptr(rstd), _ptr(workspace),
                                         _nbytes(workspace), stream))


def qlinear_group_norm_grad(desc: QlNorm, dy, dy_strides, x, x_strides, mean, rstd, dx, dx_strides,
                            dgamma, dbeta, workspace, stream) -> None:
    check(_lib.load().qlinear_group_norm_grad(_byref(desc), _ptr(dy), *dy_strides, _ptr(x),
                                              *x_strides, _ptr(mean), _ptr(rstd), _ptr(dx),
                                              *dx_strides, _ptr(dgamma), _ptr(dbeta),
                                              _ptr(workspace), _nbytes(workspace), stream))


def qlinear_grad_norm(table, n: int, units: int, partials, stream) -> None:
    check(_lib.load().qlinear_grad_norm(_ptr(table), n, units, _ptr(partials), stream))


def qlinear_grad_clip(table, n: int, units: int, partials, max_norm: float, norm, stream) -> None:
    check(_lib.load().qlinear_grad_clip(_ptr(table), n, units, _ptr(partials), float(max_norm),
                                        _ptr(norm), stream))


# ---------------------------------------------------------------- adapters ----

class LoraAdapters:
    """Adapters A [n, rank, K], B [n, N, rank] (f32 or bf16) of one projection.

    ``scales`` f32 [n] (None: 1) and ``ranks`` int32 [n] (None: all of the
    stored rank) are device tensors. The rows of a call belong to requests:
    request i owns rows [row_offsets[i], row_offsets[i+1]) and runs adapter
    ``adapter[i]`` (-1: none); both are int32 device tensors."""

    def __init__(self, A, B, scales=None, ranks=None, x_dtype: str = "f32"):
        _need(x_dtype in _NAMES, f"x_dtype {x_dtype!r} is not one of {sorted(_NAMES)}")
        _need(A.dim() == 3 and B.dim() == 3 and A.shape[0] == B.shape[0]
              and A.shape[1] == B.shape[2], "A and B must be [n, rank, K] and [n, N, rank]")
        _need(A.dtype in _DT, f"A is {A.dtype}: f32 or bf16 only")
        _flat(A, "A", A.dtype)
        _flat(B, "B", A.dtype)
        n, self.rank, self.K = A.shape
        self.N = B.shape[1]
        if scales is not None:
            _flat(scales, "scales", torch.float32, (n,))
        if ranks is not None:
            _flat(ranks, "ranks", torch.int32, (n,))
        self.A, self.B, self.scales, self.ranks = A, B, scales, ranks
        self.x_dtype = _NAMES[x_dtype]
        self.desc = QlLora(N=self.N, K=self.K, rank=self.rank, n_adapters=n,
                           x_dtype=_DT[self.x_dtype], w_dtype=_DT[A.dtype], A=_ptr(A), B=_ptr(B),
                           scales=_ptr(scales), ranks=_ptr(ranks))
        qlinear_lora_workspace(self.desc, 0, 1)  # its checks

    def _requests(self, row_offsets, adapter) -> QlRequests:
        n = adapter.numel()
        _flat(row_offsets, "row_offsets", torch.int32, (n + 1,))
        _flat(adapter, "adapter", torch.int32, (n,))
        return QlRequests(n_requests=n, row_offsets=_ptr(row_offsets), adapter=_ptr(adapter))

    def apply(self, X, row_offsets, adapter, base=None, out=None, cfg: int = 0, w: float = 1.0,
              save: bool = False, stream=None):
        """base + scale_a (X A_a^T) B_a^T, f32 [M, N] ([M/2, N] with cfg = 1, whose
        offsets partition M/2 rows). ``out`` may be ``base``; None allocates. With
        ``save`` returns (out, S), S f32 [M, rank] for :meth:`grad`."""
        M = X.shape[0]
        rows = M // 2 if cfg else M
        ldx = _rows(X, "X", self.x_dtype, (M, self.K))
        q = self._requests(row_offsets, adapter)
        ctx, s = _on(stream)
        with ctx:
            if out is None:
                out = torch.empty((rows, self.N), dtype=torch.float32, device="cuda")
            S = torch.empty((M, self.rank), dtype=torch.float32, device="cuda") if save else None
            ws = _workspace(qlinear_lora_workspace(self.desc, M, q.n_requests, cfg))
        ldy = _rows(out, "out", torch.float32, (rows, self.N))
        ldb = 0 if base is None else _rows(base, "base", torch.float32, (rows, self.N))
        qlinear_lora(self.desc, X, ldx, M, q, cfg, w, base, ldb, out, ldy, S, ws, s)
        return (out, S) if save else out

    def grad(self, X, row_offsets, adapter, S, dY, need_dx: bool = True, stream=None):
        """(dX, dA, dB) of :meth:`apply` (cfg = 0): dX is the adapters' part only
        (None without ``need_dx``); dA, dB in the adapters' type."""
        M = X.shape[0]
        ldx = _rows(X, "X", self.x_dtype, (M, self.K))
        lddy = _rows(dY, "dY", torch.float32, (M, self.N))
        _flat(S, "S", torch.float32, (M, self.rank))
        q = self._requests(row_offsets, adapter)
        ctx, s = _on(stream)
        with ctx:
            dX = torch.empty((M, self.K), dtype=self.x_dtype, device="cuda") if need_dx else None
            dA, dB = torch.empty_like(self.A), torch.empty_like(self.B)
            ws = _workspace(qlinear_lora_workspace(self.desc, M, q.n_requests, 0, 1))
        qlinear_lora_grad(self.desc, X, ldx, M, q, S, dY, lddy, dX, self.K, dA, dB, ws, s)
        return dX, dA, dB


# -------------------------------------------------------------- group norm ----

def _image(t, name: str, dtype, shape=None):
    """(batch, positions, channels, (batch stride, row stride)) of [B, L, C], or
    of [B, C, H, W] in channels-last order."""
    _check(t, name, dtype, shape)
    if t.dim() == 4:
        B, C, H, W = t.shape
        _need(H == 1 or W == 1 or t.stride(2) == W * t.stride(3),
              f"{name}: positions are not evenly spaced")
        L, c_st = H * W, t.stride(1)
        row = t.stride(3) if W > 1 else t.stride(2) if H > 1 else C
    else:
        _need(t.dim() == 3, f"{name} must be [B, L, C] or channels-last [B, C, H, W]")
        B, L, C = t.shape
        c_st, row = t.stride(2), t.stride(1) if L > 1 else C
    _need(C == 1 or c_st == 1, f"{name}: channels are not contiguous")
    return B, L, C, (t.stride(0) if B > 1 else 0, row)


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
        w = given[0].dtype if given else torch.float32
        _need(w in _DT, f"gamma is {w}: f32 or bf16 only")
        for t, name in ((gamma, "gamma"), (beta, "beta")):
            if t is not None:
                _flat(t, name, w, (self.C,))
        self.gamma, self.beta, self.groups = gamma, beta, groups
        self.desc = QlNorm(batch=0, positions=0, channels=self.C, groups=groups,
                           x_dtype=_lib.QL_F32, w_dtype=_DT[w], act=_ACTS[act], eps=eps,
                           gamma=_ptr(gamma), beta=_ptr(beta))
        self.w_dtype = w
        qlinear_group_norm_workspace(self.desc)  # its checks

    def _desc(self, dtype, B, L, C) -> QlNorm:
        _need(C == self.C, f"x has {C} channels, not {self.C}")
        d = QlNorm.from_buffer_copy(self.desc)
        d.batch, d.positions, d.x_dtype = B, L, _DT[dtype]
        return d

    def forward(self, x, out=None, stats: bool = False, stream=None):
        """act(norm(x)); ``out`` may be ``x``. With ``stats`` returns (out, mean,
        rstd), f32 [B, groups] each, for :meth:`grad`."""
        _need(x.dtype in _DT, f"x is {x.dtype}: f32 or bf16 only")
        B, L, C, xs = _image(x, "x", x.dtype)
        d = self._desc(x.dtype, B, L, C)
        ctx, s = _on(stream)
        with ctx:
            out = _like(x) if out is None else out
            mean, rstd = ((torch.empty((B, self.groups), dtype=torch.float32, device="cuda")
                           for _ in range(2)) if stats else (None, None))
            ws = _workspace(qlinear_group_norm_workspace(d))
        ys = _image(out, "out", x.dtype, x.shape)[3]
        qlinear_group_norm(d, x, xs, out, ys, mean, rstd, ws, s)
        return (out, mean, rstd) if stats else out

    def grad(self, dy, x, mean, rstd, stream=None):
        """(dx, dgamma, dbeta); the last two in gamma's type, None where the
        parameter is."""
        _need(x.dtype in _DT, f"x is {x.dtype}: f32 or bf16 only")
        B, L, C, xs = _image(x, "x", x.dtype)
        d = self._desc(x.dtype, B, L, C)
        ds = _image(dy, "dy", x.dtype, x.shape)[3]
        _flat(mean, "mean", torch.float32, (B, self.groups))
        _flat(rstd, "rstd", torch.float32, (B, self.groups))
        ctx, s = _on(stream)
        with ctx:
            dx = _like(x)
            dgamma = None if self.gamma is None else torch.empty_like(self.gamma)
            dbeta = None if self.beta is None else torch.empty_like(self.beta)
            ws = _workspace(qlinear_group_norm_workspace(d, 1))
        qlinear_group_norm_grad(d, dy, ds, x, xs, mean, rstd, dx, _image(dx, "dx", x.dtype)[3],
                                dgamma, dbeta, ws, s)
        return dx, dgamma, dbeta


# ---------------------------------------------------------------- clipping ----

class GradSet:
    """Gradients to be clipped by their global norm, in place or into ``out``
    (tensors of the same sizes, f32 or bf16 each).

    Made once for gradients that stay where they are (the set holds the tensors
    and a device table of their addresses); make a new one when a tensor is
    replaced."""

    def __init__(self, grads: Sequence, out: Optional[Sequence] = None):
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        _need(len(self.grads) == len(self.out), "out must list one tensor for each gradient")
        rows, unit = [], 0
        for g, o in zip(self.grads, self.out):
            for t, name in ((g, "gradient"), (o, "out")):
                _need(t.dtype in _DT, f"{name} is {t.dtype}: f32 or bf16 only")
                _flat(t, name, t.dtype)
            n = g.numel()
            _need(o.numel() == n, "out and its gradient differ in size")
            _need(_ptr(g) != _ptr(o) or g.dtype == o.dtype or n == 0,
                  "out is its gradient with another type")
            rows.append((_ptr(g), _ptr(o), n, unit, _DT[g.dtype] | _DT[o.dtype] << 32))
            unit += -(-n // _lib.QL_GRAD_UNIT)
        self.units = unit
        self.table = torch.tensor(rows, dtype=torch.int64).reshape(-1, 5).cuda()

    def partials(self, stream=None):
        """f64 [QL_GRAD_PARTIALS], adding up to the squared norm. Gradients sharded
        over processes: all-reduce them and hand them to :meth:`clip`."""
        ctx, s = _on(stream)
        with ctx:
            p = torch.empty(_lib.QL_GRAD_PARTIALS, dtype=torch.float64, device="cuda")
        qlinear_grad_norm(self.table, len(self.grads), self.units, p, s)
        return p

    def clip(self, max_norm: float, partials=None, stream=None):
        """out = gradient * min(1, max_norm / (norm + 1e-6)); the norm before, f32 []."""
        if partials is None:
            partials = self.partials(stream)
        _flat(partials, "partials", torch.float64, (_lib.QL_GRAD_PARTIALS,))
        ctx, s = _on(stream)
        with ctx:
            norm = torch.empty((), dtype=torch.float32, device="cuda")
        qlinear_grad_clip(self.table, len(self.grads), self.units, partials, max_norm, norm, s)
        return norm
