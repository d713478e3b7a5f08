"""ctypes binding of libqlinear.so (declared in include/qlinear.h).

Argument marshalling only: every step of the quantized linear runs in the
library's HIP kernels. The library is loaded from this package directory;
if it has not been built, loading raises instead of falling back to
anything else.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libqlinear.so")

QL_OK, QL_ERR_ARG, QL_ERR_UNSUPPORTED, QL_ERR_OOM, QL_ERR_HIP = range(5)
QL_F32, QL_BF16 = 0, 1
QL_WSCALE_PER_TENSOR, QL_WSCALE_PER_SEGMENT, QL_WSCALE_PER_CHANNEL = 0, 1, 2
QL_ASCALE_DUAL, QL_ASCALE_SYMMETRIC = 0, 1
QL_ACT_NONE, QL_ACT_SILU = 0, 1
QL_HEADS_NONE, QL_HEADS_RMS = 0, 1
QL_PAIRS_ADJACENT, QL_PAIRS_HALVES = 0, 1
QL_POS_I32, QL_POS_F32 = 0, 1
QL_MAX_AXES = 4
QL_GRAD_UNIT, QL_GRAD_PARTIALS = 4096, 1024

EXPORTS = (
    "qlinear_plan", "qlinear_plan_destroy", "qlinear_plan_weights", "qlinear_quantize_act",
    "qlinear_gemm", "qlinear_cfg_combine", "qlinear_last_error", "qlinear_version",
    "qlinear_plan_lsb_view", "qlinear_plan_lsb_update", "qlinear_gamp_allocate",
    "qlinear_quantize_act_noalloc", "qlinear_probe_mfma",
    "qlinear_lora_workspace", "qlinear_lora", "qlinear_lora_grad",
    "qlinear_group_norm_workspace", "qlinear_group_norm", "qlinear_group_norm_grad",
    "qlinear_grad_norm", "qlinear_grad_clip",
    "qlinear_rows4_bytes", "qlinear_rows4_pack", "qlinear_rows4_quantize", "qlinear_rows4_unpack",
    "qlinear_rows4_workspace", "qlinear_rows4",
    "qlinear_heads_workspace", "qlinear_heads", "qlinear_heads_grad",
    "qlinear_attention_workspace", "qlinear_attention", "qlinear_attention_grad",
)


class QlDesc(ctypes.Structure):
    _fields_ = [
        ("N", ctypes.c_int32), ("K", ctypes.c_int32),
        ("w_bits", ctypes.c_int32), ("a_bits", ctypes.c_int32),
        ("hadamard_block", ctypes.c_int32), ("n_segments", ctypes.c_int32),
        ("seg_offsets", ctypes.POINTER(ctypes.c_int32)),
        ("w_scale_mode", ctypes.c_int), ("a_scale_mode", ctypes.c_int),
        ("x_dtype", ctypes.c_int), ("single_hadamard", ctypes.c_int32),
        ("n_k_segments", ctypes.c_int32), ("k_seg_offsets", ctypes.POINTER(ctypes.c_int32)),
    ]


class QlLora(ctypes.Structure):
    _fields_ = [
        ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("rank", ctypes.c_int32),
        ("n_adapters", ctypes.c_int32), ("x_dtype", ctypes.c_int), ("w_dtype", ctypes.c_int),
        ("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("scales", ctypes.c_void_p),
        ("ranks", ctypes.c_void_p),
    ]


class QlRequests(ctypes.Structure):
    _fields_ = [("n_requests", ctypes.c_int32), ("row_offsets", ctypes.c_void_p),
                ("adapter", ctypes.c_void_p)]


class QlNorm(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("positions", ctypes.c_int32), ("channels", ctypes.c_int32),
        ("groups", ctypes.c_int32), ("x_dtype", ctypes.c_int), ("w_dtype", ctypes.c_int),
        ("act", ctypes.c_int), ("eps", ctypes.c_float), ("gamma", ctypes.c_void_p),
        ("beta", ctypes.c_void_p),
    ]


class QlRows4(ctypes.Structure):
    _fields_ = [
        ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("group", ctypes.c_int32),
        ("x_dtype", ctypes.c_int), ("s_dtype", ctypes.c_int), ("act", ctypes.c_int),
        ("packed", ctypes.c_void_p), ("bias", ctypes.c_void_p),
    ]


class QlHeadsView(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("batch", ctypes.c_int64), ("row", ctypes.c_int64),
                ("head", ctypes.c_int64)]


class QlHeads(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("positions", ctypes.c_int32), ("q_heads", ctypes.c_int32),
        ("k_heads", ctypes.c_int32), ("v_heads", ctypes.c_int32), ("dim", ctypes.c_int32),
        ("x_dtype", ctypes.c_int), ("y_dtype", ctypes.c_int), ("w_dtype", ctypes.c_int),
        ("norm", ctypes.c_int), ("eps", ctypes.c_float), ("gamma_q", ctypes.c_void_p),
        ("gamma_k", ctypes.c_void_p), ("n_axes", ctypes.c_int32),
        ("axis_dims", ctypes.c_int32 * QL_MAX_AXES), ("pairs", ctypes.c_int),
        ("freqs", ctypes.c_void_p), ("pos_dtype", ctypes.c_int),
    ]


class QlAttn(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("q_len", ctypes.c_int32), ("k_len", ctypes.c_int32),
        ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("dim", ctypes.c_int32),
        ("dtype", ctypes.c_int), ("scale", ctypes.c_float), ("k_lens", ctypes.c_void_p),
        ("k_mask", ctypes.c_void_p), ("mask_batch", ctypes.c_int64),
    ]


class QLError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"qlinear status {status}: {msg}")
        self.status = status


_lib = None


def load() -> ctypes.CDLL:
    """Load libqlinear.so (built in-tree by the package's _build.build())."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it first (python -m bit_post_quantization_amd._build)")
    L = ctypes.CDLL(LIB_PATH)
    P, I32, I64, F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    LORA, REQ, NORM = (ctypes.POINTER(t) for t in (QlLora, QlRequests, QlNorm))
    ROWS4, HEADS, ATTN, VIEW, SIZE = (ctypes.POINTER(t) for t in (QlRows4, QlHeads, QlAttn,
                                                                  QlHeadsView, I64))
    sig = {
        "qlinear_plan": ([ctypes.POINTER(QlDesc), P, P, ctypes.POINTER(P)], ctypes.c_int),
        "qlinear_plan_destroy": ([P], ctypes.c_int),
        "qlinear_plan_weights": ([P, P, P, P], ctypes.c_int),
        "qlinear_plan_lsb_view": ([P, I32, P, ctypes.POINTER(P)], ctypes.c_int),
        "qlinear_plan_lsb_update": ([P, P, I32, P], ctypes.c_int),
        "qlinear_gamp_allocate": ([I32, P, P, I32, ctypes.c_int64, P, P], ctypes.c_int),
        "qlinear_quantize_act": ([P, P, I32, I32, P, P, P, P], ctypes.c_int),
        "qlinear_quantize_act_noalloc": ([P, P, I32, I32, P, P, P, P], ctypes.c_int),
        "qlinear_gemm": ([P, P, P, I32, I32, F32, P, P, P], ctypes.c_int),
        "qlinear_cfg_combine": ([P, I32, I32, F32, P, P], ctypes.c_int),
        "qlinear_probe_mfma": ([P, I32, I32, P, ctypes.c_int64, P], ctypes.c_int),
        "qlinear_lora_workspace": ([LORA, I32, I32, I32, I32, ctypes.POINTER(I64)], ctypes.c_int),
        "qlinear_lora": ([LORA, P, I64, I32, REQ, I32, F32, P, I64, P, I64, P, P, I64, P],
                         ctypes.c_int),
        "qlinear_lora_grad": ([LORA, P, I64, I32, REQ, P, P, I64, P, I64, P, P, P, I64, P],
                              ctypes.c_int),
        "qlinear_group_norm_workspace": ([NORM, I32, ctypes.POINTER(I64)], ctypes.c_int),
        "qlinear_group_norm": ([NORM, P, I64, I64, P, I64, I64, P, P, P, I64, P], ctypes.c_int),
        "qlinear_group_norm_grad": ([NORM, P, I64, I64, P, I64, I64, P, P, P, I64, I64, P, P, P,
                                     I64, P], ctypes.c_int),
        "qlinear_grad_norm": ([P, I32, I64, P, P], ctypes.c_int),
        "qlinear_grad_clip": ([P, I32, I64, P, F32, P, P], ctypes.c_int),
        "qlinear_rows4_bytes": ([ROWS4, SIZE], ctypes.c_int),
        "qlinear_rows4_pack": ([ROWS4, P, P, P, P], ctypes.c_int),
        "qlinear_rows4_quantize": ([ROWS4, P, ctypes.c_int, P, P], ctypes.c_int),
        "qlinear_rows4_unpack": ([ROWS4, P, P, P], ctypes.c_int),
        "qlinear_rows4_workspace": ([ROWS4, I32, SIZE], ctypes.c_int),
        "qlinear_rows4": ([ROWS4, P, I64, I32, P, I64, P, I64, P], ctypes.c_int),
        "qlinear_heads_workspace": ([HEADS, SIZE], ctypes.c_int),
        "qlinear_heads": ([HEADS, P, I64, I64, P, I64, VIEW, VIEW, VIEW, P], ctypes.c_int),
        "qlinear_heads_grad": ([HEADS, VIEW, VIEW, VIEW, P, I64, I64, P, I64, P, I64, I64, P, P, P,
                                I64, P], ctypes.c_int),
        "qlinear_attention_workspace": ([ATTN, I32, SIZE], ctypes.c_int),
        "qlinear_attention": ([ATTN, VIEW, VIEW, VIEW, VIEW, P, P, I64, P], ctypes.c_int),
        "qlinear_attention_grad": ([ATTN, VIEW, VIEW, VIEW, VIEW, VIEW, P, VIEW, VIEW, VIEW, P,
                                    I64, P], ctypes.c_int),
        "qlinear_last_error": ([], ctypes.c_char_p),
        "qlinear_version": ([], ctypes.c_char_p),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return L


def check(status: int) -> None:
    if status != QL_OK:
        msg = load().qlinear_last_error().decode()
        raise QLError(status, msg)
