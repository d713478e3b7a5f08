"""MI355X-native quantized linear layer for diffusion transformers.

DualScale (polarity-aware) activation quantization with optional block
Walsh-Hadamard rotation and LSB truncation (of activation codes per call,
of the stored weight codes per step through plan views), an int8-MFMA GEMM
over both polarity planes with per-channel / per-segment weight scales, and
an fp32 epilogue with the classifier-free-guidance combine -- all in hand-written
HIP kernels for gfx950 behind the C ABI of include/qlinear.h.

Beside the layer: low-rank adapters of many requests (forward and backward),
group normalisation with an activation over channels-last images (forward and
backward), and clipping of many gradients by their global norm. In the block
around it: few rows against 4-bit weights with group scales, norms of queries and
keys for each head with the rotation by positions of several axes, and attention to
another sequence's states (the last two forward and backward).
"""
from .qlinear import (  # noqa: F401
    Plan, QLError, QuantLinear, qlinear_cfg_combine, qlinear_gamp_allocate, qlinear_gemm,
    qlinear_plan,
    qlinear_plan_destroy, qlinear_plan_lsb_update, qlinear_plan_lsb_view, qlinear_plan_weights,
    qlinear_probe_mfma, qlinear_quantize_act, qlinear_quantize_act_noalloc, qlinear_version,
)

_OPS = ("GradSet", "GroupNormAct", "LoraAdapters", "qlinear_grad_clip", "qlinear_grad_norm",
        "qlinear_group_norm", "qlinear_group_norm_grad", "qlinear_group_norm_workspace",
        "qlinear_lora", "qlinear_lora_grad", "qlinear_lora_workspace")

_BLOCK = ("CrossAttention", "GroupLinear4", "HeadNormRope", "qlinear_attention",
          "qlinear_attention_grad", "qlinear_attention_workspace", "qlinear_heads",
          "qlinear_heads_grad", "qlinear_heads_workspace", "qlinear_rows4", "qlinear_rows4_bytes",
          "qlinear_rows4_pack", "qlinear_rows4_quantize", "qlinear_rows4_unpack",
          "qlinear_rows4_workspace")


def __getattr__(name):  # ops.py and block.py need torch, which the layer's binding imports when used
    if name in _OPS:
        from . import ops
        return getattr(ops, name)
    if name in _BLOCK:
        from . import block
        return getattr(block, name)
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


def __dir__():
    return sorted(list(globals()) + list(_OPS) + list(_BLOCK))
