"""The microscaled-format operators on torch tensors (include/moe_mx.h).

The calls are in csrc/mx_torch.cpp: each checks its tensors (ValueError), allocates what it returns and launches on the
current stream, or on `stream`; the library's own refusals raise MoeError.  This module adds what they work on.
"""

from __future__ import annotations

import torch

from . import MOE_MX_PRODUCT_WORKSPACE, MoeError, load_library, moe_mx_pack_weights, moe_mx_packed_bytes, moe_mx_weights

load_library()  # says what to build where it is missing; the module below links to it
try:
    from . import _mx_torch
except ImportError as e:
    raise ImportError("the module of the calls on torch tensors is missing or does not fit this torch; build it with "
                      "`python -m mixture_experts_ffn_infer_gb300.build` (which needs g++ and the headers of Python and "
                      "torch)") from e

_U8 = torch.uint8
_BITS = (16, 8, 4, 4)
_GROUP = (0, 32, 32, 16)


def _on(stream, fn, *args):
    """fn on another stream than the current one: what it allocates belongs to the stream that it launches on.  The
    stream (an object, or a handle; 0 is the device's default stream) is of the device of fn's first argument."""
    at = getattr(args[0], "codes", args[0]) if args else None
    device = getattr(at, "device", None)
    if device is None or device.type != "cuda":
        return fn(*args)                         # which refuses them
    if not hasattr(stream, "cuda_stream"):
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError(f"stream: of {stream.device}, the tensors are on {device}")
    with torch.cuda.stream(stream):
        return fn(*args)


class MxRows:
    """Rows of `cols` columns in a microscaled format: uint8 codes [rows, .] and scales [rows, pitch] (None for
    bf16), and NVFP4's fp32 factor [1] (None = 1)."""

    __slots__ = ("fmt", "cols", "codes", "scales", "global_scale")

    def __init__(self, fmt, cols, codes, scales=None, global_scale=None):
        self.fmt = fmt
        self.cols = cols
        self.codes = codes
        self.scales = scales
        self.global_scale = global_scale

    @property
    def rows(self):
        return self.codes.shape[0]


class MxWeights:
    """Experts' matrices [num_experts, n_out, k] (two of them, gate and up, with swiglu) in the packed layout;
    alpha, alpha_up: fp32 [num_experts] factors of the products (None = 1)."""

    __slots__ = ("fmt", "num_experts", "n_out", "k", "packed", "alpha", "alpha_up", "swiglu")

    def __init__(self, fmt, num_experts, n_out, k, packed, alpha=None, alpha_up=None, swiglu=False):
        self.fmt = fmt
        self.num_experts = num_experts
        self.n_out = n_out
        self.k = k
        self.packed = packed
        self.alpha = alpha
        self.alpha_up = alpha_up
        self.swiglu = swiglu

    def struct(self) -> moe_mx_weights:
        """The C struct (its pointers are those of the tensors held here)."""
        ptr = [None if t is None else t.data_ptr() for t in (self.packed, self.alpha, self.alpha_up)]
        return moe_mx_weights(self.fmt, self.num_experts, self.n_out, self.k, bool(self.swiglu), *ptr)


def mx_rows(fmt, rows, cols, device="cuda", global_scale=None) -> MxRows:
    """Uninitialised rows."""
    if not 0 <= fmt <= 3 or cols <= 0 or cols & 31:
        raise MoeError(2, "moe_mx_code_bytes")
    codes = torch.empty((rows, cols * _BITS[fmt] >> 3), dtype=_U8, device=device)
    pitch = cols // _GROUP[fmt] + 15 & -16 if fmt else 0
    return MxRows(fmt, cols, codes, torch.empty((rows, pitch), dtype=_U8, device=device) if pitch else None, global_scale)


def mx_workspace(device="cuda"):
    """A workspace of the grouped products (its error word starts at zero)."""
    return torch.zeros(MOE_MX_PRODUCT_WORKSPACE, dtype=_U8, device=device)


def mx_get_error(device=None) -> int:
    """The first error (MOE_ERR_*) that the device recorded in calls without a workspace since the last time, MOE_OK if
    none; waits for the device.  (Calls with a workspace record theirs in it: moe_get_error.)"""
    torch.cuda.synchronize(device)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return _mx_torch.default_error()


def _check_rows(r: MxRows, like=None):
    """Rows that are what their format and width say (and what `like` is)."""
    want = mx_rows(r.fmt, r.codes.shape[0], r.cols, "meta")
    for name in ("codes", "scales"):
        t, w = getattr(r, name), getattr(want, name)
        if (t is None) != (w is None):
            raise ValueError(f"{name}: missing, or there without a use")
        if t is not None and (t.dtype != _U8 or t.shape != w.shape or not t.is_contiguous()
                              or t.device != r.codes.device):
            raise ValueError(f"{name}: expected contiguous uint8 {tuple(w.shape)} on {r.codes.device}")
    if like is not None and (r.fmt, r.cols, r.rows, r.codes.device) != (like.fmt, like.cols, like.rows, like.codes.device):
        raise ValueError("up: not like the first matrix")


def mx_pack(rows: MxRows, num_experts, up=None, alpha=None, alpha_up=None, stream=None) -> MxWeights:
    """Packed weights from rows [num_experts * n_out] of a format (up: the SwiGLU pair's second matrix)."""
    if stream is not None:
        return _on(stream, mx_pack, rows, num_experts, up, alpha, alpha_up)
    _check_rows(rows)
    if up is not None:
        _check_rows(up, rows)
    if num_experts < 1 or rows.rows % num_experts != 0:
        raise ValueError("rows: not a multiple of num_experts")
    w = MxWeights(rows.fmt, num_experts, rows.rows // num_experts, rows.cols, None, alpha, alpha_up, up is not None)
    nbytes = moe_mx_packed_bytes(w.struct())
    if nbytes == 0:
        raise MoeError(2, "moe_mx_packed_bytes")
    device = rows.codes.device
    for name, t in (("alpha", alpha), ("alpha_up", alpha_up)):
        if t is not None and (t.dtype != torch.float32 or t.numel() != num_experts or t.device != device):
            raise ValueError(f"{name}: expected {num_experts} fp32 values on {device}")
    if device.type != "cuda":
        raise ValueError("expected tensors on a CUDA device")
    w.packed = torch.empty(nbytes, dtype=_U8, device=device)
    with torch.cuda.device(device):
        moe_mx_pack_weights(w.struct(), rows.codes, rows.scales, up.codes if up else None, up.scales if up else None,
                            w.packed)
    return w


_mx_torch.setup(MxRows, MoeError, _on)
mx_quantise = _mx_torch.mx_quantise
mx_add_rmsnorm = _mx_torch.mx_add_rmsnorm
mx_dequantise = _mx_torch.mx_dequantise
mx_grouped_product = _mx_torch.mx_grouped_product
mx_grouped_swiglu = _mx_torch.mx_grouped_swiglu
mx_layer_forward = _mx_torch.mx_layer_forward
