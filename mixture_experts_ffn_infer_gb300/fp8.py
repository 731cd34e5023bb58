"""The router's and the FP8 operators on torch tensors (include/moe_router.h, include/moe_fp8.h).

The calls are in csrc/fp8_torch.cpp: each checks its tensors (ValueError), allocates what it returns and launches on the
current stream, or on `stream`; the library's own refusals raise MoeError.  None is recorded by autograd: gradients are
calls of their own (route_backward; the product of the transposed weights).  This module adds what they work on.
"""

from __future__ import annotations

import torch

from . import MoeError, moe_fp8_pack_weights, moe_fp8_packed_bytes, moe_fp8_scale_pitch, moe_fp8_weights
from .mx import _mx_torch, _on

_CODES = (torch.uint8, torch.float8_e4m3fn)


class Fp8Rows:
    """Rows of e4m3 codes [rows, cols] (as bytes or float8_e4m3fn) with one fp32 scale per 128 columns,
    [rows, moe_fp8_scale_pitch(cols)]."""

    __slots__ = ("codes", "scales")

    def __init__(self, codes, scales):
        self.codes = codes
        self.scales = scales

    @property
    def rows(self):
        return self.codes.shape[0]

    @property
    def cols(self):
        return self.codes.shape[1]


class Fp8Weights:
    """Experts' matrices [num_experts, n_out, k] of e4m3 codes in the packed layout, with one fp32 scale per 128 x 128
    block [num_experts, ceil(n_out / 128), ceil(k / 128)]."""

    __slots__ = ("num_experts", "n_out", "k", "packed", "scales")

    def __init__(self, num_experts, n_out, k, packed, scales):
        self.num_experts = num_experts
        self.n_out = n_out
        self.k = k
        self.packed = packed
        self.scales = scales

    def struct(self) -> moe_fp8_weights:
        """The C struct (its pointers are those of the tensors held here)."""
        ptr = [None if t is None else t.data_ptr() for t in (self.packed, self.scales)]
        return moe_fp8_weights(self.num_experts, self.n_out, self.k, *ptr)


def fp8_rows(rows, cols, device="cuda") -> Fp8Rows:
    """Uninitialised rows."""
    pitch = moe_fp8_scale_pitch(cols)
    if pitch == 0:
        raise MoeError(2, "moe_fp8_scale_pitch")
    return Fp8Rows(torch.empty((rows, cols), dtype=torch.uint8, device=device),
                   torch.empty((rows, pitch), dtype=torch.float32, device=device))


def fp8_pack(codes, scales, transpose=False, stream=None) -> Fp8Weights:
    """Packed weights from e4m3 codes [E, rows, cols] (a matrix [rows, cols]: one expert) and their blocks' scales
    [E, ceil(rows / 128), ceil(cols / 128)]: out = x W^T.  With transpose those of out = x W, by which the gradient of
    the rows goes back."""
    if stream is not None:
        return _on(stream, fp8_pack, codes, scales, transpose)
    if codes.dim() == 2 and scales.dim() == 2:
        codes, scales = codes[None], scales[None]
    if codes.dim() != 3 or codes.dtype not in _CODES or not codes.is_contiguous():
        raise ValueError("codes: expected contiguous e4m3 codes (as bytes or float8_e4m3fn) [E, rows, cols]")
    experts, rows, cols = codes.shape
    blocks = (experts, -(-rows // 128), -(-cols // 128))
    if scales.dtype != torch.float32 or tuple(scales.shape) != blocks or not scales.is_contiguous() \
            or scales.device != codes.device:
        raise ValueError(f"scales: expected contiguous fp32 {blocks} on {codes.device}")
    w = Fp8Weights(experts, *((cols, rows) if transpose else (rows, cols)), None, scales)
    if max(experts, rows, cols) >= 1 << 31:
        raise MoeError(2, "moe_fp8_packed_bytes")
    nbytes = moe_fp8_packed_bytes(w.struct())
    if nbytes == 0:
        raise MoeError(2, "moe_fp8_packed_bytes")
    device = codes.device
    if device.type != "cuda":
        raise ValueError("expected tensors on a CUDA device")
    w.packed = torch.empty(nbytes, dtype=torch.uint8, device=device)
    if transpose:
        w.scales = torch.empty((experts, blocks[2], blocks[1]), dtype=torch.float32, device=device)
    with torch.cuda.device(device):
        moe_fp8_pack_weights(w.struct(), codes, scales, transpose, w.packed, w.scales if transpose else None)
    return w


_mx_torch.fp8_setup(Fp8Rows)
fp8_quantise = _mx_torch.fp8_quantise
fp8_dequantise = _mx_torch.fp8_dequantise
fp8_grouped_product = _mx_torch.fp8_grouped_product
route = _mx_torch.route
balance_loss = _mx_torch.balance_loss
route_backward = _mx_torch.route_backward
