"""GB300 routed-expert forward of a Kimi K2 MoE block.

A thin ctypes binding over ``libmoe_ffn.so`` (declared in ``include/moe_ffn.h``).
The functions carry the C names and only marshal arguments: torch tensors are
passed by device pointer together with the current CUDA stream; every step of
the computation runs in the library's sm_103a kernels.  There is no fallback:
if the library is missing or cannot load, every call raises.

PyTorch supplies device memory and streams.  Convenience helpers
(``workspace``, ``infer``, ``layer_forward``, ``permute``) allocate outputs with
torch and then call the same entry points.
"""

from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_ffn.so")

MOE_TRACE_MAX = 16

STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE",
          4: "MOE_ERR_ROUTING", 5: "MOE_ERR_TIMEOUT", 6: "MOE_ERR_RANGE", 7: "MOE_ERR_CUDA"}
MOE_OK = 0


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}")
        self.status = status


class moe_dims(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("d_ff", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("act_scheme", ctypes.c_int32)]


MOE_ACT_EXACT = 0          # activations carried exactly as e4m3 split terms
MOE_ACT_FP8_DYNAMIC = 1    # per-128-feature e4m3 activations, scale amax / 448


MOE_LAYOUT_ROW_MAJOR = 0
MOE_LAYOUT_TILED = 1


class moe_weights(ctypes.Structure):
    _fields_ = [("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("s_gate", ctypes.c_void_p), ("s_up", ctypes.c_void_p), ("s_down", ctypes.c_void_p),
                ("layout", ctypes.c_int32)]


class moe_mx_weights(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("num_experts", ctypes.c_int32), ("n_out", ctypes.c_int32),
                ("k", ctypes.c_int32), ("swiglu", ctypes.c_int32), ("packed", ctypes.c_void_p),
                ("alpha", ctypes.c_void_p), ("alpha_up", ctypes.c_void_p)]


# microscaled formats (include/moe_mx.h)
MOE_MX_BF16, MOE_MX_MXFP8, MOE_MX_MXFP4, MOE_MX_NVFP4 = range(4)
MX_FORMATS = {"bf16": MOE_MX_BF16, "mxfp8": MOE_MX_MXFP8, "mxfp4": MOE_MX_MXFP4, "nvfp4": MOE_MX_NVFP4}
MOE_MX_OUT_BF16, MOE_MX_OUT_F16 = 0, 1
MOE_MX_PRODUCT_WORKSPACE = 256


class moe_trace(ctypes.Structure):
    _fields_ = [("events", ctypes.c_void_p * MOE_TRACE_MAX), ("n_events", ctypes.c_int32),
                ("n_recorded", ctypes.c_int32), ("labels", ctypes.c_char_p * MOE_TRACE_MAX),
                ("gemms_only", ctypes.c_int32), ("n_launched", ctypes.c_int32)]


_lib = None
_lock = threading.Lock()

_SIGS = {
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(moe_dims), ctypes.c_int64, ctypes.c_int32]),
    "moe_tiled_bytes": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]),
    "moe_permute_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(moe_dims), ctypes.c_int64]),
    "moe_pack_weights": (ctypes.c_int, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(moe_weights),
                                         ctypes.POINTER(moe_weights), ctypes.c_void_p]),
    "moe_permute": (ctypes.c_int, [ctypes.POINTER(moe_dims), ctypes.c_int64] + [ctypes.c_void_p] * 5
                    + [ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "moe_experts_forward": (ctypes.c_int, [ctypes.POINTER(moe_dims), ctypes.c_int64] + [ctypes.c_void_p] * 4
                            + [ctypes.POINTER(moe_weights), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                               ctypes.c_void_p]),
    "moe_combine": (ctypes.c_int, [ctypes.POINTER(moe_dims), ctypes.c_int64] + [ctypes.c_void_p] * 4
                    + [ctypes.c_int32, ctypes.c_void_p]),
    "moe_infer": (ctypes.c_int, [ctypes.POINTER(moe_dims), ctypes.c_int64] + [ctypes.c_void_p] * 3
                  + [ctypes.POINTER(moe_weights), ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                     ctypes.c_size_t, ctypes.c_void_p, ctypes.POINTER(moe_trace)]),
    "moe_layer_forward": (ctypes.c_int, [ctypes.POINTER(moe_dims), ctypes.c_int64, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.POINTER(moe_weights), ctypes.POINTER(moe_weights), ctypes.c_int32,
                                         ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t,
                                         ctypes.c_void_p, ctypes.POINTER(moe_trace)]),
    "moe_mlp_forward": (ctypes.c_int, [ctypes.POINTER(moe_dims), ctypes.c_int64, ctypes.c_void_p,
                                       ctypes.POINTER(moe_weights), ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                       ctypes.c_size_t, ctypes.c_void_p]),
    "moe_infer_static": (ctypes.c_int, [ctypes.POINTER(moe_dims), ctypes.c_int64] + [ctypes.c_void_p] * 3
                         + [ctypes.POINTER(moe_weights), ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p]),
    "moe_ep_plan_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(moe_dims), ctypes.c_int64]),
    "moe_ep_dispatch_plan": (ctypes.c_int, [ctypes.POINTER(moe_dims), ctypes.c_int32, ctypes.c_int64]
                             + [ctypes.c_void_p] * 4 + [ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t,
                                                        ctypes.c_void_p]),
    "moe_ep_gather": (ctypes.c_int, [ctypes.POINTER(moe_dims), ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]),
    "moe_ep_regroup_workspace_size": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int32]),
    "moe_ep_regroup": (ctypes.c_int, [ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int64,
                                      ctypes.c_int64] + [ctypes.c_void_p] * 5 + [ctypes.c_size_t, ctypes.c_void_p]),
    "moe_ep_experts_forward": (ctypes.c_int, [ctypes.POINTER(moe_dims), ctypes.c_int64] + [ctypes.c_void_p] * 4
                               + [ctypes.POINTER(moe_weights), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                  ctypes.c_void_p]),
    "moe_ep_combine": (ctypes.c_int, [ctypes.POINTER(moe_dims), ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                      ctypes.c_void_p]),
    "moe_mx_code_bytes": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int64]),
    "moe_mx_scale_pitch": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int64]),
    "moe_mx_quantise": (ctypes.c_int, [ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                       ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64]
                        + [ctypes.c_void_p] * 3),
    "moe_mx_add_rmsnorm": (ctypes.c_int, [ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                          ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                          ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_int64] + [ctypes.c_void_p] * 4),
    "moe_mx_dequantise": (ctypes.c_int, [ctypes.c_int32, ctypes.c_int64, ctypes.c_int32] + [ctypes.c_void_p] * 4
                          + [ctypes.c_int64, ctypes.c_void_p]),
    "moe_mx_packed_bytes": (ctypes.c_size_t, [ctypes.POINTER(moe_mx_weights)]),
    "moe_mx_pack_weights": (ctypes.c_int, [ctypes.POINTER(moe_mx_weights)] + [ctypes.c_void_p] * 6),
    "moe_mx_grouped_product": (ctypes.c_int, [ctypes.POINTER(moe_mx_weights), ctypes.c_int64] + [ctypes.c_void_p] * 5
                               + [ctypes.c_int32, ctypes.c_int64, ctypes.c_int64] + [ctypes.c_void_p] * 3
                               + [ctypes.c_size_t, ctypes.c_void_p]),
    "moe_mx_grouped_swiglu": (ctypes.c_int, [ctypes.POINTER(moe_mx_weights), ctypes.c_int64] + [ctypes.c_void_p] * 8
                              + [ctypes.c_size_t, ctypes.c_void_p]),
    "moe_mx_layer_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(moe_mx_weights), ctypes.POINTER(moe_mx_weights),
                                                      ctypes.c_int32, ctypes.c_int64]),
    "moe_mx_layer_forward": (ctypes.c_int, [ctypes.POINTER(moe_mx_weights), ctypes.POINTER(moe_mx_weights),
                                            ctypes.c_int32, ctypes.c_int64] + [ctypes.c_void_p] * 3
                             + [ctypes.c_float] + [ctypes.c_void_p] * 6
                             + [ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "moe_check_bounded_wait": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "moe_get_error": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
}

MOE_STATIC_SCRATCH_BYTES = 8 << 20


def load_library(path: Optional[str] = None):
    """Load the CUDA library (raises if it is absent: there is no other implementation)."""
    global _lib
    with _lock:
        if _lib is None:
            p = path or LIB_PATH
            if not os.path.exists(p):
                raise RuntimeError(f"{p} is missing; build it with `python -m mixture_experts_ffn_infer_gb300.build`")
            L = ctypes.CDLL(p)
            for name, (res, args) in _SIGS.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


def exported_symbols():
    return list(_SIGS)


# ---------------------------------------------------------------- marshalling helpers

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _addr(t):
    return None if t is None else t.data_ptr()


def _raw_stream(stream, t):
    """The stream's handle; by default that of the current stream of t's device (the lookup that torch's own stream
    object wraps: a fifth of its cost)."""
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(t.get_device()) if t.is_cuda else None
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where)


def dims(d: int, d_ff: int, num_experts: int, top_k: int, act_scheme: int = MOE_ACT_EXACT) -> moe_dims:
    return moe_dims(d, d_ff, num_experts, top_k, act_scheme)


def weights(bank) -> moe_weights:
    """moe_weights from an object with w_gate/w_up/w_down/s_gate/s_up/s_down device tensors
    (and an optional ``layout`` attribute, default row-major)."""
    return moe_weights(*((t.data_ptr() if t is not None else None) for t in (bank.w_gate, bank.w_up, bank.w_down,
                                                                              bank.s_gate, bank.s_up, bank.s_down)),
                       int(getattr(bank, "layout", MOE_LAYOUT_ROW_MAJOR)))


# ---------------------------------------------------------------- C entry points (same names)

def moe_status_string(status: int) -> str:
    return load_library().moe_status_string(status).decode()


def moe_workspace_size(dm: moe_dims, n_tokens: int, d_ff_shared: int = 0) -> int:
    return load_library().moe_workspace_size(ctypes.byref(dm), n_tokens, d_ff_shared)


def moe_permute_workspace_size(dm: moe_dims, n_tokens: int) -> int:
    return load_library().moe_permute_workspace_size(ctypes.byref(dm), n_tokens)


def moe_tiled_bytes(which: int, num_experts: int, d: int, d_ff: int) -> int:
    return load_library().moe_tiled_bytes(which, num_experts, d, d_ff)


def moe_pack_weights(num_experts, d, d_ff, src: moe_weights, dst: moe_weights, stream=None):
    st = load_library().moe_pack_weights(num_experts, d, d_ff, ctypes.byref(src), ctypes.byref(dst),
                                         _stream(stream))
    _check(st, "moe_pack_weights")


def moe_permute(dm, n_tokens, topk_ids, tokens_per_expert, expert_offsets, sorted_pos, inv_pos, ws,
                validate=False, stream=None):
    st = load_library().moe_permute(ctypes.byref(dm), n_tokens, _ptr(topk_ids), _ptr(tokens_per_expert),
                                    _ptr(expert_offsets), _ptr(sorted_pos), _ptr(inv_pos), int(bool(validate)),
                                    _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "moe_permute")


def moe_experts_forward(dm, n_tokens, x, topk_weight, expert_offsets, sorted_pos, w: moe_weights, rows, ws,
                        stream=None):
    st = load_library().moe_experts_forward(ctypes.byref(dm), n_tokens, _ptr(x), _ptr(topk_weight),
                                            _ptr(expert_offsets), _ptr(sorted_pos), ctypes.byref(w), _ptr(rows),
                                            _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "moe_experts_forward")


def moe_combine(dm, n_tokens, rows, shared, residual, out, out_is_fp32=False, stream=None):
    st = load_library().moe_combine(ctypes.byref(dm), n_tokens, _ptr(rows), _ptr(shared), _ptr(residual), _ptr(out),
                                    int(bool(out_is_fp32)), _stream(stream))
    _check(st, "moe_combine")


def moe_infer(dm, n_tokens, x, topk_ids, topk_weight, w: moe_weights, out, ws, out_is_fp32=False, stream=None,
              trace: Optional[moe_trace] = None):
    st = load_library().moe_infer(ctypes.byref(dm), n_tokens, _ptr(x), _ptr(topk_ids), _ptr(topk_weight),
                                  ctypes.byref(w), _ptr(out), int(bool(out_is_fp32)), _ptr(ws),
                                  ws.numel() * ws.element_size(), _stream(stream),
                                  ctypes.byref(trace) if trace is not None else None)
    _check(st, "moe_infer")


def moe_mlp_forward(dm, n_tokens, x, w: moe_weights, out, ws, out_is_fp32=False, stream=None):
    st = load_library().moe_mlp_forward(ctypes.byref(dm), n_tokens, _ptr(x), ctypes.byref(w), _ptr(out),
                                        int(bool(out_is_fp32)), _ptr(ws), ws.numel() * ws.element_size(),
                                        _stream(stream))
    _check(st, "moe_mlp_forward")


def moe_layer_forward(dm, n_tokens, hidden, gain, eps, topk_ids, topk_weight, routed: moe_weights,
                      shared: Optional[moe_weights], d_ff_shared, out, ws, out_is_fp32=False, stream=None,
                      trace: Optional[moe_trace] = None):
    st = load_library().moe_layer_forward(ctypes.byref(dm), n_tokens, _ptr(hidden), _ptr(gain), float(eps),
                                          _ptr(topk_ids), _ptr(topk_weight), ctypes.byref(routed),
                                          ctypes.byref(shared) if shared is not None else None, int(d_ff_shared),
                                          _ptr(out), int(bool(out_is_fp32)), _ptr(ws),
                                          ws.numel() * ws.element_size(), _stream(stream),
                                          ctypes.byref(trace) if trace is not None else None)
    _check(st, "moe_layer_forward")


def moe_infer_static(dm, n_tokens, x, topk_ids, topk_weight, w: moe_weights, out, out_is_fp32=False, stream=None):
    """moe_infer on the library's built-in scratch (no workspace argument)."""
    st = load_library().moe_infer_static(ctypes.byref(dm), n_tokens, _ptr(x), _ptr(topk_ids), _ptr(topk_weight),
                                         ctypes.byref(w), _ptr(out), int(bool(out_is_fp32)), _stream(stream))
    _check(st, "moe_infer_static")


def moe_ep_plan_workspace_size(dm: moe_dims, n_tokens: int) -> int:
    return load_library().moe_ep_plan_workspace_size(ctypes.byref(dm), n_tokens)


def moe_ep_dispatch_plan(dm, ep_size, n_tokens, topk_ids, tokens_per_expert, send_counts, tok_slot, capacity, ws,
                         stream=None):
    st = load_library().moe_ep_dispatch_plan(ctypes.byref(dm), ep_size, n_tokens, _ptr(topk_ids),
                                             _ptr(tokens_per_expert), _ptr(send_counts), _ptr(tok_slot), capacity,
                                             _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "moe_ep_dispatch_plan")


def moe_ep_gather(dm, n_tokens, x, tok_slot, n_slots, send_rows, stream=None):
    st = load_library().moe_ep_gather(ctypes.byref(dm), n_tokens, _ptr(x), _ptr(tok_slot), n_slots, _ptr(send_rows),
                                      _stream(stream))
    _check(st, "moe_ep_gather")


def moe_ep_regroup_workspace_size(experts_per_rank: int, ep_size: int) -> int:
    return load_library().moe_ep_regroup_workspace_size(experts_per_rank, ep_size)


def moe_ep_regroup(experts_per_rank, ep_size, recv_counts, capacity, n_slots, local_counts, local_offsets, row_pos,
                   pos_row, ws, stream=None):
    st = load_library().moe_ep_regroup(experts_per_rank, ep_size, _ptr(recv_counts), capacity, n_slots,
                                       _ptr(local_counts), _ptr(local_offsets), _ptr(row_pos), _ptr(pos_row),
                                       _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "moe_ep_regroup")


def moe_ep_experts_forward(dm, n_slots, recv_rows, local_offsets, row_pos, pos_row, w: moe_weights, out_rows, ws,
                           stream=None):
    st = load_library().moe_ep_experts_forward(ctypes.byref(dm), n_slots, _ptr(recv_rows), _ptr(local_offsets),
                                               _ptr(row_pos), _ptr(pos_row), ctypes.byref(w), _ptr(out_rows),
                                               _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "moe_ep_experts_forward")


def moe_ep_combine(dm, n_tokens, back_rows, tok_slot, n_slots, topk_weight, out, out_is_fp32=False, stream=None):
    st = load_library().moe_ep_combine(ctypes.byref(dm), n_tokens, _ptr(back_rows), _ptr(tok_slot), n_slots,
                                       _ptr(topk_weight), _ptr(out), int(bool(out_is_fp32)), _stream(stream))
    _check(st, "moe_ep_combine")


def moe_check_bounded_wait(ws, stream=None):
    st = load_library().moe_check_bounded_wait(_ptr(ws), _stream(stream))
    _check(st, "moe_check_bounded_wait")


def moe_get_error(ws, stream=None) -> int:
    return load_library().moe_get_error(_ptr(ws), _stream(stream))


# microscaled formats

def moe_mx_code_bytes(fmt: int, cols: int) -> int:
    return load_library().moe_mx_code_bytes(fmt, cols)


def moe_mx_scale_pitch(fmt: int, cols: int) -> int:
    return load_library().moe_mx_scale_pitch(fmt, cols)


def moe_mx_quantise(fmt, n, k, d, x, x_ld, positions, global_scale, out_rows, codes, scales, stream=None):
    st = (_lib or load_library()).moe_mx_quantise(
        fmt, n, k, d, x.data_ptr(), x_ld, _addr(positions), _addr(global_scale), out_rows, codes.data_ptr(),
        _addr(scales), _raw_stream(stream, x))
    if st:
        raise MoeError(st, "moe_mx_quantise")


def moe_mx_add_rmsnorm(fmt, n, k, d, x, x_ld, residual, r_ld, gain, eps, positions, global_scale, out_rows, sum_out,
                       codes, scales, stream=None):
    st = (_lib or load_library()).moe_mx_add_rmsnorm(
        fmt, n, k, d, x.data_ptr(), x_ld, _addr(residual), r_ld, gain.data_ptr(), eps, _addr(positions),
        _addr(global_scale), out_rows, _addr(sum_out), codes.data_ptr(), _addr(scales), _raw_stream(stream, x))
    if st:
        raise MoeError(st, "moe_mx_add_rmsnorm")


def moe_mx_dequantise(fmt, rows, d, codes, scales, global_scale, out, out_ld, stream=None):
    st = (_lib or load_library()).moe_mx_dequantise(fmt, rows, d, codes.data_ptr(), _addr(scales), _addr(global_scale),
                                                    out.data_ptr(), out_ld, _raw_stream(stream, out))
    if st:
        raise MoeError(st, "moe_mx_dequantise")


def moe_mx_packed_bytes(w: moe_mx_weights) -> int:
    return load_library().moe_mx_packed_bytes(ctypes.byref(w))


def moe_mx_pack_weights(w: moe_mx_weights, codes, scales, codes_up, scales_up, packed, stream=None):
    st = load_library().moe_mx_pack_weights(ctypes.byref(w), _ptr(codes), _ptr(scales), _ptr(codes_up),
                                            _ptr(scales_up), _ptr(packed), _raw_stream(stream, packed))
    _check(st, "moe_mx_pack_weights")


def moe_mx_grouped_product(w: moe_mx_weights, rows, x_codes, x_scales, x_global, expert_offsets, out, out_type,
                           out_rows, out_ld, out_pos, row_weight, ws, stream=None):
    st = (_lib or load_library()).moe_mx_grouped_product(
        w, rows, x_codes.data_ptr(), _addr(x_scales), _addr(x_global), expert_offsets.data_ptr(), out.data_ptr(),
        out_type, out_rows, out_ld, _addr(out_pos), _addr(row_weight), ws.data_ptr(), ws.nbytes,
        _raw_stream(stream, out))
    if st:
        raise MoeError(st, "moe_mx_grouped_product")


def moe_mx_grouped_swiglu(w: moe_mx_weights, rows, x_codes, x_scales, x_global, expert_offsets, h_global, h_codes,
                          h_scales, ws, stream=None):
    st = (_lib or load_library()).moe_mx_grouped_swiglu(
        w, rows, x_codes.data_ptr(), _addr(x_scales), _addr(x_global), expert_offsets.data_ptr(), _addr(h_global),
        h_codes.data_ptr(), _addr(h_scales), ws.data_ptr(), ws.nbytes, _raw_stream(stream, h_codes))
    if st:
        raise MoeError(st, "moe_mx_grouped_swiglu")


def moe_mx_layer_workspace_size(gate_up: moe_mx_weights, down: moe_mx_weights, top_k: int, n_tokens: int) -> int:
    return load_library().moe_mx_layer_workspace_size(ctypes.byref(gate_up), ctypes.byref(down), top_k, n_tokens)


def moe_mx_layer_forward(gate_up: moe_mx_weights, down: moe_mx_weights, top_k, n_tokens, x, residual, gain, eps,
                         topk_ids, topk_weight, x_global, h_global, sum_out, out, ws, out_is_fp32=False, stream=None):
    st = (_lib or load_library()).moe_mx_layer_forward(
        gate_up, down, top_k, n_tokens, x.data_ptr(), _addr(residual), _addr(gain), eps, topk_ids.data_ptr(),
        topk_weight.data_ptr(), _addr(x_global), _addr(h_global), _addr(sum_out), out.data_ptr(), bool(out_is_fp32),
        ws.data_ptr(), ws.nbytes, _raw_stream(stream, x))
    if st:
        raise MoeError(st, "moe_mx_layer_forward")


# ---------------------------------------------------------------- allocating conveniences

class TiledBank:
    """A bank whose e4m3 codes are in the tiled streaming layout: w_gate holds gate and up
    interleaved, w_up is None, w_down holds down row blocks in pairs (flat uint8 tensors)."""

    layout = MOE_LAYOUT_TILED

    def __init__(self, w_gate, w_down, s_gate, s_up, s_down, num_experts, d_ff, d):
        self.w_gate, self.w_up, self.w_down = w_gate, None, w_down
        self.s_gate, self.s_up, self.s_down = s_gate, s_up, s_down
        self.num_experts, self.d_ff, self.d = num_experts, d_ff, d


def bank_sizes(bank):
    """(num_experts, d_ff, d) of a row-major or tiled bank."""
    if isinstance(bank, TiledBank):
        return bank.num_experts, bank.d_ff, bank.d
    return tuple(bank.w_gate.shape)


def pack_bank(bank, stream=None) -> TiledBank:
    """Tiled copy of a row-major bank's codes (scales shared with the source)."""
    import torch
    E, d_ff, d = bank.w_gate.shape
    dev = bank.w_gate.device
    gu = torch.empty(moe_tiled_bytes(0, E, d, d_ff), dtype=torch.uint8, device=dev)
    dn = torch.empty(moe_tiled_bytes(2, E, d, d_ff), dtype=torch.uint8, device=dev)
    out = TiledBank(gu, dn, bank.s_gate, bank.s_up, bank.s_down, E, d_ff, d)
    moe_pack_weights(E, d, d_ff, weights(bank), weights(out), stream)
    return out


def workspace(dm: moe_dims, n_tokens: int, d_ff_shared: int = 0, device="cuda"):
    import torch
    nbytes = moe_workspace_size(dm, n_tokens, d_ff_shared)
    if nbytes == 0:
        raise MoeError(2, "moe_workspace_size")
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def permute(topk_ids, num_experts: int, ws=None, validate=False, stream=None):
    """-> (tokens_per_expert, expert_offsets, sorted_pos, inv_pos) int32 device tensors."""
    import torch
    n, k = topk_ids.shape
    dm = moe_dims(128, 128, num_experts, k)
    if ws is None:
        nbytes = load_library().moe_permute_workspace_size(ctypes.byref(dm), n)
        if nbytes == 0:
            raise MoeError(2, "moe_permute_workspace_size")
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=topk_ids.device)
    dev = topk_ids.device
    counts = torch.empty(num_experts, dtype=torch.int32, device=dev)
    offsets = torch.empty(num_experts + 1, dtype=torch.int32, device=dev)
    sp = torch.empty(max(n * k, 1), dtype=torch.int32, device=dev)
    ip = torch.empty(max(n * k, 1), dtype=torch.int32, device=dev)
    moe_permute(dm, n, topk_ids, counts, offsets, sp, ip, ws, validate=validate, stream=stream)
    return counts, offsets, sp[: n * k], ip[: n * k]


def infer(x, topk_ids, topk_weight, bank, ws=None, out_is_fp32=False, stream=None, act_scheme=MOE_ACT_EXACT):
    import torch
    n, d = x.shape
    E, d_ff, _ = bank_sizes(bank)
    dm = moe_dims(d, d_ff, E, topk_ids.shape[1], act_scheme)
    if ws is None:
        ws = workspace(dm, n, 0, x.device)
    out = torch.empty(n, d, dtype=torch.float32 if out_is_fp32 else torch.bfloat16, device=x.device)
    moe_infer(dm, n, x, topk_ids, topk_weight, weights(bank), out, ws, out_is_fp32, stream)
    return out


def mlp_forward(x, bank, ws=None, out_is_fp32=False, stream=None, act_scheme=MOE_ACT_EXACT):
    """One SwiGLU MLP (a bank with E = 1) on every row of x."""
    import torch
    n, d = x.shape
    E, d_ff, _ = bank_sizes(bank)
    dm = moe_dims(d, d_ff, E, 1, act_scheme)
    if ws is None:
        ws = workspace(dm, n, 0, x.device)
    out = torch.empty(n, d, dtype=torch.float32 if out_is_fp32 else torch.bfloat16, device=x.device)
    moe_mlp_forward(dm, n, x, weights(bank), out, ws, out_is_fp32, stream)
    return out


def layer_forward(hidden, gain, eps, topk_ids, topk_weight, bank, shared=None, ws=None, out_is_fp32=False,
                  stream=None, act_scheme=MOE_ACT_EXACT):
    import torch
    n, d = hidden.shape
    E, d_ff, _ = bank_sizes(bank)
    dm = moe_dims(d, d_ff, E, topk_ids.shape[1], act_scheme)
    dff_sh = bank_sizes(shared)[1] if shared is not None else 0
    if ws is None:
        ws = workspace(dm, n, dff_sh, hidden.device)
    out = torch.empty(n, d, dtype=torch.float32 if out_is_fp32 else torch.bfloat16, device=hidden.device)
    moe_layer_forward(dm, n, hidden, gain, eps, topk_ids, topk_weight, weights(bank),
                      weights(shared) if shared is not None else None, dff_sh, out, ws, out_is_fp32, stream)
    return out


# ---------------------------------------------------------------- microscaled formats
# A decode step's call is a few microseconds of GPU time: the checks below are written to cost little on the host
# (no message is formatted, and no library call made, for arguments that pass).

_MX_BITS = (16, 8, 4, 4)
_MX_GROUP = (0, 32, 32, 16)


def _mx_width(fmt, cols):
    """(code bytes, scale pitch) of a row, as moe_mx_code_bytes and moe_mx_scale_pitch give them."""
    if not 0 <= fmt <= 3 or cols <= 0 or cols & 31:
        raise MoeError(2, "moe_mx_code_bytes")
    return cols * _MX_BITS[fmt] >> 3, (-(-(cols // _MX_GROUP[fmt]) // 16) * 16 if fmt else 0)


class MxRows:
    """Rows of `cols` columns in a microscaled format: uint8 codes [rows, .] and scales [rows, pitch] (None for
    bf16), and NVFP4's fp32 factor [1] (None = 1)."""

    __slots__ = ("fmt", "cols", "codes", "scales", "global_scale")

    def __init__(self, fmt, cols, codes, scales=None, global_scale=None):
        self.fmt, self.cols, self.codes, self.scales, self.global_scale = fmt, cols, codes, scales, global_scale

    @property
    def rows(self):
        return self.codes.shape[0]


class MxWeights:
    """Experts' matrices [num_experts, n_out, k] (two of them, gate and up, with swiglu) in the packed layout;
    alpha, alpha_up: fp32 [num_experts] factors of the products (None = 1)."""

    def __init__(self, fmt, num_experts, n_out, k, packed, alpha=None, alpha_up=None, swiglu=False):
        self.fmt, self.num_experts, self.n_out, self.k = fmt, num_experts, n_out, k
        self.packed, self.alpha, self.alpha_up, self.swiglu = packed, alpha, alpha_up, bool(swiglu)

    def __setattr__(self, name, value):
        self.__dict__[name] = value
        self.__dict__["_checked"] = None       # the struct below is of the attributes as they were

    def struct(self) -> moe_mx_weights:
        return moe_mx_weights(self.fmt, self.num_experts, self.n_out, self.k, int(self.swiglu), _addr(self.packed),
                              _addr(self.alpha), _addr(self.alpha_up))

    def checked(self, dev):
        """The struct, once the tensors have been checked against it."""
        got = self._checked
        if got is None or got[1] != dev:
            st = self.struct()
            nbytes = moe_mx_packed_bytes(st)
            if nbytes == 0:
                raise MoeError(2, "moe_mx_packed_bytes")
            if self.packed.nbytes != nbytes or not self.packed.is_contiguous() or self.packed.get_device() != dev:
                raise ValueError(f"packed: expected {nbytes} contiguous bytes on device {dev}")
            _mx_scalar(self.alpha, "alpha", dev, self.num_experts)
            _mx_scalar(self.alpha_up, "alpha_up", dev, self.num_experts)
            got = self.__dict__["_checked"] = (st, dev)
        return got[0]


def _on_stream(fn):
    """What the call allocates (results, a workspace of its own) belongs to the stream that it launches on."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        import torch
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream))
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _mx_tensor(t, name, dtype, shape, dev):
    """The tensor that a library call reads through its pointer: dense, on the device, of this type and shape."""
    if t.dtype != dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor {tuple(shape)} on device {dev}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")


def _mx_strided(t, name, shape, dev):
    """bf16 rows: the row stride in elements (that of a single row is not used, and torch may report any)."""
    import torch
    if t.dtype != torch.bfloat16 or t.shape != shape or t.get_device() != dev or t.stride(1) != 1:
        raise ValueError(f"{name}: expected bf16 rows {tuple(shape)} on device {dev}, got {t.dtype} {tuple(t.shape)} "
                         f"on {t.device}")
    ld = t.stride(0)
    return ld if shape[0] > 1 else max(ld, shape[1])


def _mx_scalar(t, name, dev, count=1):
    if t is not None:
        import torch
        if t.dtype != torch.float32 or t.numel() != count or t.get_device() != dev or not t.is_contiguous():
            raise ValueError(f"{name}: expected {count} fp32 value(s) on device {dev}")


def _mx_check_rows(r: MxRows, dev):
    import torch
    codes = r.codes
    n = codes.shape[0]
    cb, pitch = _mx_width(r.fmt, r.cols)
    _mx_tensor(codes, "codes", torch.uint8, (n, cb), dev)
    if pitch:
        if r.scales is None:
            raise ValueError("scales: missing")
        _mx_tensor(r.scales, "scales", torch.uint8, (n, pitch), dev)
    if r.global_scale is not None:
        _mx_scalar(r.global_scale, "global_scale", dev)
    return n


def mx_rows(fmt, rows, cols, device="cuda", global_scale=None) -> MxRows:
    """Uninitialised rows."""
    import torch
    cb, pitch = _mx_width(fmt, cols)
    codes = torch.empty((rows, cb), dtype=torch.uint8, device=device)
    return MxRows(fmt, cols, codes, torch.empty((rows, pitch), dtype=torch.uint8, device=device) if pitch else None,
                  global_scale)


def _mx_out(fmt, n, d, positions, out_rows, global_scale, out, device, dev):
    """(k, rows, the rows to write) of a call that writes n tokens' rows."""
    import torch
    if global_scale is not None:
        _mx_scalar(global_scale, "global_scale", dev)
    k = 1
    if positions is not None:
        k = positions.shape[1] if positions.dim() == 2 else 0
        _mx_tensor(positions, "positions", torch.int32, (n, k), dev)
    if out is None:
        m = n * k if out_rows is None else out_rows
        return k, m, mx_rows(fmt, m, d, device, global_scale)
    if out.fmt != fmt or out.cols != d:
        raise ValueError("out: of another format or width")
    m = _mx_check_rows(out, dev)
    out.global_scale = global_scale
    return k, m, out


@_on_stream
def mx_quantise(x, fmt, positions=None, out_rows=None, global_scale=None, out: Optional[MxRows] = None) -> MxRows:
    """bf16 rows x [n, d] (any row stride that is a multiple of 8) into a format; row t goes to each of positions[t]
    (int32 [n, k], default its own place) of `out` (out_rows rows, default n * k)."""
    n, d = x.shape
    dev = x.get_device()
    ld = _mx_strided(x, "x", (n, d), dev)
    k, m, out = _mx_out(fmt, n, d, positions, out_rows, global_scale, out, x.device, dev)
    moe_mx_quantise(fmt, n, k, d, x, ld, positions, global_scale, m, out.codes, out.scales)
    return out


@_on_stream
def mx_add_rmsnorm(x, residual, gain, eps, fmt, positions=None, out_rows=None, global_scale=None, sum_out=None,
                   out: Optional[MxRows] = None):
    """(rows of the normalised sum, the sum): sum = bf16(x + residual) (residual may be None), rows = Q(rmsnorm(sum))
    written as by mx_quantise.  sum_out may be x or residual."""
    import torch
    n, d = shape = x.shape
    dev = x.get_device()
    ld = _mx_strided(x, "x", shape, dev)
    r_ld = None if residual is None else _mx_strided(residual, "residual", shape, dev)
    _mx_tensor(gain, "gain", torch.bfloat16, (d,), dev)
    if sum_out is None:
        sum_out = torch.empty_strided(shape, (r_ld or d, 1), dtype=torch.bfloat16, device=x.device)
        r_ld = r_ld or d
    else:
        s_ld = _mx_strided(sum_out, "sum_out", shape, dev)
        if r_ld is not None and s_ld != r_ld and n > 1:
            raise ValueError("sum_out: its row stride differs from residual's")
        r_ld = r_ld or s_ld
    k, m, out = _mx_out(fmt, n, d, positions, out_rows, global_scale, out, x.device, dev)
    moe_mx_add_rmsnorm(fmt, n, k, d, x, ld, residual, r_ld, gain, eps, positions, global_scale, m, sum_out, out.codes,
                       out.scales)
    return out, sum_out


@_on_stream
def mx_dequantise(r: MxRows, out=None):
    """bf16 values of rows."""
    import torch
    dev = r.codes.get_device()
    n, d = _mx_check_rows(r, dev), r.cols
    if out is None:
        out, ld = torch.empty((n, d), dtype=torch.bfloat16, device=r.codes.device), d
    else:
        ld = _mx_strided(out, "out", (n, d), dev)
    moe_mx_dequantise(r.fmt, n, d, r.codes, r.scales, r.global_scale, out, ld)
    return out


@_on_stream
def mx_pack(rows: MxRows, num_experts, up: Optional[MxRows] = None, alpha=None, alpha_up=None) -> MxWeights:
    """Packed weights from rows [num_experts * n_out] of a format (up: the SwiGLU pair's second matrix)."""
    import torch
    dev = rows.codes.get_device()
    n = _mx_check_rows(rows, dev)
    if num_experts < 1 or n % num_experts != 0:
        raise ValueError("rows: not a multiple of num_experts")
    if up is not None:
        if (up.fmt, up.cols) != (rows.fmt, rows.cols) or _mx_check_rows(up, dev) != n:
            raise ValueError("up: not like the first matrix")
    w = MxWeights(rows.fmt, num_experts, n // num_experts, rows.cols, None, alpha, alpha_up, up is not None)
    nbytes = moe_mx_packed_bytes(w.struct())
    if nbytes == 0:
        raise MoeError(2, "moe_mx_packed_bytes")
    w.packed = torch.empty(nbytes, dtype=torch.uint8, device=rows.codes.device)
    moe_mx_pack_weights(w.checked(dev), rows.codes, rows.scales, up.codes if up else None, up.scales if up else None,
                        w.packed)
    return w


def _mx_operands(x: MxRows, w: MxWeights, offsets):
    """(device, rows, the weights' struct) of checked operands."""
    import torch
    dev = x.codes.get_device()
    n = _mx_check_rows(x, dev)
    st = w.checked(dev)
    if x.fmt != w.fmt or x.cols != w.k:
        raise ValueError("x: of another format or width than the weights")
    _mx_tensor(offsets, "offsets", torch.int32, (w.num_experts + 1,), dev)
    return dev, n, st


def mx_workspace(device="cuda"):
    import torch
    return torch.zeros(MOE_MX_PRODUCT_WORKSPACE, dtype=torch.uint8, device=device)


@_on_stream
def mx_grouped_product(x: MxRows, w: MxWeights, offsets, out=None, out_pos=None, row_weight=None, ws=None,
                       out_type=MOE_MX_OUT_BF16):
    """out[p(r)] = row_weight[p(r)] * x[r] W_e^T for the rows offsets[e] .. offsets[e + 1] - 1 of each expert e;
    p = out_pos (int32 [rows], default r)."""
    import torch
    dev, n, st = _mx_operands(x, w, offsets)
    dtype = torch.float16 if out_type == MOE_MX_OUT_F16 else torch.bfloat16
    cols = w.n_out
    if out is None:
        out, out_rows, ld = torch.empty((n, cols), dtype=dtype, device=x.codes.device), n, cols
    else:
        if out.dtype != dtype or out.dim() != 2 or out.shape[1] != cols or out.get_device() != dev or (
                cols > 1 and out.stride(1) != 1):
            raise ValueError("out: of another type, width or device")
        out_rows, ld = out.shape[0], max(out.stride(0), cols) if out.shape[0] < 2 else out.stride(0)
    if out_pos is not None:
        _mx_tensor(out_pos, "out_pos", torch.int32, (n,), dev)
    if row_weight is not None:
        _mx_scalar(row_weight, "row_weight", dev, out_rows)
    if ws is None:
        ws = mx_workspace(x.codes.device)
    moe_mx_grouped_product(st, n, x.codes, x.scales, x.global_scale, offsets, out, out_type, out_rows, ld, out_pos,
                           row_weight, ws)
    return out


@_on_stream
def mx_grouped_swiglu(x: MxRows, w: MxWeights, offsets, h_global=None, out: Optional[MxRows] = None, ws=None) -> MxRows:
    """Rows of silu(x Wg_e^T) * (x Wu_e^T) in the format of x."""
    dev, n, st = _mx_operands(x, w, offsets)
    _, m, out = _mx_out(w.fmt, n, w.n_out, None, None, h_global, out, x.codes.device, dev)
    if m != n:
        raise ValueError("out: of another number of rows")
    if ws is None:
        ws = mx_workspace(x.codes.device)
    moe_mx_grouped_swiglu(st, n, x.codes, x.scales, x.global_scale, offsets, h_global, out.codes, out.scales, ws)
    return out


@_on_stream
def mx_layer_forward(x, residual, gain, eps, topk_ids, topk_weight, gate_up: MxWeights, down: MxWeights,
                     x_global=None, h_global=None, ws=None, out_is_fp32=False):
    """The MoE block on microscaled experts: (sum, out) with sum = bf16(x + residual) and out = sum + the routed
    experts on rmsnorm(sum); with gain None (and residual None) (None, the routed experts on x)."""
    import torch
    n, d = shape = x.shape
    dev = x.get_device()
    bf16 = torch.bfloat16
    _mx_tensor(x, "x", bf16, shape, dev)
    if d != gate_up.k:
        raise ValueError("x: of another width than the experts")
    if residual is not None:
        _mx_tensor(residual, "residual", bf16, shape, dev)
    if gain is not None:
        _mx_tensor(gain, "gain", bf16, (d,), dev)
    k = topk_ids.shape[1]
    _mx_tensor(topk_ids, "topk_ids", torch.int32, (n, k), dev)
    _mx_tensor(topk_weight, "topk_weight", torch.float32, (n, k), dev)
    gs, ds = gate_up.checked(dev), down.checked(dev)
    if x_global is not None:
        _mx_scalar(x_global, "x_global", dev)
    if h_global is not None:
        _mx_scalar(h_global, "h_global", dev)
    device = x.device
    if ws is None:
        nbytes = moe_mx_layer_workspace_size(gs, ds, k, n)
        if nbytes == 0:
            raise MoeError(2, "moe_mx_layer_workspace_size")
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    total = torch.empty(shape, dtype=bf16, device=device) if gain is not None else None
    out = torch.empty(shape, dtype=torch.float32 if out_is_fp32 else bf16, device=device)
    moe_mx_layer_forward(gs, ds, k, n, x, residual, gain, eps, topk_ids, topk_weight, x_global, h_global, total, out,
                         ws, out_is_fp32)
    return total, out
