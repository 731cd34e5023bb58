"""The microscaled-format operators on torch tensors (include/moe_mx.h).

Each call checks its tensors, allocates what it returns and launches on the current stream (or on `stream`).  A decode
step's call is a few microseconds of GPU time, so the host's part is kept short: an argument that passes costs a few
attribute reads, and no message is formatted and no library call made for it.
"""

from __future__ import annotations

import torch

from . import (MOE_MX_BF16, MOE_MX_OUT_BF16, MOE_MX_OUT_F16, MOE_MX_PRODUCT_WORKSPACE, MoeError, load_library,
               moe_mx_packed_bytes, moe_mx_weights)

_BF16, _F16, _F32, _I32, _U8 = torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.uint8
_BITS = (16, 8, 4, 4)
_GROUP = (0, 32, 32, 16)
_empty = torch.empty


def _raw_stream(dev):
    """The handle of the device's current stream: what torch's own stream object wraps, at a tenth of its cost."""
    if dev < 0:
        raise ValueError("expected tensors on a CUDA device")
    return torch._C._cuda_getCurrentRawStream(dev)


def _width(fmt, cols):
    """(code bytes, scale pitch) of a row, as moe_mx_code_bytes and moe_mx_scale_pitch give them."""
    if not 0 <= fmt <= 3 or cols <= 0 or cols & 31:
        raise MoeError(2, "moe_mx_code_bytes")
    return cols * _BITS[fmt] >> 3, (cols // _GROUP[fmt] + 15 & -16) if fmt else 0


def _want(t, name, dtype, shape, dev):
    """A tensor that the library reads through its pointer: dense, on the device, of this type and shape."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor {tuple(shape)} on device {dev}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")


def _want_values(t, name, dev, count=1):
    if t.dtype is not _F32 or t.numel() != count or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: expected {count} fp32 value(s) on device {dev}")


def _row_stride(t, name, shape, dev):
    """bf16 rows: the row stride in elements (that of a single row is not used, and torch may report any)."""
    if t.dtype is not _BF16 or t.shape != shape or t.get_device() != dev or t.stride(1) != 1:
        raise ValueError(f"{name}: expected bf16 rows {tuple(shape)} on device {dev}, got {t.dtype} {tuple(t.shape)} "
                         f"on {t.device}")
    ld = t.stride(0)
    return ld if shape[0] > 1 or ld > shape[1] else shape[1]


def _on(stream, fn, *args, **kw):
    """fn on another stream than the current one: what it allocates belongs to the stream that it launches on."""
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(stream):
        return fn(*args, **kw)


class MxRows:
    """Rows of `cols` columns in a microscaled format: uint8 codes [rows, .] and scales [rows, pitch] (None for
    bf16), and NVFP4's fp32 factor [1] (None = 1).

    Rows that a call here allocates keep codes and scales in one buffer and make the two tensors when they are asked
    for; what is needed of them otherwise is where they are."""

    __slots__ = ("fmt", "cols", "global_scale", "_rows", "_dev", "_codes", "_scales", "_buf", "_addr")

    def __init__(self, fmt, cols, codes, scales=None, global_scale=None):
        self.fmt = fmt
        self.cols = cols
        self.global_scale = global_scale
        self._codes = codes
        self._scales = scales
        self._buf = None

    @property
    def codes(self):
        if self._codes is None:
            self._views()
        return self._codes

    @property
    def scales(self):
        if self._codes is None:
            self._views()
        return self._scales

    @property
    def rows(self):
        return self._rows if self._buf is not None else self._codes.shape[0]

    def _views(self):
        n = self._rows
        cb, pitch = _width(self.fmt, self.cols)
        self._codes = self._buf[:n * cb].view(n, cb)
        self._scales = self._buf[n * cb + 255 & -256:][:n * pitch].view(n, pitch) if pitch else None

    def _check(self, dev=None):
        """(rows, device index, address of the codes, address of the scales), once they are what they have to be."""
        if self._buf is not None:             # as allocated below
            if dev is not None and dev != self._dev:
                raise ValueError(f"rows: expected on device {dev}")
            return self._addr
        codes, scales = self._codes, self._scales
        n = codes.shape[0]
        if dev is None:
            dev = codes.get_device()
        cb, pitch = _width(self.fmt, self.cols)
        _want(codes, "codes", _U8, (n, cb), dev)
        if pitch:
            if scales is None:
                raise ValueError("scales: missing")
            _want(scales, "scales", _U8, (n, pitch), dev)
        return n, dev, codes.data_ptr(), scales.data_ptr() if pitch else None

    def _factor(self, dev):
        """Address of NVFP4's factor."""
        g = self.global_scale
        if g is None:
            return None
        _want_values(g, "global_scale", dev)
        return g.data_ptr()


def _new_rows(fmt, n, cols, device, dev, global_scale):
    if not 0 <= fmt <= 3 or cols <= 0 or cols & 31:
        raise MoeError(2, "moe_mx_code_bytes")
    r = MxRows(fmt, cols, None, None, global_scale)
    at = n * (cols * _BITS[fmt] >> 3)
    if fmt:
        scales = at + 255 & -256
        r._buf = buf = _empty(scales + n * (cols // _GROUP[fmt] + 15 & -16), dtype=_U8, device=device)
        base = buf.data_ptr()
        r._addr = n, dev, base, base + scales
    else:
        r._buf = buf = _empty(at, dtype=_U8, device=device)
        r._addr = n, dev, buf.data_ptr(), None
    r._rows = n
    r._dev = dev
    return r


def mx_rows(fmt, rows, cols, device="cuda", global_scale=None) -> MxRows:
    """Uninitialised rows."""
    device = torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return _new_rows(fmt, rows, cols, device, device.index if device.type == "cuda" else -1, global_scale)


class MxWeights:
    """Experts' matrices [num_experts, n_out, k] (two of them, gate and up, with swiglu) in the packed layout;
    alpha, alpha_up: fp32 [num_experts] factors of the products (None = 1)."""

    def __init__(self, fmt, num_experts, n_out, k, packed, alpha=None, alpha_up=None, swiglu=False):
        self.__dict__.update(fmt=fmt, num_experts=num_experts, n_out=n_out, k=k, packed=packed, alpha=alpha,
                             alpha_up=alpha_up, swiglu=bool(swiglu), _checked=None)

    def __setattr__(self, name, value):
        self.__dict__[name] = value
        self.__dict__["_checked"] = None       # the struct below is of the attributes as they were

    def struct(self) -> moe_mx_weights:
        p, a, b = self.packed, self.alpha, self.alpha_up
        return moe_mx_weights(self.fmt, self.num_experts, self.n_out, self.k, self.swiglu,
                              None if p is None else p.data_ptr(), None if a is None else a.data_ptr(),
                              None if b is None else b.data_ptr())

    def checked(self, dev):
        """The struct, once the tensors have been checked against it."""
        got = self._checked
        if got is None or got[1] != dev:
            st = self.struct()
            nbytes = moe_mx_packed_bytes(st)
            if nbytes == 0:
                raise MoeError(2, "moe_mx_packed_bytes")
            p = self.packed
            if p.numel() * p.element_size() != nbytes or not p.is_contiguous() or p.get_device() != dev:
                raise ValueError(f"packed: expected {nbytes} contiguous bytes on device {dev}")
            if self.alpha is not None:
                _want_values(self.alpha, "alpha", dev, self.num_experts)
            if self.alpha_up is not None:
                _want_values(self.alpha_up, "alpha_up", dev, self.num_experts)
            got = self.__dict__["_checked"] = (st, dev)
        return got[0]


def _out_rows(fmt, n, d, positions, out_rows, global_scale, out, device, dev):
    """(k, address of positions, address of the factor, rows, addresses of codes and scales, the rows to write)."""
    if global_scale is not None:
        _want_values(global_scale, "global_scale", dev)
        g = global_scale.data_ptr()
    else:
        g = None
    if positions is not None:
        k = positions.shape[1] if positions.dim() == 2 else 0
        _want(positions, "positions", _I32, (n, k), dev)
        at = positions.data_ptr()
    else:
        k, at = 1, None
    if out is None:
        out = _new_rows(fmt, n * k if out_rows is None else out_rows, d, device, dev, global_scale)
        m, _, codes, scales = out._addr
    else:
        if out.fmt != fmt or out.cols != d:
            raise ValueError("out: of another format or width")
        m, _, codes, scales = out._check(dev)
        out.global_scale = global_scale
    return k, at, g, m, codes, scales, out


def mx_quantise(x, fmt, positions=None, out_rows=None, global_scale=None, out=None, stream=None) -> MxRows:
    """bf16 rows x [n, d] (any row stride that is a multiple of 8) into a format; row t goes to each of positions[t]
    (int32 [n, k], default its own place) of `out` (out_rows rows, default n * k)."""
    if stream is not None:
        return _on(stream, mx_quantise, x, fmt, positions, out_rows, global_scale, out)
    shape = x.shape
    n, d = shape
    dev = x.get_device()
    ld = _row_stride(x, "x", shape, dev)
    k, at, g, m, codes, scales, out = _out_rows(fmt, n, d, positions, out_rows, global_scale, out, x.device, dev)
    st = load_library().moe_mx_quantise(fmt, n, k, d, x.data_ptr(), ld, at, g, m, codes, scales, _raw_stream(dev))
    if st:
        raise MoeError(st, "moe_mx_quantise")
    return out


def mx_add_rmsnorm(x, residual, gain, eps, fmt, positions=None, out_rows=None, global_scale=None, sum_out=None,
                   out=None, stream=None):
    """(rows of the normalised sum, the sum): sum = bf16(x + residual) (residual may be None), rows = Q(rmsnorm(sum))
    written as by mx_quantise.  sum_out may be x or residual."""
    if stream is not None:
        return _on(stream, mx_add_rmsnorm, x, residual, gain, eps, fmt, positions, out_rows, global_scale, sum_out, out)
    shape = x.shape
    n, d = shape
    dev, device = x.get_device(), x.device
    ld = _row_stride(x, "x", shape, dev)
    if residual is None:
        r_ld = res = None
    else:
        r_ld, res = _row_stride(residual, "residual", shape, dev), residual.data_ptr()
    _want(gain, "gain", _BF16, (d,), dev)
    if sum_out is None:
        r_ld = r_ld or d
        sum_out = _empty(shape, dtype=_BF16, device=device) if r_ld == d else torch.empty_strided(
            shape, (r_ld, 1), dtype=_BF16, device=device)
    else:
        s_ld = _row_stride(sum_out, "sum_out", shape, dev)
        if r_ld and s_ld != r_ld and n > 1:
            raise ValueError("sum_out: its row stride differs from residual's")
        r_ld = r_ld or s_ld
    k, at, g, m, codes, scales, out = _out_rows(fmt, n, d, positions, out_rows, global_scale, out, device, dev)
    st = load_library().moe_mx_add_rmsnorm(fmt, n, k, d, x.data_ptr(), ld, res, r_ld, gain.data_ptr(), eps, at, g, m,
                                           sum_out.data_ptr(), codes, scales, _raw_stream(dev))
    if st:
        raise MoeError(st, "moe_mx_add_rmsnorm")
    return out, sum_out


def mx_dequantise(r: MxRows, out=None, stream=None):
    """bf16 values of rows."""
    if stream is not None:
        return _on(stream, mx_dequantise, r, out)
    n, dev, codes, scales = r._check()
    g = r._factor(dev)
    d = ld = r.cols
    if out is None:
        out = _empty((n, d), dtype=_BF16, device=r._buf.device if r._codes is None else r._codes.device)
    else:
        ld = _row_stride(out, "out", (n, d), dev)
    st = load_library().moe_mx_dequantise(r.fmt, n, d, codes, scales, g, out.data_ptr(), ld, _raw_stream(dev))
    if st:
        raise MoeError(st, "moe_mx_dequantise")
    return out


def mx_pack(rows: MxRows, num_experts, up=None, alpha=None, alpha_up=None, stream=None) -> MxWeights:
    """Packed weights from rows [num_experts * n_out] of a format (up: the SwiGLU pair's second matrix)."""
    if stream is not None:
        return _on(stream, mx_pack, rows, num_experts, up, alpha, alpha_up)
    n, dev, codes, scales = rows._check()
    if num_experts < 1 or n % num_experts != 0:
        raise ValueError("rows: not a multiple of num_experts")
    codes_up = scales_up = None
    if up is not None:
        if (up.fmt, up.cols, up.rows) != (rows.fmt, rows.cols, n):
            raise ValueError("up: not like the first matrix")
        _, _, codes_up, scales_up = up._check(dev)
    w = MxWeights(rows.fmt, num_experts, n // num_experts, rows.cols, None, alpha, alpha_up, up is not None)
    nbytes = moe_mx_packed_bytes(w.struct())
    if nbytes == 0:
        raise MoeError(2, "moe_mx_packed_bytes")
    w.packed = _empty(nbytes, dtype=_U8, device=rows.codes.device)
    st = load_library().moe_mx_pack_weights(w.checked(dev), codes, scales, codes_up, scales_up, w.packed.data_ptr(),
                                            _raw_stream(dev))
    if st:
        raise MoeError(st, "moe_mx_pack_weights")
    return w


def mx_workspace(device="cuda"):
    """A workspace of the grouped products (its error word starts at zero)."""
    return torch.zeros(MOE_MX_PRODUCT_WORKSPACE, dtype=_U8, device=device)


def _operands(x: MxRows, w: MxWeights, offsets, ws):
    """(rows, device index, addresses of codes, scales and factor, the weights' struct, workspace), checked."""
    n, dev, codes, scales = x._check()
    g = x._factor(dev)
    st = w.checked(dev)
    if x.fmt != w.fmt or x.cols != w.k:
        raise ValueError("x: of another format or width than the weights")
    _want(offsets, "offsets", _I32, (w.num_experts + 1,), dev)
    if ws is None:
        ws = mx_workspace(offsets.device)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"ws: expected contiguous bytes on device {dev}")
    return n, dev, codes, scales, g, st, ws


def mx_grouped_product(x: MxRows, w: MxWeights, offsets, out=None, out_pos=None, row_weight=None, ws=None,
                       out_type=MOE_MX_OUT_BF16, stream=None):
    """out[p(r)] = row_weight[p(r)] * x[r] W_e^T for the rows offsets[e] .. offsets[e + 1] - 1 of each expert e;
    p = out_pos (int32 [rows], default r)."""
    if stream is not None:
        return _on(stream, mx_grouped_product, x, w, offsets, out, out_pos, row_weight, ws, out_type)
    n, dev, codes, scales, g, struct, ws = _operands(x, w, offsets, ws)
    dtype = _F16 if out_type == MOE_MX_OUT_F16 else _BF16
    cols = ld = w.n_out
    out_rows = n
    if out is None:
        out = _empty((n, cols), dtype=dtype, device=offsets.device)
    else:
        if out.dtype is not dtype or out.dim() != 2 or out.shape[1] != cols or out.get_device() != dev or (
                cols > 1 and out.stride(1) != 1):
            raise ValueError("out: of another type, width or device")
        out_rows, ld = out.shape[0], out.stride(0)
        if out_rows < 2 and ld < cols:
            ld = cols
    to = weight = None
    if out_pos is not None:
        _want(out_pos, "out_pos", _I32, (n,), dev)
        to = out_pos.data_ptr()
    if row_weight is not None:
        _want_values(row_weight, "row_weight", dev, out_rows)
        weight = row_weight.data_ptr()
    st = load_library().moe_mx_grouped_product(struct, n, codes, scales, g, offsets.data_ptr(), out.data_ptr(),
                                               out_type, out_rows, ld, to, weight, ws.data_ptr(), ws.nbytes,
                                               _raw_stream(dev))
    if st:
        raise MoeError(st, "moe_mx_grouped_product")
    return out


def mx_grouped_swiglu(x: MxRows, w: MxWeights, offsets, h_global=None, out=None, ws=None, stream=None) -> MxRows:
    """Rows of silu(x Wg_e^T) * (x Wu_e^T) in the format of x."""
    if stream is not None:
        return _on(stream, mx_grouped_swiglu, x, w, offsets, h_global, out, ws)
    n, dev, codes, scales, g, struct, ws = _operands(x, w, offsets, ws)
    _, _, hg, m, h_codes, h_scales, out = _out_rows(w.fmt, n, w.n_out, None, None, h_global, out, offsets.device, dev)
    if m != n:
        raise ValueError("out: of another number of rows")
    st = load_library().moe_mx_grouped_swiglu(struct, n, codes, scales, g, offsets.data_ptr(), hg, h_codes, h_scales,
                                              ws.data_ptr(), ws.nbytes, _raw_stream(dev))
    if st:
        raise MoeError(st, "moe_mx_grouped_swiglu")
    return out


def mx_layer_forward(x, residual, gain, eps, topk_ids, topk_weight, gate_up: MxWeights, down: MxWeights,
                     x_global=None, h_global=None, ws=None, out_is_fp32=False, stream=None):
    """The MoE block on microscaled experts: (sum, out) with sum = bf16(x + residual) and out = sum + the routed
    experts on rmsnorm(sum); with gain None (and residual None) (None, the routed experts on x)."""
    if stream is not None:
        return _on(stream, mx_layer_forward, x, residual, gain, eps, topk_ids, topk_weight, gate_up, down, x_global,
                   h_global, ws, out_is_fp32)
    shape = x.shape
    n, d = shape
    dev, device = x.get_device(), x.device
    _want(x, "x", _BF16, shape, dev)
    if d != gate_up.k:
        raise ValueError("x: of another width than the experts")
    if residual is not None:
        _want(residual, "residual", _BF16, shape, dev)
    if gain is not None:
        _want(gain, "gain", _BF16, (d,), dev)
    table = topk_ids.shape
    k = table[1]
    _want(topk_ids, "topk_ids", _I32, (n, k), dev)
    _want(topk_weight, "topk_weight", _F32, table, dev)
    gs, ds = gate_up.checked(dev), down.checked(dev)
    if x_global is not None:
        _want_values(x_global, "x_global", dev)
    if h_global is not None:
        _want_values(h_global, "h_global", dev)
    lib = load_library()
    if ws is None:
        nbytes = lib.moe_mx_layer_workspace_size(gs, ds, k, n)
        if nbytes == 0:
            raise MoeError(2, "moe_mx_layer_workspace_size")
        ws = _empty(nbytes, dtype=_U8, device=device)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"ws: expected contiguous bytes on device {dev}")
    total = _empty(shape, dtype=_BF16, device=device) if gain is not None else None
    out = _empty(shape, dtype=_F32 if out_is_fp32 else _BF16, device=device)
    st = lib.moe_mx_layer_forward(
        gs, ds, k, n, x.data_ptr(), None if residual is None else residual.data_ptr(),
        None if gain is None else gain.data_ptr(), eps, topk_ids.data_ptr(), topk_weight.data_ptr(),
        None if x_global is None else x_global.data_ptr(), None if h_global is None else h_global.data_ptr(),
        None if total is None else total.data_ptr(), out.data_ptr(), bool(out_is_fp32), ws.data_ptr(), ws.nbytes,
        _raw_stream(dev))
    if st:
        raise MoeError(st, "moe_mx_layer_forward")
    return total, out
