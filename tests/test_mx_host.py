"""What the host decides about the microscaled-format calls before anything is launched (no GPU needed): sizes, the
refusals of the C ABI, the refusals of the Python binding, and moe_mx.h as C99."""

import ctypes
import os
import subprocess

import pytest
import torch

import mixture_experts_ffn_infer_gb300 as mx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
P = ctypes.c_void_p(1 << 20)              # aligned addresses that are never read
ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_ffn_infer_gb300 import build
    build.build()
    return mx.load_library()


def W(fmt=3, E=4, n_out=256, k=512, swiglu=0, packed=P.value):
    return mx.moe_mx_weights(fmt, E, n_out, k, swiglu, packed, None, None)


def test_row_sizes(lib):
    assert [mx.moe_mx_code_bytes(f, 7168) for f in range(4)] == [14336, 7168, 3584, 3584]
    assert [mx.moe_mx_scale_pitch(f, 7168) for f in range(4)] == [0, 224, 224, 448]
    assert [mx.moe_mx_scale_pitch(f, 32) for f in range(4)] == [0, 16, 16, 16]
    for f, cols in ((4, 64), (-1, 64), (1, 0), (1, 33), (1, -32)):
        assert mx.moe_mx_code_bytes(f, cols) == 0 and mx.moe_mx_scale_pitch(f, cols) == 0


def test_packed_sizes(lib):
    assert mx.moe_mx_packed_bytes(W(3, 4, 257, 257 // 32 * 32)) == 4 * 2 * 1 * (32768 + 4096)
    assert mx.moe_mx_packed_bytes(W(2, 1, 256, 544)) == 3 * (32768 + 2048)
    assert mx.moe_mx_packed_bytes(W(1, 1, 129 // 32 * 32 + 32, 128, swiglu=1)) == 2 * (32768 + 1024)
    assert mx.moe_mx_packed_bytes(W(0, 2, 1, 64)) == 2 * 32768
    for w in (W(4), W(E=0), W(E=1025), W(n_out=0), W(n_out=65537), W(k=48), W(k=0), W(k=65568), W(n_out=100, swiglu=1)):
        assert mx.moe_mx_packed_bytes(w) == 0


def quantise(lib, fmt=3, n=4, k=1, d=64, x=P, ld=64, pos=None, out_rows=4, codes=P, scales=P):
    return lib.moe_mx_quantise(fmt, n, k, d, x, ld, pos, None, out_rows, codes, scales, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=0, x=None), 0), (dict(n=-1), INVALID), (dict(fmt=4), UNSUPPORTED), (dict(d=48), UNSUPPORTED),
    (dict(d=16416, ld=16416), UNSUPPORTED), (dict(k=0), INVALID), (dict(k=2), INVALID), (dict(x=None), INVALID),
    (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(x=ODD), INVALID), (dict(codes=ODD), INVALID),
    (dict(scales=ODD), INVALID), (dict(ld=32), INVALID), (dict(ld=68), INVALID), (dict(out_rows=-1), INVALID),
    (dict(n=1 << 31, k=1), UNSUPPORTED)])
def test_quantise_refusals(lib, kw, status):
    assert quantise(lib, **kw) == status


def norm(lib, fmt=1, n=4, d=64, x=P, x_ld=64, res=P, r_ld=64, gain=P, eps=1e-6, out=P, codes=P, scales=P):
    return lib.moe_mx_add_rmsnorm(fmt, n, 1, d, x, x_ld, res, r_ld, gain, eps, None, None, n, out, codes, scales, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), 0), (dict(gain=None), INVALID), (dict(gain=ODD), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(res=ODD), INVALID), (dict(out=ODD), INVALID), (dict(r_ld=32), INVALID),
    (dict(r_ld=68), INVALID), (dict(x_ld=128), INVALID)])        # sum is x here, with another stride
def test_norm_refusals(lib, kw, status):
    assert norm(lib, **kw) == status


def test_dequantise_refusals(lib):
    call = lambda fmt=1, rows=4, d=64, codes=P, scales=P, out=P, ld=64: lib.moe_mx_dequantise(fmt, rows, d, codes, scales,
                                                                                              None, out, ld, None)
    assert call(rows=0, codes=None) == 0 and call(rows=-1) == INVALID
    assert call(d=40) == UNSUPPORTED and call(fmt=9) == UNSUPPORTED
    for kw in (dict(codes=None), dict(scales=None), dict(out=None), dict(out=ODD), dict(ld=60), dict(ld=68)):
        assert call(**kw) == INVALID


def test_pack_refusals(lib):
    far = [ctypes.c_void_p((1 << 20) * i) for i in range(1, 6)]
    call = lambda w, *p: lib.moe_mx_pack_weights(ctypes.byref(w) if w else None, *p, None)
    assert call(None, *far) == INVALID
    assert call(W(k=33), *far) == UNSUPPORTED
    assert call(W(), None, *far[1:]) == INVALID and call(W(), far[0], None, *far[2:]) == INVALID
    assert call(W(swiglu=1), far[0], far[1], None, *far[3:]) == INVALID
    assert call(W(swiglu=1), *far[:3], None, far[4]) == INVALID
    assert call(W(), *far[:4], None) == INVALID and call(W(), *far[:4], ODD) == INVALID
    assert call(W(), far[0], far[1], None, None, far[0]) == INVALID          # in place


def product(lib, w=None, rows=8, xc=P, xs=P, off=P, out=P, kind=0, out_rows=8, ld=256, ws=P, wsb=256):
    w = W() if w is None else w
    return lib.moe_mx_grouped_product(ctypes.byref(w), rows, xc, xs, None, off, out, kind, out_rows, ld, None, None, ws,
                                      wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0, xc=None), 0), (dict(rows=-1), INVALID), (dict(w=W(swiglu=1)), INVALID), (dict(w=W(k=33)), UNSUPPORTED),
    (dict(w=W(packed=None)), INVALID), (dict(w=W(packed=ODD.value)), INVALID), (dict(xc=None), INVALID),
    (dict(xs=None), INVALID), (dict(xc=ODD), INVALID), (dict(xs=ODD), INVALID), (dict(off=None), INVALID),
    (dict(out=None), INVALID), (dict(kind=2), INVALID), (dict(ld=255), INVALID), (dict(ws=None), WORKSPACE),
    (dict(wsb=128), WORKSPACE), (dict(ws=ODD), WORKSPACE), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(out_rows=-1), INVALID)])
def test_product_refusals(lib, kw, status):
    assert product(lib, **kw) == status


def test_unit_count_stays_in_32_bits(lib):
    # 128 block rows of 256; a CTA counts past the last unit by one round, for which 4096 numbers are kept
    tiles = ((1 << 31) - 4096) // 128
    call = lambda t: product(lib, w=W(E=1, n_out=32768), rows=128 * (t - 1), ld=32768, ws=None)
    assert call(tiles - 1) == WORKSPACE         # accepted so far
    assert call(tiles) == UNSUPPORTED


def test_swiglu_refusals(lib):
    def call(w=W(swiglu=1), rows=8, xc=P, hc=P, hs=P, ws=P):
        return lib.moe_mx_grouped_swiglu(ctypes.byref(w), rows, xc, P, None, P, None, hc, hs, ws, 256, None)
    assert call(rows=0) == 0 and call(w=W()) == INVALID and call(ws=None) == WORKSPACE
    for kw in (dict(xc=None), dict(hc=None), dict(hs=None), dict(hc=ODD), dict(hs=ODD)):
        assert call(**kw) == INVALID


def test_layer_refusals(lib):
    gu, dn = W(3, 4, 256, 512, 1), W(3, 4, 512, 256)
    size = mx.moe_mx_layer_workspace_size(gu, dn, 2, 10)
    assert size > 10 * 2 * 512 * 2 and mx.moe_mx_layer_workspace_size(gu, dn, 2, 1000) > size
    for g, d, k, n in ((dn, dn, 2, 1), (gu, gu, 2, 1), (gu, W(2, 4, 512, 256), 2, 1), (gu, W(3, 5, 512, 256), 2, 1),
                       (gu, W(3, 4, 512, 128), 2, 1), (gu, dn, 0, 1), (gu, dn, 33, 1), (gu, dn, 2, -1), (gu, dn, 2, 1 << 30),
                       (W(3, 4, 256, 544, 1), W(3, 4, 544, 256), 2, 1)):
        assert mx.moe_mx_layer_workspace_size(g, d, k, n) == 0

    def call(n=10, x=P, res=P, gain=P, eps=1e-6, ids=P, wt=P, total=P, out=P, ws=P, wsb=size, g=gu):
        return lib.moe_mx_layer_forward(ctypes.byref(g), ctypes.byref(dn), 2, n, x, res, gain, eps, ids, wt, None, None,
                                        total, out, 0, ws, wsb, None)
    assert call(n=0) == 0 and call(n=-1) == INVALID and call(g=dn) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE and call(wsb=size - 1) == WORKSPACE
    for kw in (dict(x=None), dict(ids=None), dict(wt=None), dict(out=None), dict(total=None), dict(eps=-1.0),
               dict(gain=None), dict(gain=None, res=None), dict(res=ODD), dict(x=ODD), dict(out=ODD)):
        assert call(**kw) == INVALID


def test_binding_refusals(lib):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    gain = torch.ones(64, dtype=torch.bfloat16)
    bad = [lambda: mx.mx_quantise(x.float(), 1), lambda: mx.mx_quantise(x.t(), 1),
           lambda: mx.mx_quantise(x, 1, positions=torch.zeros(4, 1)),
           lambda: mx.mx_quantise(x, 1, positions=torch.zeros(3, 1, dtype=torch.int32)),
           lambda: mx.mx_quantise(x, 3, global_scale=torch.ones(2)),
           lambda: mx.mx_quantise(x, 1, out=mx.mx_rows(2, 4, 64, "cpu")),
           lambda: mx.mx_add_rmsnorm(x, x[:2], gain, 1e-6, 1), lambda: mx.mx_add_rmsnorm(x, x, gain[:32], 1e-6, 1),
           lambda: mx.mx_add_rmsnorm(x, x, gain, 1e-6, 1, sum_out=torch.zeros(4, 128, dtype=torch.bfloat16)[:, :64]),
           lambda: mx.mx_dequantise(mx.MxRows(1, 64, torch.zeros(4, 32, dtype=torch.uint8))),
           lambda: mx.mx_dequantise(mx.MxRows(1, 64, torch.zeros(4, 64, dtype=torch.uint8))),
           lambda: mx.mx_pack(mx.mx_rows(1, 4, 64, "cpu"), 3),
           lambda: mx.mx_pack(mx.mx_rows(1, 64, 64, "cpu"), 1, up=mx.mx_rows(1, 32, 64, "cpu"))]
    w = mx.MxWeights(1, 1, 64, 64, torch.zeros(mx.moe_mx_packed_bytes(W(1, 1, 64, 64)), dtype=torch.uint8))
    off = torch.zeros(2, dtype=torch.int32)
    r = mx.mx_rows(1, 4, 64, "cpu")
    bad += [lambda: mx.mx_grouped_product(mx.mx_rows(1, 4, 96, "cpu"), w, off), lambda: mx.mx_grouped_product(r, w, off.long()),
            lambda: mx.mx_grouped_product(mx.mx_rows(2, 4, 64, "cpu"), w, off),
            lambda: mx.mx_grouped_product(r, w, torch.zeros(3, dtype=torch.int32)),
            lambda: mx.mx_grouped_product(r, w, off, out=torch.zeros(4, 64)),
            lambda: mx.mx_grouped_product(r, w, off, out_pos=torch.zeros(3, dtype=torch.int32)),
            lambda: mx.mx_grouped_product(r, w, off, row_weight=torch.zeros(3)),
            lambda: mx.mx_grouped_product(r, mx.MxWeights(1, 1, 64, 64, torch.zeros(16, dtype=torch.uint8)), off)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mx.mx_quantise(x[:, :48], 1), lambda: mx.mx_rows(7, 4, 64, "cpu")):
        with pytest.raises(mx.MoeError):
            call()


def test_host_tensors_are_refused(lib):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    r = mx.mx_rows(1, 4, 64, "cpu")
    w = mx.MxWeights(1, 1, 64, 64, torch.zeros(mx.moe_mx_packed_bytes(W(1, 1, 64, 64)), dtype=torch.uint8))
    ws = torch.zeros(512, dtype=torch.uint8)
    for call in (lambda: mx.mx_quantise(x, 1), lambda: mx.mx_dequantise(r), lambda: mx.mx_pack(r, 1),
                 lambda: mx.mx_add_rmsnorm(x, x, torch.ones(64, dtype=torch.bfloat16), 1e-6, 1),
                 lambda: mx.mx_grouped_product(r, w, torch.zeros(2, dtype=torch.int32), ws=ws)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_call_signatures(lib):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: mx.mx_quantise(), lambda: mx.mx_quantise(x), lambda: mx.mx_quantise(x, 1, fmt=1),
                 lambda: mx.mx_quantise(x, 1, nothing=1), lambda: mx.mx_dequantise(1, 2, 3, 4), lambda: mx.mx_quantise(x, "a")):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: mx.mx_quantise(None, 1), lambda: mx.mx_quantise([1], 1), lambda: mx.mx_dequantise(None),
                 lambda: mx.mx_grouped_product(mx.mx_rows(1, 4, 64, "cpu"), None, x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(AttributeError):
        mx.mx_dequantise(x)


def test_header_is_c99(tmp_path):
    src = tmp_path / "a.c"
    src.write_text('#include "moe_mx.h"\nint main(void) { moe_mx_weights w = {MOE_MX_NVFP4, 1, 256, 256, 0, 0, 0, 0};\n'
                   "return (int)(sizeof w == 0) + (int)MOE_MX_PRODUCT_WORKSPACE; }\n")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-fsyntax-only", "-I", os.path.join(ROOT, "include"),
                    "-isystem", "/usr/local/cuda/include", str(src)], check=True)
