"""What the host decides about the FP8 calls before anything is launched (no GPU needed): sizes, the refusals of the C ABI
and of the binding."""

import ctypes

import pytest
import torch

import mixture_experts_ffn_infer_gb300 as mx

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = ctypes.c_void_p(1 << 20)              # aligned addresses that are never read
FAR = ctypes.c_void_p(1 << 40)
ODD = ctypes.c_void_p((1 << 20) + 8)
ODD4 = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module", autouse=True)
def lib():
    from mixture_experts_ffn_infer_gb300 import build
    build.build()
    return mx.load_library()


def W(E=4, n_out=256, k=512, packed=P.value, scales=P.value):
    return mx.moe_fp8_weights(E, n_out, k, packed, scales)


def test_sizes():
    assert [mx.moe_fp8_scale_pitch(c) for c in (16, 128, 144, 512, 528, 7168)] == [4, 4, 4, 4, 8, 56]
    assert [mx.moe_fp8_scale_pitch(c) for c in (0, -16, 8, 100)] == [0] * 4
    assert mx.moe_fp8_packed_bytes(W(3, 257, 144)) == 3 * 2 * 2 * 32768
    assert mx.moe_fp8_packed_bytes(W(1, 1, 16)) == 32768
    # of a bank's down matrices with an even number of blocks, as many as moe_pack_weights makes
    assert mx.moe_fp8_packed_bytes(W(384, 7168, 2048)) == mx.moe_tiled_bytes(2, 384, 7168, 2048)
    for w in (W(0), W(1025), W(n_out=0), W(n_out=65537), W(k=0), W(k=24), W(k=65552)):
        assert mx.moe_fp8_packed_bytes(w) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(n=0, x=None), OK), (dict(n=-1), INVALID), (dict(k=0), INVALID), (dict(k=2), INVALID), (dict(out_rows=-1), INVALID),
    (dict(d=24), UNSUPPORTED), (dict(d=0), UNSUPPORTED), (dict(d=16400, ld=16400), UNSUPPORTED), (dict(k=1025), UNSUPPORTED),
    (dict(n=1 << 31), UNSUPPORTED), (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(x=ODD), INVALID), (dict(codes=ODD), INVALID), (dict(scales=ODD), INVALID), (dict(ld=48), INVALID),
    (dict(ld=68), INVALID), (dict(pos=ODD4), INVALID)])
def test_quantise_refuses(lib, kw, status):
    a = dict(n=4, k=1, d=64, x=P, ld=64, pos=None, out_rows=4, codes=P, scales=P) | kw
    assert lib.moe_fp8_quantise(a["n"], a["k"], a["d"], a["x"], a["ld"], a["pos"], a["out_rows"], a["codes"], a["scales"],
                                None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0, codes=None), OK), (dict(rows=-1), INVALID), (dict(d=40), UNSUPPORTED), (dict(d=65552, ld=65552), UNSUPPORTED),
    (dict(codes=None), INVALID), (dict(scales=ODD), INVALID), (dict(out=ODD), INVALID), (dict(ld=48), INVALID),
    (dict(ld=68), INVALID)])
def test_dequantise_refuses(lib, kw, status):
    a = dict(rows=4, d=64, codes=P, scales=P, out=P, ld=64) | kw
    assert lib.moe_fp8_dequantise(a["rows"], a["d"], a["codes"], a["scales"], a["out"], a["ld"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(w=None), INVALID), (dict(w=W(0)), UNSUPPORTED), (dict(w=W(n_out=24), t=1), UNSUPPORTED),
    (dict(codes=None), INVALID), (dict(codes=ODD), INVALID),
    (dict(packed=None), INVALID), (dict(packed=ODD), INVALID), (dict(packed=P), INVALID), (dict(t=1, scales=None), INVALID),
    (dict(t=1, out=None), INVALID), (dict(t=1, scales=P, out=P), INVALID)])
def test_packing_refuses(lib, kw, status):
    a = dict(w=W(), codes=P, scales=P, t=0, packed=FAR, out=FAR) | kw
    w = None if a["w"] is None else ctypes.byref(a["w"])
    assert lib.moe_fp8_pack_weights(w, a["codes"], a["scales"], a["t"], a["packed"], a["out"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0, xc=None), OK), (dict(w=None), INVALID), (dict(w=W(k=24)), UNSUPPORTED), (dict(rows=-1), INVALID),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(w=W(1024, 65536, 512), rows=(1 << 31) - 5000), UNSUPPORTED),
    (dict(type=3), INVALID), (dict(type=-1), INVALID), (dict(out_rows=-1), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws=ODD), WORKSPACE), (dict(wb=255), WORKSPACE), (dict(w=W(packed=None)), INVALID), (dict(w=W(scales=None)), INVALID),
    (dict(w=W(packed=ODD.value)), INVALID), (dict(xc=None), INVALID), (dict(xc=ODD), INVALID), (dict(xs=ODD), INVALID),
    (dict(off=None), INVALID), (dict(out=None), INVALID), (dict(out=ODD4, type=2), INVALID), (dict(ld=255), INVALID),
    (dict(pos=ODD4), INVALID), (dict(rw=ODD4), INVALID)])
def test_the_product_refuses(lib, kw, status):
    a = dict(w=W(), rows=5, xc=P, xs=P, off=P, out=P, type=0, out_rows=5, ld=256, pos=None, rw=None, ws=P, wb=256) | kw
    w = None if a["w"] is None else ctypes.byref(a["w"])
    assert lib.moe_fp8_grouped_product(w, a["rows"], a["xc"], a["xs"], a["off"], a["out"], a["type"], a["out_rows"], a["ld"],
                                       a["pos"], a["rw"], a["ws"], a["wb"], None) == status


# ---------------------------------------------------------------- the binding

X = torch.zeros(5, 64, dtype=torch.bfloat16)
WEIGHTS = dict(num_experts=1, n_out=32, k=64, packed=torch.zeros(32768, dtype=torch.uint8), scales=torch.zeros(1, 1, 1))


def rows(n=5, cols=64):
    return mx.fp8_rows(n, cols, "cpu")


def weights(**kw):
    return mx.Fp8Weights(**(WEIGHTS | kw))


@pytest.mark.parametrize("call,why", [
    (lambda: mx.fp8_quantise(X.float()), "x: expected bf16"),
    (lambda: mx.fp8_quantise(X[:1].expand(5, 64)), "x: .*rows of their own"),
    (lambda: mx.fp8_quantise(X, positions=torch.zeros(4, 1, dtype=torch.int32)), "positions"),
    (lambda: mx.fp8_quantise(X, out=rows(4)), "fewer rows than x, and no positions"),
    (lambda: mx.fp8_quantise(X, out_rows=4), "fewer rows than x, and no positions"),
    (lambda: mx.fp8_quantise(X, positions=torch.zeros(5, 1, dtype=torch.int32), out_rows=-1), "out_rows"),
    (lambda: mx.fp8_quantise(X, out=rows(5, 80)), "width"),
    (lambda: mx.fp8_quantise(X, out=mx.Fp8Rows(rows().codes, torch.zeros(5, 1))), "scales"),
    (lambda: mx.fp8_quantise(X), "CUDA"),
    (lambda: mx.fp8_dequantise(mx.Fp8Rows(rows().codes.to(torch.int8), rows().scales)), "codes"),
    (lambda: mx.fp8_dequantise(rows(), out=X[:4]), "out"),
    (lambda: mx.fp8_dequantise(rows()), "CUDA"),
    (lambda: mx.fp8_grouped_product(rows(5, 80), weights()), "width"),
    (lambda: mx.fp8_grouped_product(rows(), weights(num_experts=2, packed=torch.zeros(65536, dtype=torch.uint8),
                                                    scales=torch.zeros(2, 1, 1))), "offsets: missing"),
    (lambda: mx.fp8_grouped_product(rows(), weights(packed=WEIGHTS["packed"][:100])), "packed"),
    (lambda: mx.fp8_grouped_product(rows(), weights(scales=torch.zeros(1, 1))), "scales"),
    (lambda: mx.fp8_grouped_product(rows(), weights(), torch.zeros(2)), "offsets"),
    (lambda: mx.fp8_grouped_product(rows(), weights(), out=torch.zeros(5, 32)), "out"),
    (lambda: mx.fp8_grouped_product(rows(), weights(), out=X[:1, :32].expand(5, 32)), "overlap"),
    (lambda: mx.fp8_grouped_product(rows(), weights(), out_pos=torch.zeros(4, dtype=torch.int32)), "out_pos"),
    (lambda: mx.fp8_grouped_product(rows(), weights(), row_weight=torch.zeros(4)), "row_weight"),
    (lambda: mx.fp8_grouped_product(rows(), weights()), "CUDA"),
    (lambda: mx.fp8_pack(torch.zeros(2, 32, 64), torch.zeros(2, 1, 1)), "codes"),
    (lambda: mx.fp8_pack(rows().codes, torch.zeros(2, 1)), "scales"),
    (lambda: mx.fp8_pack(rows().codes, torch.zeros(1, 1)), "CUDA")])
def test_the_binding_refuses(call, why):
    with pytest.raises(ValueError, match=why):
        call()


def test_unsupported_sizes():
    for call in (lambda: mx.fp8_quantise(X[:, :40]), lambda: mx.fp8_rows(4, 40), lambda: mx.fp8_grouped_product(rows(), weights(k=40)),
                 lambda: mx.fp8_grouped_product(rows(), weights(n_out=1 << 32)),
                 lambda: mx.fp8_grouped_product(rows(), weights(), out_type=3),
                 lambda: mx.fp8_quantise(torch.empty(1, (1 << 32) + 64, dtype=torch.bfloat16, device="meta")),
                 lambda: mx.fp8_pack(torch.zeros(40, 40, dtype=torch.uint8), torch.zeros(1, 1))):
        with pytest.raises(mx.MoeError):
            call()
