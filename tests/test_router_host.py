"""What the host decides about the router's calls before anything is launched (no GPU needed): sizes, the refusals of the
C ABI and of the binding, and moe_router.h as C99."""

import ctypes
import os
import subprocess

import pytest
import torch

import mixture_experts_ffn_infer_gb300 as mx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = ctypes.c_void_p(1 << 20)              # an aligned address that is never read
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module", autouse=True)
def lib():
    from mixture_experts_ffn_infer_gb300 import build
    build.build()
    return mx.load_library()


def R(E=64, k=4, score=0, type=0, groups=1, top=1, normalise=1, scale=1.0):
    return mx.moe_router(E, k, score, type, groups, top, normalise, scale)


BAD = [(dict(E=0), UNSUPPORTED), (dict(E=1025), UNSUPPORTED), (dict(k=0), UNSUPPORTED), (dict(k=33), UNSUPPORTED),
       (dict(E=3), UNSUPPORTED), (dict(score=2), UNSUPPORTED), (dict(score=-1), UNSUPPORTED), (dict(type=2), UNSUPPORTED)]


@pytest.mark.parametrize("r,status", BAD + [(dict(groups=0), UNSUPPORTED), (dict(groups=3), UNSUPPORTED),
                                            (dict(groups=64), UNSUPPORTED), (dict(groups=4, top=5), UNSUPPORTED),
                                            (dict(groups=4, top=0), UNSUPPORTED), (dict(groups=32, top=1), UNSUPPORTED)])
def test_route_refuses_routers(lib, r, status):
    assert lib.moe_route(ctypes.byref(R(**r)), 0, P, 64, None, P, P, None) == status


@pytest.mark.parametrize("kw,status", [(dict(n=0, l=None, i=None, w=None), OK), (dict(n=-1), INVALID), (dict(l=None), INVALID),
                                       (dict(l=ODD), INVALID), (dict(ld=63), INVALID), (dict(i=None), INVALID),
                                       (dict(w=None), INVALID), (dict(i=ODD), INVALID), (dict(w=ODD), INVALID),
                                       (dict(b=ODD), INVALID), (dict(n=1 << 30), UNSUPPORTED)])
def test_route_refuses(lib, kw, status):
    a = dict(n=5, l=P, ld=64, b=None, i=P, w=P) | kw
    assert lib.moe_route(ctypes.byref(R()), a["n"], a["l"], a["ld"], a["b"], a["i"], a["w"], None) == status
    assert lib.moe_route(None, 5, P, 64, None, P, P, None) == INVALID


@pytest.mark.parametrize("r,status", BAD)
def test_the_loss_and_the_gradient_refuse_routers(lib, r, status):
    assert mx.moe_balance_workspace_size(R(**r), 5, 1) == 0
    assert lib.moe_balance_loss(ctypes.byref(R(**r)), 5, P, 64, P, 1.0, None, 1, P, P, P, 1 << 40, None) == status
    assert lib.moe_route_backward(ctypes.byref(R(**r)), 5, P, 64, P, P, 1.0, P, None, None, 1, P, 64, None) == status


@pytest.mark.parametrize("kw,status", [(dict(n=-1), INVALID), (dict(S=0), INVALID), (dict(S=2), INVALID),
                                       (dict(o=P, S=65537), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(ws=ODD), WORKSPACE),
                                       (dict(wb=255), WORKSPACE), (dict(l=None), INVALID), (dict(l=ODD), INVALID),
                                       (dict(ld=8), INVALID), (dict(i=None), INVALID), (dict(i=ODD), INVALID),
                                       (dict(c=None), INVALID), (dict(c=ODD), INVALID), (dict(loss=None), INVALID),
                                       (dict(loss=ODD), INVALID), (dict(o=ODD), INVALID)])
def test_the_loss_refuses(lib, kw, status):
    a = dict(n=5, l=P, ld=64, i=P, o=None, S=1, c=P, loss=P, ws=P, wb=1 << 40) | kw
    assert lib.moe_balance_loss(ctypes.byref(R()), a["n"], a["l"], a["ld"], a["i"], 1.0, a["o"], a["S"], a["c"], a["loss"],
                                a["ws"], a["wb"], None) == status


@pytest.mark.parametrize("kw,status", [(dict(n=0, l=None, g=None), OK), (dict(n=-1), INVALID), (dict(l=None), INVALID),
                                       (dict(g=None), INVALID), (dict(gld=63), INVALID), (dict(ld=63), INVALID),
                                       (dict(i=None), INVALID), (dict(g=P, ld=64, gld=65), INVALID),
                                       (dict(S=2), INVALID), (dict(S=0), INVALID), (dict(o=P, S=65537), UNSUPPORTED),
                                       (dict(dw=ODD), INVALID), (dict(c=ODD), INVALID), (dict(dl=ODD), INVALID)])
def test_the_gradient_refuses(lib, kw, status):
    a = dict(n=5, l=P, ld=64, i=P, dw=P, c=P, dl=None, o=None, S=1, g=P, gld=64) | kw
    assert lib.moe_route_backward(ctypes.byref(R()), a["n"], a["l"], a["ld"], a["i"], a["dw"], 1.0, a["c"], a["dl"], a["o"],
                                  a["S"], a["g"], a["gld"], None) == status


def test_workspace_sizes():
    # a ticket; the sequences' parts (32 experts each); a sum and a count an expert of every piece
    assert mx.moe_balance_workspace_size(R(), 0, 1) > 0
    small, large = (mx.moe_balance_workspace_size(R(384, 8), n, 1) for n in (1, 1 << 20))
    assert small < large <= 256 + 512 + 2 * (610 * 384 * 4 + 256)
    assert mx.moe_balance_workspace_size(R(384, 8), 1 << 20, 4096) > 4096 * 384 * 8
    assert mx.moe_balance_workspace_size(R(), 5, 0) == 0 and mx.moe_balance_workspace_size(R(), 5, 65537) == 0
    assert mx.moe_balance_workspace_size(R(), -1, 1) == 0


# ---------------------------------------------------------------- the binding

L, I, F = torch.zeros(5, 16), torch.zeros(5, 2, dtype=torch.int32), torch.zeros(5, 2)


@pytest.mark.parametrize("call,why", [
    (lambda: mx.route(L.double(), 2, 0), "logits: expected fp32 or bf16"),
    (lambda: mx.route(L[0], 2, 0), "logits: expected two dimensions"),
    (lambda: mx.route(L.T, 2, 0), "logits"),
    (lambda: mx.route(L[:1].expand(5, 16), 2, 0), "logits: .*rows of their own"),
    (lambda: mx.route(L, 2, 0, bias=torch.zeros(15)), "bias"),
    (lambda: mx.route(L, 2, 0, ids=I[:4]), "ids"),
    (lambda: mx.route(L, 2, 0, ids=I.long()), "ids"),
    (lambda: mx.route(L, 2, 0, weights=F.double()), "weights"),
    (lambda: mx.route(L, 2, 0), "CUDA"),
    (lambda: mx.route(L, 40, 0), "CUDA"),
    (lambda: mx.balance_loss(L, I[:4], 1.0, 0), "ids"),
    (lambda: mx.balance_loss(L, I[0], 1.0, 0), "ids"),
    (lambda: mx.balance_loss(L, I, 1.0, 0, seq_offsets=torch.zeros(1, dtype=torch.int32)), "seq_offsets"),
    (lambda: mx.balance_loss(L, I, 1.0, 0, seq_offsets=torch.zeros(3)), "seq_offsets"),
    (lambda: mx.balance_loss(L, I, 1.0, 0), "CUDA"),
    (lambda: mx.route_backward(L, I, 0, d_weights=F[:, :1]), "d_weights"),
    (lambda: mx.route_backward(L, I, 0, counts=torch.zeros(2, 16, dtype=torch.int32), coef=1.0), "counts"),
    (lambda: mx.route_backward(L, I, 0, counts=torch.zeros(1, 16, dtype=torch.int32)), "coef"),
    (lambda: mx.route_backward(L, I, 0, d_loss=torch.zeros(2)), "d_loss"),
    (lambda: mx.route_backward(L, I, 0, out=L.bfloat16()), "out"),
    (lambda: mx.route_backward(L, I, 0, out=torch.zeros(1, 16).expand(5, 16)), "out: .*rows of their own"),
    (lambda: mx.route_backward(L, I, 0, d_weights=F), "CUDA")])
def test_the_binding_refuses(call, why):
    with pytest.raises(ValueError, match=why):
        call()


def test_sizes_past_32_bits_are_unsupported():
    wide = torch.empty(1, (1 << 32) + 16, device="meta")
    ids = torch.empty(5, (1 << 32) + 2, dtype=torch.int32, device="meta")
    for call in (lambda: mx.route(wide, 2, 0), lambda: mx.route(L, (1 << 32) + 2, 0), lambda: mx.route(L, 2, 1 << 32),
                 lambda: mx.route(L, 0, 0), lambda: mx.balance_loss(L, ids, 1.0, 0)):
        with pytest.raises(mx.MoeError):
            call()


def test_the_header_is_c99(tmp_path):
    src = tmp_path / "a.c"
    src.write_text('#include "moe_router.h"\n#include "moe_fp8.h"\nint main(void) { moe_router r = {0}; moe_fp8_weights w = {0};'
                   ' return r.groups + w.k; }\n')
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-isystem",
                    "/usr/local/cuda/include", "-c", str(src), "-o", str(tmp_path / "a.o")], check=True)
