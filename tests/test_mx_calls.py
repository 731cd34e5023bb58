"""The microscaled-format calls on the GPU as a program makes them: views, other streams, errors without a workspace."""

import pytest
import torch

import mixture_experts_ffn_infer_gb300 as mx

pytestmark = pytest.mark.gpu


def bf16(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def same(a, b):
    groups = 0 if a.scales is None else a.cols // (16 if a.fmt == mx.MOE_MX_NVFP4 else 32)
    return torch.equal(a.codes, b.codes) and (not groups or torch.equal(a.scales[:, :groups], b.scales[:, :groups]))


# ---------------------------------------------------------------- strides

@pytest.mark.parametrize("fmt", [mx.MOE_MX_BF16, mx.MOE_MX_NVFP4])
def test_a_single_row_of_any_pitch(fmt):
    # the stride of one row is not used: 100 is no multiple of 8, and x and the residual differ
    x, r, gain = bf16(1, 3, 100)[:1, :96], bf16(2, 1, 96), bf16(3, 96)
    want, total = mx.mx_add_rmsnorm(x.contiguous(), r, gain, 1e-6, fmt)
    rows, got = mx.mx_add_rmsnorm(x, r, gain, 1e-6, fmt)
    assert same(rows, want) and torch.equal(got, total)
    assert same(mx.mx_quantise(x, fmt), mx.mx_quantise(x.contiguous(), fmt))
    buf = bf16(4, 3, 100)
    mx.mx_dequantise(rows, out=buf[:1, :96])
    assert torch.equal(buf[:1, :96], mx.mx_dequantise(rows))
    into = x.clone()                                             # in place, the residual of another pitch
    rows, got = mx.mx_add_rmsnorm(into, bf16(5, 3, 100)[:1, :96], gain, 1e-6, fmt, sum_out=into)
    want, total = mx.mx_add_rmsnorm(x.contiguous(), bf16(5, 3, 100)[:1, :96].contiguous(), gain, 1e-6, fmt)
    assert got is into and torch.equal(into, total) and same(rows, want)


@pytest.mark.parametrize("own_sum", [False, True])
def test_residual_and_sum_keep_their_own_stride(own_sum):
    n, d = 7, 64
    x, wide, gain = bf16(1, n, d), bf16(2, n, 2 * d), bf16(3, d)
    total = bf16(4, n, 2 * d)
    before = total.clone()
    rows, got = mx.mx_add_rmsnorm(x, wide[:, :d], gain, 1e-6, 1, sum_out=total[:, :d] if own_sum else None)
    want, sums = mx.mx_add_rmsnorm(x, wide[:, :d].contiguous(), gain, 1e-6, 1)
    assert same(rows, want) and torch.equal(got, sums)
    assert torch.equal(total[:, d:], before[:, d:])


# ---------------------------------------------------------------- the caller's rows

def test_out_gets_its_factor_with_the_rows():
    x, gain = bf16(1, 5, 64), bf16(2, 64)
    old, new = torch.full((1,), 2.0**-4, device="cuda"), torch.full((1,), 2.0**-8, device="cuda")
    out = mx.mx_quantise(x, 3, global_scale=old)
    codes = out.codes.clone()
    with pytest.raises(mx.MoeError):                             # refused by the library: rows not on 16 bytes
        mx.mx_quantise(bf16(1, 5, 66)[:, 1:65], 3, global_scale=new, out=out)
    assert out.global_scale is old and torch.equal(out.codes, codes)
    assert mx.mx_quantise(x, 3, global_scale=new, out=out) is out
    assert out.global_scale is new and same(out, mx.mx_quantise(x, 3, global_scale=new))
    rows, _ = mx.mx_add_rmsnorm(x, None, gain, 1e-6, 3, out=out)
    assert rows is out and out.global_scale is None


# ---------------------------------------------------------------- other streams

@pytest.mark.parametrize("kind", ["object", "handle", "default"])
def test_the_stream_argument(kind):
    x, s = bf16(1, 2000, 4096), torch.cuda.Stream()
    want = mx.mx_quantise(x, 1)
    torch.cuda.synchronize()
    stream = {"object": s, "handle": s.cuda_stream, "default": 0}[kind]
    runs_on = torch.cuda.default_stream() if kind == "default" else s
    with torch.cuda.stream(runs_on):
        late = torch.zeros_like(x)
        for _ in range(20):                      # work in front, so that a call elsewhere would read the zeros
            torch.mm(x[:, :2000], x)
        late.copy_(x)
    with torch.cuda.stream(torch.cuda.Stream()):  # another one is current
        rows = mx.mx_quantise(late, 1, stream=stream)
    torch.cuda.synchronize()
    assert same(rows, want)
