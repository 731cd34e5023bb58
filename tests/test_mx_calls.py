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


# ---------------------------------------------------------------- errors where no workspace is given

def weights(fmt, E, n_out, k, seed, up=False):
    mats = [mx.mx_quantise(bf16(seed + i, E * n_out, k) * 0.05, fmt) for i in range(1 + up)]
    return mx.mx_pack(mats[0], E, up=mats[1] if up else None)


def offsets(*o):
    return torch.tensor(o, dtype=torch.int32, device="cuda")


@pytest.fixture
def clean():
    mx.mx_get_error()
    yield
    assert mx.mx_get_error() == mx.MOE_OK                       # each test read what it caused


@pytest.mark.parametrize("bad", [(0, 5, 3, 8), (-1, 2, 4, 8), (0, 2, 4, 9)])
def test_bad_offsets_are_reported_without_a_workspace(clean, bad):
    x = mx.mx_quantise(bf16(1, 8, 64), 1)
    mx.mx_grouped_product(x, weights(1, 3, 64, 64, 2), offsets(*bad))
    assert mx.mx_get_error() == 4 and mx.mx_get_error() == 0    # MOE_ERR_ROUTING, once
    mx.mx_grouped_swiglu(x, weights(1, 3, 64, 64, 2, up=True), offsets(*bad))
    assert mx.mx_get_error("cuda:0") == 4


def test_errors_stay_until_they_are_read(clean):
    x, w = mx.mx_quantise(bf16(1, 8, 64), 1), weights(1, 1, 64, 64, 2)
    good = mx.mx_grouped_product(x, w, offsets(0, 8))
    assert mx.mx_get_error() == 0
    s = torch.cuda.Stream()
    mx.mx_grouped_product(x, w, offsets(0, 9), stream=s)        # on another stream, then good calls
    assert torch.equal(mx.mx_grouped_product(x, w, offsets(0, 8)), good)
    ws = mx.mx_workspace()
    mx.mx_grouped_product(x, w, offsets(0, 9), ws=ws)
    assert mx.mx_get_error() == 4 and mx.moe_get_error(ws) == 4


def test_values_beyond_f16_are_reported_without_a_workspace(clean):
    big = mx.mx_quantise(torch.full((4, 256), 300.0, device="cuda").to(torch.bfloat16), 0)
    w = mx.mx_pack(mx.mx_quantise(torch.full((32, 256), 300.0, device="cuda").to(torch.bfloat16), 0), 1)
    mx.mx_grouped_product(big, w, offsets(0, 4), out_type=mx.MOE_MX_OUT_F16)
    assert mx.mx_get_error() == 6


@pytest.mark.parametrize("n", [40, 5000])                        # the routing plan in one kernel, and in several
def test_layer_errors_without_a_workspace(clean, n):
    d, f, E, k = 128, 64, 4, 2
    gate_up, down = weights(1, E, f, d, 1, up=True), weights(1, E, d, f, 3)
    x, r, gain, w = bf16(4, n, d), bf16(5, n, d), bf16(6, d), torch.full((n, k), 0.5, device="cuda")
    ids = torch.rand(n, E, generator=torch.Generator().manual_seed(7)).topk(k, 1).indices.to(torch.int32).cuda()
    call = lambda i, **kw: mx.mx_layer_forward(x, r, gain, 1e-6, i, w, gate_up, down, **kw)[1]
    good = call(ids)
    assert mx.mx_get_error() == 0
    bad = ids.clone()
    bad[3, 1] = E
    out = call(bad)
    others = [t for t in range(n) if t != 3]
    assert torch.equal(out[others], good[others])
    assert torch.equal(call(ids), good)                          # a good call leaves the error
    assert mx.mx_get_error() == 4
    ws = torch.full((1 << 24,), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(call(ids, ws=ws), good) and mx.moe_get_error(ws) == 0   # the word is reset there


def test_captured_calls_without_a_workspace(clean):
    x, w, off = mx.mx_quantise(bf16(1, 8, 64), 1), weights(1, 1, 64, 64, 2), offsets(0, 8)
    want = mx.mx_grouped_product(x, w, off)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mx.mx_grouped_product(x, w, off)
    graph.replay()
    assert mx.mx_get_error() == 0 and torch.equal(out, want)
    off.copy_(offsets(0, 9))
    graph.replay()
    assert mx.mx_get_error() == 4


# ---------------------------------------------------------------- the C ABI one to one

@pytest.mark.parametrize("fmt", range(4))
def test_the_unchecked_wrappers_do_the_same(fmt):
    n, d, f, E = 9, 64, 96, 2
    x, r, gain, g = bf16(1, n, d), bf16(2, n, d), bf16(3, d), torch.full((1,), 2.0**-6, device="cuda")
    pos, off = torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda")[:, None].contiguous(), offsets(0, 4, n)
    new = lambda cols: mx.mx_rows(fmt, n, cols)
    a, ws = new(d), mx.mx_workspace()
    mx.moe_mx_quantise(fmt, n, 1, d, x, d, pos, g, n, a.codes, a.scales)
    want = mx.mx_quantise(x, fmt, positions=pos, global_scale=g)
    assert same(a, want)
    back = torch.empty_like(x)
    mx.moe_mx_dequantise(fmt, n, d, a.codes, a.scales, g, back, d)
    assert torch.equal(back, mx.mx_dequantise(want))
    total = torch.empty_like(x)
    mx.moe_mx_add_rmsnorm(fmt, n, 1, d, x, d, r, d, gain, 1e-6, pos, g, n, total, a.codes, a.scales)
    want, sums = mx.mx_add_rmsnorm(x, r, gain, 1e-6, fmt, positions=pos, global_scale=g)
    assert same(a, want) and torch.equal(total, sums)
    gate_up, down = weights(fmt, E, f, d, 4, up=True), weights(fmt, E, d, f, 6)
    h = new(f)
    mx.moe_mx_grouped_swiglu(gate_up.struct(), n, a.codes, a.scales, g, off, g, h.codes, h.scales, ws)
    hidden = mx.mx_grouped_swiglu(want, gate_up, off, h_global=g)
    assert same(h, hidden)
    y = torch.empty(n, d, dtype=torch.bfloat16, device="cuda")
    mx.moe_mx_grouped_product(down.struct(), n, h.codes, h.scales, g, off, y, mx.MOE_MX_OUT_BF16, n, d, None, None, ws)
    assert torch.equal(y, mx.mx_grouped_product(hidden, down, off)) and mx.moe_get_error(ws) == mx.MOE_OK
    with pytest.raises(mx.MoeError):
        mx.moe_mx_quantise(fmt, n, 0, d, x, d, pos, g, n, a.codes, a.scales)
