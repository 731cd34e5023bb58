"""Paths of the microscaled products and the layer that depend on sizes: clusters inside the layer and with positions,
weights and unaligned rows, long rows whose weights are prefetched, factors that are no power of two, two host threads,
and the layer beside the framework's FP8 block.  Tolerances as in test_mx.py, where the helpers are."""

import threading

import pytest
import torch

import mixture_experts_ffn_infer_gb300 as mx
from mixture_experts_ffn_infer_gb300 import synthetic as syn
from tests import mx_plain as plain
from tests.test_mx import check_codes, close, dev_scalar, gen, grouped, make, offsets_of, rows_of

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- factors

@pytest.mark.parametrize("g", [0.0031, 1.7e-3])
def test_norm_with_a_factor_that_is_no_power_of_two(g):
    n, d = 40, 2080
    x, r, gain = (torch.randn(*s, generator=gen(i)).to(torch.bfloat16) for i, s in enumerate(((n, d), (n, d), (d,))))
    rows, total = mx.mx_add_rmsnorm(x.cuda(), r.cuda(), gain.cuda(), 1e-6, mx.MOE_MX_NVFP4, global_scale=dev_scalar(g))
    v = total.cpu().double()
    check_codes(rows, v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * gain.double(), "nvfp4", rel=40 * 2.0**-24, g=g)


@pytest.mark.parametrize("counts,f,k", [([3, 0, 50], 160, 288), ([20], 160, 3104)])
def test_swiglu_with_a_factor_that_is_no_power_of_two(counts, f, k):
    E, R, hg = len(counts), sum(counts), 0.0021
    x, xv = rows_of(torch.randn(R, k, generator=gen(7), dtype=torch.float64), "nvfp4", 0.002)
    gr, ga, gv = make("nvfp4", E, f, k, 9)
    ur, ua, uv = make("nvfp4", E, f, k, 10, g=0.0007)
    off = offsets_of(counts)
    h = mx.mx_grouped_swiglu(x, mx.mx_pack(gr, E, up=ur, alpha=ga, alpha_up=ua), off.cuda(), h_global=dev_scalar(hg))
    (gy, gabs), (uy, uabs) = grouped(xv, gv, off, R), grouped(xv, uv, off, R)
    acc = (k / 32 + 8) * 2.0**-23
    absolute = 1.1 * gabs * acc * uy.abs() + (gy * torch.sigmoid(gy)).abs() * uabs * acc
    check_codes(h, gy * torch.sigmoid(gy) * uy, "nvfp4", rel=2.0**-20 + gy.abs().max().item() * 2.0**-22,
                absolute=absolute, g=hg)


# ---------------------------------------------------------------- clusters: where the rows go

@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("k", [3104, 6176])       # few units, long rows: clusters of two to eight by format
@pytest.mark.parametrize("out_type,half", [(mx.MOE_MX_OUT_F16, 2.0**-11), (mx.MOE_MX_OUT_BF16, 2.0**-8)])
def test_clusters_with_positions_weights_and_strides(fmt, k, out_type, half):
    counts, n_out, R = [3, 0, 9], 144, 20          # rows 0, 1 and 14.. belong to no expert
    dtype = torch.float16 if out_type == mx.MOE_MX_OUT_F16 else torch.bfloat16
    x, xv = rows_of(torch.randn(R, k, generator=gen(1), dtype=torch.float64), fmt, 0.002)
    wr, alpha, wv = make(fmt, 3, n_out, k, 2)
    off = offsets_of(counts, start=2)
    pos = torch.randperm(R, generator=gen(3)).to(torch.int32)
    pos[3], pos[7] = -1, 30
    weight = torch.rand(30, generator=gen(4)) + 0.5
    w, ws = mx.mx_pack(wr, 3, alpha=alpha), mx.mx_workspace()
    y, a = grouped(xv, wv, off, R)
    for lead in (0, 3, 8):                         # the rows' alignment: vector and scalar stores
        buf = torch.full((30, 160), 7.0, dtype=dtype, device="cuda")
        out = buf[:, lead:lead + n_out]
        mx.mx_grouped_product(x, w, off.cuda(), out=out, out_pos=pos.cuda(), row_weight=weight.cuda(), out_type=out_type,
                              ws=ws)
        assert mx.moe_get_error(ws) == mx.MOE_OK
        left = torch.ones(30, dtype=torch.bool)
        for r in range(2, 14):
            p = int(pos[r])
            if 0 <= p < 30:
                left[p] = False
                f = float(weight[p])
                close(out[p].cpu(), y[r] * f, a[r] * f, k, half)
        keep = torch.ones(160, dtype=torch.bool)
        keep[lead:lead + n_out] = False
        assert (out.cpu()[left] == 7).all() and (buf.cpu()[:, keep] == 7).all()


# ---------------------------------------------------------------- the layer with long rows

D, F, E = 3200, 3104, 2                            # 13 chunks of a 4-bit row, 25 of MXFP8, 50 of bf16


@pytest.fixture(scope="module", params=plain.FORMATS)
def wide(request):
    """Weights of the layer, packed, and their 64-bit values on the GPU."""
    fmt = request.param
    F_ = mx.MX_FORMATS[fmt]
    g = torch.Generator("cuda").manual_seed(5)
    mats = [mx.mx_quantise((torch.randn(E * r, c, generator=g, device="cuda") * 1.2).to(torch.bfloat16), F_)
            for r, c in ((F, D), (F, D), (D, F))]
    # without a factor (1) every value is exact in bf16; the factor, no power of two, comes with the products
    scale = 0.0107
    alpha = torch.full((E,), scale, dtype=torch.float32, device="cuda")
    val = [mx.mx_dequantise(m).double().view(E, -1, m.cols) * alpha.double()[0] for m in mats]
    return {"fmt": fmt, "val": val, "xg": 0.0031 if fmt == "nvfp4" else None, "hg": 0.0021 if fmt == "nvfp4" else None,
            "gate_up": mx.mx_pack(mats[0], E, up=mats[1], alpha=alpha, alpha_up=alpha), "down": mx.mx_pack(mats[2], E, alpha=alpha)}


def inputs(n, k, seed):
    g = gen(seed)
    x, r = (torch.randn(n, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    gain = (1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda()
    ids = torch.rand(n, E, generator=g).topk(k, 1).indices.to(torch.int32).cuda()
    return x, r, gain, ids, torch.softmax(torch.randn(n, k, generator=g), -1).cuda()


def forward(c, x, r, gain, ids, w, **kw):
    return mx.mx_layer_forward(x, r, gain, 1e-6, ids, w, c["gate_up"], c["down"], x_global=dev_scalar(c["xg"]),
                               h_global=dev_scalar(c["hg"]), **kw)


def held(v, fmt, g):
    """64-bit rows as the format holds them."""
    g = 1.0 if g is None else g
    return plain.decode(*plain.encode(v.cpu(), fmt, g), fmt, v.shape[1], g).cuda()


def exact(c, x, r, gain, ids, w):
    total = (x.float() + r.float()).to(torch.bfloat16)
    v = total.double()
    v = held(v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * gain.double(), c["fmt"], c["xg"])
    out = torch.zeros_like(v)
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if len(t):
            gate, up = v[t] @ c["val"][0][e].T, v[t] @ c["val"][1][e].T
            h = held(gate * torch.sigmoid(gate) * up, c["fmt"], c["hg"])
            out.index_add_(0, t, w[t, j].double()[:, None] * (h @ c["val"][2][e].T))
    return total, out


@pytest.mark.parametrize("n,k", [(1, 1), (3, 2), (70, 2), (600, 2)])   # clusters in both products, in one, in none
def test_layer_with_long_rows(wide, n, k):
    args = inputs(n, k, 10 + n)
    total, out = forward(wide, *args, out_is_fp32=True)
    sums, want = exact(wide, *args)
    assert torch.equal(total, sums)
    got = out.double() - total.double()
    # f16 rows (2^-11) and fp32 sums; bf16: h by its last bit.  Else codes of h next to a border: h is off by about
    # 2^-19, and a border lies within that of one value in 2^16 (four times as many and two are allowed); a code off by
    # a step is off by the codes' root mean square at most.
    steps = (2 / (n * k * F) + 2.0**-14) ** 0.5
    assert ((got - want).norm() / want.norm()).item() < 2.0**-9 + (2.0**-8 if wide["fmt"] == "bf16" else steps)
    assert torch.equal(forward(wide, *args, out_is_fp32=True)[1], out)  # bit for bit the same again


@pytest.mark.parametrize("n,k", [(1, 1), (3, 2), (70, 2)])
def test_clusters_in_a_captured_layer_from_a_cleared_workspace(wide, n, k):
    # each replay has other tokens and routing, and nothing of the one before in the workspace
    x, r, gain, ids, w = inputs(n, k, 3)
    ws = torch.zeros(1 << 25, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    xg, hg = dev_scalar(wide["xg"]), dev_scalar(wide["hg"])
    call = lambda **kw: mx.mx_layer_forward(x, r, gain, 1e-6, ids, w, wide["gate_up"], wide["down"], x_global=xg,
                                            h_global=hg, **kw)[1]
    call(ws=ws, stream=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ws.zero_()
        outs = [call(ws=ws) for _ in range(3)]
    for seed in range(20, 24):
        for a, b in zip((x, r, gain, ids, w), inputs(n, k, seed)):
            a.copy_(b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert mx.moe_get_error(ws) == mx.MOE_OK
        want = call()
        for out in outs:
            assert torch.equal(out, want)


def test_two_threads_on_two_streams(wide):
    cases = [inputs(n, 2, 40 + n) for n in (3, 70)]
    want = [forward(wide, *c)[1] for c in cases]
    torch.cuda.synchronize()
    failed = []

    def work(c, y):
        try:
            s, ws = torch.cuda.Stream(), torch.zeros(1 << 25, dtype=torch.uint8, device="cuda")
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                for i in range(40):
                    out = forward(wide, *c, ws=ws if i % 2 else None)[1]
                    if i % 10 == 0 and not torch.equal(out, y):
                        failed.append(i)
            s.synchronize()
            if mx.moe_get_error(ws) != mx.MOE_OK:
                failed.append("error word")
        except Exception as e:  # noqa: BLE001 - reported below
            failed.append(repr(e))

    threads = [threading.Thread(target=work, args=a) for a in zip(cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and mx.mx_get_error() == mx.MOE_OK


# ---------------------------------------------------------------- beside the FP8 block

def test_layer_beside_the_framework_s_block():
    """bf16 experts that hold an FP8 bank's exact values, against the oracle's block.  The block rounds its norm twice to
    bf16 (the normalised row, then its product with the gain); mx_layer_forward rounds once, into the format.  Without
    its norm, on the block's own normalised rows, it is the block."""
    import oracle
    wl = syn.Workload("mx_beside", 24, 512, 256, 6, 2, full_block=True, d_ff_shared=128, seed=12)
    b = syn.make_inputs(wl)
    for s in (b.bank.s_gate, b.bank.s_up, b.bank.s_down):
        s.copy_(torch.exp2(torch.round(torch.log2(s))))          # then code * scale is exact in bf16
    hidden = b.x.cuda()
    want = torch.from_numpy(oracle.layer_forward(b.x, b.gain, b.eps, b.topk_ids, b.topk_weight, b.bank)).cuda()
    routed = want - hidden.double()

    def rows(q, s):
        v = q.view(torch.float8_e4m3fn).float() * s.repeat_interleave(128, 1).repeat_interleave(128, 2)
        held = v.to(torch.bfloat16)
        assert torch.equal(held.float(), v)
        return mx.mx_quantise(held.flatten(0, 1).cuda(), mx.MOE_MX_BF16)

    gate_up = mx.mx_pack(rows(b.bank.w_gate, b.bank.s_gate), 6, up=rows(b.bank.w_up, b.bank.s_up))
    down = mx.mx_pack(rows(b.bank.w_down, b.bank.s_down), 6)
    ids, w, gain = b.topk_ids.cuda(), b.topk_weight.cuda(), b.gain.cuda()
    xn = torch.from_numpy(oracle.rmsnorm(b.x, b.gain, b.eps)).to(torch.bfloat16).cuda()
    _, same = mx.mx_layer_forward(xn, None, None, 0.0, ids, w, gate_up, down, out_is_fp32=True)
    # h once to bf16 (2^-8 of each value at most), f16 rows (2^-11)
    assert ((same.double() - routed).norm() / routed.norm()).item() < 2.0**-8 + 2.0**-11
    total, out = mx.mx_layer_forward(hidden, None, gain, b.eps, ids, w, gate_up, down, out_is_fp32=True)
    assert torch.equal(total, hidden)
    # y differs by three roundings of 2^-8 at most, which silu(gate) * up doubles
    assert ((out.double() - total.double() - routed).norm() / routed.norm()).item() < 7 * 2.0**-8 + 2.0**-11
