"""Microscaled formats on the GPU: rows in and out, the norm, the packed layout, the grouped products and the layer,
against plain 64-bit statements (tests/mx_plain.py).

Quantising bf16 rows has one right answer per bit (correctly rounded divisions, ties to even), so codes and scales are
compared exactly.  Behind an fp32 computation (the norm, the SwiGLU epilogue) the exact value may lie within the
computation's error of a rounding border: there a code must be nearest to the exact quotient to within that error.
Products: half a step of the output type (bf16 2^-8, f16 2^-11) plus fp32 accumulation, at most one rounding of 2^-23
of the absolute sum per 32 columns and a few for the factors."""

import pytest
import torch

import mixture_experts_ffn_infer_gb300 as mx
from tests import mx_plain as plain

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


def bf16(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)


def dev_scalar(v):
    return None if v is None else torch.tensor([v], dtype=torch.float32, device="cuda")


def rows_of(v, fmt, g=None):
    """Library rows from a float64 CPU matrix through the plain encoder, and the values they stand for."""
    g1 = 1.0 if g is None else g
    codes, scales = plain.encode(v, fmt, g1)
    val = plain.decode(codes, scales, fmt, v.shape[1], g1)
    if scales is not None:
        scales = torch.nn.functional.pad(scales, (0, -scales.shape[1] % 16), value=0xA5).cuda()   # padding is ignored
    return mx.MxRows(mx.MX_FORMATS[fmt], v.shape[1], codes.contiguous().cuda(), scales,
                     dev_scalar(g) if fmt == "nvfp4" else None), val


def bits_equal(rows, codes, scales):
    assert torch.equal(rows.codes.cpu(), codes)
    if scales is not None:
        assert torch.equal(rows.scales.cpu()[:, :scales.shape[1]], scales)


# ---------------------------------------------------------------- rows

@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("n,d", [(1, 32), (3, 96), (2, 7168), (33, 2080), (5, 8224), (2, 16384)])
def test_quantise_bits(fmt, n, d):
    x = bf16(gen(n * d), n, d) * torch.exp2(torch.randint(-9, 9, (n, 1), generator=gen(1))).to(torch.bfloat16)
    r = mx.mx_quantise(x.cuda(), mx.MX_FORMATS[fmt])
    bits_equal(r, *plain.encode(x.double(), fmt))
    back = mx.mx_dequantise(r).cpu()
    want = plain.decode(*plain.encode(x.double(), fmt), fmt, d)
    assert torch.equal(back, want.to(torch.bfloat16))


@pytest.mark.parametrize("g", [2.0**-8, 0.0031, 1.7e-3, 11.0])
def test_quantise_nvfp4_factor_bits(g):
    x = bf16(gen(5), 64, 1024, std=1.5)
    r = mx.mx_quantise(x.cuda(), mx.MOE_MX_NVFP4, global_scale=dev_scalar(g))
    bits_equal(r, *plain.encode(x.double(), "nvfp4", g))
    back = mx.mx_dequantise(r).cpu().double()
    want = plain.decode(*plain.encode(x.double(), "nvfp4", g), "nvfp4", 1024, g)
    # the factor times the scale is rounded to 32 bits, then one rounding to bf16
    assert ((back - want).abs() <= want.abs() * (2.0**-8 + 2.0**-22)).all()


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
def test_quantise_ends_of_the_range(fmt):
    x = torch.zeros(1, 512)
    x[0, 32:64] = 3.3e38                       # the largest magnitudes
    x[0, 64:96] = torch.linspace(-1e-38, 1e-38, 32)
    x[0, 96] = 1e-40                            # subnormal
    x[0, 128:160] = -448.0
    x[0, 160:192] = 6.0 * torch.exp2(torch.arange(32.0) - 16)
    x[0, 192:224] = torch.arange(32.0) / 4      # ties
    x[0, 224:256] = 1e-3
    x[0, 224] = 400.0                           # everything else rounds to zero or near it
    x = x.to(torch.bfloat16)
    r = mx.mx_quantise(x.cuda(), mx.MX_FORMATS[fmt])
    bits_equal(r, *plain.encode(x.double(), fmt))


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
def test_quantise_non_finite_stays_in_its_group(fmt):
    x = bf16(gen(2), 4, 256)
    x[0, 40] = float("nan")
    x[1, 100] = float("inf")
    x[2, 255] = float("-inf")
    r = mx.mx_quantise(x.cuda(), mx.MX_FORMATS[fmt])
    bits_equal(r, *plain.encode(x.double(), fmt))
    bad = ~torch.isfinite(x.float()).reshape(4, -1, plain.GROUP[fmt]).all(-1).repeat_interleave(plain.GROUP[fmt], 1)
    assert torch.equal(torch.isnan(mx.mx_dequantise(r).float().cpu()), bad)


@pytest.mark.parametrize("fmt", plain.FORMATS)
def test_quantise_strides_and_positions(fmt):
    wide = bf16(gen(3), 7, 200)
    x = wide.cuda()[:, 8:168]                   # 16-byte aligned rows, 200 apart
    pos = torch.tensor([[3, 20], [0, -1], [99, 7], [1, 2], [4, 5], [6, 8], [10, 24]], dtype=torch.int32)
    out = mx.mx_rows(mx.MX_FORMATS[fmt], 25, 160)
    out.codes.fill_(0x5A)
    mx.mx_quantise(x, mx.MX_FORMATS[fmt], positions=pos.cuda(), out=out)
    codes, scales = plain.encode(wide[:, 8:168].double(), fmt)
    seen = set()
    for t in range(7):
        for p in pos[t].tolist():
            if 0 <= p < 25:
                seen.add(p)
                assert torch.equal(out.codes[p].cpu(), codes[t])
                if scales is not None:
                    assert torch.equal(out.scales[p].cpu()[:scales.shape[1]], scales[t])
    for p in set(range(25)) - seen:
        assert (out.codes[p] == 0x5A).all()


def check_codes(rows, exact, fmt, rel, absolute=0.0, g=1.0):
    """rows' codes are nearest to the 64-bit values `exact`, up to an error of rel * |value| + absolute in them."""
    codes, scales = rows.codes.cpu(), rows.scales.cpu() if rows.scales is not None else None
    err = exact.abs() * rel + absolute
    if fmt == "bf16":
        got = plain.decode(codes, None, fmt, rows.cols)
        assert ((got - exact).abs() <= exact.abs() * 2.0**-8 + err * (1 + 2.0**-8) + 1e-38).all()
        return
    G = plain.GROUP[fmt]
    grp, gerr = exact.reshape(exact.shape[0], -1, G), err.reshape(exact.shape[0], -1, G)
    byte = scales[:, :grp.shape[1]].long()
    low, high = (grp.abs() - gerr).clamp(min=0).amax(-1), (grp.abs() + gerr).amax(-1)
    lo, hi = plain.group_divisor(low, fmt, g)[0], plain.group_divisor(high, fmt, g)[0]
    assert ((lo <= byte) & (byte <= hi)).all()
    div = plain.scale_values(byte, fmt, g)[..., None]
    code = plain.code_values(codes, fmt).reshape(grp.shape)
    lv = plain.levels(fmt)
    at = torch.searchsorted(lv, code.abs())
    up = torch.where(at + 1 < len(lv), (lv[(at + 1).clamp(max=len(lv) - 1)] + lv[at]) / 2, torch.inf)
    dn = torch.where(at > 0, (lv[at] + lv[(at - 1).clamp(min=0)]) / 2, -torch.inf)
    live = div > 0
    t = torch.where(live, grp.abs() / torch.where(live, div, 1.0), 0.0)
    slack = torch.where(live, gerr / torch.where(live, div, 1.0), 0.0) + t * 2.0**-22
    assert ((t >= dn - slack) & (t <= up + slack)).all()
    wrong_sign = (code != 0) & (torch.sign(code) != torch.sign(grp)) & (grp.abs() > gerr)
    assert not wrong_sign.any()


# ---------------------------------------------------------------- norm

@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("n,d,residual", [(1, 7168, True), (9, 32, True), (4, 2080, False), (3, 8192, True), (2, 12000, True)])
def test_add_rmsnorm(fmt, n, d, residual):
    g = gen(d + n)
    x, r, gain = bf16(g, n, d), bf16(g, n, d) if residual else None, (1 + bf16(g, d, std=0.1)).to(torch.bfloat16)
    pos = torch.randperm(n, generator=g).to(torch.int32)[:, None]
    rows, total = mx.mx_add_rmsnorm(x.cuda(), r.cuda() if residual else None, gain.cuda(), 1e-6, mx.MX_FORMATS[fmt],
                                    positions=pos.cuda())
    want = (x.float() + r.float()).to(torch.bfloat16) if residual else x   # one bf16 rounding of an exact fp32 sum
    assert torch.equal(total.cpu(), want)
    v = want.double()
    y = v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * gain.double()
    exact = torch.empty_like(y)
    exact[pos[:, 0].long()] = y
    # fp32: a thread's 8 or 16 squares, ten shuffle sums (each 2^-24), rsqrtf (2 ulp), two products
    check_codes(rows, exact, fmt, rel=40 * 2.0**-24)


@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("d", [32, 512, 544, 1024, 1056, 4128])
def test_many_rows(fmt, d):
    """More rows than SMs: a row to a warp up to 1024 columns (here with a last CTA of three), wider ones a CTA."""
    g = gen(d)
    n, k = 611, 9                               # positions past the eighth as well
    x, r, gain = bf16(g, n, d), bf16(g, n, d), (1 + bf16(g, d, std=0.1)).to(torch.bfloat16)
    F = mx.MX_FORMATS[fmt]
    bits_equal(mx.mx_quantise(x.cuda(), F), *plain.encode(x.double(), fmt))
    pos = torch.full((n, k), -1, dtype=torch.int32)
    pos[:, 8] = torch.randperm(n, generator=g).to(torch.int32)
    pos[:, 3] = pos[:, 8] + n
    out = mx.mx_rows(F, 2 * n, d)
    rows, total = mx.mx_add_rmsnorm(x.cuda(), r.cuda(), gain.cuda(), 1e-6, F, positions=pos.cuda(), out=out)
    want = (x.float() + r.float()).to(torch.bfloat16)
    assert torch.equal(total.cpu(), want)
    v = want.double()
    exact = torch.empty(2 * n, d, dtype=torch.float64)
    exact[pos[:, 8].long()] = exact[pos[:, 3].long()] = v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * gain.double()
    check_codes(rows, exact, fmt, rel=40 * 2.0**-24)


@pytest.mark.parametrize("fmt,g", [("mxfp8", 1.0), ("mxfp4", 1.0), ("nvfp4", 2.0**-8)])
def test_add_rmsnorm_few_codes_off_the_exact_values(fmt, g):
    # y is off by four fp32 roundings (the sum, rsqrtf's two units, two products): 2^-22 at most.  A code differs only
    # with its quotient that near a border, at most 8 borders a binade: 2^-18 of the codes, 14 of 3.7 million, and a
    # group's scale as often, for which its 16 or 32 codes may follow.
    gg = gen(77)
    n, d = 512, 7168
    x, r, gain = bf16(gg, n, d), bf16(gg, n, d), (1 + bf16(gg, d, std=0.1)).to(torch.bfloat16)
    rows, total = mx.mx_add_rmsnorm(x.cuda(), r.cuda(), gain.cuda(), 1e-6, mx.MX_FORMATS[fmt],
                                    global_scale=dev_scalar(g) if fmt == "nvfp4" else None)
    v = total.cpu().double()
    codes, scales = plain.encode(v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * gain.double(), fmt, g)
    groups = rows.scales.cpu()[:, :scales.shape[1]] != scales
    assert groups.sum().item() <= 14
    off = rows.codes.cpu() != codes
    off &= ~groups.repeat_interleave(off.shape[1] // groups.shape[1], 1)
    assert off.sum().item() <= 42               # three times the mean


def test_add_rmsnorm_in_place_and_strided():
    g = gen(8)
    d = 256
    x, r, gain = bf16(g, 6, d), bf16(g, 6, 2 * d), torch.ones(d, dtype=torch.bfloat16)
    a, b = x.cuda(), r.cuda()
    rows, total = mx.mx_add_rmsnorm(a, b[:, :d], gain.cuda(), 1e-6, mx.MOE_MX_MXFP8, sum_out=b[:, :d])
    want = (x.float() + r[:, :d].float()).to(torch.bfloat16)
    assert torch.equal(b.cpu()[:, :d], want) and torch.equal(b.cpu()[:, d:], r[:, d:])
    ref, _ = mx.mx_add_rmsnorm(want.cuda(), None, gain.cuda(), 1e-6, mx.MOE_MX_MXFP8)
    assert torch.equal(rows.codes, ref.codes)


def test_add_rmsnorm_zero_and_non_finite_rows():
    x = torch.zeros(3, 128, dtype=torch.bfloat16)
    x[1, 5] = float("inf")
    x[2] = 1.0
    rows, _ = mx.mx_add_rmsnorm(x.cuda(), None, torch.ones(128, dtype=torch.bfloat16).cuda(), 1e-6, mx.MOE_MX_MXFP4)
    v = mx.mx_dequantise(rows).float().cpu()
    assert (v[0] == 0).all() and (v[2] == 1).all()
    assert torch.isnan(v[1, :32]).all()         # inf / inf; the other groups are finite / inf = 0
    assert (v[1, 32:] == 0).all()


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
def test_add_rmsnorm_groups_near_zero(fmt):
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    x[0, 64:] = bf16(gen(1), 192)               # zero groups beside others
    x[1] = 1e-30 * bf16(gen(2), 256)            # rs = 1000: all of it eps
    x[2, :32] = 2e-39                            # subnormal
    x[3, 5] = 1e-38
    x[3, 200] = -3.0
    rows, _ = mx.mx_add_rmsnorm(x.cuda(), None, torch.ones(256, dtype=torch.bfloat16).cuda(), 1e-6, mx.MX_FORMATS[fmt])
    v = x.double()
    check_codes(rows, v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6), fmt, rel=40 * 2.0**-24, absolute=1e-44)


# ---------------------------------------------------------------- packed weights

@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("pair", [False, True])
def test_pack_layout_bytes(fmt, pair):
    E, n, k = 2, 160 if pair else 300, 352
    g = gen(4)
    mats = [rows_of(torch.randn(E * n, k, generator=g, dtype=torch.float64), fmt)[0] for _ in range(1 + pair)]
    w = mx.mx_pack(mats[0], E, up=mats[1] if pair else None)
    parts = [(m.codes.cpu(), m.scales.cpu() if m.scales is not None else None) for m in mats]
    assert torch.equal(w.packed.cpu(), plain.pack(parts, fmt, E))


# ---------------------------------------------------------------- products

def make(fmt, E, n_out, k, seed, g=0.0009):
    """Packed weights and their float64 values [E, n_out, k]."""
    rows, val = rows_of(torch.randn(E * n_out, k, generator=gen(seed), dtype=torch.float64) * 0.05, fmt,
                        g if fmt == "nvfp4" else None)
    alpha = torch.full((E,), g, dtype=torch.float32, device="cuda") if fmt == "nvfp4" else None
    rows.global_scale = None
    return rows, alpha, val.reshape(E, n_out, k)


def offsets_of(counts, start=0):
    o = [start]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32)


def grouped(x, w, off, rows):
    """(product, sum of absolute terms) in 64 bits; NaN where a row has no expert."""
    y = torch.full((rows, w.shape[1]), torch.nan, dtype=torch.float64)
    a = y.clone()
    for e in range(w.shape[0]):
        lo, hi = int(off[e]), int(off[e + 1])
        y[lo:hi] = x[lo:hi] @ w[e].T
        a[lo:hi] = x[lo:hi].abs() @ w[e].abs().T
    return y, a


def close(got, want, absum, k, half_step):
    tol = want.abs() * half_step * 1.001 + absum * (k / 32 + 8) * 2.0**-23 + 1e-30
    err = (got.double() - want).abs()
    assert (err <= tol).all(), (err / tol).max()


CASES = [  # counts per expert, n_out, k
    ([1], 1, 32),
    ([1], 256, 256),
    ([5], 100, 96),
    ([0, 17, 0, 128, 1, 129], 300, 544),
    ([300, 0, 64], 257, 1056),
    ([33] * 9, 512, 1024),
    ([1300], 300, 288),           # eleven tiles of one expert: two chunks
    ([3], 300, 3104),             # few units, long rows: clusters of two, four and eight by format
    ([100, 0, 1], 257, 6176),
    ([1], 96, 7168),
]


@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("counts,n_out,k", CASES)
def test_grouped_product(fmt, counts, n_out, k):
    E, R = len(counts), sum(counts)
    x, xv = rows_of(torch.randn(R, k, generator=gen(7), dtype=torch.float64), fmt, 0.002)
    wr, alpha, wv = make(fmt, E, n_out, k, 9)
    w = mx.mx_pack(wr, E, alpha=alpha)
    off = offsets_of(counts)
    ws = mx.mx_workspace()
    y = mx.mx_grouped_product(x, w, off.cuda(), ws=ws)
    assert mx.moe_get_error(ws) == mx.MOE_OK
    want, absum = grouped(xv, wv, off, R)
    close(y.cpu(), want, absum, k, 2.0**-8)
    # twice the same: bit for bit
    assert torch.equal(y, mx.mx_grouped_product(x, w, off.cuda(), ws=ws))


@pytest.mark.parametrize("fmt", plain.FORMATS)
def test_grouped_product_positions_weights_f16_strides(fmt):
    counts, n_out, k = [3, 40, 0, 9], 144, 320
    R, E = 60, 4                                   # rows 0, 1 and 54.. belong to no expert
    x, xv = rows_of(torch.randn(R, k, generator=gen(1), dtype=torch.float64), fmt, 0.002)
    wr, alpha, wv = make(fmt, E, n_out, k, 2)
    off = offsets_of(counts, start=2)
    pos = torch.randperm(R, generator=gen(3)).to(torch.int32)
    pos[10] = -1
    pos[11] = 70
    weight = torch.rand(70, generator=gen(4)) + 0.5
    for out_type, dtype, half in ((mx.MOE_MX_OUT_F16, torch.float16, 2.0**-11), (mx.MOE_MX_OUT_BF16, torch.bfloat16, 2.0**-8)):
        for lead in (0, 3, 8):                     # the rows' alignment: vector and scalar stores
            buf = torch.full((70, 160), 7.0, dtype=dtype, device="cuda")
            out = buf[:, lead:lead + n_out]
            ws = mx.mx_workspace()
            mx.mx_grouped_product(x, mx.mx_pack(wr, E, alpha=alpha), off.cuda(), out=out, out_pos=pos.cuda(),
                                  row_weight=weight.cuda(), out_type=out_type, ws=ws)
            assert mx.moe_get_error(ws) == mx.MOE_OK
            y, a = grouped(xv, wv, off, R)
            left = torch.ones(70, dtype=torch.bool)
            for r in range(2, 54):
                p = int(pos[r])
                if 0 <= p < 70:
                    left[p] = False
                    f = float(weight[p])
                    close(out[p].cpu(), y[r] * f, a[r] * f, k, half)
            assert (out.cpu()[left] == 7).all()
            keep = torch.ones(160, dtype=torch.bool)
            keep[lead:lead + n_out] = False
            assert (buf.cpu()[:, keep] == 7).all()


def test_grouped_product_nan_scale_stays_in_its_row():
    x, _ = rows_of(torch.randn(40, 512, generator=gen(1), dtype=torch.float64), "nvfp4")
    x.scales[7, 3] = 0x7F
    wr, alpha, _ = make("nvfp4", 1, 256, 512, 2)
    y = mx.mx_grouped_product(x, mx.mx_pack(wr, 1, alpha=alpha), offsets_of([40]).cuda()).float().cpu()
    bad = torch.zeros(40, dtype=torch.bool)
    bad[7] = True
    assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()


def test_grouped_product_f16_overflow_is_reported():
    x, _ = rows_of(torch.full((4, 256), 300.0, dtype=torch.float64), "bf16")
    w, _ = rows_of(torch.full((32, 256), 300.0, dtype=torch.float64), "bf16")
    ws = mx.mx_workspace()
    y = mx.mx_grouped_product(x, mx.mx_pack(w, 1), offsets_of([4]).cuda(), out_type=mx.MOE_MX_OUT_F16, ws=ws)
    assert mx.moe_get_error(ws) == 6 and torch.isinf(y).all()


@pytest.mark.parametrize("bad", [[0, 5, 3, 8], [-1, 2, 4, 8], [0, 2, 4, 9]])
def test_grouped_product_bad_offsets(bad):
    x, _ = rows_of(torch.randn(8, 64, generator=gen(1), dtype=torch.float64), "mxfp8")
    wr, _, _ = make("mxfp8", 3, 64, 64, 2)
    ws = mx.mx_workspace()
    out = torch.full((8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    mx.mx_grouped_product(x, mx.mx_pack(wr, 3), torch.tensor(bad, dtype=torch.int32).cuda(), out=out, ws=ws)
    assert mx.moe_get_error(ws) == 4 and (out == 7).all()


@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("counts,f,k", [([1], 32, 32), ([3, 0, 50], 160, 288), ([130, 7], 256, 1024), ([20], 160, 3104),
                                        ([1, 0, 2], 96, 7168)])
def test_grouped_swiglu(fmt, counts, f, k):
    E, R = len(counts), sum(counts)
    x, xv = rows_of(torch.randn(R, k, generator=gen(7), dtype=torch.float64), fmt, 0.002)
    gr, ga, gv = make(fmt, E, f, k, 9)
    ur, ua, uv = make(fmt, E, f, k, 10, g=0.0007)
    off = offsets_of(counts)
    hg = 2.0**-9
    h = mx.mx_grouped_swiglu(x, mx.mx_pack(gr, E, up=ur, alpha=ga, alpha_up=ua), off.cuda(),
                             h_global=dev_scalar(hg) if fmt == "nvfp4" else None)
    (gy, gabs), (uy, uabs) = grouped(xv, gv, off, R), grouped(xv, uv, off, R)
    exact = gy * torch.sigmoid(gy) * uy
    acc = (k / 32 + 8) * 2.0**-23
    # d silu / dg is at most 1.1; the fast exponential and division add a few parts in 2^22
    absolute = 1.1 * gabs * acc * uy.abs() + (gy * torch.sigmoid(gy)).abs() * uabs * acc
    rel = 2.0**-20 + gy.abs().max().item() * 2.0**-22
    check_codes(h, exact, fmt, rel=rel, absolute=absolute, g=hg if fmt == "nvfp4" else 1.0)


# ---------------------------------------------------------------- large offsets

def test_offsets_past_32_bits():
    rows, n_out, k = 300_032, 7168, 32             # 2.15e9 output elements; 64-bit row offsets everywhere
    x = torch.randn(rows, k, generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    r = mx.mx_quantise(x, mx.MOE_MX_MXFP8)
    wr, _, wv = make("mxfp8", 1, n_out, k, 2)
    y = mx.mx_grouped_product(r, mx.mx_pack(wr, 1), torch.tensor([0, rows], dtype=torch.int32).cuda())
    back = mx.mx_quantise(y, mx.MOE_MX_MXFP8)
    for at in (0, 299_593, rows - 1):
        xv = plain.decode(r.codes[at:at + 1].cpu(), r.scales[at:at + 1].cpu(), "mxfp8", k)
        close(y[at:at + 1].cpu(), xv @ wv[0].T, xv.abs() @ wv[0].abs().T, k, 2.0**-8)
        codes, scales = plain.encode(y[at:at + 1].cpu().double(), "mxfp8")
        assert torch.equal(back.codes[at:at + 1].cpu(), codes)
        assert torch.equal(back.scales[at:at + 1].cpu()[:, :scales.shape[1]], scales)
    del y
    v = mx.mx_dequantise(back)
    want = plain.decode(back.codes[-1:].cpu(), back.scales[-1:].cpu(), "mxfp8", n_out)
    assert torch.equal(v[-1:].cpu(), want.to(torch.bfloat16))


# ---------------------------------------------------------------- the layer

def layer_case(fmt, n, d, E, k, f, seed):
    g = gen(seed)
    c = {"x": bf16(g, n, d), "res": bf16(g, n, d), "gain": (1 + bf16(g, d, std=0.1)).to(torch.bfloat16)}
    c["ids"] = torch.rand(n, E, generator=g).topk(k, 1).indices.to(torch.int32)
    c["w"] = torch.softmax(torch.randn(n, k, generator=g), -1)
    gr, ga, gv = make(fmt, E, f, d, seed + 1)
    ur, ua, uv = make(fmt, E, f, d, seed + 2)
    dr, da, dv = make(fmt, E, d, f, seed + 3)
    c["gate_up"], c["down"] = mx.mx_pack(gr, E, up=ur, alpha=ga, alpha_up=ua), mx.mx_pack(dr, E, alpha=da)
    c["val"] = gv, uv, dv
    c["xg"], c["hg"] = (2.0**-8, 2.0**-9) if fmt == "nvfp4" else (None, None)
    return c


def layer_exact(c, fmt, norm=True):
    v = c["x"].double()
    if norm:
        total = (c["x"].float() + c["res"].float()).to(torch.bfloat16).double()
        v = total / torch.sqrt((total * total).mean(1, keepdim=True) + 1e-6) * c["gain"].double()
    def q(t, g):
        g = 1.0 if g is None else g
        return plain.decode(*plain.encode(t, fmt, g), fmt, t.shape[1], g)
    v = q(v, c["xg"])
    gv, uv, dv = c["val"]
    out = total.clone() if norm else torch.zeros_like(v)
    for t in range(v.shape[0]):
        for j, e in enumerate(c["ids"][t].tolist()):
            gy, uy = gv[e] @ v[t], uv[e] @ v[t]
            out[t] += float(c["w"][t, j]) * (dv[e] @ q((gy * torch.sigmoid(gy) * uy)[None], c["hg"])[0])
    return out


def run_layer(c, fmt, norm=True, **kw):
    return mx.mx_layer_forward(c["x"].cuda(), c["res"].cuda() if norm else None, c["gain"].cuda() if norm else None, 1e-6,
                               c["ids"].cuda(), c["w"].cuda(), c["gate_up"], c["down"],
                               x_global=dev_scalar(c["xg"]), h_global=dev_scalar(c["hg"]), **kw)


@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("n,d,E,k,f", [(1, 256, 5, 3, 96), (70, 384, 6, 2, 160), (300, 128, 2, 1, 64)])
def test_layer(fmt, n, d, E, k, f):
    c = layer_case(fmt, n, d, E, k, f, 3)
    total, out = run_layer(c, fmt, out_is_fp32=True)
    assert torch.equal(total.cpu(), (c["x"].float() + c["res"].float()).to(torch.bfloat16))
    want = layer_exact(c, fmt) - total.cpu().double()
    got = out.cpu().double() - total.cpu().double()
    # f16 rows (2^-11), fp32 sums; a code of the few that lie within 2^-20 of a border may differ by a step
    # (at most a quarter of its value), as bf16's h may by its last bit
    assert ((got - want).norm() / want.norm()).item() < 2.0**-9 + (2.0**-8 if fmt == "bf16" else 0.25 * 2.0**-7)
    _, plainly = run_layer(c, fmt, norm=False, out_is_fp32=True)
    want = layer_exact(c, fmt, norm=False)
    assert ((plainly.cpu().double() - want).norm() / want.norm()).item() < 2.0**-9 + (2.0**-8 if fmt == "bf16" else 0.25 * 2.0**-7)
    _, half = run_layer(c, fmt)
    assert torch.equal(half, out.to(torch.bfloat16))


def test_layer_bad_ids_are_reported_and_skipped():
    c = layer_case("mxfp8", 40, 128, 4, 2, 64, 6)
    _, good = run_layer(c, "mxfp8")
    c["ids"][3, 1] = 4
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    _, out = run_layer(c, "mxfp8", ws=ws)
    assert mx.moe_get_error(ws) == 4
    others = [t for t in range(40) if t != 3]
    assert torch.equal(out[others], good[others])


def test_layer_graph_and_other_stream():
    c = layer_case("nvfp4", 20, 256, 8, 4, 128, 12)
    _, want = run_layer(c, "nvfp4")
    x, res, gain, ids, w = (c[p].cuda() for p in ("x", "res", "gain", "ids", "w"))
    xg, hg = dev_scalar(c["xg"]), dev_scalar(c["hg"])
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    call = lambda: mx.mx_layer_forward(x, res, gain, 1e-6, ids, w, c["gate_up"], c["down"], x_global=xg, h_global=hg,
                                       ws=ws, stream=s)
    _, eager = call()
    s.synchronize()
    assert torch.equal(eager, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        _, out = call()
    x.copy_(x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    _, again = mx.mx_layer_forward(x, res, gain, 1e-6, ids, w, c["gate_up"], c["down"], x_global=xg, h_global=hg)
    assert torch.equal(out, again) and not torch.equal(out, want)


@pytest.mark.parametrize("n", [1, 20, 3000])   # the routing plan in one kernel, and in several
def test_layer_graph_with_nothing_left_in_the_workspace(n):
    # each replay starts from a cleared workspace and other routing: a kernel that read the plan, or the rows, before
    # they are written would give something else
    c = layer_case("mxfp8", n, 256, 8, 4, 128, 21)
    x, res, gain, ids, w = (c[p].cuda() for p in ("x", "res", "gain", "ids", "w"))
    ws = torch.zeros(1 << 25, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    args = (x, res, gain, 1e-6, ids, w, c["gate_up"], c["down"])
    mx.mx_layer_forward(*args, ws=ws, stream=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ws.zero_()
        outs = [mx.mx_layer_forward(*args, ws=ws)[1] for _ in range(3)]
    for k in range(4):
        ids.copy_(torch.rand(n, 8, generator=gen(k)).topk(4, 1).indices.to(torch.int32))
        x.copy_(bf16(gen(50 + k), n, 256))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        fresh = torch.zeros(1 << 25, dtype=torch.uint8, device="cuda")
        _, want = mx.mx_layer_forward(*args, ws=fresh)
        torch.cuda.synchronize()
        for out in outs:
            assert torch.equal(out, want)


def test_layer_inputs_written_right_before_the_call():
    # weights, rows and routing overwritten by the kernels in front of the call: nothing may be read ahead of them
    c, o = layer_case("mxfp4", 40, 256, 8, 4, 128, 31), layer_case("mxfp4", 40, 256, 8, 4, 128, 41)
    _, want = run_layer(o, "mxfp4")
    names = ("x", "res", "gain", "ids", "w")
    a, b = [[t[p].cuda() for p in names] for t in (c, o)]
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    call = lambda: mx.mx_layer_forward(a[0], a[1], a[2], 1e-6, a[3], a[4], c["gate_up"], c["down"], ws=ws)[1]
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        for t, u in zip(a, b):
            t.copy_(u)
        c["gate_up"].packed.copy_(o["gate_up"].packed)
        c["down"].packed.copy_(o["down"].packed)
        out = call()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


class Guarded:
    """Device buffers with 4 KB of a fixed pattern on either side of each."""

    def __init__(self):
        self.all = []

    def bytes(self, *shape):
        n = 1
        for v in shape:
            n *= v
        buf = torch.full((8192 + (n + 255) // 256 * 256,), 0xC3, dtype=torch.uint8, device="cuda")
        self.all.append((buf, n))
        return buf[4096:4096 + n].view(*shape)

    def like(self, dtype, *shape):
        size = torch.empty(0, dtype=dtype).element_size()
        return self.bytes(*shape[:-1], shape[-1] * size).view(dtype)

    def rows(self, fmt, n, cols):
        pitch = mx.moe_mx_scale_pitch(fmt, cols)
        return mx.MxRows(fmt, cols, self.bytes(n, mx.moe_mx_code_bytes(fmt, cols)), self.bytes(n, pitch) if pitch else None)

    def check(self):
        torch.cuda.synchronize()
        for buf, n in self.all:
            assert (buf[:4096] == 0xC3).all() and (buf[4096 + n:] == 0xC3).all()


@pytest.mark.parametrize("fmt", plain.FORMATS)
def test_nothing_is_written_beside_the_outputs(fmt):
    F, g = mx.MX_FORMATS[fmt], gen(6)
    n, k, d, f, E = 45, 2, 256, 160, 3
    m = Guarded()
    x, res, gain = bf16(g, n, d).cuda(), bf16(g, n, d).cuda(), torch.ones(d, dtype=torch.bfloat16).cuda()
    pos = torch.randperm(n * k, generator=g).to(torch.int32).reshape(n, k).cuda()
    q = m.rows(F, n * k, d)
    mx.mx_quantise(x, F, positions=pos, out=q)
    mx.mx_add_rmsnorm(x, res, gain, 1e-6, F, positions=pos, out=q, sum_out=m.like(torch.bfloat16, n, d))
    mx.mx_dequantise(q, out=m.like(torch.bfloat16, n * k, d))
    gu = [rows_of(torch.randn(E * f, d, generator=g, dtype=torch.float64), fmt)[0] for _ in range(2)]
    dn = rows_of(torch.randn(E * d, f, generator=g, dtype=torch.float64), fmt)[0]
    w1, w2 = mx.mx_pack(gu[0], E, up=gu[1]), mx.mx_pack(dn, E)
    for w, parts in ((w1, gu), (w2, [dn])):
        packed = m.bytes(w.packed.numel())
        mx.moe_mx_pack_weights(w.struct(), parts[0].codes, parts[0].scales, parts[-1].codes, parts[-1].scales, packed)
        assert torch.equal(packed, w.packed)
    off = offsets_of([40, 0, 50]).cuda()
    h, ws = m.rows(F, n * k, f), m.bytes(256)
    ws.zero_()
    mx.mx_grouped_swiglu(q, w1, off, out=h, ws=ws)
    mx.mx_grouped_product(h, w2, off, out=m.like(torch.bfloat16, n * k, d), ws=ws)
    assert mx.moe_get_error(ws) == mx.MOE_OK
    size = mx.moe_mx_layer_workspace_size(w1.struct(), w2.struct(), k, n)
    ids = torch.rand(n, E, generator=g).topk(k, 1).indices.to(torch.int32).cuda()
    wt = torch.rand(n, k, generator=g).cuda()
    total, out, lws = m.like(torch.bfloat16, n, d), m.like(torch.bfloat16, n, d), m.bytes(size)
    mx.moe_mx_layer_forward(w1.struct(), w2.struct(), k, n, x, res, gain, 1e-6, ids, wt, None, None, total, out, lws)
    assert mx.moe_get_error(lws) == mx.MOE_OK
    m.check()


def test_calls_hold_no_references():
    import sys
    x = torch.randn(4, 64, device="cuda").to(torch.bfloat16)
    gain, pos, g = torch.ones(64, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 1, dtype=torch.int32, device="cuda"), dev_scalar(1.0)
    w = mx.mx_pack(make("nvfp4", 1, 64, 64, 1)[0], 1, alpha=dev_scalar(2.0))
    off = offsets_of([4]).cuda()
    held = [x, gain, pos, g, w, w.packed, w.alpha, off]
    before = None
    for i in range(60):
        rows, total = mx.mx_add_rmsnorm(x, x, gain, 1e-6, 3, positions=pos, global_scale=g)
        out = mx.mx_quantise(x, 3, global_scale=g, out=rows)
        assert out is rows
        y = mx.mx_grouped_product(rows, w, off)
        mx.mx_dequantise(rows, out=total)
        with pytest.raises(ValueError):
            mx.mx_grouped_product(rows, w, off.long())
        counts = [sys.getrefcount(o) for o in (*held, rows, rows.codes, total, y, None, mx.MxRows)]
        if i == 5:
            before = torch.cuda.memory_allocated(), counts
    assert torch.cuda.memory_allocated() == before[0]
    assert all(abs(a - b) < 10 for a, b in zip(counts, before[1]))


def test_rows_of_nothing():
    w = mx.mx_pack(make("mxfp4", 2, 64, 64, 1)[0], 2)
    x = mx.mx_rows(mx.MOE_MX_MXFP4, 0, 64)
    assert mx.mx_grouped_product(x, w, torch.zeros(3, dtype=torch.int32, device="cuda")).shape == (0, 64)
    r = mx.mx_quantise(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), mx.MOE_MX_MXFP4)
    assert mx.mx_dequantise(r).shape == (0, 64)
