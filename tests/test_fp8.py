"""The FP8 operators on the GPU against plain statements (fp8_plain.py)."""

import math

import pytest
import torch

import mixture_experts_ffn_infer_gb300 as mx
from tests import fp8_plain as plain

pytestmark = pytest.mark.gpu
DTYPES = {mx.MOE_FP8_OUT_BF16: torch.bfloat16, mx.MOE_FP8_OUT_F16: torch.float16, mx.MOE_FP8_OUT_F32: torch.float32}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def bf16(seed, *shape):
    return torch.randn(*shape, generator=gen(seed)).to(torch.bfloat16)


def codes_of(seed, *shape):
    return (torch.randn(*shape, generator=gen(seed)) * 100).to(torch.float8_e4m3fn).view(torch.uint8)


def finite_codes(seed, *shape):
    return (torch.randn(*shape, generator=gen(seed)) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def scales_of(seed, *shape):
    return torch.rand(*shape, generator=gen(seed)) * 0.01 + 1e-4


def within(got, want, tol, slack=0.0):
    """NaN where want is (the random codes hold e4m3's NaN here and there), within tol elsewhere."""
    nan = want.isnan()
    assert torch.equal(got.isnan(), nan)
    return bool(((got - want).abs() <= tol + slack)[~nan].all())


def same_bits(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


def ragged(seed, rows, experts):
    cut = torch.randint(0, rows + 1, (experts - 1,), generator=gen(seed)).sort().values
    return [0, *cut.tolist(), rows]


def same_rows(got, codes, scales):
    # (a quotient of -0 keeps no sign)
    a, b = (t.cpu().view(torch.float8_e4m3fn).float() for t in (got.codes, codes))
    n = scales.shape[1]
    assert torch.equal(a, b)
    assert torch.equal(got.scales.cpu()[:, :n].nan_to_num(-1.0), scales.nan_to_num(-1.0))


# ---------------------------------------------------------------- rows

@pytest.mark.parametrize("n", [1, 5, 400])
@pytest.mark.parametrize("d", [16, 112, 128, 144, 1024, 2080, 7168, 16384])
def test_rows(n, d):
    if n * d > 1 << 22:
        n = 310
    x = bf16(n + d, n, d)
    r = mx.fp8_quantise(x.cuda())
    codes, scales = plain.quantise(x)
    same_rows(r, codes, scales)
    back = mx.fp8_dequantise(r).cpu()
    assert torch.equal(back, plain.values(codes, scales).float().to(torch.bfloat16))


def test_rows_of_odd_values():
    d = 128 * 9
    x = bf16(1, 12, d)
    x[0] = 0
    x[1, 130] = math.nan
    x[2, 5] = math.inf
    x[3, 1000] = -math.inf
    x[4] = torch.finfo(torch.bfloat16).max
    x[5] = 2.0**-133                              # the smallest bf16
    x[6, :128] = 2.0**-130
    x[7] *= 2.0**100
    x[8] *= 2.0**-100
    x[9, ::128] = 1e30                            # one large value a block
    # ties of every kind: 448 makes the scale 1
    x[10] = (torch.arange(d) % 2048 / 16.0).to(torch.bfloat16)
    x[10, ::128] = 448.0
    x[11] = (torch.arange(d) / 1024.0).to(torch.bfloat16)
    x[11, ::128] = -448.0
    r = mx.fp8_quantise(x.cuda())
    codes, scales = plain.quantise(x)
    same_rows(r, codes, scales)
    back = mx.fp8_dequantise(r).cpu()
    want = plain.values(codes, scales).float().to(torch.bfloat16)
    assert torch.equal(back.nan_to_num(7.0), want.nan_to_num(7.0))


def test_values_are_rounded_to_fp32_and_then_to_bf16():
    # scales by which some codes' products have more bits than fp32 and round there to halfway between two bf16
    codes = torch.arange(0x78, 0x7f, dtype=torch.uint8)                    # 256 to 448: four bits
    scales = (2**23 + torch.randint(0, 2**23, (1 << 18,), generator=gen(1))).float() * 2.0**-30
    v = codes.view(torch.float8_e4m3fn).double()[None] * scales.double()[:, None]
    half = (v.float().view(torch.int32) & 0xffff == 0x8000) & (v.float().double() != v)
    scales = scales[half.any(1)]
    assert len(scales) > 4
    r = mx.Fp8Rows(torch.zeros(len(scales), 16, dtype=torch.uint8), torch.zeros(len(scales), 4))
    r.codes[:, :7], r.codes[:, 8:15] = codes, codes | 0x80
    r.scales[:, 0] = scales
    got = mx.fp8_dequantise(mx.Fp8Rows(r.codes.cuda(), r.scales.cuda())).cpu()
    want = (r.codes.view(torch.float8_e4m3fn).float() * r.scales[:, :1]).to(torch.bfloat16)
    assert torch.equal(got, want)


@pytest.mark.parametrize("n,k,d", [(1, 1, 256), (7, 3, 400), (350, 8, 128), (320, 9, 1040), (33, 20, 2048)])
def test_positions(n, k, d):
    x = bf16(n, n, d)
    out_rows = n * k + 5
    at = torch.randperm(out_rows, generator=gen(k))[:n * k].reshape(n, k).to(torch.int32)
    if n > 3:
        at[0, 0], at[1, -1], at[2, 0] = -1, out_rows, 1 << 30
    codes, scales = plain.quantise(x)
    out = mx.fp8_rows(out_rows, d)
    out.codes.fill_(0x11)
    out.scales.fill_(-5.0)
    got = mx.fp8_quantise(x.cuda(), positions=at.cuda(), out=out)
    assert got is out
    want_c, want_s = torch.full((out_rows, d), 0x11, dtype=torch.uint8), torch.full(tuple(out.scales.shape), -5.0)
    for t in range(n):
        for j in range(k):
            if 0 <= at[t, j] < out_rows:
                want_c[at[t, j]] = codes[t]
                want_s[at[t, j], :scales.shape[1]] = scales[t]
    same_rows(out, want_c, want_s)


def test_strided_rows():
    for a, d, width in ((0, 256, 264), (8, 400, 1000), (16, 128, 144)):
        x = bf16(d, 330, width).cuda()
        for n in (330, 3, 1):
            rows = x[:n, a:a + d]
            same_rows(mx.fp8_quantise(rows), *plain.quantise(rows.cpu()))
        r = mx.fp8_quantise(x[:, a:a + d])
        room = torch.full_like(x, 3.0)
        mx.fp8_dequantise(r, out=room[:, a:a + d])
        assert torch.equal(room[:, a:a + d], mx.fp8_dequantise(r))
        assert (room[:, :a] == 3).all() and (room[:, a + d:] == 3).all()


# ---------------------------------------------------------------- packing

@pytest.mark.parametrize("E,n_out,k", [(1, 1, 16), (2, 256, 128), (3, 257, 144), (1, 130, 400), (2, 1000, 272)])
def test_packed_bytes(E, n_out, k):
    codes, scales = codes_of(E, E, n_out, k), scales_of(1, E, plain.blocks(n_out), plain.blocks(k))
    w = mx.fp8_pack(codes.cuda(), scales.cuda())
    assert (w.num_experts, w.n_out, w.k) == (E, n_out, k) and torch.equal(w.packed.cpu(), plain.packed(codes))
    if n_out % 16 == 0:
        t = mx.fp8_pack(codes.cuda().view(torch.float8_e4m3fn), scales.cuda(), transpose=True)
        assert (t.num_experts, t.n_out, t.k) == (E, k, n_out)
        assert torch.equal(t.packed.cpu(), plain.packed(codes.transpose(1, 2).contiguous()))
        assert torch.equal(t.scales.cpu(), scales.transpose(1, 2))


def test_the_banks_tiled_layout_is_the_packed_one():
    # moe_pack_weights' down matrix, as a serving program already holds it
    E, d, f = 2, 384, 256
    codes = codes_of(3, E, d, f).cuda()
    bank = type("Bank", (), dict(w_gate=codes.view(E, f, d), w_up=codes.view(E, f, d), w_down=codes, s_gate=None, s_up=None, s_down=None))
    tiled = mx.pack_bank(bank).w_down
    assert torch.equal(tiled, mx.fp8_pack(codes, scales_of(1, E, 3, 2).cuda()).packed)


# ---------------------------------------------------------------- products

def make(seed, rows, E, n_out, k):
    x = mx.Fp8Rows(codes_of(seed, rows, k).cuda(), torch.full((rows, mx.moe_fp8_scale_pitch(k)), math.nan).cuda())
    x.scales[:, :plain.blocks(k)] = scales_of(seed + 1, rows, plain.blocks(k)).cuda()
    codes, scales = codes_of(seed + 2, E, n_out, k), scales_of(seed + 3, E, plain.blocks(n_out), plain.blocks(k))
    return x, mx.fp8_pack(codes.cuda(), scales.cuda()), plain.weight_values(codes, scales)


def check_product(x, w, wv, offsets, out_type=mx.MOE_FP8_OUT_BF16):
    xv = plain.values(x.codes.cpu(), x.scales.cpu())
    out = torch.full((x.rows, -(-w.n_out // 16) * 16), -77.0, dtype=DTYPES[out_type], device="cuda")[:, :w.n_out]
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    ws = mx.mx_workspace()
    got = mx.fp8_grouped_product(x, w, off, out=out, out_type=out_type, ws=ws)
    assert mx.moe_get_error(ws) == mx.MOE_OK and got is out
    want, size = plain.product(xv, wv, offsets)
    got = got.cpu().double()
    mine = torch.zeros(x.rows, dtype=torch.bool)
    mine[offsets[0]:offsets[-1]] = True
    assert within(got[mine], want[mine], plain.tolerance(want, size, w.k, DTYPES[out_type])[mine])
    assert (got[~mine] == -77).all()
    return got


@pytest.mark.parametrize("out_type", DTYPES)
@pytest.mark.parametrize("rows,E,n_out,k", [(1, 1, 16, 16), (1, 1, 256, 128), (8, 3, 300, 272), (16, 1, 1, 144),
                                            (129, 1, 128, 256), (257, 2, 513, 400), (300, 7, 1001, 1040),
                                            (700, 1, 384, 640), (64, 64, 128, 128), (40, 1024, 32, 32),
                                            (2500, 5, 272, 160), (5000, 2, 640, 304)])
def test_product(out_type, rows, E, n_out, k):
    x, w, wv = make(rows + n_out, rows, E, n_out, k)
    check_product(x, w, wv, ragged(rows, rows, E), out_type)


@pytest.mark.parametrize("rows,E,n_out,k", [(3000, 1, 1500, 512), (1300, 3, 2000, 256), (152 * 64, 2, 512, 128)])
def test_product_of_many_units(rows, E, n_out, k):
    x, w, wv = make(1, rows, E, n_out, k)
    check_product(x, w, wv, ragged(2, rows, E))


@pytest.mark.parametrize("rows,E,n_out,k,sizes", [
    (100, 19, 2048, 272, None),                    # few rows of many experts
    (1300, 4, 2001, 7168, [130, 0, 1, 1169]),      # tiles of 256 rows: their second half with 2 rows, none, 17
    (1400, 3, 2000, 7168, [0, 511, 777]),
    (6000, 3, 1000, 2064, [257, 3000, 2500])])     # (rows that no expert has)
def test_product_of_each_tile(rows, E, n_out, k, sizes):
    x, w, wv = make(7, rows, E, n_out, k)
    offsets = ragged(3, rows, E) if sizes is None else [sum(sizes[:e]) for e in range(E + 1)]
    for out_type in DTYPES:
        check_product(x, w, wv, offsets, out_type)


def test_large_tiles_with_positions_weights_and_values_that_are_not_finite():
    rows, E, n_out, k = 1300, 2, 2003, 7168
    x, w, wv = make(8, rows, E, n_out, k)
    x.scales[700, 3], x.codes[20, 7000] = math.inf, 0x7f
    offsets = [0, 645, rows]
    want, size = plain.product(plain.values(x.codes.cpu(), x.scales.cpu()), wv, offsets)
    at = torch.randperm(rows + 9, generator=gen(1))[:rows].to(torch.int32)
    at[130], at[900] = rows + 9, -5
    weight = torch.rand(rows + 9, generator=gen(2)) * 3 - 1
    room = torch.full((rows + 9, n_out + 5), 9.0, dtype=torch.bfloat16, device="cuda")
    mx.fp8_grouped_product(x, w, torch.tensor(offsets, dtype=torch.int32, device="cuda"), out=room[:, 3:3 + n_out],
                           out_pos=at.cuda(), row_weight=weight.cuda())
    got = room.cpu().double()
    assert (got[:, :3] == 9).all() and (got[:, 3 + n_out:] == 9).all()
    on = (at >= 0) & (at < rows + 9)
    odd = torch.zeros(rows, dtype=torch.bool)
    odd[[20, 700]] = True
    assert not got[at[odd].long(), 3:3 + n_out].isfinite().any()
    on &= ~odd
    to, f = at[on].long(), weight.double()[at[on].long()][:, None]
    tol = plain.tolerance(want, size, k, torch.bfloat16)
    assert within(got[to, 3:3 + n_out], want[on] * f, tol[on] * f.abs(), 1e-30)
    rest = torch.ones(rows + 9, dtype=torch.bool)
    rest[at[(at >= 0) & (at < rows + 9)].long()] = False
    assert (got[rest] == 9).all()


@pytest.mark.parametrize("out_type", DTYPES)
@pytest.mark.parametrize("sizes,n_out,k", [([32], 300, 272), ([17], 1001, 144), ([33, 0, 16, 41], 129, 1552), ([64], 64, 640)])
def test_few_rows_with_positions_and_weights(out_type, sizes, n_out, k):
    rows, E = sum(sizes), len(sizes)
    x, w, wv = make(rows, rows, E, n_out, k)
    offsets = [sum(sizes[:e]) for e in range(E + 1)]
    check_product(x, w, wv, offsets, out_type)
    want, size = plain.product(plain.values(x.codes.cpu(), x.scales.cpu()), wv, offsets)
    tol = plain.tolerance(want, size, k, DTYPES[out_type])
    at = torch.randperm(rows + 6, generator=gen(1))[:rows].to(torch.int32)
    at[2], at[rows - 1] = -1, rows + 6
    weight = torch.rand(rows + 6, generator=gen(2)) * 3 - 1
    room = torch.full((rows + 6, n_out + 3), 9.0, dtype=DTYPES[out_type], device="cuda")
    mx.fp8_grouped_product(x, w, torch.tensor(offsets, dtype=torch.int32, device="cuda"), out=room[:, 1:1 + n_out],
                           out_pos=at.cuda(), row_weight=weight.cuda(), out_type=out_type)
    got = room.cpu().double()
    on = (at >= 0) & (at < rows + 6)
    to, f = at[on].long(), weight.double()[at[on].long()][:, None]
    assert within(got[to, 1:1 + n_out], want[on] * f, tol[on] * f.abs(), 1e-30)
    rest = torch.ones(rows + 6, dtype=torch.bool)
    rest[to] = False
    assert (got[rest] == 9).all() and (got[:, 0] == 9).all() and (got[:, 1 + n_out:] == 9).all()


def test_rows_of_no_expert_stay():
    x, w, wv = make(5, 400, 3, 260, 144)
    for offsets in ([7, 7, 150, 390], [0, 0, 0, 0], [400, 400, 400, 400], [129, 130, 131, 132]):
        check_product(x, w, wv, offsets)


@pytest.mark.parametrize("offsets", [[0, 20, 10, 40], [-1, 10, 20, 40], [0, 10, 20, 41]])
def test_offsets_that_do_not_ascend_compute_nothing(offsets):
    x, w, _ = make(5, 40, 3, 64, 48)
    out, ws = torch.full((40, 64), 5.0, dtype=torch.bfloat16, device="cuda"), mx.mx_workspace()
    mx.fp8_grouped_product(x, w, torch.tensor(offsets, dtype=torch.int32, device="cuda"), out=out, ws=ws)
    assert (out == 5).all() and mx.moe_get_error(ws) == 4 and mx.moe_get_error(ws) == mx.MOE_OK
    mx.mx_get_error()
    mx.fp8_grouped_product(x, w, torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    assert mx.mx_get_error() == 4 and mx.mx_get_error() == mx.MOE_OK


@pytest.mark.parametrize("out_type", DTYPES)
def test_positions_weights_and_unaligned_rows(out_type):
    rows, n_out, k = 300, 333, 272
    x, w, wv = make(9, rows, 2, n_out, k)
    offsets = [0, 170, rows]
    want, size = plain.product(plain.values(x.codes.cpu(), x.scales.cpu()), wv, offsets)
    tol = plain.tolerance(want, size, k, DTYPES[out_type])
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    at = torch.randperm(rows + 20, generator=gen(1))[:rows].to(torch.int32)
    at[3], at[200] = -1, rows + 20
    weight = torch.rand(rows + 20, generator=gen(2)) * 3 - 1
    for width, first in ((n_out, 0), (n_out + 1, 1), (352, 0), (368, 5), (368, 16)):
        room = torch.full((rows + 20, width), 9.0, dtype=DTYPES[out_type], device="cuda")
        out = room[:, first:first + n_out]
        mx.fp8_grouped_product(x, w, off, out=out, out_pos=at.cuda(), row_weight=weight.cuda(), out_type=out_type)
        got = room.cpu().double()
        assert (got[:, :first] == 9).all() and (got[:, first + n_out:] == 9).all()
        on = (at >= 0) & (at < rows + 20)
        to = at[on].long()
        f = weight.double()[to][:, None]
        assert within(got[to, first:first + n_out], want[on] * f, tol[on] * f.abs(), 1e-30)
        rest = torch.ones(rows + 20, dtype=torch.bool)
        rest[to] = False
        assert (got[rest] == 9).all()


def test_values_that_are_not_finite_stay_in_their_rows():
    rows, n_out, k = 140, 200, 400
    x, w, wv = make(2, rows, 1, n_out, k)
    clean = mx.fp8_grouped_product(x, w)
    x.scales[5, 1] = math.nan
    x.codes[17, 3] = 0x7f
    x.scales[130, 0] = math.inf
    got = mx.fp8_grouped_product(x, w)
    keep = torch.ones(rows, dtype=torch.bool)
    keep[[5, 17, 130]] = False
    assert same_bits(got[keep.cuda()], clean[keep.cuda()])
    assert got[5].isnan().all() and got[17].isnan().all() and not got[130].isfinite().any()


def test_f16_beyond_its_range_is_reported():
    x, w, _ = make(3, 20, 1, 64, 128)
    x.scales[7] = 1e6
    ws = mx.mx_workspace()
    got = mx.fp8_grouped_product(x, w, out_type=mx.MOE_FP8_OUT_F16, ws=ws)
    assert not got[7].isfinite().all() and mx.moe_get_error(ws) == 6
    mx.fp8_grouped_product(x, w, ws=ws)
    assert mx.moe_get_error(ws) == mx.MOE_OK


def test_one_expert_needs_no_offsets():
    x, w, wv = make(4, 150, 1, 96, 208)
    got = mx.fp8_grouped_product(x, w)
    assert same_bits(got, mx.fp8_grouped_product(x, w, torch.tensor([0, 150], dtype=torch.int32, device="cuda")))
    none = mx.fp8_grouped_product(mx.Fp8Rows(x.codes[:0], x.scales[:0]), w)
    assert none.shape == (0, 96)


def test_the_rows_gradient_by_the_transposed_weights():
    # y = x W^T, so dL/dx = dy W: against the formula and against differences of sum(dy * y)
    E, n_out, k, rows = 2, 272, 400, 90
    codes, scales = finite_codes(1, E, n_out, k), scales_of(2, E, plain.blocks(n_out), plain.blocks(k))
    back = mx.fp8_pack(codes.cuda(), scales.cuda(), transpose=True)
    offsets = [0, 50, rows]
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    dy = mx.fp8_quantise(bf16(3, rows, n_out).cuda())
    got = mx.fp8_grouped_product(dy, back, off, out_type=mx.MOE_FP8_OUT_F32).cpu().double()
    wv = plain.weight_values(codes, scales)
    dyv = plain.values(dy.codes.cpu(), dy.scales.cpu())
    want, size = plain.product(dyv, wv.transpose(1, 2), offsets)
    assert within(got, want, plain.tolerance(want, size, n_out, torch.float32))
    x, step = torch.randn(rows, k, generator=gen(4), dtype=torch.float64), torch.randn(rows, k, generator=gen(5), dtype=torch.float64)
    f = lambda v: (dyv * plain.product(v, wv, offsets)[0]).sum()
    slope = (f(x + step) - f(x - step)) / 2      # y is linear
    assert abs(slope - (got * step).sum()) <= (plain.tolerance(want, size, n_out, torch.float32) * step.abs()).sum() + 1e-9 * abs(f(x))


def test_offsets_past_32_bits():
    # 40,000 rows of 65,536 codes: their bytes pass 2^31, the output's elements 2^31 as well
    rows, k = 40000, 65536
    codes = torch.randint(0, 100, (rows, k), dtype=torch.uint8, device="cuda")
    x = mx.Fp8Rows(codes, torch.rand(rows, 512, device="cuda") * 0.01)
    wc = codes_of(1, 1, 256, k)
    w = mx.fp8_pack(wc.cuda(), scales_of(2, 1, 2, 512).cuda())
    room = torch.zeros(rows, 60000, dtype=torch.bfloat16, device="cuda")
    got = mx.fp8_grouped_product(x, w, out=room[:, 59000:59256])
    pick = torch.tensor([0, 1, 20000, 32767, 32768, 35000, 39999])
    xv = plain.values(codes[pick.cuda()].cpu(), x.scales[pick.cuda()].cpu())
    want, size = plain.product(xv, plain.weight_values(wc, w.scales.cpu()), [0, len(pick)])
    assert within(got[pick.cuda()].cpu().double(), want, plain.tolerance(want, size, k, torch.bfloat16))
    assert (room[:, :59000] == 0).all() and (room[:, 59256:] == 0).all()
    q = mx.fp8_quantise(room[:, :16384], positions=torch.arange(rows, dtype=torch.int32, device="cuda")[:, None])
    assert (q.codes == 0).all() and (q.scales == 1).all()


# ---------------------------------------------------------------- as a program runs them

def block(x, logits, gate_up, down, k, ws):
    """An FP8 expert block from the operators: route, plan, rows to their positions, products, SwiGLU, back, sum."""
    n, E, d = x.shape[0], down.num_experts, x.shape[1]
    ids, weight = mx.route(logits, k, mx.MOE_SCORE_SIGMOID, scale=2.5)
    _, offsets, sorted_pos, inv_pos = mx.permute(ids, E)
    rows = mx.fp8_quantise(x, positions=inv_pos.view(n, k))
    gu = mx.fp8_grouped_product(rows, gate_up, offsets, ws=ws).float()
    f = gu.shape[1] // 2
    h = (gu[:, :f] * torch.sigmoid(gu[:, :f]) * gu[:, f:]).to(torch.bfloat16)
    out_rows = torch.empty(n * k, d, dtype=torch.float16, device="cuda")
    mx.fp8_grouped_product(mx.fp8_quantise(h), down, offsets, out=out_rows, out_pos=sorted_pos, row_weight=weight.view(-1),
                           out_type=mx.MOE_FP8_OUT_F16, ws=ws)
    out = torch.empty(n, d, dtype=torch.float32, device="cuda")
    mx.moe_combine(mx.dims(d, 128, E, k), n, out_rows, None, None, out, out_is_fp32=True)
    return out, ids, weight


def test_a_block_of_them_beside_the_librarys_own():
    # the same FP8 experts through moe_infer with dynamic activations: same quantisation, other roundings in between
    n, d, f, E, k = 200, 512, 256, 8, 3
    gate, up, down = finite_codes(1, E, f, d), finite_codes(2, E, f, d), finite_codes(3, E, d, f)
    sg, su, sd = (scales_of(s, E, a // 128, b // 128) * 0.01 for s, a, b in ((4, f, d), (5, f, d), (6, d, f)))
    bank = type("Bank", (), {})()
    for name, t in dict(w_gate=gate, w_up=up, w_down=down, s_gate=sg, s_up=su, s_down=sd).items():
        setattr(bank, name, t.cuda())
    gate_up = mx.fp8_pack(torch.cat([gate, up], 1).cuda(), torch.cat([sg, su], 1).cuda())
    dn = mx.fp8_pack(down.cuda(), sd.cuda())
    x, logits, ws = bf16(7, n, d).cuda(), torch.randn(n, E, generator=gen(8)).cuda(), mx.mx_workspace()
    out, ids, weight = block(x, logits, gate_up, dn, k, ws)
    want = mx.infer(x, ids, weight, bank, out_is_fp32=True, act_scheme=mx.MOE_ACT_FP8_DYNAMIC)
    # h differs by two bf16 roundings (2^-8 each) before its e4m3 one, whose half step is 2^-4: a few codes move a step
    assert ((out - want).norm() / want.norm()).item() < 2.0**-4
    held, graph = x.clone(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = block(held, logits, gate_up, dn, k, ws)[0]
    for seed in (11, 7):
        held.copy_(bf16(seed, n, d))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, block(held, logits, gate_up, dn, k, ws)[0])
    assert torch.equal(got, out) and mx.moe_get_error(ws) == mx.MOE_OK


@pytest.mark.parametrize("rows,E,n_out,k", [(1300, 1, 2048, 7168), (5000, 2, 640, 304), (700, 1, 384, 640), (40, 3, 512, 400)])
def test_captured_products_follow_their_inputs(rows, E, n_out, k):
    # each kind of tile, captured and replayed on other rows and other offsets, with another product in front
    x, w, _ = make(1, rows, E, n_out, k)
    other, _, _ = make(2, rows, E, n_out, k)
    first, second = ragged(1, rows, E), ragged(2, rows, E)
    off = torch.tensor(first, dtype=torch.int32, device="cuda")
    held = mx.Fp8Rows(x.codes.clone(), x.scales.clone())
    out, ws = torch.zeros(rows, n_out, dtype=torch.float32, device="cuda"), mx.mx_workspace()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for _ in range(2):
            mx.fp8_grouped_product(held, w, off, out=out, out_type=mx.MOE_FP8_OUT_F32, ws=ws)
    for rows_now, offsets in ((x, first), (other, second), (x, second)):
        held.codes.copy_(rows_now.codes)
        held.scales.copy_(rows_now.scales)
        off.copy_(torch.tensor(offsets, dtype=torch.int32))
        graph.replay()
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        want = mx.fp8_grouped_product(rows_now, w, off, out_type=mx.MOE_FP8_OUT_F32, ws=ws, stream=stream.cuda_stream)
        torch.cuda.synchronize()
        assert same_bits(out, want)
    assert mx.moe_get_error(ws) == mx.MOE_OK


def test_other_streams_share_a_workspace():
    x, w, _ = make(1, 2000, 2, 600, 512)
    off = torch.tensor([0, 900, 2000], dtype=torch.int32, device="cuda")
    want = mx.fp8_grouped_product(x, w, off)
    ws, streams = mx.mx_workspace(), [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [mx.fp8_grouped_product(x, w, off, ws=ws, stream=s) for s in streams for _ in range(4)]
    rows = mx.fp8_quantise(mx.fp8_dequantise(x, stream=streams[0]), stream=streams[0])
    torch.cuda.synchronize()
    assert all(same_bits(g, want) for g in got) and mx.moe_get_error(ws) == mx.MOE_OK and rows.rows == 2000
