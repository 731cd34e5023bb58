"""The router's choice, balance loss and gradient on the GPU against plain 64-bit statements (router_plain.py)."""

import math

import pytest
import torch

import mixture_experts_ffn_infer_gb300 as mx
from tests import router_plain as plain
from tests.router_plain import EPS

pytestmark = pytest.mark.gpu
INF = math.inf


def gen(seed):
    return torch.Generator().manual_seed(seed)


def logits_of(seed, n, E, dtype=torch.float32, std=1.5):
    return (torch.randn(n, E, generator=gen(seed)) * std).to(dtype)


def check_choice(logits, k, kind, bias=None, groups=1, top_groups=1, normalise=True, scale=1.0, on_gpu=None):
    x = logits.cuda() if on_gpu is None else on_gpu
    ids, w = mx.route(x, k, mx.MOE_SCORES[kind], bias=None if bias is None else bias.cuda(), groups=groups,
                      top_groups=top_groups, normalise=normalise, scale=scale)
    want_ids, want_w = plain.choice(logits, k, kind, bias, groups, top_groups, normalise, scale)
    assert ids.dtype == torch.int32 and torch.equal(ids.cpu(), want_ids)
    w = w.cpu().double()
    nan = want_w.isnan()
    assert torch.equal(w.isnan(), nan)
    # a score, the chosen ones' sum (their errors and k + 5 additions), a quotient and a product
    tol = (2 * plain.score_error(logits) + k + 9) * EPS
    err = ((w - want_w).abs() - tol * want_w.abs())[~nan]
    assert err.numel() == 0 or err.max() <= 1e-37
    return ids, w


# ---------------------------------------------------------------- the choice

@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,E,k,bias", [(1, 1, 1, False), (1, 384, 8, True), (5, 384, 8, False), (3, 7, 7, True),
                                        (40, 60, 3, True), (7, 128, 4, False), (9, 129, 16, True), (4, 256, 32, False),
                                        (3, 32, 32, True), (3, 500, 32, True), (2, 1024, 9, True), (400, 16, 4, False),
                                        (33, 1000, 5, False), (2000, 66, 2, True)])
def test_choice(kind, dtype, n, E, k, bias):
    b = torch.randn(E, generator=gen(E)) * 0.1 if bias else None
    check_choice(logits_of(n + E, n, E, dtype), k, kind, b, normalise=n % 2 == 0, scale=2.5)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top,k,bias", [(256, 8, 4, 8, True), (256, 8, 4, 8, False), (96, 6, 2, 5, True),
                                                 (60, 5, 3, 7, False), (32, 32, 3, 3, True), (64, 2, 1, 32, True),
                                                 (30, 10, 10, 12, False), (1024, 32, 5, 9, True), (93, 31, 7, 4, False)])
def test_groups(kind, E, groups, top, k, bias):
    b = torch.randn(E, generator=gen(E)) * 0.1 if bias else None
    for dtype in (torch.float32, torch.bfloat16):
        check_choice(logits_of(E + top, 50, E, dtype), k, kind, b, groups, top, normalise=top % 2 == 0)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_strides_and_alignments(kind):
    wide = logits_of(1, 30, 203)
    for dtype in (torch.float32, torch.bfloat16):
        x = wide.to(dtype).cuda()
        for a, E in ((0, 64), (1, 64), (2, 64), (3, 200), (0, 203)):
            rows = x[:, a:a + E]
            check_choice(rows.cpu(), 6, kind, on_gpu=rows)
            check_choice(rows[:1].cpu(), 6, kind, on_gpu=rows[:1])


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top", [(1, 1), (4, 2)])
def test_equal_values_go_to_the_lowest_index(kind, groups, top):
    E, k = 64, 8
    flat = torch.zeros(3, E)
    few = (torch.randint(0, 3, (20, E), generator=gen(1)).float() - 1).to(torch.bfloat16)
    for logits in (flat, few):
        for bias in (None, torch.zeros(E), torch.randint(0, 2, (E,), generator=gen(2)).float() * 0.25):
            check_choice(logits, k, kind, bias, groups, top)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top", [(24, 1, 1), (64, 1, 1), (384, 1, 1), (64, 8, 3)])
def test_scores_closer_than_fp32_tells_apart(kind, E, groups, top):
    # biases that bring every expert's choice to the same value within fp32's rounding: the order is in the bits below
    logits = logits_of(E + top, 1, E, std=1.0)
    bias = (1.0 - plain.scores(logits, kind)[0]).float()
    check_choice(logits, 8, kind, bias, groups, top)
    # and pairs of them among others
    many = logits_of(E, 40, E, std=1.0)
    s = plain.scores(many, kind)[0]
    pairs = torch.randn(E, generator=gen(3)) * 0.05
    pairs[1::2] = (s[0::2] + pairs[0::2].double() - s[1::2]).float()
    check_choice(many, 8, kind, pairs, groups, top)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masks_and_values_that_are_not_finite(kind, groups, with_bias):
    E, k = 40, 6
    x = logits_of(5, 12, E)
    x[0] = -INF                                   # nothing left
    x[1, 3:] = -INF                               # fewer than k
    x[2, ::2] = -INF
    x[3, 7] = math.nan
    x[4, 9] = INF
    x[5] = torch.finfo(torch.float32).min         # the type's lowest value masks nothing: all equal
    x[6, 1:] = torch.finfo(torch.float32).min
    x[7] = 200.0
    x[8] = -200.0                                 # sigmoid: below fp32
    x[9, :10] = -INF                              # a whole group
    bias = None
    if with_bias:
        bias = torch.randn(E, generator=gen(6)) * 0.1
        bias[5], bias[11], bias[30] = -INF, math.nan, INF
    if kind == "sigmoid":
        x[8] = -60.0 - torch.arange(E) / 64       # in range, and apart in 64 bits
    check_choice(x, k, kind, bias, groups, max(1, groups // 2))
    check_choice(x, k, kind, bias, groups, max(1, groups // 2), normalise=False)


def check_many(x, k, kind, bias, normalise):
    """check_choice, without groups, by one stable sort of all rows."""
    ids, w = mx.route(x.cuda(), k, mx.MOE_SCORES[kind], bias=None if bias is None else bias.cuda(), normalise=normalise)
    l, s = x.double(), plain.scores(x, kind)
    by = l if bias is None else s + bias.double()
    off = (l == -INF) | by.isnan() | (by == -INF)
    got = by.masked_fill(off, -INF).sort(dim=1, descending=True, stable=True).indices[:, :k]
    none, bad = off.gather(1, got), l.isnan().any(1) | ((l == INF).any(1) & (kind == "softmax"))
    got = got.masked_fill(none | bad[:, None], -1).int()
    assert torch.equal(ids.cpu(), got)
    want = s.gather(1, got.clamp(min=0).long()).masked_fill(got < 0, 0.0)
    if normalise:
        want = want / (want.sum(1, keepdim=True) + plain.TINY)
    w = w.cpu().double()
    assert w[bad].isnan().all()
    tol = (2 * plain.score_error(x) + k + 9) * EPS
    assert ((w - want).abs() <= tol * want.abs() + 1e-37)[~bad].all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,E,k,bias", [(5000, 384, 8, True), (4865, 60, 3, True), (6001, 256, 9, False), (5001, 512, 8, True),
                                        (20001, 16, 4, False), (5500, 128, 8, True), (9001, 32, 9, False), (5003, 388, 1, True),
                                        (5600, 8, 8, True), (5500, 384, 9, True), (5500, 386, 8, True)])
def test_choice_of_many_rows(kind, dtype, n, E, k, bias):
    b = torch.randn(E, generator=gen(E)) * 0.1 if bias else None
    x = logits_of(n + E, n, E, dtype)
    check_many(x, k, kind, b, n % 2 == 0)
    # neighbouring rows of which one or both are out of the ordinary
    x[0] = -INF
    x[7, 2] = math.nan
    x[8, 1], x[9, 3] = INF, INF
    x[100:130] = 0.25                                                    # more equal ones than a half has room for
    x[130:400:3] = torch.randint(0, 3, (90, E), generator=gen(1)).to(dtype)
    x[400:500, ::2] = -INF
    x[501:600:2, 3:] = -INF                                              # fewer than k
    x[700:800] = torch.finfo(dtype).min
    x[n - 1, 1:] = -INF
    check_many(x, k, kind, b, n % 2 == 1)
    if b is not None:
        b[:] = 0.5                                                       # masked ones' choices are above the others'
        b[2], b[5] = -INF, math.nan
        b[1::2] += 8
        check_many(x, k, kind, b, True)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_close_scores_among_many_rows(kind):
    n, E, k = 5200, 64, 6
    x = logits_of(9, n, E, std=1.0)
    x[::5] = x[0]
    b = torch.randn(E, generator=gen(3)) * 0.05
    s = plain.scores(x, kind)[0]
    b[1::2] = (s[0::2] + b[0::2].double() - s[1::2]).float()
    check_many(x, k, kind, b, True)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top,k,with_bias", [(64, 8, 3, 6, True), (64, 8, 3, 6, False), (40, 5, 2, 4, True), (32, 32, 5, 4, True)])
def test_groups_closer_than_fp32_tells_apart(kind, E, groups, top, k, with_bias):
    # groups of the same logits, moved by less than fp32 scores tell apart, by nothing, or masked
    size = E // groups
    x = logits_of(E, 1, size, std=1.0).repeat(1, groups).repeat(30, 1)
    x[10:] *= 1 + torch.randint(-2, 3, (20, E), generator=gen(1)) * 2.0**-23
    x[5, :size], x[6, size:2 * size], x[7, ::2] = -INF, -INF, -INF
    x[8, 0], x[9, E - 1] = 9.0, 9.0
    x[25:] = logits_of(2, 5, E)
    b = None
    if with_bias:
        b = (torch.randn(size, generator=gen(2)) * 0.1).repeat(groups)
        b[1] += 2.0**-20
    check_choice(x, k, kind, b, groups, top)
    if with_bias:
        b[3], b[E // 2] = INF, -INF
        check_choice(x, k, kind, b, groups, top)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_rows_of_more_candidates_than_lanes(kind):
    # the largest values all in a few lanes' columns, so that what the shorter sort bounds are more than 32
    n, E, k = 30, 512, 12
    x = logits_of(3, n, E, std=0.5)
    for t in range(n):
        x[t, torch.arange(E) % 128 // 4 % 16 < 3 + t % 9] += 4
    check_choice(x, k, kind)
    check_choice(x, k, kind, torch.randn(E, generator=gen(1)) * 0.01)
    check_choice(x.to(torch.bfloat16), k, kind)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("infinite", [1, 5, 8, 9, 40])
def test_infinite_biases_among_many_rows(kind, infinite):
    n, E, k = 6000, 384, 8
    x = logits_of(infinite, n, E)
    x[:3000] = x[:3000].round()                   # many equal ones: more candidates than a half has room for
    x[::7, 3] = -INF                              # masked, whatever the bias
    b = torch.randn(E, generator=gen(5)) * 0.05
    b[torch.randperm(E, generator=gen(infinite))[:infinite]] = INF
    b[3] = INF
    check_many(x, k, kind, b, True)
    b[b == INF] = 1e30
    check_many(x, k, kind, b, False)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top,k,infinite", [
    (32, 32, 1, 1, [5]), (32, 32, 3, 2, [9, 4, 31, 17, 2]),                   # groups of one expert
    (64, 8, 1, 4, [8, 13]), (64, 8, 2, 6, [8, 13]), (64, 8, 2, 6, [40, 41, 42, 9, 10]),
    (64, 8, 4, 8, [8, 9, 26, 31, 40, 45, 56, 63]),                            # two in each of as many as are kept
    (64, 8, 2, 8, [8, 9, 26, 31, 40, 45, 56, 63]), (64, 8, 3, 20, [1, 2, 12, 30, 62, 63]),
    (256, 8, 1, 8, [255, 254]), (60, 2, 1, 7, [59, 31])])
def test_groups_of_infinite_biases(kind, E, groups, top, k, infinite):
    x = logits_of(E + top, 20, E)
    x[3, infinite[0]] = -INF                      # masked, whatever the bias
    x[4] = 0.25
    b = torch.randn(E, generator=gen(2)) * 0.1
    b[infinite] = INF
    check_choice(x, k, kind, b, groups, top)
    b[b == INF] = 3e38                            # in range each, and not their sum
    check_choice(x, k, kind, b, groups, top)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top,k", [(64, 8, 3, 5), (32, 4, 2, 3), (256, 8, 4, 8)])
@pytest.mark.parametrize("large", [1000.0, 3e5])
def test_groups_whose_sums_are_small_beside_their_choices(kind, E, groups, top, k, large):
    # a group's two largest choices are near +large and -large: each rounds by large 2^-24, and their sum is small
    size, n = E // groups, 300
    for noise in (1e-4, 1e-3):
        x = (logits_of(E, 1, size).repeat(1, groups) * (1 + noise * torch.randn(n, E, generator=gen(1)))).float()
        x[n - 1] = x[n - 1, :size].repeat(groups)                             # equal groups
        sums = torch.full((groups, size), -INF)
        sums[:, 1], sums[:, 4] = large, -large
        check_choice(x, k, kind, sums.flatten(), groups, top)
        sums[:, 2:] = -large                                                  # which one is second is unsure too
        check_choice(x, k, kind, sums.flatten(), groups, top)
        sums[::2] = 0.0                                                       # beside groups of ordinary choices
        check_choice(x, k, kind, sums.flatten(), groups, top)
        sums[1::2, 1] = INF
        check_choice(x, k, kind, sums.flatten(), groups, top)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_scores_that_64_bits_do_not_tell_apart(kind):
    # sigmoids that are 1, softmax scores that are 0: equal, so that the lowest index goes first (without a bias the logits')
    E, k = 64, 6
    order = torch.stack([torch.randperm(E, generator=gen(s)) for s in range(30)])
    x = (40.0 + order) if kind == "sigmoid" else -800.0 * order
    b = torch.zeros(E)
    for bias in (None, b, b.index_fill(0, torch.arange(20, 50), 0.5)):
        check_choice(x.float(), k, kind, bias)
        check_many(x.float().repeat(200, 1), k, kind, bias, True)
    for bias in (None, b):
        check_choice(x.float(), k, kind, bias, 8, 3)


def test_the_callers_tensors_and_nothing_around_them():
    n, E, k = 70, 48, 5
    x = logits_of(1, n, E).cuda()
    want = mx.route(x, k, mx.MOE_SCORE_SIGMOID)
    room_i, room_w = torch.full((n + 2, k), -7, dtype=torch.int32).cuda(), torch.full((n + 2, k), -7.0).cuda()
    got = mx.route(x, k, mx.MOE_SCORE_SIGMOID, ids=room_i[1:-1], weights=room_w[1:-1])
    assert got[0].data_ptr() == room_i[1:].data_ptr() and torch.equal(room_i[1:-1], want[0]) and torch.equal(room_w[1:-1], want[1])
    for room in (room_i, room_w):
        assert (room[0] == -7).all() and (room[-1] == -7).all()
    empty = mx.route(x[:0], k, mx.MOE_SCORE_SIGMOID)
    assert empty[0].shape == (0, k) and empty[1].shape == (0, k)


# ---------------------------------------------------------------- the loss

def ragged(seed, n, S):
    cut = torch.randint(0, n + 1, (S - 1,), generator=gen(seed)).sort().values
    if S > 3:
        cut[1] = cut[0]
    return torch.cat([torch.tensor([0]), cut, torch.tensor([n])]).to(torch.int32)


def ids_of(seed, n, k, E):
    return torch.rand(n, E, generator=gen(seed)).topk(k, 1).indices.to(torch.int32)


def loss_error(logits, live_rows):
    """Relative: a share (a sigmoid's e^-l is within |l| 2^-24, below the 2 spread + 5 units that score_error has for more:
    these logits have both signs), and sums of positive values: a CTA's run of max(8, n / 608) rows, 8 to 32 at a time, as many
    sums to join, up to 609 pieces by eight warps, 32 experts, E / 32 parts and the sequences by 256 threads (24 for up to 6000 of them and
    13 to join), besides a handful of products."""
    n, E = logits.shape
    run = max(8, n / 608)
    return (2 * plain.score_error(logits) + run / 8 + 32 + 77 + 8 + 5 + E / 32 + 24 + 13 + 10) * EPS


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,E,k,S,pad", [(1, 1, 1, 1, 0), (1, 384, 8, 1, 0), (64, 16, 4, 1, 0), (65, 33, 2, 3, 1),
                                         (1001, 60, 3, 5, 37), (500, 384, 8, 500, 0), (3000, 130, 6, 40, 5),
                                         (130, 1024, 32, 2, 0), (2000, 8, 2, 6000, 300),
                                         (20001, 64, 6, 7, 13), (12000, 384, 8, 3001, 0), (10001, 256, 16, 1, 0),
                                         (9999, 500, 3, 9000, 77), (70001, 8, 1, 50, 1), (10000, 130, 9, 11, 0),
                                         (9800, 64, 17, 5, 0), (6000, 9, 5, 3, 0), (7001, 50, 12, 400, 6), (5500, 24, 12, 50, 0),
                                         (5001, 32, 8, 5001, 0), (6000, 1, 1, 2, 5)])
def test_loss_and_counts(kind, dtype, n, E, k, S, pad):
    logits, ids = logits_of(n + E, n, E, dtype), ids_of(n, n, k, E)
    offsets = None if S == 1 and pad == 0 else ragged(S, n - pad, S)
    loss, counts = mx.balance_loss(logits.cuda(), ids.cuda(), 0.01, mx.MOE_SCORES[kind],
                                   seq_offsets=None if offsets is None else offsets.cuda())
    want, want_counts = plain.balance(logits, ids, 0.01, kind, offsets)
    assert loss.shape == () and counts.dtype == torch.int32 and torch.equal(counts.cpu(), want_counts)
    assert abs(loss.item() - want.item()) <= loss_error(logits, n) * abs(want.item())


def test_even_shares_cost_the_coefficient():
    n, E, k = 96, 48, 4
    ids = torch.arange(n * k).reshape(n, k).remainder(E).to(torch.int32).cuda()
    for score in (mx.MOE_SCORE_SOFTMAX, mx.MOE_SCORE_SIGMOID):
        loss, counts = mx.balance_loss(torch.zeros(n, E).cuda(), ids, 0.125, score)
        assert (counts == n * k // E).all() and abs(loss.item() - 0.125) < 0.125 * 100 * EPS


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_loss_of_odd_rows(kind):
    n, E, k = 50, 20, 3
    logits, ids = logits_of(1, n, E), ids_of(2, n, k, E)
    logits[3] = -INF
    logits[4, 5:] = -INF
    ids[7] = torch.tensor([-1, E, 1 << 30], dtype=torch.int32)   # counted nowhere
    ids[8] = 4                                                    # one expert three times
    offsets = torch.tensor([5, 5, 30, 45], dtype=torch.int32)     # rows in front of the first and behind the last
    for o in (None, offsets):
        args = dict(seq_offsets=None if o is None else o.cuda())
        loss, counts = mx.balance_loss(logits.cuda(), ids.cuda(), 1.0, mx.MOE_SCORES[kind], **args)
        want, want_counts = plain.balance(logits, ids, 1.0, kind, o)
        assert torch.equal(counts.cpu(), want_counts)
        assert abs(loss.item() - want.item()) <= loss_error(logits, n) * want.item()
    logits[10, 2] = math.nan
    loss, counts = mx.balance_loss(logits.cuda(), ids.cuda(), 1.0, mx.MOE_SCORES[kind])
    assert loss.isnan() and torch.equal(counts.cpu(), plain.balance(logits, ids, 1.0, kind)[1])
    loss, _ = mx.balance_loss(logits.cuda(), ids.cuda(), 1.0, mx.MOE_SCORES[kind],      # the NaN is padding
                              seq_offsets=torch.tensor([0, 10], dtype=torch.int32).cuda())
    assert loss.isfinite()


@pytest.mark.parametrize("offsets", [[0, 30, 20, 50], [-1, 10, 20, 50], [0, 10, 20, 51], [60, 10, 5, 0]])
def test_offsets_that_do_not_ascend_give_nan(offsets):
    n, E, k = 50, 20, 3
    logits, ids = logits_of(1, n, E).cuda(), ids_of(2, n, k, E).cuda()
    o = torch.tensor(offsets, dtype=torch.int32).cuda()
    loss, counts = mx.balance_loss(logits, ids, 1.0, mx.MOE_SCORE_SOFTMAX, seq_offsets=o)
    assert loss.isnan()
    grad = mx.route_backward(logits, ids, mx.MOE_SCORE_SOFTMAX, counts=counts, coef=1.0, seq_offsets=o)
    assert grad.shape == (n, E)
    torch.cuda.synchronize()


def test_no_rows():
    E, k = 12, 2
    for o in (None, torch.zeros(4, dtype=torch.int32).cuda()):
        loss, counts = mx.balance_loss(torch.zeros(0, E).cuda(), torch.zeros(0, k, dtype=torch.int32).cuda(), 1.0, 0, seq_offsets=o)
        assert loss.item() == 0.0 and (counts == 0).all() and counts.shape[1] == E
    assert mx.route_backward(torch.zeros(0, E).cuda(), torch.zeros(0, k, dtype=torch.int32).cuda(), 0).shape == (0, E)


def test_the_callers_workspace_again_and_again():
    # one buffer, of the size that is asked for, for calls of all sizes one behind the other: nothing of the last is left
    calls = []
    for seed, (n, E, k, S, kind) in enumerate([(20000, 384, 8, 9, "sigmoid"), (3, 16, 2, 1, "softmax"), (6000, 8, 2, 3000, "sigmoid"),
                                               (0, 64, 4, 5, "softmax"), (5001, 1000, 32, 2, "softmax"), (40, 33, 3, 60, "sigmoid"),
                                               (20000, 384, 8, 9, "sigmoid"), (1, 1, 1, 1, "sigmoid")]):
        offsets = None if S == 1 else ragged(seed, n, S).cuda()
        r = mx.moe_router(E, k, mx.MOE_SCORES[kind], mx.MOE_LOGITS_F32, 1, 1, 1, 1.0)
        calls.append((mx.moe_balance_workspace_size(r, n, S), (logits_of(seed, n, E).cuda(), ids_of(seed, n, k, E).cuda(), 0.5,
                                                               mx.MOE_SCORES[kind]), offsets))
    want = [mx.balance_loss(*args, seq_offsets=offsets) for _, args, offsets in calls]
    room = torch.full((256 + max(b for b, _, _ in calls) + 512,), 0xff, dtype=torch.uint8, device="cuda")

    def all_calls():
        return [mx.balance_loss(*args, seq_offsets=offsets, ws=room[256:256 + b]) for b, args, offsets in calls]

    def same(got):
        return all(torch.equal(a, b) and torch.equal(c, d) for (a, c), (b, d) in zip(got, want))

    assert same(all_calls()) and same(all_calls())
    assert (room[:256] == 0xff).all() and (room[-512:] == 0xff).all()
    for (b, args, offsets), (loss, counts) in zip(calls, want):
        room.fill_(0xff)
        got = mx.balance_loss(*args, seq_offsets=offsets, ws=room[256:256 + b])
        assert torch.equal(got[0], loss) and torch.equal(got[1], counts)
        assert (room[:256] == 0xff).all() and (room[256 + b:] == 0xff).all()
    with pytest.raises(mx.MoeError):
        mx.balance_loss(*calls[0][1], seq_offsets=calls[0][2], ws=room[256:256 + calls[0][0] - 1])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = all_calls()
    for _ in range(3):
        room.fill_(0x7f)
        graph.replay()
        torch.cuda.synchronize()
        assert same(got)


# ---------------------------------------------------------------- the gradient

def check_gradient(logits, ids, kind, offsets=None, coef=None, d_loss=None, out=None, **kw):
    cuda = lambda t: None if t is None else t.cuda()
    x = logits.cuda()
    args = dict(kw, d_weights=cuda(kw.get("d_weights")))
    if coef is not None:
        _, counts = mx.balance_loss(x, ids.cuda(), coef, mx.MOE_SCORES[kind], seq_offsets=cuda(offsets))
        args |= dict(counts=counts, coef=coef, seq_offsets=cuda(offsets), d_loss=cuda(d_loss))
    got = mx.route_backward(x, ids.cuda(), mx.MOE_SCORES[kind], out=out(x) if out else None, **args)
    assert got.dtype == logits.dtype
    scale = 1.0 if d_loss is None else d_loss.item()
    want = plain.gradient(logits, ids, kind, coef=coef, d_loss=scale, offsets=offsets, **kw)
    size = plain.gradient_size(logits, ids, kind, coef=coef, d_loss=scale, offsets=offsets, **kw)
    # every factor of every term is a score, a sum of scores or a product with one; the counts' factor has eight roundings
    tol = (6 * plain.score_error(logits) + 2 * ids.shape[1] + 30) * EPS
    half = torch.finfo(logits.dtype).eps / 2
    err = (got.cpu().double() - want).abs() - tol * size - half * (want.abs() + tol * size)
    assert err.max() <= 1e-37, (err.max(), want.abs().max())
    return got, want


CASES = [(1, 1, 1, 1, 0), (1, 384, 8, 1, 0), (64, 16, 4, 1, 0), (65, 33, 2, 3, 1), (1001, 60, 3, 5, 37),
         (300, 384, 8, 300, 0), (3000, 130, 6, 40, 5), (130, 1024, 32, 2, 0), (500, 8, 2, 2000, 100),
         # several rows to a warp
         (6001, 8, 2, 7, 9), (5003, 9, 5, 3000, 0), (7001, 50, 12, 400, 6), (5500, 24, 12, 1, 0), (5001, 64, 16, 3, 100),
         (5001, 32, 8, 5001, 0), (9000, 48, 13, 31, 0)]


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,E,k,S,pad", CASES)
def test_gradient(kind, dtype, n, E, k, S, pad):
    logits, ids = logits_of(n + E, n, E, dtype), ids_of(n, n, k, E)
    offsets = None if S == 1 and pad == 0 else ragged(S, n - pad, S)
    d_weights = torch.randn(n, k, generator=gen(4))
    both = dict(d_weights=d_weights, coef=0.7, d_loss=torch.tensor([3.0]), offsets=offsets, scale=2.5)
    check_gradient(logits, ids, kind, normalise=True, **both)
    check_gradient(logits, ids, kind, normalise=False, **both)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_gradient_of_each_part_alone(kind):
    n, E, k = 90, 40, 4
    logits, ids = logits_of(1, n, E), ids_of(2, n, k, E)
    d_weights = torch.randn(n, k, generator=gen(4))
    check_gradient(logits, ids, kind, d_weights=d_weights, normalise=True)
    check_gradient(logits, ids, kind, d_weights=d_weights, normalise=False, scale=0.5)
    offsets = torch.tensor([10, 10, 60, 80], dtype=torch.int32)
    got, _ = check_gradient(logits, ids, kind, coef=2.0, offsets=offsets)
    assert (got[:10] == 0).all() and (got[80:] == 0).all() and (got[10:80] != 0).any()
    nothing = mx.route_backward(logits.cuda(), ids.cuda(), mx.MOE_SCORES[kind])
    assert (nothing == 0).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_gradient_against_differences(kind):
    n, E, k = 40, 24, 3
    logits, ids = logits_of(1, n, E), ids_of(2, n, k, E)
    offsets = torch.tensor([0, 15, 33], dtype=torch.int32)
    kw = dict(d_weights=torch.randn(n, k, generator=gen(4)), normalise=True, scale=2.5, coef=5.0, offsets=offsets)
    got, _ = check_gradient(logits, ids, kind, **kw)
    step = torch.randn(n, E, generator=gen(5), dtype=torch.float64)
    h = 1e-5
    up, down = (plain.objective(logits.double() + s * h * step, ids, kind, **kw) for s in (1, -1))
    along = (got.cpu().double() * step).sum()
    # h^2 times the third derivative (below 10 a term of order 1), the difference's rounding, the gradient's own error
    size = (plain.gradient_size(logits, ids, kind, **kw) * step.abs()).sum()
    assert abs((up - down) / (2 * h) - along) <= 10 * h * h * size + 1e-15 / h * n + 400 * EPS * size


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalise", [False, True])
def test_gradient_of_odd_rows(kind, normalise):
    n, E, k = 30, 40, 6
    logits, ids = logits_of(1, n, E), ids_of(2, n, k, E)
    logits[0] = -INF
    logits[1, 3:] = -INF
    ids[1] = torch.tensor([0, 1, 2, -1, -1, -1], dtype=torch.int32)
    logits[2, ::2] = -INF
    ids[3] = torch.tensor([5, 5, 5, 7, 7, E], dtype=torch.int32)    # named twice, and none
    ids[4] = -1
    logits[5] = 30.0
    logits[6] = -30.0
    d_weights = torch.randn(n, k, generator=gen(4))
    finite = logits.clone()
    finite[logits == -INF] = -1e4                                   # the same scores of 0, without inf - inf in the formula
    cuda = logits.cuda()
    for row in range(7):
        one, i, g = logits[row:row + 1], ids[row:row + 1], d_weights[row:row + 1]
        got = mx.route_backward(cuda[row:row + 1], i.cuda(), mx.MOE_SCORES[kind], d_weights=g.cuda(), normalise=normalise)
        if row == 0:
            assert (got == 0).all()
            continue
        kw = dict(d_weights=g, normalise=normalise)
        want, size = (f(finite[row:row + 1], i, kind, **kw) for f in (plain.gradient, plain.gradient_size))
        tol = (6 * plain.score_error(one) + 2 * k + 30) * EPS
        assert ((got.cpu().double() - want).abs() - tol * size - EPS * want.abs()).max() <= 1e-37
        assert (got.cpu()[one == -INF] == 0).all()
    bad = logits.clone()
    bad[9, 1] = math.nan
    grads = [mx.route_backward(x.cuda(), ids.cuda(), mx.MOE_SCORES[kind], d_weights=d_weights.cuda(), normalise=normalise)
             for x in (bad, logits)]
    assert grads[0][9].isnan().all()
    keep = torch.arange(n) != 9
    assert torch.equal(grads[0][keep], grads[1][keep])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_gradient_into_strided_rows_and_in_place(dtype, kind):
    n, E, k = 60, 36, 4
    ids, d_weights = ids_of(2, n, k, E), torch.randn(n, k, generator=gen(4))
    logits = logits_of(1, n, E, dtype)
    for a, width in ((0, 40), (1, 41), (4, 48)):
        room = torch.full((n, width), 9.0, dtype=dtype).cuda()
        check_gradient(logits, ids, kind, d_weights=d_weights, coef=1.0, out=lambda x: room[:, a:a + E])
        assert (room[:, :a] == 9).all() and (room[:, a + E:] == 9).all()
    got, _ = check_gradient(logits, ids, kind, d_weights=d_weights, coef=1.0, out=lambda x: x)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,E,k", [(60, 384, 8), (33, 61, 3), (6000, 8, 2), (5001, 50, 12), (5600, 256, 8)])
@pytest.mark.parametrize("level", [-35.0, -44.0, -60.0, -87.0, -89.0, -95.0, -300.0, -600.0])
def test_sigmoid_shares_of_low_rows(dtype, n, E, k, level):
    # A share does not depend on whether fp32 holds the scores that it is of.
    logits = (logits_of(n + E, n, E) * 2 + level).to(dtype)
    logits[::3] = logits_of(n, len(logits[::3]), E, dtype)                  # beside ordinary rows
    logits[4, 1:] = -INF
    ids, offsets = ids_of(n, n, k, E), ragged(3, n, 4)
    loss, counts = mx.balance_loss(logits.cuda(), ids.cuda(), 0.01, mx.MOE_SCORE_SIGMOID, seq_offsets=offsets.cuda())
    want, want_counts = plain.balance(logits, ids, 0.01, "sigmoid", offsets)
    assert torch.equal(counts.cpu(), want_counts)
    # shares as loss_error has them, of rows of a spread below 20; e^-l of low rows is within |l| 2^-24, of those that go by the
    # sigmoid up to 64 of these, in a score and in its row's sum
    low = (2 * (12 + 2 * 20 + E / 32 + 5) + 2 * 64) * EPS
    assert abs(loss.item() - want.item()) <= (loss_error(logits[::3], n) + low) * want.item()
    # The gradient of the loss; and with that of weights whose scores are above 2^-126 (below, weights are 0).
    finite = logits.clone()
    finite[logits == -INF] = -690.0
    for d_weights in (None, torch.randn(n, k, generator=gen(4))):
        kw = dict(coef=5.0, offsets=offsets, d_weights=d_weights)
        got = mx.route_backward(logits.cuda(), ids.cuda(), mx.MOE_SCORE_SIGMOID, counts=counts, coef=5.0, seq_offsets=offsets.cuda(),
                                d_weights=None if d_weights is None else d_weights.cuda()).cpu().double()
        grad, size = (f(finite, ids, "sigmoid", **kw) for f in (plain.gradient, plain.gradient_size))
        tol = (6 * (12 + 2 * 20 + E / 32 + 5 + 64) + 2 * k + 30) * EPS
        err = (got - grad).abs() - tol * size - torch.finfo(dtype).eps / 2 * (grad.abs() + tol * size)
        none = 0.0 if d_weights is None else 1.2e-38 * 1e20 * d_weights.abs().sum(1, keepdim=True)
        assert (err <= 1e-37 + none).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("level", [-1000.0, -1e4, None])
def test_sigmoid_shares_of_rows_below_every_float(dtype, level):
    # there the shares are a softmax's; the type's lowest value masks nothing
    n, E, k = 90, 40, 4
    logits = torch.full((n, E), torch.finfo(dtype).min, dtype=dtype) if level is None else (logits_of(1, n, E) + level).to(dtype)
    ids = ids_of(2, n, k, E)
    loss, counts = mx.balance_loss(logits.cuda(), ids.cuda(), 1.0, mx.MOE_SCORE_SIGMOID)
    want, _ = plain.balance(logits, ids, 1.0, "softmax")
    assert abs(loss.item() - want.item()) <= loss_error(logits, n) * want.item()
    got = mx.route_backward(logits.cuda(), ids.cuda(), mx.MOE_SCORE_SIGMOID, counts=counts, coef=3.0).cpu().double()
    grad, size = (f(logits, ids, "softmax", coef=3.0) for f in (plain.gradient, plain.gradient_size))
    tol = (6 * plain.score_error(logits) + 2 * k + 30) * EPS
    assert ((got - grad).abs() - tol * size - torch.finfo(dtype).eps / 2 * (grad.abs() + tol * size)).max() <= 1e-37


# ---------------------------------------------------------------- as a program runs them

def test_the_same_bits_each_time_and_in_a_graph():
    n, E, k = 5000, 384, 8
    x, x2 = logits_of(1, n, E).cuda(), logits_of(2, n, E).cuda()
    offsets = ragged(3, n, 7).cuda()
    bias = (torch.randn(E, generator=gen(4)) * 0.05).cuda()
    d_weights, d_loss = torch.randn(n, k, generator=gen(5)).cuda(), torch.tensor([0.5]).cuda()

    def step(x):
        ids, w = mx.route(x, k, mx.MOE_SCORE_SIGMOID, bias=bias, scale=2.5)
        loss, counts = mx.balance_loss(x, ids, 1e-3, mx.MOE_SCORE_SIGMOID, seq_offsets=offsets)
        grad = mx.route_backward(x, ids, mx.MOE_SCORE_SIGMOID, d_weights=d_weights, scale=2.5, counts=counts, coef=1e-3,
                                 d_loss=d_loss, seq_offsets=offsets)
        return ids, w, loss, counts, grad

    want = [step(x), step(x2)]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(step(x), want[0]))
    held = x.clone()
    torch.cuda.synchronize()
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(held)
    with torch.cuda.graph(other):
        got2 = step(held)
    for data, w in ((x2, want[1]), (x, want[0]), (x2, want[1])):
        held.copy_(data)
        graph.replay()
        other.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, w)) and all(torch.equal(a, b) for a, b in zip(got2, w))


def test_another_stream():
    n, E, k = 3000, 100, 4
    x, s = logits_of(1, n, E).cuda(), torch.cuda.Stream()
    want_ids, want_w = mx.route(x, k, mx.MOE_SCORE_SOFTMAX)
    want_loss, want_counts = mx.balance_loss(x, want_ids, 1.0, mx.MOE_SCORE_SOFTMAX)
    want_grad = mx.route_backward(x, want_ids, mx.MOE_SCORE_SOFTMAX, counts=want_counts, coef=1.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        late = torch.zeros_like(x)
        big = torch.zeros(4096, 4096, device="cuda")
        for _ in range(20):
            big = big @ big
        late.copy_(x)
    ids, w = mx.route(late, k, mx.MOE_SCORE_SOFTMAX, stream=s)
    loss, counts = mx.balance_loss(late, ids, 1.0, mx.MOE_SCORE_SOFTMAX, stream=s.cuda_stream)
    grad = mx.route_backward(late, ids, mx.MOE_SCORE_SOFTMAX, counts=counts, coef=1.0, stream=s)
    s.synchronize()
    for a, b in ((ids, want_ids), (w, want_w), (loss, want_loss), (counts, want_counts), (grad, want_grad)):
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    # 4,400,000 rows of 512: 2.25e9 logits, and as many gradients
    n, E, k = 4_400_000, 512, 8
    x = torch.empty(n, E, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    bias = (torch.randn(E, generator=gen(2)) * 0.05).cuda()
    ids, w = mx.route(x, k, mx.MOE_SCORE_SIGMOID, bias=bias)
    offsets = torch.tensor([0, n - 70, n - 5], dtype=torch.int32).cuda()
    loss, counts = mx.balance_loss(x, ids, 1.0, mx.MOE_SCORE_SIGMOID, seq_offsets=offsets)
    q, want = torch.zeros(E, dtype=torch.float64, device="cuda"), 0.0
    for a in range(0, n - 70, 1 << 18):
        s = torch.sigmoid(x[a:min(a + (1 << 18), n - 70)].double())
        q += (s / s.sum(1, keepdim=True)).sum(0)
    full = ids[:n - 70].flatten().bincount(minlength=E)
    assert torch.equal(counts[0].long(), full)
    want = ((full.double() * q).sum() * E / (k * (n - 70.0) ** 2)).item()
    tail = slice(n - 70, n - 5)
    last, last_counts = plain.balance(x[tail].cpu(), ids[tail].cpu(), 1.0, "sigmoid")
    assert torch.equal(counts[1].cpu(), last_counts[0])
    assert abs(loss.item() - (want + last.item()) / 2) <= loss_error(x[tail].cpu(), n) * want
    grad = mx.route_backward(x, ids, mx.MOE_SCORE_SIGMOID, d_weights=w)
    for a in (0, 4_194_304 - 20, n - 40):      # 2^31 elements lie at row 4,194,304
        rows = slice(a, a + 40)
        some, some_w = mx.route(x[rows], k, mx.MOE_SCORE_SIGMOID, bias=bias)
        assert torch.equal(ids[rows], some) and ((w[rows] - some_w).abs() <= 32 * EPS * some_w).all()
        assert torch.equal(grad[rows], mx.route_backward(x[rows], some, mx.MOE_SCORE_SIGMOID, d_weights=w[rows]))
    assert torch.equal(mx.route_backward(x, ids, mx.MOE_SCORE_SIGMOID, d_weights=w, out=x), grad)


def test_the_routing_plan_takes_the_choice():
    n, E, k = 600, 48, 5
    x = logits_of(1, n, E).cuda()
    ids, _ = mx.route(x, k, mx.MOE_SCORE_SOFTMAX)
    _, counts = mx.balance_loss(x, ids, 1.0, mx.MOE_SCORE_SOFTMAX)
    assert torch.equal(mx.permute(ids, E, validate=True)[0], counts[0])
