"""What is measured of the router's operators (choice, balance loss, gradient) and of the FP8 ones (rows, products by expert).

A case names an operator ("op") and its sizes.

    route    scores of n rows of logits over E experts (softmax or sigmoid), the k largest of score + bias within the best groups,
             and their weights
    balance  the loss sum_s E / (k T_s^2) sum_e count_se sum_t q_te over sequences s of T_s rows, and the counts
    grad     the logits' gradient from that of the weights and that of the loss
    rows     bf16 rows to e4m3 with one fp32 scale per 128 columns, at their routed positions, and back
    product  such rows, grouped by expert, times e4m3 matrices with one fp32 scale per 128 x 128 block
"""

import math

import torch

own = False

BLOCK = 128
TOP = 448.0
COEF = 1e-3
TINY = 1e-20


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decoded token's eight experts: latency alone
        {"name": "route_token", "op": "route", "n": 1, "experts": 384, "k": 8, "score": "sigmoid", "type": "fp32", "bias": True,
         "groups": 1, "top_groups": 1, "normalise": True},
        # a long prompt's routing
        {"name": "route_prompt", "op": "route", "n": 32768, "experts": 384, "k": 8, "score": "sigmoid", "type": "fp32", "bias": True,
         "groups": 1, "top_groups": 1, "normalise": True},
        # a few ragged sequences, one of them empty, padding behind the last, a small model's experts
        {"name": "balance_odd", "op": "balance", "n": 1001, "experts": 60, "k": 3, "score": "softmax", "type": "bf16", "sequences": 5, "padding": 37},
        # a training step's batch of sequences
        {"name": "balance_batch", "op": "balance", "n": 65536, "experts": 384, "k": 8, "score": "sigmoid", "type": "fp32", "sequences": 16, "padding": 0},
        # both gradients over ragged sequences
        {"name": "grad_odd", "op": "grad", "n": 1001, "experts": 60, "k": 3, "score": "softmax", "type": "bf16", "sequences": 5, "padding": 37,
         "normalise": False},
        # both gradients of a training step's batch
        {"name": "grad_batch", "op": "grad", "n": 65536, "experts": 384, "k": 8, "score": "sigmoid", "type": "fp32", "sequences": 16, "padding": 0,
         "normalise": True},
        # a decode batch's tokens to their eight routed positions
        {"name": "rows_decode", "op": "rows", "n": 16, "k": 8, "d": 7168},
        # a prompt's tokens to their eight routed positions
        {"name": "rows_prompt", "op": "rows", "n": 4096, "k": 8, "d": 7168},
        # one token's eight experts, down projection: the weights of eight experts and nothing else
        {"name": "product_token", "op": "product", "rows": 8, "experts": 384, "n_out": 7168, "k": 2048, "skew": 0.0},
        # ragged experts, some of them empty, sizes that end inside every tile and block
        {"name": "product_odd", "op": "product", "rows": 1000, "experts": 16, "n_out": 1001, "k": 1040, "skew": 1.2},
        # a prompt's routed rows through the down projection
        {"name": "product_prompt", "op": "product", "rows": 32768, "experts": 384, "n_out": 7168, "k": 2048, "skew": 0.0},
        # one matrix for every row, as in a dense layer: the tensor cores alone
        {"name": "product_dense", "op": "product", "rows": 8192, "experts": 1, "n_out": 7168, "k": 7168, "skew": 0.0},
    ]


def draw(rng):
    def spread(lo, hi, step=1):
        return max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + step)))) // step * step)

    op = rng.choice(["route", "balance", "grad", "rows", "product", "product"])
    c = {"op": op}
    if op in ("route", "balance", "grad"):
        group = spread(1, 64)
        groups = rng.choice([1, 1, rng.randint(2, 8)])
        experts = max(2, group * groups if groups > 1 else spread(2, 512))
        n = spread(1, 65536)
        while n * experts > 32768 * 384:
            n //= 2
        c |= {"n": n, "experts": experts, "score": rng.choice(["sigmoid", "softmax"]), "type": rng.choice(["fp32", "bf16"])}
        if op == "route":
            top = rng.randint(1, groups)
            c |= {"k": rng.randint(1, min(16, top * (experts // groups))), "bias": rng.random() < 0.6, "groups": groups, "top_groups": top}
        else:
            sequences = min(n, spread(1, 64))
            c |= {"k": rng.randint(1, min(16, experts)), "sequences": sequences, "padding": rng.choice([0, n // 10])}
        if op != "balance":
            c["normalise"] = rng.random() < 0.5
    elif op == "rows":
        n, d = spread(1, 32768), spread(16, 8192, 16)
        c |= {"n": n, "k": rng.choice([1, 1, 2, 3, 8]) if n <= 4096 else 1, "d": d}
    else:
        experts = rng.choice([1, spread(2, 384)])
        n_out, k = spread(16, 7168), spread(16, 7168, 16)
        while experts * n_out * k > 384 * 7168 * 2048 // 2:
            experts = max(1, experts // 2)
        rows = spread(1, 32768)
        while rows * n_out * k > 32768 * 7168 * 1024:
            rows //= 2
        c |= {"rows": rows, "experts": experts, "n_out": n_out, "k": k, "skew": rng.choice([0.0, 1.2])}
    return c


# ---------------------------------------------------------------- inputs

def _gen(case, seed):
    text = repr(sorted((k, v) for k, v in case.items() if k != "name"))
    return torch.Generator(device="cuda").manual_seed((seed * 1000003 + sum((i + 1) * ord(ch) for i, ch in enumerate(text))) % (1 << 62))


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _choice(gen, n, k, experts):
    return torch.rand(n, experts, generator=gen, device="cuda").topk(k, dim=1).indices.to(torch.int32)


def _positions(ids):
    """Where each (token, slot) lands when the entries are sorted by expert (stable), as an [n, k] table."""
    order = torch.sort(ids.flatten(), stable=True).indices
    at = torch.empty_like(order)
    at[order] = torch.arange(order.numel(), device=order.device)
    return at.reshape(ids.shape).to(torch.int32)


def _sequences(gen, n, count):
    """Offsets of `count` ragged sequences over n rows, the second of them empty where there are three or more."""
    cut = torch.randint(0, n + 1, (count - 1,), generator=gen, device="cuda").sort().values
    if count >= 3:
        cut[1] = cut[0]
    off = torch.zeros(count + 1, dtype=torch.int32, device="cuda")
    off[1:-1] = cut
    off[-1] = n
    return off


def _offsets(gen, rows, experts, skew):
    """Rows by expert: even odds, or by a power law that leaves some experts empty."""
    odds = torch.arange(1, experts + 1, device="cuda", dtype=torch.float32) ** -skew
    odds = odds[torch.randperm(experts, generator=gen, device="cuda")]
    who = torch.multinomial(odds, rows, replacement=True, generator=gen)
    count = torch.bincount(who, minlength=experts)
    return torch.nn.functional.pad(count.cumsum(0), (1, 0)).to(torch.int32)


def _round_e4m3(t):
    a = t.abs()
    step = torch.ldexp(torch.ones_like(a), (torch.frexp(a).exponent - 1).clamp(min=-6) - 3)
    return torch.copysign((torch.round(a / step) * step).clamp(max=TOP), t)


def _blocks(cols):
    return -(-cols // BLOCK)


def _quantise(v):
    """fp32 rows -> (codes' values, scales [rows, blocks])."""
    rows, cols = v.shape
    g = torch.nn.functional.pad(v, (0, -cols % BLOCK)).reshape(rows, -1, BLOCK)
    amax = g.abs().amax(-1)
    scale = torch.where(amax > 0, amax / TOP, 1.0)
    return _round_e4m3(g / scale[..., None]).reshape(rows, -1)[:, :cols], scale


def _bytes(q):
    return q.to(torch.float8_e4m3fn).view(torch.uint8)


def _weights(gen, experts, rows, cols):
    """Experts' matrices as a checkpoint holds them: codes [E, rows, cols] and scales of 128 x 128 blocks."""
    codes = torch.empty(experts, rows, cols, dtype=torch.uint8, device="cuda")
    scales = torch.empty(experts, _blocks(rows), _blocks(cols), device="cuda")
    for e in range(experts):
        w = torch.nn.functional.pad(_randn(gen, rows, cols) * 0.02, (0, -cols % BLOCK, 0, -rows % BLOCK))
        t = w.reshape(_blocks(rows), BLOCK, _blocks(cols), BLOCK)
        s = t.abs().amax((1, 3)) / TOP
        codes[e] = (t / s[:, None, :, None]).reshape(w.shape)[:rows, :cols].to(torch.float8_e4m3fn).view(torch.uint8)
        scales[e] = s
    return codes, scales


def _packed(codes):
    """The codes as a serving program keeps them once they are loaded: blocks of 256 rows by 128 columns, consecutive along the
    row, zeros past the matrix. A block holds row r's 16-byte piece j at piece j ^ (r % 8) of its 128 bytes."""
    experts, rows, cols = codes.shape
    up, chunks = -(-rows // 256), _blocks(cols)
    row = torch.arange(256, device=codes.device)[:, None]
    piece = torch.arange(8, device=codes.device) ^ (row % 8)
    packed = torch.empty(experts, up, chunks, 256, 8, 16, dtype=torch.uint8, device=codes.device)
    for e in range(experts):
        t = torch.nn.functional.pad(codes[e], (0, chunks * 128 - cols, 0, up * 256 - rows))
        packed[e] = t.reshape(up, 256, chunks, 8, 16).transpose(1, 2)[:, :, row, piece]
    return packed.flatten()


def prepare(case, seed):
    gen, op = _gen(case, seed), case["op"]
    s = {"case": case}
    if op in ("route", "balance", "grad"):
        n, experts, k = case["n"], case["experts"], case["k"]
        logits = _randn(gen, n, experts) * 1.5 + _randn(gen, experts)  # some experts are liked better
        s["logits"] = logits if case["type"] == "fp32" else logits.to(torch.bfloat16)
        if op == "route":
            s["bias"] = _randn(gen, experts) * 0.05 if case["bias"] else None
        else:
            s["ids"] = torch.topk(s["logits"].float() + _randn(gen, n, experts) * 0.1, k, dim=1).indices.to(torch.int32)
            s["offsets"] = _sequences(gen, n - case["padding"], case["sequences"])
            s["ends"] = s["offsets"].tolist()
        if op == "grad":
            s["d_weights"] = _randn(gen, n, k)
            s["d_loss"] = torch.rand(1, generator=gen, device="cuda") + 0.5
            counts = [torch.bincount(s["ids"][a:b].flatten(), minlength=experts) for a, b in zip(s["ends"], s["ends"][1:])]
            s["counts"] = torch.stack(counts).to(torch.int32)  # kept from the forward pass
    elif op == "rows":
        s["x"] = _randn(gen, case["n"], case["d"]).to(torch.bfloat16)
        s["positions"] = _positions(_choice(gen, case["n"], case["k"], 64))
    else:
        rows, experts, n_out, k = case["rows"], case["experts"], case["n_out"], case["k"]
        q, scale = _quantise(_randn(gen, rows, k))
        s["codes"] = _bytes(q)
        s["scales"] = torch.nn.functional.pad(scale, (0, -scale.shape[1] % 4))  # rows of scales start on 16 bytes
        s["w_codes"], s["w_scales"] = _weights(gen, experts, n_out, k)
        s["packed"] = _packed(s["w_codes"])
        s["offsets"] = _offsets(gen, rows, experts, case["skew"])
        s["ends"] = s["offsets"].tolist()
        s["workspace"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass, plain

def _scores(logits, kind):
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _route(s):
    case = s["case"]
    n, experts, k, groups = case["n"], case["experts"], case["k"], case["groups"]
    score = _scores(s["logits"].double(), case["score"])  # 64 bits: which of two close ones is larger
    by = score if s["bias"] is None else score + s["bias"].double()
    if groups > 1:
        size = experts // groups
        best = by.reshape(n, groups, size).topk(min(2, size), dim=2).values.sum(2)
        keep = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        on = torch.zeros(n, groups, dtype=torch.bool, device="cuda")
        on[torch.arange(n, device="cuda")[:, None], keep] = True
        by = torch.where(on.repeat_interleave(size, 1), by, -math.inf)
    ids = torch.sort(by, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(_scores(s["logits"].float(), case["score"]), 1, ids)
    if case["normalise"]:
        w = w / (w.sum(1, keepdim=True) + TINY)
    return ids.to(torch.int32), w * 2.5


def _shares(case, logits):
    q = _scores(logits, case["score"])
    return q / q.sum(1, keepdim=True) if case["score"] == "sigmoid" else q


def _balance(s):
    case = s["case"]
    q = _shares(case, s["logits"].float())
    counts, loss, live = [], torch.zeros((), device="cuda"), 0
    for a, b in zip(s["ends"], s["ends"][1:]):
        c = (s["ids"][a:b].flatten()[:, None] == torch.arange(case["experts"], device="cuda", dtype=torch.int32)).sum(0)
        counts.append(c.to(torch.int32))
        if b > a:
            loss = loss + (c.float() * q[a:b].sum(0)).sum() * (case["experts"] / (case["k"] * float(b - a) ** 2))
            live += 1
    return loss * (COEF / max(live, 1)), torch.stack(counts)


def _grad(s):
    case = s["case"]
    logits = s["logits"].float()
    score = _scores(logits, case["score"])
    ids = s["ids"].long()
    chosen, g = torch.gather(score, 1, ids), s["d_weights"] * 2.5
    if case["normalise"]:
        total = chosen.sum(1, keepdim=True) + TINY
        g = (g - (g * chosen).sum(1, keepdim=True) / total) / total
    d = torch.zeros_like(score).scatter_add_(1, ids, g)
    c = torch.zeros_like(score)
    live = sum(b > a for a, b in zip(s["ends"], s["ends"][1:]))
    for i, (a, b) in enumerate(zip(s["ends"], s["ends"][1:])):
        if b > a:
            c[a:b] = s["counts"][i].float() * (s["d_loss"] * (COEF * case["experts"] / (case["k"] * float(b - a) ** 2 * live)))
    if case["score"] == "softmax":
        d = d + c
        out = score * (d - (d * score).sum(1, keepdim=True))
    else:
        total = score.sum(1, keepdim=True)
        d = d + (c - (c * score).sum(1, keepdim=True) / total) / total
        out = d * score * (1 / (1 + torch.exp(logits)))
    return out.to(s["logits"].dtype)


def _values(codes, scales):
    """fp32 values of rows of codes with scales by blocks of columns."""
    return codes.view(torch.float8_e4m3fn).float() * scales.repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op in ("route", "balance", "grad"):
        return {"route": _route, "balance": _balance, "grad": _grad}[op](s)
    if op == "rows":
        at = s["positions"]
        q, scale = _quantise(s["x"].float())
        v = (q * scale.repeat_interleave(BLOCK, 1)[:, :q.shape[1]]).to(torch.bfloat16)
        rows = torch.empty(at.numel(), v.shape[1], dtype=torch.bfloat16, device="cuda")
        rows[at.flatten().long()] = v.repeat_interleave(at.shape[1], 0)
        return rows
    x = _values(s["codes"], s["scales"])
    out = torch.empty(case["rows"], case["n_out"], device="cuda")
    for e, (a, b) in enumerate(zip(s["ends"], s["ends"][1:])):
        if b > a:
            w = _values(s["w_codes"][e], s["w_scales"][e].repeat_interleave(BLOCK, 0)[:case["n_out"]])
            out[a:b] = x[a:b] @ w.T
    return out.to(torch.bfloat16)


# ---------------------------------------------------------------- one pass, the framework's calls

def _kernels(s):
    import mixture_experts_ffn_infer_gb300 as mx

    case = s["case"]
    op = case["op"]
    if op in ("route", "balance", "grad"):
        score = mx.MOE_SCORES[case["score"]]
    if op == "route":
        return mx.route(s["logits"], case["k"], score, bias=s["bias"], groups=case["groups"], top_groups=case["top_groups"],
                        normalise=case["normalise"], scale=2.5)
    if op == "balance":
        return mx.balance_loss(s["logits"], s["ids"], COEF, score, seq_offsets=s["offsets"])
    if op == "grad":
        return mx.route_backward(s["logits"], s["ids"], score, d_weights=s["d_weights"], normalise=case["normalise"], scale=2.5,
                                 counts=s["counts"], coef=COEF, d_loss=s["d_loss"], seq_offsets=s["offsets"])
    if op == "rows":
        return mx.fp8_dequantise(mx.fp8_quantise(s["x"], positions=s["positions"]))
    x = mx.Fp8Rows(s["codes"], s["scales"])
    w = mx.Fp8Weights(case["experts"], case["n_out"], case["k"], s["packed"], s["w_scales"])
    return mx.fp8_grouped_product(x, w, s["offsets"], ws=s["workspace"])


def run(state):
    return _kernels(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def _row_bytes(cols):
    return cols + 4 * _blocks(cols)


def work(case):
    op = case["op"]
    if op in ("route", "balance", "grad"):
        n, experts, k = case["n"], case["experts"], case["k"]
        held = n * experts * (4 if case["type"] == "fp32" else 2)
        if op == "route":
            return {"bytes": held + 8 * n * k + (4 * experts if case["bias"] else 0), "flops": 8 * n * experts}
        live = n - case["padding"]
        if op == "balance":
            return {"bytes": held * live // n + 4 * live * k + 4 * case["sequences"] * (experts + 1), "flops": 8 * live * experts}
        return {"bytes": 2 * held + 8 * n * k + 4 * case["sequences"] * (experts + 1), "flops": 12 * n * experts}
    if op == "rows":
        n, k, d = case["n"], case["k"], case["d"]
        return {"bytes": 2 * n * d + 2 * n * k * _row_bytes(d) + 2 * n * k * d + 4 * n * k, "flops": 4 * n * d}
    rows, n_out, k = case["rows"], case["n_out"], case["k"]
    touched = _touched(rows, case["experts"], case["skew"])
    return {"bytes": touched * (n_out * k + 4 * _blocks(n_out) * _blocks(k)) + rows * _row_bytes(k) + 2 * rows * n_out, "flops": 2 * rows * n_out * k}


def _touched(rows, experts, skew):
    odds = [(i + 1) ** -skew for i in range(experts)]
    return sum(1 - (1 - o / sum(odds)) ** rows for o in odds)


# ---------------------------------------------------------------- in 64 bits, from the definition

def _exact_scores(case, logits):
    return torch.sigmoid(logits) if case["score"] == "sigmoid" else torch.softmax(logits, 1)


def _exact_route(s):
    case = s["case"]
    score = _exact_scores(case, s["logits"].double())
    by = score + (0 if s["bias"] is None else s["bias"].double())
    size = case["experts"] // case["groups"]
    if case["groups"] > 1:
        # a group's rank: how many are better, or as good and in front of it
        top = by.reshape(case["n"], -1, size).sort(2).values[:, :, -2:].sum(2)
        better = (top[:, None, :] > top[:, :, None]).sum(2)
        for g in range(case["groups"]):
            better[:, g] += (top[:, :g] == top[:, g:g + 1]).sum(1)
        by = by.masked_fill((better >= case["top_groups"]).repeat_interleave(size, 1), -math.inf)
    ids = []
    for _ in range(case["k"]):
        top = by.max(1, keepdim=True).values
        first = (by == top).to(torch.uint8).argmax(1, keepdim=True)
        ids.append(first)
        by = by.scatter(1, first, -math.inf)
    ids = torch.cat(ids, 1)
    w = score.gather(1, ids)
    return ids.to(torch.int32), 2.5 * (w / (w.sum(1, keepdim=True) + TINY) if case["normalise"] else w)


def _exact_loss(s, logits, counts):
    case = s["case"]
    q = _exact_scores(case, logits)
    q = q / q.sum(1, keepdim=True)
    total, live = 0, 0
    for i, (a, b) in enumerate(zip(s["ends"], s["ends"][1:])):
        if b > a:
            f = counts[i].double() * case["experts"] / (case["k"] * (b - a))
            total = total + (f * q[a:b].mean(0)).sum()
            live += 1
    return total * COEF / max(live, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s)
    if op == "balance":
        counts = torch.stack([torch.bincount(s["ids"][a:b].flatten().long(), minlength=case["experts"]) for a, b in zip(s["ends"], s["ends"][1:])])
        return _exact_loss(s, s["logits"].double(), counts), counts.to(torch.int32)
    if op == "grad":
        with torch.enable_grad():
            logits = s["logits"].double().requires_grad_()
            w = _exact_scores(case, logits).gather(1, s["ids"].long())
            if case["normalise"]:
                w = w / (w.sum(1, keepdim=True) + TINY)
            both = (w * 2.5 * s["d_weights"].double()).sum() + _exact_loss(s, logits, s["counts"]) * s["d_loss"].double()[0]
            return torch.autograd.grad(both, logits)[0]
    if op == "rows":
        levels = torch.tensor([(c % 8) * 2.0**-9 if c < 8 else (1 + c % 8 / 8) * 2.0 ** (c // 8 - 7) for c in range(127)], dtype=torch.float64, device="cuda")
        mids = (levels[1:] + levels[:-1]) / 2
        out = torch.empty(case["n"] * case["k"], case["d"], dtype=torch.float64, device="cuda")
        for a in range(0, case["d"], BLOCK):
            v = s["x"][:, a:a + BLOCK].double()
            top = v.abs().amax(1, keepdim=True)
            scale = torch.where(top > 0, (top / TOP).float().double(), 1.0)  # held in 32 bits
            t = v.abs() / scale
            low, high = torch.bucketize(t, mids), torch.bucketize(t, mids, right=True)
            v = levels[torch.where(low % 2 == 0, low, high)] * v.sign() * scale
            for j in range(case["k"]):
                out[s["positions"][:, j].long(), a:a + BLOCK] = v
        return out
    if 2 * case["rows"] * case["n_out"] * case["k"] > 1 << 43:
        return None
    out = torch.zeros(case["rows"], case["n_out"], dtype=torch.float64, device="cuda")
    x = s["codes"].view(torch.float8_e4m3fn).double()
    for e in range(case["experts"]):
        a, b = s["ends"][e], s["ends"][e + 1]
        if b == a:
            continue
        w = s["w_codes"][e].view(torch.float8_e4m3fn).double()
        for j, at in enumerate(range(0, case["k"], BLOCK)):
            part = torch.mm(x[a:b, at:at + BLOCK], w[:, at:at + BLOCK].t()) * s["scales"][a:b, j:j + 1].double()
            out[a:b] += part * s["w_scales"][e, :, j].double().repeat_interleave(BLOCK)[:case["n_out"]]
    return out
