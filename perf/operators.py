"""What is measured of the microscaled-format operators: norm, rows, products by expert and the layer made of them.

A case names an operator ("op"), a format ("fmt": bf16, mxfp8, mxfp4 or nvfp4) and sizes. The formats hold a row as

    bf16   bf16 values
    mxfp8  e4m3 codes, one power of two (biased by 127) per 32 columns
    mxfp4  e2m1 codes, two to a byte (the lower column in the low half), one power of two per 32 columns
    nvfp4  e2m1 codes, one e4m3 scale per 16 columns, times one fp32 factor for the tensor

The power of two is the smallest that brings the group's largest magnitude to the format's largest value or below; the e4m3 scale
is the group's largest magnitude over 6 times the factor. Codes are rounded to nearest, ties to even.
"""

import math

import torch

own = False

GROUP = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
TOP = {"mxfp8": 448.0, "mxfp4": 6.0}
#: columns in the 128 bytes of codes that a packed block holds of a row, and bytes of scales beside them
CHUNK = {"bf16": 64, "mxfp8": 128, "mxfp4": 256, "nvfp4": 256}
WORDS = {"bf16": 0, "mxfp8": 1, "mxfp4": 2, "nvfp4": 4}
EPS = 1e-6


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decoded token ahead of a 7168-wide block: latency alone
        {"name": "norm_token", "op": "norm", "fmt": "nvfp4", "n": 1, "k": 1, "d": 7168},
        # an odd batch of an odd width, each row copied to its three routed positions
        {"name": "norm_odd", "op": "norm", "fmt": "mxfp4", "n": 333, "k": 3, "d": 2080},
        # a long prompt's rows, 8 bits out
        {"name": "norm_prompt", "op": "norm", "fmt": "mxfp8", "n": 32768, "k": 1, "d": 7168},
        # a decode batch's tokens to their eight routed positions
        {"name": "rows_decode", "op": "rows", "fmt": "nvfp4", "n": 16, "k": 8, "d": 7168},
        # a prompt's tokens to their eight routed positions
        {"name": "rows_prompt", "op": "rows", "fmt": "mxfp4", "n": 4096, "k": 8, "d": 7168},
        # one token's eight experts, down projection: the weights of eight experts and nothing else
        {"name": "product_token", "op": "product", "fmt": "nvfp4", "rows": 8, "experts": 384, "n_out": 7168, "k": 2048, "skew": 0.0},
        # ragged experts, some of them empty, sizes that end inside every tile
        {"name": "product_odd", "op": "product", "fmt": "mxfp8", "rows": 1000, "experts": 16, "n_out": 1001, "k": 1056, "skew": 1.2},
        # unquantised experts, a few hundred rows each
        {"name": "product_bf16", "op": "product", "fmt": "bf16", "rows": 4096, "experts": 16, "n_out": 2048, "k": 1024, "skew": 0.0},
        # a prompt's routed rows through the down projection
        {"name": "product_prompt", "op": "product", "fmt": "mxfp4", "rows": 32768, "experts": 384, "n_out": 7168, "k": 2048, "skew": 0.0},
        # the block for one decoded token
        {"name": "layer_token", "op": "layer", "fmt": "nvfp4", "n": 1, "d": 7168, "experts": 384, "topk": 8, "d_ff": 2048},
        # a small model's block
        {"name": "layer_tiny", "op": "layer", "fmt": "mxfp8", "n": 128, "d": 1024, "experts": 16, "topk": 4, "d_ff": 256},
        # the block for a prompt
        {"name": "layer_prompt", "op": "layer", "fmt": "nvfp4", "n": 4096, "d": 7168, "experts": 384, "topk": 8, "d_ff": 2048},
    ]


def draw(rng):
    def spread(lo, hi, step=1):
        return max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + step)))) // step * step)

    op = rng.choice(["norm", "rows", "product", "layer"])
    c = {"op": op, "fmt": rng.choice(["bf16", "mxfp8", "mxfp4", "nvfp4"])}
    if op in ("norm", "rows"):
        n, d = spread(1, 32768), spread(32, 8192, 32)
        c |= {"n": n, "k": rng.choice([1, 1, 2, 3, 8]) if n <= 4096 else 1, "d": d}
    elif op == "product":
        experts = rng.choice([1, spread(2, 384)])
        n_out, k = spread(64, 7168), spread(64, 7168, 32)
        while experts * n_out * k > 384 * 7168 * 2048 // (4 if c["fmt"] == "bf16" else 1):
            experts = max(1, experts // 2)
        rows = spread(1, 32768)
        while rows * n_out * k > 32768 * 7168 * 2048:
            rows //= 2
        c |= {"rows": rows, "experts": experts, "n_out": n_out, "k": k, "skew": rng.choice([0.0, 1.2])}
    else:
        experts = spread(4, 384)
        d, d_ff = spread(128, 7168, 128), spread(128, 2048, 128)
        while c["fmt"] == "bf16" and experts * d * d_ff > 96 * 7168 * 2048:
            experts //= 2
        c |= {"n": spread(1, 4096), "d": d, "experts": experts, "topk": rng.randint(1, min(8, experts)), "d_ff": d_ff}
    return c


# ---------------------------------------------------------------- the formats in elementary operations

def _round_e2m1(t):
    a = t.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp(max=6.0), t)


def _round_e4m3(t):
    a = t.abs()
    step = torch.ldexp(torch.ones_like(a), (torch.frexp(a).exponent - 1).clamp(min=-6) - 3)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), t)


def _quantise(v, fmt, factor):
    """fp32 rows -> (codes' values, scales, the values they stand for), groups along the last axis."""
    if fmt == "bf16":
        q = v.to(torch.bfloat16)
        return q, None, q.float()
    g = v.reshape(*v.shape[:-1], -1, GROUP[fmt])
    amax = g.abs().amax(-1, keepdim=True)
    if fmt == "nvfp4":
        scale = _round_e4m3(amax / (6.0 * factor))
        by = scale * factor
    else:
        m, e = torch.frexp(amax / TOP[fmt])
        e = torch.where(amax > 0, torch.where(m > 0.5, e, e - 1).clamp(min=-126), -126)
        scale = by = torch.ldexp(torch.ones_like(amax), e)
    t = torch.where(by > 0, g / torch.where(by > 0, by, 1.0), 0.0)
    q = _round_e4m3(t) if fmt == "mxfp8" else _round_e2m1(t)
    return q.reshape(v.shape), scale.squeeze(-1), (q * by).reshape(v.shape)


def _codes(q, scale, fmt):
    """The bytes that hold the codes, and the scales' bytes."""
    if fmt == "bf16":
        return q.view(torch.uint8), None
    if fmt == "mxfp8":
        codes = q.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        at = torch.tensor([0, 1, 2, 3, 4, 0, 5, 0, 6, 0, 0, 0, 7], dtype=torch.uint8, device=q.device)
        half = at[(q.abs() * 2).to(torch.int32)] | (torch.signbit(q).to(torch.uint8) << 3)
        codes = half[..., 0::2] | (half[..., 1::2] << 4)
    if fmt == "nvfp4":
        return codes, scale.to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, (torch.frexp(scale).exponent + 126).to(torch.uint8)


def _values(codes, scales, fmt, factor):
    """fp32 values of rows of codes and scales."""
    if fmt == "bf16":
        return codes.view(torch.bfloat16).float()
    if fmt == "mxfp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        level = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
        level = torch.cat([level, -level])
        v = level[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int32)]
    groups = v.shape[-1] // GROUP[fmt]
    scales = scales[..., :groups]
    if fmt == "nvfp4":
        s = scales.view(torch.float8_e4m3fn).float() * factor
    else:
        s = torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.to(torch.int32) - 127)
    return (v.reshape(*v.shape[:-1], groups, GROUP[fmt]) * s[..., None]).flatten(-2)


# ---------------------------------------------------------------- inputs

def _gen(case, seed):
    text = repr(sorted((k, v) for k, v in case.items() if k != "name"))
    return torch.Generator(device="cuda").manual_seed((seed * 1000003 + sum((i + 1) * ord(ch) for i, ch in enumerate(text))) % (1 << 62))


def _bf16(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def _route(gen, n, k, experts):
    return torch.rand(n, experts, generator=gen, device="cuda").topk(k, dim=1).indices.to(torch.int32)


def _positions(ids):
    """Where each (token, slot) lands when the entries are sorted by expert (stable), as an [n, k] table."""
    order = torch.sort(ids.flatten(), stable=True).indices
    at = torch.empty_like(order)
    at[order] = torch.arange(order.numel(), device=order.device)
    return at.reshape(ids.shape).to(torch.int32)


def _factor(v):
    """The tensor's fp32 factor of nvfp4: its largest magnitude at the top of codes times scales."""
    return v.abs().amax().float() / (6.0 * 448.0)


def _weights(gen, experts, rows, cols, fmt, std=0.02):
    """Experts' weights as a checkpoint holds them: codes [E, rows, .], scales [E, rows, .] and nvfp4's factor per expert."""
    made = []
    for _ in range(experts):
        w = torch.randn(rows, cols, generator=gen, device="cuda") * std
        f = _factor(w)
        q, s, _ = _quantise(w, fmt, f)
        made.append((*_codes(q, s, fmt), f))
    codes = torch.stack([m[0] for m in made])
    scales = torch.stack([m[1] for m in made]) if fmt != "bf16" else None
    return {"codes": codes, "scales": scales, "factor": torch.stack([m[2] for m in made]) if fmt == "nvfp4" else torch.ones(experts, device="cuda")}


def _packed(parts, fmt):
    """The weights as a serving program keeps them once they are loaded: blocks of 256 rows by 128 bytes of codes with their scales,
    consecutive along the row. Two parts (gate, up) share a block, 128 rows of each. A block holds row r's 16-byte piece j at piece
    j ^ (r % 8) of its 128 bytes, then word w of the row's scales at 1024 w + 512 (r / 128) + 16 (r % 32) + 4 (r / 32 % 4)."""
    tall = 256 // len(parts)
    blocks = []
    for p in parts:
        codes, scales = p["codes"], p["scales"]
        experts, rows, width = codes.shape
        up, chunks = -(-rows // tall), -(-width // 128)
        codes = torch.nn.functional.pad(codes, (0, chunks * 128 - width, 0, up * tall - rows))
        codes = codes.reshape(experts, up, tall, chunks, 8, 16).transpose(2, 3)
        row = torch.arange(tall, device=codes.device)[:, None]
        codes = codes[:, :, :, row, torch.arange(8, device=codes.device) ^ (row % 8)]
        if scales is not None:
            w = WORDS[fmt]
            scales = torch.nn.functional.pad(scales, (0, chunks * w * 4 - scales.shape[-1], 0, up * tall - rows))
            scales = scales.reshape(experts, up, tall, chunks, w, 4).permute(0, 1, 3, 4, 2, 5)
        blocks.append((codes, scales))
    codes = torch.cat([b[0] for b in blocks], 3).flatten(3)
    if fmt == "bf16":
        return codes.contiguous()
    scales = torch.cat([b[1] for b in blocks], 4)
    scales = scales.reshape(*scales.shape[:4], 2, 4, 32, 4).transpose(5, 6).flatten(3)
    return torch.cat([codes, scales], 3)


def _offsets(gen, rows, experts, skew):
    """Rows by expert: even odds, or by a power law that leaves some experts empty."""
    odds = torch.arange(1, experts + 1, device="cuda", dtype=torch.float32) ** -skew
    odds = odds[torch.randperm(experts, generator=gen, device="cuda")]
    who = torch.multinomial(odds, rows, replacement=True, generator=gen)
    count = torch.bincount(who, minlength=experts)
    return torch.nn.functional.pad(count.cumsum(0), (1, 0)).to(torch.int32)


def prepare(case, seed):
    gen, fmt, op = _gen(case, seed), case["fmt"], case["op"]
    s = {"case": case}
    if op in ("norm", "rows", "layer"):
        n, d = case["n"], case["d"]
        s["x"] = _bf16(gen, n, d)
        if op != "rows":
            s["residual"] = _bf16(gen, n, d)
            s["gain"] = 1 + _bf16(gen, d, std=0.1)
        s["factor"] = torch.tensor(2.0**-8, device="cuda")  # calibrated: values up to 10; a power of two adds no rounding of its own
    if op in ("norm", "rows"):
        s["positions"] = _positions(_route(gen, n, case["k"], 64))
    elif op == "product":
        rows, experts, n_out, k = case["rows"], case["experts"], case["n_out"], case["k"]
        x = torch.randn(rows, k, generator=gen, device="cuda")
        s["factor"] = _factor(x)
        q, scale, _ = _quantise(x, fmt, s["factor"])
        s["codes"], scale = _codes(q, scale, fmt)
        if scale is not None:  # rows of scales start on 16 bytes
            scale = torch.nn.functional.pad(scale, (0, -scale.shape[1] % 16))
        s["scales"] = scale
        s["w"] = _weights(gen, experts, n_out, k, fmt)
        s["packed"] = _packed([s["w"]], fmt)
        s["offsets"] = _offsets(gen, rows, experts, case["skew"])
        s["ends"] = s["offsets"].tolist()
    if op == "layer":
        experts, f = case["experts"], case["d_ff"]
        s["gate"], s["up"] = (_weights(gen, experts, f, d, fmt) for _ in range(2))
        s["down"] = _weights(gen, experts, d, f, fmt)
        s["packed_gate_up"], s["packed_down"] = _packed([s["gate"], s["up"]], fmt), _packed([s["down"]], fmt)
        s["ids"] = _route(gen, n, case["topk"], experts)
        s["topk_weight"] = torch.softmax(torch.randn(n, case["topk"], generator=gen, device="cuda"), -1)
        s["h_factor"] = torch.tensor(2.0**-6, device="cuda")
        count = torch.bincount(s["ids"].flatten(), minlength=experts)
        s["ends"] = torch.nn.functional.pad(count.cumsum(0), (1, 0)).tolist()
    # a workspace that a serving program allocates once
    rows = case["n"] * case["topk"] if op == "layer" else 0
    s["workspace"] = torch.zeros((1 << 24) + rows * (5 * case.get("d", 0) + 3 * case.get("d_ff", 0) + 64), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass, plain

def _norm(s):
    total = (s["x"].float() + s["residual"].float()).to(torch.bfloat16)
    v = total.float()
    return total, v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * s["gain"].float()


def _product(x, w, ends, fmt):
    """fp32 rows times each row's expert, expert after expert."""
    out = torch.empty(x.shape[0], w["codes"].shape[1], device="cuda")
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        if b > a:
            m = _values(w["codes"][e], None if fmt == "bf16" else w["scales"][e], fmt, w["factor"][e])
            out[a:b] = x[a:b] @ m.T
    return out


def _plain(s):
    case, fmt = s["case"], s["case"]["fmt"]
    op = case["op"]
    if op == "product":
        return _product(_values(s["codes"], s["scales"], fmt, s["factor"]), s["w"], s["ends"], fmt).to(torch.bfloat16)
    total, v = _norm(s) if op != "rows" else (None, s["x"].float())
    v = _quantise(v, fmt, s["factor"])[2]
    if op != "layer":
        at = s["positions"]
        rows = torch.empty(at.numel(), v.shape[1], dtype=torch.bfloat16, device="cuda")
        rows[at.flatten().long()] = v.to(torch.bfloat16).repeat_interleave(at.shape[1], 0)
        return rows if op == "rows" else (total, rows)
    k = case["topk"]
    order = torch.sort(s["ids"].flatten(), stable=True).indices
    x = v[order // k]
    g, u = _product(x, s["gate"], s["ends"], fmt), _product(x, s["up"], s["ends"], fmt)
    h = _quantise(g / (1 + torch.exp(-g)) * u, fmt, s["h_factor"])[2]
    y = torch.empty(order.numel(), case["d"], device="cuda")
    y[order] = _product(h, s["down"], s["ends"], fmt)
    y = (y.reshape(case["n"], k, -1) * s["topk_weight"][..., None]).sum(1)
    return total, (total.float() + y).to(torch.bfloat16)


# ---------------------------------------------------------------- one pass, the framework's calls

def _kernels(s):
    import mixture_experts_ffn_infer_gb300 as mx

    case = s["case"]
    fmt, op = mx.MX_FORMATS[case["fmt"]], case["op"]
    factor = s["factor"] if case["fmt"] == "nvfp4" else None
    if op == "product":
        x = mx.MxRows(fmt, case["k"], s["codes"], s["scales"], factor)
        w = mx.MxWeights(fmt, case["experts"], case["n_out"], case["k"], s["packed"], s["w"]["factor"] if factor is not None else None)
        return mx.mx_grouped_product(x, w, s["offsets"], ws=s["workspace"])
    if op == "rows":
        return mx.mx_dequantise(mx.mx_quantise(s["x"], fmt, positions=s["positions"], global_scale=factor))
    if op == "norm":
        rows, total = mx.mx_add_rmsnorm(s["x"], s["residual"], s["gain"], EPS, fmt, positions=s["positions"], global_scale=factor)
        return total, mx.mx_dequantise(rows)
    alpha = [s[p]["factor"] if factor is not None else None for p in ("gate", "up", "down")]
    gate_up = mx.MxWeights(fmt, case["experts"], case["d_ff"], case["d"], s["packed_gate_up"], alpha[0], alpha[1], swiglu=True)
    down = mx.MxWeights(fmt, case["experts"], case["d"], case["d_ff"], s["packed_down"], alpha[2])
    return mx.mx_layer_forward(s["x"], s["residual"], s["gain"], EPS, s["ids"], s["topk_weight"], gate_up, down, x_global=factor,
                               h_global=s["h_factor"] if factor is not None else None, ws=s["workspace"])


def run(state):
    return _kernels(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def _row_bytes(fmt, cols):
    return {"bf16": 2.0, "mxfp8": 1 + 1 / 32, "mxfp4": 0.5 + 1 / 32, "nvfp4": 0.5 + 1 / 16}[fmt] * cols


def work(case):
    fmt, op = case["fmt"], case["op"]
    if op in ("norm", "rows"):
        n, k, d = case["n"], case["k"], case["d"]
        held = 2 * n * k * _row_bytes(fmt, d) if fmt != "bf16" else 0  # the quantised rows, written and read; bf16 rows are the output
        return {"bytes": (6 if op == "norm" else 2) * n * d + held + 2 * n * k * d + 4 * n * k, "flops": 8 * n * d}
    if op == "product":
        rows, n_out, k = case["rows"], case["n_out"], case["k"]
        touched = _touched(rows, case["experts"], case["skew"])
        return {"bytes": touched * n_out * _row_bytes(fmt, k) + rows * _row_bytes(fmt, k) + 2 * rows * n_out, "flops": 2 * rows * n_out * k}
    n, d, f, rows = case["n"], case["d"], case["d_ff"], case["n"] * case["topk"]
    touched = case["experts"] * (1 - (1 - case["topk"] / case["experts"]) ** n)
    return {"bytes": touched * (2 * f * _row_bytes(fmt, d) + d * _row_bytes(fmt, f)) + 8 * n * d, "flops": 6 * rows * d * f}


def _touched(rows, experts, skew):
    odds = [(i + 1) ** -skew for i in range(experts)]
    return sum(1 - (1 - o / sum(odds)) ** rows for o in odds)


# ---------------------------------------------------------------- in 64 bits, from the definition

def _nearest(t, levels):
    """Index of the nearest of the ascending levels (from 0), ties to the even index."""
    mids = (levels[1:] + levels[:-1]) / 2
    low, high = torch.bucketize(t, mids), torch.bucketize(t, mids, right=True)
    return torch.where(low % 2 == 0, low, high)


def _levels(kind):
    if kind == "e2m1":
        return torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    return torch.tensor([(c % 8) * 2.0**-9 if c < 8 else (1 + c % 8 / 8) * 2.0 ** (c // 8 - 7) for c in range(127)], dtype=torch.float64, device="cuda")


def _exact_rows(v, fmt, factor):
    """The values that 64-bit rows stand for once they are held in the format (bf16 rows: unrounded)."""
    if fmt == "bf16":
        return v
    parts = []
    for p in v.split(1024):
        g = p.reshape(p.shape[0], -1, GROUP[fmt])
        top = g.abs().max(-1, keepdim=True).values
        if fmt == "nvfp4":
            e4m3 = _levels("e4m3")
            by = e4m3[_nearest(top / (6 * factor.double()), e4m3)] * factor.double()
        else:
            by = torch.exp2(torch.ceil(torch.log2(top / TOP[fmt])).clamp(min=-126))
            by = torch.where(top > TOP[fmt] * by, by * 2, torch.where(top <= TOP[fmt] * by / 2, by / 2, by))
        levels = _levels("e4m3" if fmt == "mxfp8" else "e2m1")
        t = torch.where(by > 0, g.abs() / by, 0.0)
        parts.append((levels[_nearest(t, levels)] * g.sign() * by).reshape(p.shape))
    return torch.cat(parts)


def _exact_weight(w, e, fmt):
    codes = w["codes"][e]
    if fmt == "bf16":
        return codes.view(torch.bfloat16).double()
    if fmt == "mxfp8":
        e4m3 = torch.cat([_levels("e4m3"), torch.zeros(1, dtype=torch.float64, device="cuda")])
        v = torch.cat([e4m3, -e4m3])[codes.long()]
    else:
        level = _levels("e2m1")
        v = torch.cat([level, -level])[torch.stack((codes % 16, codes // 16), 2).reshape(codes.shape[0], -1).long()]
    scale = w["scales"][e].long()
    scale = _levels("e4m3")[scale.clamp(max=126)] * w["factor"][e].double() if fmt == "nvfp4" else torch.exp2(scale.double() - 127)
    return v * scale.repeat_interleave(GROUP[fmt], 1)[:, :v.shape[1]]


def _exact_product(x, w, ends, fmt):
    out = torch.zeros(x.shape[0], w["codes"].shape[1], dtype=torch.float64, device="cuda")
    for e in range(len(ends) - 1):
        if ends[e + 1] > ends[e]:
            out[ends[e]:ends[e + 1]] = torch.mm(x[ends[e]:ends[e + 1]], _exact_weight(w, e, fmt).t())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    fmt, op = case["fmt"], case["op"]
    if op == "product":
        held = {"codes": s["codes"][None], "scales": None if fmt == "bf16" else s["scales"][None, :, :case["k"] // GROUP[fmt]], "factor": s["factor"][None]}
        return _exact_product(_exact_weight(held, 0, fmt), s["w"], s["ends"], fmt)
    total, v = None, s["x"].double()
    if op != "rows":
        total = v + s["residual"].double()
        v = total.to(torch.bfloat16).double()  # the norm is that of the sum as it is stored
        v = v / torch.sqrt((v * v).sum(1, keepdim=True) / case["d"] + EPS) * s["gain"].double()
    v = _exact_rows(v, fmt, s["factor"])
    if op != "layer":
        rows = torch.empty(case["n"] * case["k"], case["d"], dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            rows[s["positions"][:, j].long()] = v
        return rows if op == "rows" else (total, rows)
    flat = s["ids"].flatten()
    order = flat.argsort(stable=True)
    x = v[torch.div(order, case["topk"], rounding_mode="floor")]
    g, u = (_exact_product(x, s[p], s["ends"], fmt) for p in ("gate", "up"))
    h = _exact_rows(g * torch.sigmoid(g) * u, fmt, s["h_factor"])
    y = _exact_product(h, s["down"], s["ends"], fmt) * s["topk_weight"].double().flatten()[order][:, None]
    out = total.to(torch.bfloat16).double()
    return total, out.index_add(0, torch.div(order, case["topk"], rounding_mode="floor"), y)
