"""The router's operators stated plainly in 64 bits (CPU tensors), and the errors that fp32 arithmetic may make."""

import math

import torch

EPS = 2.0**-24
TINY = 1e-20


def scores(logits, kind):
    l = logits.double()
    if kind == "sigmoid" and l.requires_grad:
        # autograd's own derivative of a sigmoid is s (1 - s), which at a logit of 30 keeps ten bits of 1 - s; this one's
        # is s times 1 / (1 + e^l)
        return torch.exp(torch.nn.functional.logsigmoid(l))
    return torch.sigmoid(l) if kind == "sigmoid" else torch.nan_to_num(torch.softmax(l, 1))


def choice(logits, k, kind, bias=None, groups=1, top_groups=1, normalise=True, scale=1.0):
    """ids and weights, one row after the other."""
    n, E = logits.shape
    s = scores(logits, kind)
    by = s if bias is None else s + bias.double()
    size = E // groups
    ids, weights = torch.full((n, k), -1, dtype=torch.int32), torch.zeros(n, k, dtype=torch.float64)
    for t in range(n):
        l = logits[t].double()
        if l.isnan().any() or (kind == "softmax" and (l == math.inf).any()):
            weights[t] = math.nan
            continue
        left = [e for e in range(E) if l[e] > -math.inf and by[t, e] > -math.inf]
        if groups > 1:
            value = {}
            for g in range(groups):
                best = sorted((by[t, e].item() for e in left if e // size == g), reverse=True)[:2]
                if best:
                    value[g] = sum(best)
            kept = sorted(value, key=lambda g: (-value[g], g))[:top_groups]
            left = [e for e in left if e // size in kept]
        of = l if bias is None else by[t]
        got = sorted(left, key=lambda e: (-of[e].item(), e))[:k]
        ids[t, :len(got)] = torch.tensor(got, dtype=torch.int32)
        w = s[t, got]
        weights[t, :len(got)] = scale * (w / (w.sum() + TINY) if normalise else w)
    return ids, weights


def score_error(logits):
    """A bound of an fp32 score's relative error, in units of 2^-24: expf within 2 ulp (4 of them), the sum of 1 and it,
    the reciprocal within an ulp (2); under softmax also the difference's rounding, once for the expert and once for the
    row's sum, and that sum's E / 32 + 5 additions; a product."""
    finite = logits.double()[logits.isfinite()]
    spread = (finite.max() - finite.min()).item() if finite.numel() else 0.0
    return 12 + 2 * spread + logits.shape[1] / 32 + 5


def sequences(offsets, n):
    if offsets is None:
        return [(0, n)]
    o = offsets.tolist()
    return list(zip(o, o[1:]))


def shares(logits, kind):
    s = scores(logits, kind)
    return torch.nan_to_num(s / s.sum(1, keepdim=True)) if kind == "sigmoid" else s


def balance(logits, ids, coef, kind, offsets=None):
    """loss and counts (the loss differentiable where logits are)."""
    n, E = logits.shape
    q = shares(logits, kind)
    k = ids.shape[1]
    total, live, counts = torch.zeros((), dtype=torch.float64), 0, []
    for a, b in sequences(offsets, n):
        part = ids[a:b]
        c = torch.bincount(part[(part >= 0) & (part < E)].long(), minlength=E)
        counts.append(c)
        if b > a:
            total = total + (c.double() * q[a:b].sum(0)).sum() * E / (k * (b - a) ** 2)
            live += 1
    return coef * total / max(live, 1), torch.stack(counts).to(torch.int32)


def objective(logits, ids, kind, d_weights=None, normalise=True, scale=1.0, coef=None, d_loss=1.0, offsets=None):
    """What route_backward is the gradient of: sum d_weights * weights(ids) + d_loss * loss."""
    s = scores(logits, kind)
    total = torch.zeros((), dtype=torch.float64)
    if d_weights is not None:
        on = (ids >= 0) & (ids < logits.shape[1])
        w = torch.where(on, s.gather(1, torch.where(on, ids, 0).long()), 0.0)
        if normalise:
            w = w / (w.sum(1, keepdim=True) + TINY)
        total = total + (scale * w * d_weights.double()).sum()
    if coef is not None:
        total = total + d_loss * balance(logits, ids, coef, kind, offsets)[0]
    return total


def gradient(logits, ids, kind, **kw):
    l = logits.double().requires_grad_()
    return torch.autograd.grad(objective(l, ids, kind, **kw), l)[0]


def gradient_size(logits, ids, kind, d_weights=None, normalise=True, scale=1.0, coef=None, d_loss=1.0, offsets=None):
    """The gradient's formula with every term's magnitude: what its rounding errors are relative to."""
    n, E = logits.shape
    s = scores(logits, kind)
    d = torch.zeros(n, E, dtype=torch.float64)
    if d_weights is not None:
        on = (ids >= 0) & (ids < E)
        at = torch.where(on, ids, 0).long()
        g = torch.where(on, d_weights.double().abs() * scale, 0.0)
        if normalise:
            chosen = torch.where(on, s.gather(1, at), 0.0)
            total = chosen.sum(1, keepdim=True) + TINY
            g = torch.where(on, (g + (g * chosen).sum(1, keepdim=True) / total) / total, 0.0)
        d.scatter_add_(1, at, g)
    c = torch.zeros(n, E, dtype=torch.float64)
    if coef is not None:
        seqs = sequences(offsets, n)
        live = sum(b > a for a, b in seqs)
        counts = balance(logits, ids, coef, kind, offsets)[1]
        for i, (a, b) in enumerate(seqs):
            if b > a:
                c[a:b] = counts[i].double() * abs(d_loss * coef) * E / (ids.shape[1] * (b - a) ** 2 * live)
    if kind == "softmax":
        d = d + c
        return s * (d + (d * s).sum(1, keepdim=True))
    total = s.sum(1, keepdim=True).clamp(min=1e-300)
    return (d + (c + (c * s).sum(1, keepdim=True) / total) / total) * s * torch.sigmoid(-logits.double())
