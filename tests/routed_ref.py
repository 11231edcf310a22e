"""Plain 64-bit statements of the routed layer's operators (CPU tensors): scores and
choices, their gradient, the row exchange and its gradients, and the AdamW step."""
from __future__ import annotations

import math

import torch

LOWEST = float(torch.finfo(torch.bfloat16).min)
Q_BLOCK = 256


def scores(x, score):
    x = x.double()
    ok = (x > LOWEST) & (x < math.inf)
    if score == "sigmoid":
        return torch.where(ok, torch.sigmoid(x), 0.0), ok
    xs = torch.where(ok, x, -math.inf)
    s = torch.softmax(xs, dim=1)
    return torch.where(ok, s, 0.0), ok


def route(x, k, *, score="softmax", groups=1, top_groups=1, group_top=1, renorm=False, scale=1.0,
          bias=None):
    """One token after the other, by sorting (value descending, index ascending)."""
    T, E = x.shape
    s, ok = scores(x, score)
    limited = top_groups < groups
    if bias is None and not (limited and group_top == 2):
        c = x.double().clone()
    else:
        c = s + (0 if bias is None else bias.double())
    if bias is not None:
        ok = ok & torch.isfinite(bias)
    idx = torch.full((T, k), -1, dtype=torch.int32)
    w = torch.zeros(T, k, dtype=torch.float64)
    per = E // groups
    cl, okl = c.tolist(), ok.tolist()
    for t in range(T):
        allowed = [e for e in range(E) if okl[t][e]]
        if limited:
            value = []
            for q in range(groups):
                best = sorted((cl[t][e] for e in allowed if e // per == q), reverse=True)
                value.append((-sum(best[:group_top]) if best else math.inf, q))
            stay = {q for _, q in sorted(value)[:top_groups]}
            allowed = [e for e in allowed if e // per in stay]
        chosen = sorted(allowed, key=lambda e: (-cl[t][e], e))[:k]
        for j, e in enumerate(chosen):
            idx[t, j] = e
            w[t, j] = s[t, e]
        if renorm and chosen:
            # through the ratio of the scores, which survives their underflow
            xs = x[t, chosen].double()
            if score == "softmax":
                w[t, :len(chosen)] = torch.softmax(xs, 0)
            else:
                w[t, :len(chosen)] = torch.softmax(torch.nn.functional.logsigmoid(xs), 0)
    return idx, scale * w


def gates(x, idx, *, score="softmax", renorm=False, scale=1.0):
    """The weights of fixed choices as a differentiable function of 64-bit logits."""
    ok = (x > LOWEST) & (x < math.inf)
    xs = torch.where(ok, x, torch.full_like(x, -math.inf))
    if score == "sigmoid":
        s = torch.sigmoid(xs)
    else:  # a row with nothing left has no scores at all
        some = ok.any(dim=1, keepdim=True)
        s = torch.softmax(torch.where(some, xs, torch.zeros_like(xs)), dim=1) * some
    there = idx >= 0
    w = torch.where(there, s.gather(1, idx.clamp(min=0).long()), torch.zeros((), dtype=x.dtype))
    if renorm:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total == 0, torch.ones_like(total), total)
    return scale * w


def route_backward(x, idx, dgate, **kw):
    x = x.double().clone().requires_grad_(True)
    w = gates(x, idx, **kw)
    (g,) = torch.autograd.grad((w * dgate.double()).sum(), x)
    return torch.nan_to_num(g, nan=0.0)


def assign(idx, E, C):
    T, k = idx.shape
    seen = [0] * E
    slot = torch.full((T, k), 2 ** 31 - 1, dtype=torch.int32)
    kept = torch.zeros(T, k, dtype=torch.uint8)
    tok = torch.full((E * C,), -1, dtype=torch.int32)
    for t, row in enumerate(idx.tolist()):
        for j, e in enumerate(row):
            if 0 <= e < E:
                slot[t, j] = seen[e]
                if seen[e] < C:
                    kept[t, j] = 1
                    tok[e * C + seen[e]] = t
                seen[e] += 1
    arrivals = torch.tensor(seen, dtype=torch.int32)
    kept_cnt = arrivals.clamp(max=C)
    return dict(slot=slot, kept=kept, tok_of_row=tok, arrivals=arrivals, kept_cnt=kept_cnt,
                n_dropped=(arrivals - kept_cnt).sum().to(torch.int32).view(1))


def rows_of(idx, slot, kept, C):
    """(tokens, choices, expert rows) of the kept choices."""
    t, j = torch.nonzero(kept, as_tuple=True)
    return t, j, idx[t, j].long() * C + slot[t, j].long()


def gather(rows, idx, slot, kept, gate=None):
    T, C, d = idx.shape[0], rows.shape[1], rows.shape[2]
    t, j, r = rows_of(idx, slot, kept, C)
    val = rows.reshape(-1, d)[r].double()
    if gate is not None:
        val = val * gate[t, j, None].double()
    return torch.zeros(T, d, dtype=torch.float64).index_add_(0, t, val)


def combine_backward(dy, ye, idx, gate, slot, kept):
    E, C, d = ye.shape
    t, j, r = rows_of(idx, slot, kept, C)
    dye = torch.zeros(E * C, d, dtype=torch.float64)
    dye[r] = gate[t, j, None].double() * dy[t].double()
    dgate = torch.zeros(idx.shape, dtype=torch.float64)
    dgate[t, j] = (dy[t].double() * ye.reshape(-1, d)[r].double()).sum(1)
    return dye.view(E, C, d), dgate


def dequantize(q, scale):
    q = q.float().double()
    return q * scale.double().repeat_interleave(Q_BLOCK)[:q.numel()]


def adamw(p, g, m, v, *, step, lr, betas, eps, weight_decay, coef=1.0):
    """New (p, m, v) in 64 bits."""
    b1, b2 = betas
    g = g.double() * coef
    m = b1 * m.double() + (1 - b1) * g
    v = b2 * v.double() + (1 - b2) * g * g
    mh, vh = m / (1 - b1 ** step), v / (1 - b2 ** step)
    p = p.double() * (1 - lr * weight_decay) - lr * mh / (vh.sqrt() + eps)
    return p, m, v
