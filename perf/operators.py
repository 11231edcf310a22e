"""Operator cases: routing scores, the row exchange for several choices a token,
and the AdamW step, each in plain torch and through the library's entry points.

``run`` computes an operator from elementary torch operations, or with
``own = True`` calls the library.  Both work on the same state.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
# a logit at or below bf16's lowest value masks its expert, like -inf
LOWEST = float(torch.finfo(torch.bfloat16).min)
BLOCK = 256  # elements that share one scale of the 8-bit states


# ---- cases ---------------------------------------------------------------------

def listed():
    return [
        # one decoding step of four sequences: launch and latency only
        dict(name="route_decode", op="route", T=4, E=256, k=8, score="sigmoid", groups=8,
             top_groups=4, group_top=2, renorm=True, bias=True, dtype="f32", pad=False),
        # a large training batch: sigmoid scores, balance bias, 4 of 8 groups stay
        dict(name="route_train", op="route", T=65536, E=256, k=8, score="sigmoid", groups=8,
             top_groups=4, group_top=2, renorm=True, bias=True, dtype="f32", pad=False),
        # ragged prefill with padded rows: softmax, no groups, bf16 logits (exact ties occur)
        dict(name="route_prefill_pad", op="route", T=8191, E=60, k=6, score="softmax", groups=1,
             top_groups=1, group_top=1, renorm=False, bias=False, dtype="bf16", pad=True),
        # gradient of plain softmax gates: every logit gets one
        dict(name="route_bwd_softmax", op="route_backward", T=32768, E=64, k=6, score="softmax",
             groups=1, top_groups=1, group_top=1, renorm=False, bias=False, dtype="f32", pad=False),
        # gradient of renormalised sigmoid gates, odd batch, bf16
        dict(name="route_bwd_sigmoid", op="route_backward", T=4097, E=256, k=8, score="sigmoid",
             groups=8, top_groups=4, group_top=2, renorm=True, bias=True, dtype="bf16", pad=False),
        # rows of a training batch into expert order: slots, then the copy
        dict(name="dispatch_train", op="dispatch", T=16384, E=64, k=8, d=1024, cf=1.25,
             dtype="bf16"),
        # a few decoding tokens over many experts, nothing dropped
        dict(name="dispatch_decode", op="dispatch", T=5, E=128, k=4, d=768, cf=0.0, dtype="bf16"),
        # weighted sum of eight expert rows a token, odd batch, wide rows
        dict(name="combine_wide", op="combine", T=8191, E=256, k=8, d=2560, cf=1.5, dtype="bf16"),
        # gradients of the weighted sum: expert rows and weights
        dict(name="combine_bwd", op="combine_backward", T=16384, E=64, k=6, d=1024, cf=1.25,
             dtype="bf16"),
        # a sparse layer's parameters: one dense set and sixteen experts, clipped, bf16 copies
        dict(name="adamw_experts", op="adamw", bits=32, dense=50_000_000, n=16, lo=8_388_608,
             hi=8_388_608, grad="f32", copy=True, clip=True),
        # the same with 8-bit states and bf16 gradients
        dict(name="adamw8_experts", op="adamw", bits=8, dense=50_000_000, n=16, lo=8_388_608,
             hi=8_388_608, grad="bf16", copy=False, clip=True),
        # many small tensors of odd sizes: launches, not bytes
        dict(name="adamw_small", op="adamw", bits=32, dense=0, n=120, lo=1, hi=20_011, grad="f32",
             copy=False, clip=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route", "route_backward", "dispatch", "dispatch_backward",
                     "combine", "combine_backward", "adamw", "adamw"])
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 1, 2, 3, 4, 8])
        per = rng.randint(4, 256 // groups)
        top_groups = rng.randint(1, groups)
        E = groups * per
        return dict(op=op, T=_log_int(rng, 1, 65536), E=E,
                    k=rng.randint(1, min(16, top_groups * per)),
                    score=rng.choice(["softmax", "sigmoid"]), groups=groups, top_groups=top_groups,
                    group_top=rng.choice([1, 2]), renorm=rng.random() < 0.5,
                    bias=rng.random() < 0.6, dtype=rng.choice(["f32", "bf16"]),
                    pad=rng.random() < 0.3)
    if op == "adamw":
        bits = rng.choice([32, 8])
        n = rng.randint(1, 100)
        lo = _log_int(rng, 1, 2000)
        hi = max(lo, min(_log_int(rng, 1000, 4_000_000), 60_000_000 // n))
        return dict(op=op, bits=bits, dense=rng.choice([0, _log_int(rng, 1000, 40_000_000)]), n=n,
                    lo=lo, hi=hi, grad=rng.choice(["f32", "bf16"]), copy=rng.random() < 0.4,
                    clip=rng.random() < 0.6)
    E = rng.randint(2, 256)
    k = rng.randint(1, min(16, E))
    d = 64 * _log_int(rng, 1, 40)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    room = 100_000_000 // (k * d * (1 if dtype == "bf16" else 2))
    T = _log_int(rng, 1, max(1, min(65536, room)))
    return dict(op=op, T=T, E=E, k=k, d=d, cf=rng.choice([0.75, 1.0, 1.25, 1.5]), dtype=dtype)


# ---- inputs --------------------------------------------------------------------

def _dt(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _capacity(c):
    """Rows an expert takes: floor(T k / E * cf), at least 1; cf = 0: every token fits."""
    if c["cf"] == 0.0:
        return c["T"]
    return max(1, int(c["T"] * c["k"] / c["E"] * c["cf"]))


def _lengths(c):
    """The tensors' lengths: `dense` if any, then n from lo to hi, evenly in their logarithm."""
    n, lo, hi = c["n"], c["lo"], c["hi"]
    step = (hi / lo) ** (1.0 / max(1, n - 1))
    return ([c["dense"]] if c["dense"] else []) + [int(lo * step ** i) for i in range(n)]


def _prepare_route(c, g):
    T, E = c["T"], c["E"]
    x = torch.randn(T, E, generator=g, device=DEV)
    x += 0.5 * torch.randn(E, generator=g, device=DEV)  # experts of unlike popularity
    if c["pad"]:
        x[16::17] = -math.inf                                   # padded tokens
        x[::5, torch.randint(E, (1,), generator=g, device=DEV)] = torch.finfo(torch.float32).min
    x = x.clamp(min=LOWEST).to(_dt(c["dtype"])) if c["dtype"] == "bf16" else x
    if c["pad"]:
        x[16::17] = -math.inf
    b = 0.05 * torch.randn(E, generator=g, device=DEV) if c["bias"] else None
    s = dict(c=c, logits=x, bias=b)
    if c["op"] == "route":
        s["expert_idx"] = torch.empty(T, c["k"], dtype=torch.int32, device=DEV)
        s["gate"] = torch.empty(T, c["k"], device=DEV)
    else:
        s["expert_idx"] = _plain_route(c, x, b)[0]
        s["dgate"] = torch.randn(T, c["k"], generator=g, device=DEV)
        s["dlogits"] = torch.empty_like(x)
    return s


def _prepare_rows(c, g):
    T, E, k, d, C = c["T"], c["E"], c["k"], c["d"], _capacity(c)
    dt = _dt(c["dtype"])
    liking = torch.rand(T, E, generator=g, device=DEV) + 0.3 * torch.rand(E, generator=g, device=DEV)
    idx = liking.sort(dim=1, descending=True).indices[:, :k].to(torch.int32).contiguous()
    s = dict(c=c, expert_idx=idx)
    if c["op"] == "dispatch":
        s["x"] = torch.randn(T, d, generator=g, device=DEV).to(dt)
        s["xe"] = torch.zeros(E * C + 1, d, dtype=dt, device=DEV)  # the last row takes dropped choices
        return s
    a = _plain_assign(c, idx)
    s.update(slot=a["slot"], kept=a["kept"])
    if c["op"] == "dispatch_backward":
        s["dxe"] = torch.randn(E, C, d, generator=g, device=DEV, dtype=torch.float32).to(dt)
        s["dx"] = torch.empty(T, d, dtype=dt, device=DEV)
        return s
    w = torch.rand(T, k, generator=g, device=DEV) + 0.05
    s["gate"] = w / w.sum(1, keepdim=True)
    s["ye"] = torch.empty(E, C, d, dtype=dt, device=DEV)
    s["ye"].normal_(generator=g)
    if c["op"] == "combine":
        s["y"] = torch.empty(T, d, dtype=dt, device=DEV)
    else:
        s["dy"] = torch.randn(T, d, generator=g, device=DEV).to(dt)
        s["dye"] = torch.zeros(E * C + 1, d, dtype=dt, device=DEV)
        s["dgate"] = torch.empty(T, k, device=DEV)
    return s


def _prepare_adamw(c, g):
    lens = _lengths(c)
    starts, total = [], 0
    for n in lens:  # every tensor starts a block of its own; the rest of its last block is zero
        starts.append(total)
        total += -(-n // BLOCK) * BLOCK
    p = 0.02 * torch.randn(total, generator=g, device=DEV)
    gr = 1e-3 * torch.randn(total, generator=g, device=DEV)
    m = 2e-4 * torch.randn(total, generator=g, device=DEV)
    v = (1e-3 * torch.randn(total, generator=g, device=DEV)).square_().add_(1e-8)
    for a, n in zip(starts, lens):
        end = a + -(-n // BLOCK) * BLOCK
        for t in (p, gr, m, v):
            t[a + n:end] = 0
    s = dict(c=c, lens=lens, starts=starts, p=p, g=gr.to(_dt(c["grad"])), step=1000, lr=3e-4,
             copy=torch.zeros(total, dtype=torch.bfloat16, device=DEV) if c["copy"] else None)
    s["norm"] = s["g"].double().square().sum().sqrt().reshape(1) if c["clip"] else None
    s["max_norm"] = 0.5 * float(s["norm"]) if c["clip"] else 0.0
    if c["bits"] == 32:
        s.update(m=m, v=v, m_scale=None, v_scale=None)
    else:
        s["m"], s["m_scale"] = _to_e4m3(m)
        s["v"], s["v_scale"] = _to_e4m3(v.sqrt())
    if own:
        import sparse_mixture_experts_fwd_b200 as moe

        def cut(t, per=1):
            if t is None:
                return None
            return [t[a // per:a // per + -(-n // per)] for a, n in zip(starts, lens)]

        s["tensors"] = moe.adamw_tensors(
            cut(p), cut(s["g"]), cut(s["m"]), cut(s["v"]), exp_avg_scale=cut(s["m_scale"], BLOCK),
            exp_avg_sq_scale=cut(s["v_scale"], BLOCK), bf16_copies=cut(s["copy"]))
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    if case["op"] in ("route", "route_backward"):
        return _prepare_route(case, g)
    if case["op"] == "adamw":
        return _prepare_adamw(case, g)
    return _prepare_rows(case, g)


# ---- plain forms ---------------------------------------------------------------

def _plain_scores(c, x):
    """Scores in 64 bits and which logits count (not masked, not NaN or +inf)."""
    x = x.double()
    ok = (x > LOWEST) & (x < math.inf)
    x = torch.where(ok, x, -math.inf)
    if c["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x)), ok, x
    top = x.max(dim=1, keepdim=True).values
    e = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(dim=1, keepdim=True)
    return e / torch.where(total == 0, 1.0, total), ok, x


def _plain_route(c, x, bias):
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    s, ok, x = _plain_scores(c, x)
    by_group = c["top_groups"] < G
    if bias is None and not (by_group and c["group_top"] == 2):
        v = x  # the scores grow with the logits
    else:
        v = s if bias is None else s + bias.double()
    v = torch.where(ok, v, -math.inf)
    if by_group:
        best = v.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :c["group_top"]]
        none = best[:, :, 0] == -math.inf
        best = torch.where(best == -math.inf, 0.0, best).sum(dim=2)
        best = torch.where(none, -math.inf, best)
        first = best.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        stays = (first[:, :, None] == torch.arange(G, device=x.device)).any(dim=1)
        v = torch.where(stays.repeat_interleave(E // G, dim=1), v, -math.inf)
    v, idx = v.sort(dim=1, descending=True, stable=True)
    left = v[:, :k] != -math.inf
    idx = idx[:, :k]
    w = torch.where(left, s.gather(1, idx), 0.0)
    if c["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = w / torch.where(total == 0, 1.0, total)
    return torch.where(left, idx, -1).to(torch.int32), w.float()


def _plain_route_backward(c, x, idx, dw):
    x = x.float()
    ok = (x > LOWEST) & (x < math.inf)
    x = torch.where(ok, x, -math.inf)
    there = idx >= 0
    at = idx.clamp(min=0).long()
    dw = torch.where(there, dw, 0.0)
    if c["score"] == "softmax" and not c["renorm"]:
        top = x.max(dim=1, keepdim=True).values
        e = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
        total = e.sum(dim=1, keepdim=True)
        s = e / torch.where(total == 0, 1.0, total)
        a = torch.zeros_like(s).scatter_add_(1, at, dw)
        return s * (a - (a * s).sum(dim=1, keepdim=True))
    xs = torch.where(there, x.gather(1, at), -math.inf)
    if c["score"] == "softmax":
        top = xs.max(dim=1, keepdim=True).values
        s = torch.exp(xs - torch.where(top == -math.inf, 0.0, top))
        slope = 1.0
    else:
        s = 1.0 / (1.0 + torch.exp(-xs))
        slope = 1.0 / (1.0 + torch.exp(xs))
    if c["renorm"]:
        total = s.sum(dim=1, keepdim=True)
        q = s / torch.where(total == 0, 1.0, total)
        d = q * slope * (dw - (dw * q).sum(dim=1, keepdim=True))
    else:
        d = dw * s * slope
    return torch.zeros_like(x).scatter_add_(1, at, torch.where(there, d, 0.0))


def _plain_assign(c, idx):
    E, C = c["E"], _capacity(c)
    e = idx.reshape(-1).long()
    took = torch.arange(E, device=e.device)[:, None] == e
    before = took.cumsum(dim=1, dtype=torch.int32)
    slot = before.gather(0, e[None, :])[0] - 1
    kept = slot < C
    arrivals = before[:, -1].clone()
    kept_cnt = arrivals.clamp(max=C)
    row = torch.where(kept, e * C + slot, E * C)
    tok = torch.full((E * C + 1,), -1, dtype=torch.int32, device=e.device)
    tok[row] = torch.arange(e.numel(), dtype=torch.int32, device=e.device) // c["k"]
    shape = idx.shape
    return dict(slot=slot.to(torch.int32).view(shape), kept=kept.to(torch.uint8).view(shape),
                tok_of_row=tok[:-1], arrivals=arrivals, kept_cnt=kept_cnt,
                n_dropped=(arrivals - kept_cnt).sum().to(torch.int32).view(1))


def _rows(c, s):
    """Row of the expert buffer for each choice; the one past its end where it was dropped."""
    C = _capacity(c)
    return torch.where(s["kept"] != 0, s["expert_idx"].long() * C + s["slot"], c["E"] * C)


def _plain_dispatch(c, s):
    a = _plain_assign(c, s["expert_idx"])
    row = _rows(c, dict(expert_idx=s["expert_idx"], slot=a["slot"], kept=a["kept"]))
    s["xe"][row.reshape(-1)] = s["x"].repeat_interleave(c["k"], dim=0)
    a["xe"] = s["xe"][:-1]
    return a


def _gathered(c, rows, s):
    """[T, k, d] in 32 bits: the rows of the kept choices, zeros for the others."""
    flat = rows.reshape(-1, rows.shape[-1])
    kept = s["kept"] != 0
    at = torch.where(kept, _rows(c, s), 0)
    return torch.where(kept[:, :, None], flat[at].float(), 0.0)


def _plain_combine_backward(c, s):
    dy = s["dy"].float()
    dgate = (dy[:, None, :] * _gathered(c, s["ye"], s)).sum(dim=2)
    dye = s["gate"][:, :, None] * dy[:, None, :]
    s["dye"][_rows(c, s).reshape(-1)] = dye.to(s["dye"].dtype).view(-1, c["d"])
    return dict(dye=s["dye"][:-1], dgate=dgate)


def _to_e4m3(t):
    """Codes and one scale for each block of BLOCK values."""
    t = t.view(-1, BLOCK)
    scale = t.abs().max(dim=1, keepdim=True).values / 448.0
    q = t / torch.where(scale == 0, 1.0, scale)
    # what is not zero in the second moment stays so: 2^-9 is the smallest code
    q = torch.where((t > 0) & (t.min() >= 0), q.clamp(min=2.0 ** -9), q)
    return q.to(torch.float8_e4m3fn).view(-1), scale.view(-1)


def _of_e4m3(q, scale):
    return (q.float().view(-1, BLOCK) * scale[:, None]).view(-1)


BETA1, BETA2, EPS, DECAY = 0.9, 0.95, 1e-8, 0.1


def _plain_adamw(c, s):
    t, lr = s["step"], s["lr"]
    g = s["g"].float()
    if c["clip"]:
        g = g * (s["max_norm"] / s["norm"]).clamp(max=1.0).float()
    m, v = s["m"], s["v"]
    if c["bits"] == 8:
        m = _of_e4m3(m, s["m_scale"])
        v = _of_e4m3(v, s["v_scale"]).square()
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    root = v.sqrt()
    denom = root / math.sqrt(1 - BETA2 ** t) + EPS
    p = s["p"] * (1 - lr * DECAY) - (lr / (1 - BETA1 ** t)) * (m / denom)
    s["p"].copy_(p)
    out = dict(p=s["p"])
    if c["bits"] == 8:
        qm, sm = _to_e4m3(m)
        qv, sv = _to_e4m3(root)
        for name, x in (("m", qm), ("v", qv), ("m_scale", sm), ("v_scale", sv)):
            s[name].copy_(x)
            out[name] = s[name]
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
        out.update(m=s["m"], v=s["v"])
    if c["copy"]:
        s["copy"].copy_(p)
        out["copy"] = s["copy"]
    return out


# ---- the library's calls -------------------------------------------------------

def _own_route_config(moe, c):
    return moe.make_route_config(c["T"], c["E"], c["k"], score=c["score"], num_groups=c["groups"],
                                 top_groups=c["top_groups"], group_top=c["group_top"],
                                 renorm=c["renorm"], dtype=_dt(c["dtype"]))


def _own_run(s):
    import sparse_mixture_experts_fwd_b200 as moe
    c = s["c"]
    op = c["op"]
    if op == "route":
        idx, gate = moe.route(_own_route_config(moe, c), s["logits"], s["bias"],
                              expert_idx=s["expert_idx"], gate=s["gate"])
        return dict(expert_idx=idx, gate=gate)
    if op == "route_backward":
        return dict(dlogits=moe.route_backward(_own_route_config(moe, c), s["logits"],
                                               s["expert_idx"], s["dgate"], dlogits=s["dlogits"]))
    if op == "adamw":
        moe.adamw_step(s["tensors"], step=s["step"], lr=s["lr"], betas=(BETA1, BETA2), eps=EPS,
                       weight_decay=DECAY, norm=s["norm"], max_norm=s["max_norm"])
        out = dict(p=s["p"], m=s["m"], v=s["v"])
        if c["bits"] == 8:
            out.update(m_scale=s["m_scale"], v_scale=s["v_scale"])
        if c["copy"]:
            out["copy"] = s["copy"]
        return out
    cfg = moe.make_config(c["T"], c["d"], 64, c["E"], c["k"], _capacity(c), dtype=_dt(c["dtype"]))
    if op == "dispatch":
        a = moe.assign(cfg, s["expert_idx"])
        xe = s["xe"][:-1]
        moe.dispatch(cfg, s["x"], s["expert_idx"], a["slot"], a["kept"], xe=xe)
        return dict(a, xe=xe)
    if op == "dispatch_backward":
        return dict(dx=moe.dispatch_backward(cfg, s["dxe"], s["expert_idx"], s["slot"], s["kept"],
                                             dx=s["dx"]))
    if op == "combine":
        return dict(y=moe.combine(cfg, s["ye"], s["expert_idx"], s["gate"], s["slot"], s["kept"],
                                  y=s["y"]))
    dye = s["dye"][:-1]
    _, dgate = moe.combine_backward(cfg, s["dy"], s["ye"], s["expert_idx"], s["gate"], s["slot"],
                                    s["kept"], dye=dye, dgate=s["dgate"])
    return dict(dye=dye, dgate=dgate)


def run(state):
    c = state["c"]
    if c["op"] == "adamw":
        state["step"] += 1
    if own:
        return _own_run(state)
    if c["op"] == "route":
        idx, gate = _plain_route(c, state["logits"], state["bias"])
        return dict(expert_idx=idx, gate=gate)
    if c["op"] == "route_backward":
        d = _plain_route_backward(c, state["logits"], state["expert_idx"], state["dgate"])
        return dict(dlogits=d.to(state["logits"].dtype))
    if c["op"] == "adamw":
        return _plain_adamw(c, state)
    if c["op"] == "dispatch":
        return _plain_dispatch(c, state)
    if c["op"] == "dispatch_backward":
        return dict(dx=_gathered(c, state["dxe"], state).sum(dim=1).to(state["dx"].dtype))
    if c["op"] == "combine":
        y = (state["gate"][:, :, None] * _gathered(c, state["ye"], state)).sum(dim=1)
        return dict(y=y.to(state["y"].dtype))
    return _plain_combine_backward(c, state)


# ---- what a pass cannot do without ----------------------------------------------

def work(case):
    c = case
    if c["op"] in ("route", "route_backward"):
        T, E, k, es = c["T"], c["E"], c["k"], _dt(c["dtype"]).itemsize
        if c["op"] == "route":
            return dict(bytes=T * E * es + (E * 4 if c["bias"] else 0) + T * k * 8,
                        flops=12 * T * E)
        dense = c["score"] == "softmax" and not c["renorm"]
        return dict(bytes=(T * E if dense else T * k) * es + T * k * 8 + T * E * es,
                    flops=(10 * T * E if dense else 12 * T * k))
    if c["op"] == "adamw":
        n = sum(_lengths(c))
        per = 4 + 4 + (4 if c["grad"] == "f32" else 2) + (2 if c["copy"] else 0)
        per += 16 if c["bits"] == 32 else 4 + 16 / BLOCK
        return dict(bytes=per * n, flops=16 * n)
    T, k, d, es = c["T"], c["k"], c["d"], _dt(c["dtype"]).itemsize
    kept = min(T * k, c["E"] * _capacity(c))  # the most choices that can be kept
    if c["op"] == "dispatch":
        return dict(bytes=(T + kept) * d * es + T * k * 9 + c["E"] * _capacity(c) * 4, flops=T * k)
    if c["op"] == "combine_backward":
        return dict(bytes=(T + 2 * kept) * d * es + T * k * 17, flops=3 * kept * d)
    return dict(bytes=(T + kept) * d * es + T * k * (13 if c["op"] == "combine" else 9),
                flops=2 * kept * d)


# ---- the definitions in 64 bits -------------------------------------------------

def _exact_scores(c, x):
    ok = (x > LOWEST) & (x < np.inf)
    with np.errstate(over="ignore"):
        if c["score"] == "sigmoid":
            return np.where(ok, 1.0 / (1.0 + np.exp(-np.where(ok, x, 0.0))), 0.0), ok
        top = np.max(np.where(ok, x, -np.inf), axis=1, keepdims=True)
        e = np.where(ok, np.exp(np.where(ok, x, 0.0) - np.where(np.isfinite(top), top, 0.0)), 0.0)
    return e / np.maximum(e.sum(axis=1, keepdims=True), 1e-300), ok


def _exact_route(c, s):
    x = s["logits"].double().cpu().numpy()
    T, E = x.shape
    score, ok = _exact_scores(c, x)
    two = c["group_top"] == 2 and c["top_groups"] < c["groups"]
    v = score + s["bias"].double().cpu().numpy() if s["bias"] is not None else score if two else x
    v = np.where(ok, v, -np.inf)
    rows = np.arange(T)
    if c["top_groups"] < c["groups"]:
        per = E // c["groups"]
        left = v.reshape(T, c["groups"], per).copy()
        total = np.zeros((T, c["groups"]))
        for i in range(c["group_top"]):
            best = left.max(axis=2)
            total += np.where((best == -np.inf) & (i > 0), 0.0, best)
            np.put_along_axis(left, left.argmax(axis=2)[:, :, None], -np.inf, axis=2)
        stays = np.zeros((T, c["groups"]), bool)
        for _ in range(c["top_groups"]):
            stays[rows, np.where(stays, -np.inf, total).argmax(axis=1)] = True
            total = np.where(stays, -np.inf, total)
        v = np.where(np.repeat(stays, per, axis=1), v, -np.inf)
    idx, w = np.empty((T, c["k"]), np.int32), np.zeros((T, c["k"]))
    for j in range(c["k"]):
        e = v.argmax(axis=1)
        there = v[rows, e] != -np.inf
        idx[:, j] = np.where(there, e, -1)
        w[:, j] = np.where(there, score[rows, e], 0.0)
        v[rows, e] = -np.inf
    if c["renorm"]:
        w = w / np.maximum(w.sum(axis=1, keepdims=True), 1e-300)
    return dict(expert_idx=idx, gate=w)


def _exact_route_backward(c, s):
    """Through the chosen scores: dL/dscore first, then the scores' own derivative."""
    x = s["logits"].double().cpu().numpy()
    idx, dw = s["expert_idx"].cpu().numpy(), s["dgate"].double().cpu().numpy()
    score, ok = _exact_scores(c, x)
    there = idx >= 0
    at = np.where(there, idx, 0)
    chosen = np.where(there, np.take_along_axis(score, at, axis=1), 0.0)
    dw = np.where(there, dw, 0.0)
    if c["renorm"]:
        total = np.maximum(chosen.sum(axis=1, keepdims=True), 1e-300)
        dw = (dw - (dw * chosen).sum(axis=1, keepdims=True) / total) / total
    ds = np.zeros_like(score)
    for j in range(c["k"]):
        ds[np.arange(len(ds)), at[:, j]] += np.where(there[:, j], dw[:, j], 0.0)
    if c["score"] == "sigmoid":
        return dict(dlogits=np.where(ok, ds * score * (1 - score), 0.0))
    return dict(dlogits=score * (ds - (ds * score).sum(axis=1, keepdims=True)))


def _exact_assign(c, idx):
    """By sorting: a choice's slot is its place among its expert's, in token order."""
    E, C, k = c["E"], _capacity(c), c["k"]
    e = idx.cpu().numpy().reshape(-1)
    order = np.argsort(e, kind="stable")
    arrivals = np.bincount(e, minlength=E).astype(np.int32)
    first = np.concatenate([[0], np.cumsum(arrivals)[:-1]])
    slot = np.empty(e.size, np.int32)
    slot[order] = np.arange(e.size) - np.repeat(first, arrivals)
    kept = slot < C
    tok = np.full(E * C, -1, np.int32)
    tok[e[kept].astype(np.int64) * C + slot[kept]] = np.arange(e.size)[kept] // k
    kept_cnt = np.minimum(arrivals, C)
    return dict(slot=slot.reshape(-1, k), kept=kept.reshape(-1, k).astype(np.uint8), tok_of_row=tok,
                arrivals=arrivals, kept_cnt=kept_cnt,
                n_dropped=np.array([(arrivals - kept_cnt).sum()], np.int32), xe=None)


def _exact_rows(c, s):
    """One choice after the other, in 64 bits on the GPU."""
    E, C, d = c["E"], _capacity(c), c["d"]
    kept = s["kept"].bool()
    total = torch.zeros(c["T"], d, dtype=torch.float64, device=DEV)
    dgate = torch.zeros(c["T"], c["k"], dtype=torch.float64, device=DEV)
    dye = torch.zeros(E * C, d, dtype=torch.float64, device=DEV) if "dy" in s else None
    for j in range(c["k"]):
        t = kept[:, j].nonzero()[:, 0]
        row = s["expert_idx"][t, j].long() * C + s["slot"][t, j]
        if "dy" in s:
            dgate[t, j] = (s["dy"][t].double() * s["ye"].view(E * C, d)[row].double()).sum(1)
            dye[row] = s["gate"][t, j, None].double() * s["dy"][t].double()
        else:
            x = s["dxe" if "dxe" in s else "ye"].view(E * C, d)[row].double()
            total.index_add_(0, t, x * s["gate"][t, j, None].double() if "gate" in s else x)
    if "dy" in s:
        return dict(dye=dye, dgate=dgate)
    return dict(dx=total) if "dxe" in s else dict(y=total)


def _exact_adamw(c, s):
    f = torch.float64
    t, lr = s["step"] + 1, s["lr"]
    g = s["g"].to(f)
    if c["clip"]:
        g = g * min(1.0, s["max_norm"] / float(s["norm"]))
    if c["bits"] == 8:
        m = (s["m"].float().to(f).view(-1, BLOCK) * s["m_scale"].to(f)[:, None]).view(-1)
        v = (s["v"].float().to(f).view(-1, BLOCK) * s["v_scale"].to(f)[:, None]).view(-1) ** 2
    else:
        m, v = s["m"].to(f), s["v"].to(f)
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g ** 2 * (1 - BETA2)
    step = m / (1 - BETA1 ** t) / ((v / (1 - BETA2 ** t)) ** 0.5 + EPS)
    p = s["p"].to(f) - lr * DECAY * s["p"].to(f) - lr * step
    out = dict(p=p, copy=p) if c["copy"] else dict(p=p)
    if c["bits"] == 8:
        for name, x in (("m", m), ("v", v ** 0.5)):
            x = x.view(-1, BLOCK)
            scale = x.abs().amax(1, keepdim=True) / 448.0
            q = x / scale.clamp(min=1e-300)
            if name == "v":
                q = torch.where(x > 0, q.clamp(min=2.0 ** -9), q)
            out[name] = q.float().to(torch.float8_e4m3fn).to(f).view(-1)
            out[name + "_scale"] = scale.view(-1)
        return out
    return dict(out, m=m, v=v)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(case, s)
    if case["op"] == "route_backward":
        return _exact_route_backward(case, s)
    if case["op"] == "adamw":
        return _exact_adamw(case, s)
    if case["op"] == "dispatch":
        return _exact_assign(case, s["expert_idx"])
    return _exact_rows(case, s)
