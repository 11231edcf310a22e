"""moe_adamw_step against the formula in 64 bits (tests/routed_ref.py).

Tolerances, u = 2^-24.  m: two products and a sum of fp32 values, 4 u of the terms' magnitudes
(clip coefficient included).  v: the same with a square, 6 u.  The step lr m^/(sqrt v^ + eps):
m's and half of v's error, sqrt.approx 2 u, the quotient 4 u, the scalars 3 u: 20 u of the step's
size computed from the magnitudes; p adds 2 u |p|.  bf16 copies: 2^-8.  8-bit codes: the nearest
e4m3 value, 2^-4 relative or half the smallest code (2^-10) of the scale, with 8 u for the fp32
value itself and 2 u for the scale."""
import math

import pytest
import torch

import routed_ref as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
LENS = [0, 1, 3, 255, 256, 257, 1000, 2047, 2048, 2049, 4096 + 17, 70001]
HYPER = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module")
def moe(cuda_device):
    import sparse_mixture_experts_fwd_b200 as m
    return m


def quantize(x):
    """e4m3 codes and scales of 256-element blocks (CPU)."""
    n = x.numel()
    blocks = -(-n // 256)
    pad = torch.zeros(blocks * 256)
    pad[:n] = x
    pad = pad.view(blocks, 256)
    scale = pad.abs().amax(1) / 448.0
    q = pad / torch.where(scale == 0, 1.0, scale)[:, None]
    return q.view(-1)[:n].to(torch.float8_e4m3fn), scale


def make(lens, bits, grad_dtype, seed=0, copies=False):
    g = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(lens):
        s = 10.0 ** (i % 4)
        p = 0.02 * torch.randn(n, generator=g)
        gr = (1e-4 * s * torch.randn(n, generator=g)).to(grad_dtype)
        m = 2e-5 * s * torch.randn(n, generator=g)
        v = (1e-4 * s * torch.randn(n, generator=g)).square()
        t = dict(p=p, g=gr, m=m, v=v)
        if bits == 8:
            t["m"], t["ms"] = quantize(m)
            t["v"], t["vs"] = quantize(v.sqrt())
        if copies:
            t["copy"] = torch.zeros(n, dtype=torch.bfloat16)
        out.append(t)
    return out


def guarded(t):
    """A device copy with a canary behind it (16-byte aligned)."""
    raw = torch.full((t.numel() * t.element_size() + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    view = raw[:t.numel() * t.element_size()].view(t.dtype) if t.numel() else \
        torch.empty(0, dtype=t.dtype, device="cuda")
    view.copy_(t)
    return view, raw


def on_device(moe, ts, bits):
    D, raws = [], []
    for t in ts:
        d = {}
        for n, x in t.items():
            d[n], raw = guarded(x)
            raws.append((raw, x.numel() * x.element_size()))
        D.append(d)
    col = lambda n: [d[n] for d in D]  # noqa: E731
    kw = dict(exp_avg_scale=col("ms"), exp_avg_sq_scale=col("vs")) if bits == 8 else {}
    if "copy" in D[0]:
        kw["bf16_copies"] = col("copy")
    return D, moe.adamw_tensors(col("p"), col("g"), col("m"), col("v"), **kw), raws


def check(before, D, raws, bits, step, coef=1.0, hyper=HYPER):
    torch.cuda.synchronize()
    lr, (b1, b2), eps, wd = hyper["lr"], hyper["betas"], hyper["eps"], hyper["weight_decay"]
    for raw, n in raws:
        assert bool((raw[n:] == 0x5A).all()), "wrote behind a tensor"
    for t, d in zip(before, D):
        if t["p"].numel() == 0:
            continue
        g = t["g"].double()
        if bits == 8:
            m0 = ref.dequantize(t["m"], t["ms"])
            v0 = ref.dequantize(t["v"], t["vs"]).square()
        else:
            m0, v0 = t["m"].double(), t["v"].double()
        p, m, v = ref.adamw(t["p"], g, m0, v0, step=step, coef=coef, **hyper)
        msize = b1 * m0.abs() + (1 - b1) * (g * coef).abs()
        stepsize = lr * msize / (1 - b1 ** step) / ((v / (1 - b2 ** step)).sqrt() + eps)
        err = (d["p"].cpu().double() - p).abs()
        assert bool((err <= 2 * U * t["p"].abs() + 24 * U * stepsize + U * p.abs()).all()), float(err.max())
        if bits == 32:
            assert bool(((d["m"].cpu().double() - m).abs() <= 4 * U * msize + 1e-44).all())
            assert bool(((d["v"].cpu().double() - v).abs() <= 6 * U * v + 1e-44).all())
        else:
            for name, x, s in (("m", m, "ms"), ("v", v.sqrt(), "vs")):
                n = x.numel()
                blocks = -(-n // 256)
                pad = torch.zeros(blocks * 256, dtype=torch.float64)
                pad[:n] = x.abs()
                scale = pad.view(blocks, 256).amax(1) / 448
                got_scale = d[s].cpu().double()
                assert bool(((got_scale - scale).abs() <= 16 * U * scale + 1e-44).all())
                got = ref.dequantize(d[name].cpu(), d[s].cpu())
                one = got_scale.repeat_interleave(256)[:n]
                bound = 2.0 ** -4 * x.abs() + 2.0 ** -10 * one + 32 * U * (x.abs() + msize)
                if name == "v":  # what is above 0 is never stored as 0
                    bound = torch.where((x > 0) & (x < 2.0 ** -9 * one), 2.0 ** -9 * one, bound)
                    assert bool((got[x > 0] > 0).all())
                assert bool(((got - x).abs() <= bound).all()), name
        if "copy" in d:
            assert torch.equal(d["copy"].cpu(), d["p"].cpu().bfloat16())


@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16], ids=["g32", "g16"])
@pytest.mark.parametrize("bits", [32, 8])
def test_step_on_many_lengths(moe, bits, grad_dtype):
    before = make(LENS, bits, grad_dtype, seed=bits, copies=True)
    D, ts, raws = on_device(moe, before, bits)
    moe.adamw_step(ts, step=3, **HYPER)
    check(before, D, raws, bits, 3)
    # a second step from what the first one left
    now = [{n: x.cpu().clone() for n, x in d.items()} for d in D]
    moe.adamw_step(ts, step=4, **HYPER)
    check(now, D, raws, bits, 4)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("n", [1, 24, 25, 32, 33, 128, 129, 384, 385, 900])
def test_tensor_counts(moe, bits, n):
    before = make([(37 * i) % 700 for i in range(n)], bits, torch.float32, seed=n)
    D, ts, raws = on_device(moe, before, bits)
    moe.adamw_step(ts, step=1, **HYPER)
    check(before, D, raws, bits, 1)


@pytest.mark.parametrize("bits", [32, 8])
def test_long_tensors_equal_their_pieces(moe, bits):
    """One call on 45 M elements (long chunks) gives the bits of calls on its pieces (short ones)."""
    n, cuts = 45_000_123, [0, 15_000_064, 30_000_128, 45_000_123]   # cuts at blocks of 256
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(3)
    p = 0.02 * torch.randn(n, generator=gen, device=dev)
    g = (1e-3 * torch.randn(n, generator=gen, device=dev)).bfloat16()
    state = moe.adamw_state([p], bits)
    whole = moe.adamw_tensors([p], [g], **state)
    q, other = p.clone(), {}
    other = moe.adamw_state([q], bits)
    parts = []
    for a, b in zip(cuts, cuts[1:]):
        cut = {k: [v[0][a // 256:-(-b // 256)] if k.endswith("scale") else v[0][a:b]]
               for k, v in other.items()}
        parts.append(moe.adamw_tensors([q[a:b]], [g[a:b]], **cut))
    for step in (1, 2):
        moe.adamw_step(whole, step=step, **HYPER)
        for ts in parts:
            moe.adamw_step(ts, step=step, **HYPER)
        assert torch.equal(p, q)
        for k in state:
            assert torch.equal(state[k][0].view(torch.uint8), other[k][0].view(torch.uint8)), k
    assert not torch.equal(p[:1000], torch.zeros(1000, device=dev))


@pytest.mark.parametrize("bits", [32, 8])
def test_clip_by_the_sparseclip_norm(moe, bits):
    before = make([5000, 777, 2048], bits, torch.float32, seed=5)
    D, ts, raws = on_device(moe, before, bits)
    out = moe.sparseclip_norm([D[0]["g"]], [D[1]["g"], D[2]["g"]], 2)
    norm = float(out[0])
    for max_norm in (0.25 * norm, 4.0 * norm):
        now = [{n: x.cpu().clone() for n, x in d.items()} for d in D]
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        moe.adamw_step(ts, step=2, norm=out, max_norm=max_norm, status=st, **HYPER)
        check(now, D, raws, bits, 2, coef=min(1.0, max_norm / norm))
        assert int(st) == 0


@pytest.mark.parametrize("bits", [32, 8])
def test_unusable_norm_or_step_writes_nothing(moe, bits):
    before = make([3000, 5], bits, torch.float32, seed=6, copies=True)
    D, ts, raws = on_device(moe, before, bits)
    dev = "cuda"
    cases = [dict(norm=torch.tensor([v], dtype=torch.float64, device=dev), max_norm=1.0)
             for v in (math.nan, math.inf, -math.inf)]
    cases += [dict(step_lr=torch.tensor(v, dtype=torch.float64, device=dev))
              for v in ((0.0, 1e-3), (math.nan, 1e-3), (2.0, math.inf))]
    for kw in cases:
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        moe.adamw_step(ts, step=2, status=st, **{**HYPER, **kw})
        assert int(st) == moe.STATUS_NONFINITE
        moe.adamw_step(ts, step=2, **{**HYPER, **kw})  # without a status word too
        torch.cuda.synchronize()
        for t, d in zip(before, D):
            for n in t:
                assert torch.equal(d[n].cpu().view(torch.uint8), t[n].view(torch.uint8)), n


def test_captured_step_follows_step_and_rate(moe):
    before = make([5000, 300], 32, torch.float32, seed=7)
    D, ts, raws = on_device(moe, before, 32)
    sl = torch.tensor([1.0, HYPER["lr"]], dtype=torch.float64, device="cuda")
    rest = {k: v for k, v in HYPER.items() if k != "lr"}
    moe.adamw_step(ts, step_lr=sl, **rest)  # eager once first
    check(before, D, raws, 32, 1)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s, capture_error_mode="global"):
        moe.adamw_step(ts, step_lr=sl, stream=torch.cuda.current_stream(), **rest)
    for t, lr in ((2, 1e-3), (3, 5e-4)):
        sl.copy_(torch.tensor([float(t), lr], dtype=torch.float64))
        now = [{n: x.cpu().clone() for n, x in d.items()} for d in D]
        graph.replay()
        check(now, D, raws, 32, t, hyper={**HYPER, "lr": lr})
    del graph


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_state_and_zero_gradients(moe, bits):
    n = 1000
    p = torch.randn(n, generator=torch.Generator().manual_seed(1)).cuda()
    g = torch.zeros(n, device="cuda")
    g[300:310] = 1e-3
    state = moe.adamw_state([p], bits)
    ts = moe.adamw_tensors([p], [g], **state)
    q = p.clone()
    moe.adamw_step(ts, step=1, lr=1e-2, weight_decay=0.0)
    torch.cuda.synchronize()
    moved = (p != q).cpu()
    assert moved[300:310].all() and not moved[:300].any() and not moved[310:].any()
    # the first step has the length of the rate: lr * g / (|g| + eps), eps = 1e-8 of 1e-3
    assert bool(((p - q).cpu()[300:310].abs() - 1e-2).abs().max() < 1e-2 * 2e-5 + 4 * U * 4)


def test_eight_bits_tiny_and_poisoned_blocks(moe):
    n = 1024
    p = torch.zeros(n, device="cuda")
    g = torch.zeros(n, device="cuda")
    g[:256] = 1e-33                                # below what a scale can hold: m stays 0
    g[256:512] = 1e-3
    g[600] = float("nan")
    g[800], g[801] = 1.0, 1e-9                     # the smaller second moment is not lost
    state = moe.adamw_state([p], 8)
    ts = moe.adamw_tensors([p], [g], **state)
    moe.adamw_step(ts, step=1, lr=1e-3, weight_decay=0.0)
    torch.cuda.synchronize()
    m, v = state["exp_avg"][0].cpu().float(), state["exp_avg_sq"][0].cpu().float()
    ms = state["exp_avg_scale"][0].cpu()
    assert float(m[:256].abs().max()) == 0 and float(ms[0]) == 0
    assert torch.isfinite(p[:600]).all() and torch.isnan(p[600])
    assert float(v[801]) > 0
    assert torch.isfinite(ms[[0, 1, 3]]).all() and not torch.isfinite(ms[2])
    moe.adamw_step(ts, step=2, lr=1e-3, weight_decay=0.0)
    torch.cuda.synchronize()
    assert torch.isfinite(p[:512]).all() and torch.isfinite(p[768:]).all()


def test_eight_bit_codes_are_the_formulas(moe):
    """Every operation of the moments rounded by itself (as separate fp32 operations are here), so
    that the codes and scales are bit for bit those of the formula, over two steps of 20 M
    elements: a contracted product and sum moves one code in half a million across a border."""
    n, dev = 20_000_000, "cuda"
    gen = torch.Generator(device=dev).manual_seed(5)
    p = torch.zeros(n, device=dev)
    g = (1e-3 * torch.randn(n, generator=gen, device=dev)).bfloat16()
    state = moe.adamw_state([p], 8)
    q = {k: v[0] for k, v in state.items()}
    b1, b2 = HYPER["betas"]
    ts = moe.adamw_tensors([p], [g], **state)
    norm = torch.full((1,), 3.0, dtype=torch.float64, device=dev)
    clip = torch.tensor(1.0 / 3.0, dtype=torch.float64).float().to(dev)
    m = torch.zeros(n, device=dev)
    r = torch.zeros(n, device=dev)
    for step in (1, 2, 3):
        moe.adamw_step(ts, step=step, norm=norm, max_norm=1.0, **HYPER)
        gc = g.float() * clip
        m = m * b1 + gc * (1 - b1)
        r = ((r * r) * b2 + ((1 - b2) * gc) * gc).sqrt()
        for name, x in (("exp_avg", m), ("exp_avg_sq", r)):
            blocks = x.view(-1, 256)
            scale = blocks.abs().amax(1, keepdim=True) * torch.tensor(1 / 448, device=dev)
            code = blocks / scale
            if name == "exp_avg_sq":
                code = torch.where(blocks > 0, code.clamp(min=2.0 ** -9), code)
            code = code.to(torch.float8_e4m3fn)
            assert torch.equal(q[name + "_scale"], scale.view(-1)), (name, step)
            differ = int((q[name].view(torch.uint8) != code.view(-1).view(torch.uint8)).sum())
            assert differ == 0, (name, step, differ)
            back = code.float() * scale
            m, r = (back.view(-1), r) if name == "exp_avg" else (m, back.view(-1))


def test_refusals(moe):
    f = lambda n: torch.zeros(n, device="cuda")  # noqa: E731
    p, g, m, v = f(100), f(100), f(100), f(100)
    moe.adamw_tensors([p], [g], [m], [v])
    with pytest.raises(moe.MoEError, match="overlaps"):
        moe.adamw_tensors([p, p], [g, g], [m, f(100)], [v, f(100)])
    with pytest.raises(moe.MoEError, match="overlaps"):
        moe.adamw_tensors([p], [g], [m], [m])
    with pytest.raises(moe.MoEError, match="overlaps"):
        moe.adamw_tensors([p], [p], [m], [v])
    big = f(200)
    with pytest.raises(moe.MoEError, match="overlaps"):
        moe.adamw_tensors([big[:104], big[100:]], [f(104), f(100)], [f(104), f(100)],
                          [f(104), f(100)])
    # one gradient for two parameters is only read
    moe.adamw_tensors([p, f(100)], [g, g], [m, f(100)], [v, f(100)])
    with pytest.raises(moe.MoEError, match="aligned"):
        moe.adamw_tensors([f(101)[1:]], [g], [m], [v])
    with pytest.raises(ValueError, match="elements"):
        moe.adamw_tensors([p], [f(99)], [m], [v])
    with pytest.raises(TypeError, match="exp_avg_sq"):
        moe.adamw_tensors([p], [g], [m], [v.to(torch.float8_e4m3fn)])
    with pytest.raises(ValueError, match="contiguous"):
        moe.adamw_tensors([f(200)[::2]], [g], [m], [v])
    with pytest.raises(ValueError, match="CUDA|is on"):
        moe.adamw_tensors([p], [torch.zeros(100)], [m], [v])
    ts = moe.adamw_tensors([p], [g], [m], [v])
    for kw in (dict(step=0), dict(betas=(1.0, 0.9)), dict(eps=0.0), dict(lr=math.nan),
               dict(weight_decay=-1.0),
               dict(norm=torch.ones(1, dtype=torch.float64, device="cuda"), max_norm=0.0)):
        with pytest.raises(moe.MoEError):
            moe.adamw_step(ts, **kw)
    moe.adamw_step(moe.adamw_tensors([], [], [], []))  # nothing to do


def test_router_weights_are_trained(moe):
    """One step on the router's weights from the routed layer's own gradients: logits, routing,
    combine's and routing's gradients, the SparseClip norm, the clipped AdamW step."""
    gen = torch.Generator().manual_seed(11)
    T, d, E, k, C = 120, 64, 16, 4, 60
    x = torch.randn(T, d, generator=gen).bfloat16().cuda()
    W = (torch.randn(E, d, generator=gen) / 8).cuda()
    Wr = W.bfloat16()
    ye = torch.randn(E, C, d, generator=gen).bfloat16().cuda()
    dy = torch.randn(T, d, generator=gen).bfloat16().cuda()
    cfg = moe.make_config(T, d, 64, E, k, C)
    rcfg = moe.make_route_config(T, E, k, renorm=True)
    ffn = moe.ep_ffn_config(cfg, 1)
    logits = moe.router(ffn, x, Wr)
    idx, gate = moe.route(rcfg, logits)
    a = moe.assign(cfg, idx)
    dye, dgate = moe.combine_backward(cfg, dy, ye, idx, gate, a["slot"], a["kept"])
    dlogits = moe.route_backward(rcfg, logits, idx, dgate)
    dW = (dlogits.t() @ x.float()).contiguous()
    norm = moe.sparseclip_norm([dW], [], E)
    state = moe.adamw_state([W], 32)
    ts = moe.adamw_tensors([W], [dW], bf16_copies=[Wr], **state)
    before, max_norm = W.cpu().clone(), 0.5 * float(norm[0])
    moe.adamw_step(ts, step=1, norm=norm, max_norm=max_norm, **HYPER)
    torch.cuda.synchronize()
    zero = torch.zeros_like(before)
    p, m, v = ref.adamw(before, dW.cpu(), zero, zero, step=1, coef=0.5, **HYPER)
    assert bool(((W.cpu().double() - p).abs() <= 4 * U * p.abs() + 24 * U * HYPER["lr"]).all())
    assert torch.equal(Wr, W.bfloat16())


@pytest.mark.parametrize("bits", [32, 8])
def test_elements_past_32_bits(moe, bits):
    """A tensor of more than 2^31 elements (30 and 17 GB in all): its last elements come out as
    those of a short tensor do, which sees nothing of the others."""
    n, tail, dev = 2 ** 31 + 1000, 2024, "cuda"     # the tail starts at a block of 256
    gen = torch.Generator(device=dev).manual_seed(4)
    p = torch.zeros(n, device=dev)
    g = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    p[-tail:].normal_(generator=gen)
    g[-tail:].normal_(generator=gen)
    state = moe.adamw_state([p], bits)
    q, h = p[-tail:].clone(), g[-tail:].clone()
    short = moe.adamw_state([q], bits)
    whole, part = moe.adamw_tensors([p], [g], **state), moe.adamw_tensors([q], [h], **short)
    for step in (1, 2):
        moe.adamw_step(whole, step=step, **HYPER)
        moe.adamw_step(part, step=step, **HYPER)
    assert (n - tail) % 256 == 0
    assert torch.equal(p[-tail:], q) and not bool(torch.equal(q, torch.zeros_like(q)))
    for name, v in short.items():
        assert torch.equal(state[name][0][-v[0].numel():].view(torch.uint8), v[0].view(torch.uint8)), name
    assert int(torch.count_nonzero(p[:-tail])) == 0
