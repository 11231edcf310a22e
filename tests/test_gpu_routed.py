"""Routing by scores and the row exchange for up to 16 choices a token, forward and backward,
against 64-bit statements (tests/routed_ref.py).

Tolerances.  u = 2^-24 is half a step of fp32, h = 2^-8 of bf16 (finfo.eps / 2).
 * gates: the logit difference in the exponent is off by |x - m| u <= 32 u for the inputs here,
   expf by 4 u, a sum of at most 256 terms (8 per lane, 5 shuffles) by 13 u, a division and two
   products by 3 u, and for renormalised sigmoids two such quotients: under 128 u relative.
 * dlogits: a product of up to three such factors with a difference a - dot, where dot (16 terms)
   is off by its terms' magnitudes: 512 u of (|a| + sum |a_i s_i|) s.  bf16: plus h of the value.
 * gathered rows: k terms in order, k u of the sum of magnitudes, plus h (bf16) or u (fp32) of
   the result.  dgate: a row of d products: (d / 32 + 16) u of the sum of magnitudes.
"""
import math

import pytest
import torch

import routed_ref as ref

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8
DTYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module")
def moe(cuda_device):
    import sparse_mixture_experts_fwd_b200 as m
    return m


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def check_route(moe, x, k, bias=None, want_status=0, **kw):
    """Choices equal, gates within 128 u; canaries behind the outputs untouched."""
    T, E = x.shape
    dev = "cuda"
    names = dict(groups="num_groups")
    cfg = moe.make_route_config(T, E, k, dtype=x.dtype,
                                **{names.get(n, n): v for n, v in kw.items()})
    idx = torch.full((T + 1, k), -77, dtype=torch.int32, device=dev)
    gate = torch.full((T + 1, k), -77.0, device=dev)
    st = status_word()
    moe.route(cfg, x.to(dev), None if bias is None else bias.to(dev), expert_idx=idx[:T],
              gate=gate[:T], status=st)
    ri, rw = ref.route(x, k, bias=bias, **kw)
    assert int(st) == want_status
    assert bool((idx[T] == -77).all()) and bool((gate[T] == -77).all())
    assert torch.equal(idx[:T].cpu(), ri)
    err = (gate[:T].cpu().double() - rw).abs()
    assert bool((err <= 128 * U * rw.abs() + 1e-37).all()), float(err.max())
    return idx[:T], gate[:T]


SHAPES = [
    # T, E, k, groups, top_groups, group_top
    (1, 1, 1, 1, 1, 1), (3, 2, 2, 1, 1, 1), (17, 8, 3, 1, 1, 1), (65, 60, 6, 1, 1, 1),
    (33, 64, 8, 8, 3, 2), (129, 256, 8, 8, 4, 2), (40, 256, 16, 1, 1, 1), (50, 255, 5, 5, 2, 2),
    (41, 240, 7, 15, 4, 1), (37, 100, 16, 4, 2, 2), (29, 96, 4, 32, 9, 2), (31, 252, 9, 9, 3, 2),
    (23, 37, 2, 1, 1, 1), (1200, 128, 4, 2, 1, 1), (19, 12, 4, 3, 2, 1), (64, 129, 16, 3, 3, 2),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=[str(s) for s in SHAPES])
def test_route_shapes(moe, shape, dtype):
    T, E, k, G, tg, gt = shape
    g = torch.Generator().manual_seed(T * 1000 + E)
    x = (1.5 * torch.randn(T, E, generator=g)).to(dtype)
    b = 0.1 * torch.randn(E, generator=g)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            for bias in (None, b):
                check_route(moe, x, k, bias, score=score, renorm=renorm, groups=G, top_groups=tg,
                            group_top=gt, scale=2.5 if renorm else 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_equal_candidates(moe, score):
    """All logits equal: the lowest experts of the lowest groups, in order."""
    x = torch.full((5, 64), 0.75)
    b = torch.full((64,), 0.01)
    for bias in (None, b):
        idx, _ = check_route(moe, x, 6, bias, score=score)
        assert idx[0].tolist() == [0, 1, 2, 3, 4, 5]
        idx, _ = check_route(moe, x, 12, bias, score=score, groups=8, top_groups=2, group_top=2)
        assert idx[0].tolist() == list(range(12))
    # zeros of both signs are equal
    z = torch.zeros(3, 16)
    z[:, ::2] = -0.0
    for dt in DTYPES:
        idx, _ = check_route(moe, z.to(dt), 4, score=score)
        assert idx[0].tolist() == [0, 1, 2, 3]


@pytest.mark.parametrize("bias_on", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_candidates_one_step_apart(moe, score, bias_on):
    """Logits whose scores fp32 cannot tell apart: neighbours in fp32 around one value, shuffled,
    the order is the exact one; the same across the border of the top groups."""
    g = torch.Generator().manual_seed(4)
    E, T = 64, 48
    base = torch.tensor([0.5, 2.0, 7.0, -3.0]).repeat(T // 4)[:, None]
    x = base.clone().expand(T, E).contiguous()
    bits = x.view(torch.int32) + torch.stack([torch.randperm(E, generator=g) for _ in range(T)]).int()
    x = bits.view(torch.float32)
    b = torch.full((E,), 0.03125) if bias_on else None
    check_route(moe, x, 7, b, score=score)
    check_route(moe, x, 5, b, score=score, groups=8, top_groups=3, group_top=2)
    check_route(moe, x, 5, b, score=score, groups=8, top_groups=3, group_top=1)
    # equal pairs at the border, with a third candidate one step above them
    y = torch.full((T, 16), -1.0)
    y[:, 3] = y[:, 9] = 1.0
    y[:, 12] = torch.nextafter(torch.tensor(1.0), torch.tensor(2.0))
    check_route(moe, y, 1, None if b is None else b[:16], score=score)
    check_route(moe, y, 2, None if b is None else b[:16], score=score)


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_twins(moe, score, dtype):
    """Every expert has a twin whose logit is one step of its type away (up, down or equal), and
    with groups every group has a twin that differs in one expert: few candidates are close, at
    every place of the order and at its borders."""
    g = torch.Generator().manual_seed(12)
    T, E = 150, 64
    base = (1.2 * torch.randn(T, E // 2, generator=g)).to(dtype)
    move = torch.randint(-1, 2, (T, E // 2), generator=g)
    it = torch.int32 if dtype == torch.float32 else torch.int16
    twin = (base.view(it) + move.to(it)).view(dtype)
    x = torch.stack([base, twin], dim=2).view(T, E).contiguous()
    groups = x.view(T, 4, 2, 8)[:, :, :1].expand(T, 4, 2, 8).clone()
    one = torch.randint(0, 8, (T, 4), generator=g)
    t, q = torch.arange(T)[:, None], torch.arange(4)[None, :]
    bumped = (groups[:, :, 1].clone().view(it).gather(2, one[:, :, None])[:, :, 0] + 1).view(dtype)
    groups[t, q, 1, one] = bumped
    y = groups.reshape(T, E)[:, torch.randperm(8, generator=g).repeat_interleave(8) * 8
                             + torch.arange(8).repeat(8)].contiguous()
    flat = torch.full((E,), 0.015625)
    for b in (None, flat):
        for k in (1, 2, 7, 16):
            check_route(moe, x, k, b, score=score)
            for gt in (1, 2):
                check_route(moe, x, min(k, 12), b, score=score, groups=8, top_groups=3, group_top=gt)
                check_route(moe, y, min(k, 12), b, score=score, groups=8, top_groups=3, group_top=gt)


@pytest.mark.parametrize("shape", [(255, 5, 2, 2), (240, 3, 2, 2), (252, 9, 9, 1), (256, 1, 1, 1)],
                         ids=str)
@pytest.mark.parametrize("top", [0.05, 0.6], ids=["flat", "peaked"])
def test_route_softmax_and_bias_make_near_sums(moe, shape, top):
    """Softmax scores whose sums with the bias come in pairs, a large part of them closer than fp32
    shows (2^-23 and below), for layers of 8 and of up to 16 logits a lane: flat rows, and rows of
    one likely expert and many unlikely ones, whose sum is most wrong.  The likely expert's
    neighbour in the order has little score and a large bias, so that the sum's error moves one of
    them and not the other."""
    E, G, tg, gt = shape
    g = torch.Generator().manual_seed(E + int(100 * top))
    T, k = 60, 8
    s = torch.rand(T, E, generator=g, dtype=torch.float64) + 0.5
    s[:, E - 1] = 0
    s = 0.9 * (1 - top) * s / s.sum(1, keepdim=True)
    b = torch.empty(E)
    n = E // 2
    b[0::2] = 0.02 * torch.rand(E - n, generator=g)
    even = b[0::2][:n].double() + s[:, 0:2 * n:2]
    b[1::2] = (even.mean(0) - s[:, 1::2].mean(0)).float()
    s[:, 1::2] = (even - b[1::2].double()).clamp(min=1e-4)        # s + b of a pair: equal
    b[0], b[E - 1] = top, 0.0
    s[:, E - 1] = s[:, 0] + b[0].double()
    b[1], s[:, 1] = -1.0, 0
    s[:, 1] = 1 - s.sum(1)                                        # never chosen; the sum is 1
    assert float(s.min()) > 0
    x = s.log().float()                                           # ... up to the logits' rounding
    check_route(moe, x, k, b, score="softmax", groups=G, top_groups=tg, group_top=gt)
    check_route(moe, x, 1, b, score="softmax", groups=G, top_groups=tg, group_top=gt)


def test_route_border_hidden_behind_equal_ones(moe):
    """Many exactly equal candidates at the last place, and one that differs from them by less
    than fp32 shows (its bias makes up for a smaller logit)."""
    E, k = 32, 4
    x = torch.full((8, E), 0.25)
    b = torch.full((E,), 0.5)
    x[:, 20] = 0.25 + 2.0 ** -20
    b[20] = 0.5 - 2.0 ** -23
    for t in range(8):
        x[t, :t] += 1.0
    check_route(moe, x, k, b, score="sigmoid")
    check_route(moe, x, k, b, score="softmax")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_every_token_open(moe, score):
    """More tokens that only fp64 can order than a block's list takes (every one of 400000)."""
    g = torch.Generator().manual_seed(3)
    E, distinct, T = 48, 40, 400_000
    x = torch.full((distinct, E), 0.5).view(torch.int32)
    x = (x + torch.stack([torch.randperm(E, generator=g) for _ in range(distinct)]).int()).view(torch.float32)
    b = torch.full((E,), 0.25)
    ri, rw = ref.route(x, 3, score=score, bias=b)
    many = x.cuda().repeat(T // distinct, 1)
    cfg = moe.make_route_config(T, E, 3, score=score)
    idx, gate = moe.route(cfg, many, b.cuda())
    assert torch.equal(idx, ri.cuda().repeat(T // distinct, 1))
    err = (gate.double() - rw.cuda().repeat(T // distinct, 1)).abs()
    assert float((err / rw.cuda().repeat(T // distinct, 1)).max()) <= 128 * U


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_masks(moe, score, dtype):
    g = torch.Generator().manual_seed(9)
    T, E, k = 40, 48, 6
    x = torch.randn(T, E, generator=g).to(dtype)
    x[3] = -math.inf                                # nothing left
    x[4] = torch.finfo(dtype).min                   # the same by the type's lowest value
    x[5, 2:] = -math.inf                            # two left of six
    x[6, 1:] = torch.finfo(torch.bfloat16).min
    x[7, 5:] = -math.inf
    x[7, 0] = 3.0e4                                 # a large logit among few
    x[8, :] = -200.0                                # scores that underflow in fp32
    x[8, 11] = -190.0
    b = 0.2 * torch.randn(E, generator=g)
    bm = b.clone()
    bm[10:20] = -math.inf
    for bias in (None, b, bm):
        for renorm in (False, True):
            idx, gate = check_route(moe, x, k, bias, score=score, renorm=renorm)
            assert idx[3].tolist() == [-1] * k == idx[4].tolist() and float(gate[3].abs().sum()) == 0
            check_route(moe, x, k, bias, score=score, renorm=renorm, groups=4, top_groups=2,
                        group_top=2)
            check_route(moe, x, 3, bias, score=score, renorm=renorm, groups=4, top_groups=1,
                        group_top=1)
    idx, _ = check_route(moe, x, k, bm, score=score)
    assert not bool(((idx >= 10) & (idx < 20)).any())


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups_with_few_left(moe, score, dtype):
    """The groups that stay hold fewer experts than k while those left out hold more: the rest of
    the choices is -1, not an expert of a group that was left out."""
    g = torch.Generator().manual_seed(21)
    T, E, per = 60, 64, 8
    x = torch.randn(T, E, generator=g)
    left = torch.randint(0, 4, (T, E // per), generator=g)      # 0 to 3 of 8 left in each group
    order = torch.rand(T, E // per, per, generator=g).argsort(2)
    x = torch.where(order.view(T, E) < left.repeat_interleave(per, 1), x, -math.inf).to(dtype)
    b = 0.1 * torch.randn(E, generator=g)
    for bias in (None, b):
        for gt in (1, 2):
            for k, tg in ((8, 1), (16, 2), (16, 3), (5, 2)):
                idx, _ = check_route(moe, x, k, bias, score=score, groups=8, top_groups=tg,
                                     group_top=gt)
                assert bool((idx == -1).any())


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
def test_route_nan_and_inf_are_masked_and_reported(moe, dtype):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(20, 24, generator=g).to(dtype)
    for t, v in ((0, math.nan), (7, math.inf)):
        y = x.clone()
        y[t, 5] = v
        idx, _ = check_route(moe, y, 4, want_status=moe.STATUS_BAD_LOGIT, score="softmax")
        assert not bool((idx[t] == 5).any())
    for v in (math.nan, math.inf):
        b = torch.zeros(24)
        b[9] = v
        idx, _ = check_route(moe, x, 4, b, want_status=moe.STATUS_BAD_LOGIT, score="sigmoid")
        assert not bool((idx == 9).any())


FEW = [
    # E, k, groups, top_groups, group_top
    (1, 1, 1, 1, 1), (5, 3, 1, 1, 1), (8, 2, 1, 1, 1), (8, 4, 4, 2, 1), (12, 3, 3, 2, 2),
    (15, 4, 5, 2, 1), (16, 16, 1, 1, 1), (16, 4, 8, 3, 2), (16, 6, 2, 1, 2), (13, 2, 13, 4, 1),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shape", FEW, ids=[str(s) for s in FEW])
def test_route_few_experts(moe, shape, score, dtype):
    """Long batches over few experts: empty and short rows, ties, a masked expert, NaN and +inf.
    403 rows are repeated to a batch, and every repetition gives the same bits."""
    E, k, G, tg, gt = shape
    n, T = 403, 33001
    g = torch.Generator().manual_seed(E * 100 + k)
    x = 1.5 * torch.randn(n, E, generator=g)
    x[1::3] = torch.round(2 * x[1::3]) / 2 + 0.125               # equal logits, none opposite
    x[2::5] = x[2::5].masked_fill(torch.rand(len(x[2::5]), E, generator=g) < 0.6, -math.inf)
    x[3::97] = torch.finfo(torch.bfloat16).min
    x[4::101] = -200.0                                           # scores that underflow in fp32
    x = x.to(dtype)
    b = 0.1 * torch.randn(E, generator=g)
    kw = dict(score=score, groups=G, top_groups=tg, group_top=gt)
    bm = b.clone()
    bm[E // 2] = -math.inf
    rows = torch.arange(T) % n

    def check(bias, renorm, status=0):
        cfg = moe.make_route_config(T, E, k, dtype=dtype, score=score, num_groups=G, top_groups=tg,
                                    group_top=gt, renorm=renorm, scale=1.5)
        st = status_word()
        idx, gate = moe.route(cfg, x[rows].cuda(), None if bias is None else bias.cuda(), status=st)
        ri, rw = ref.route(x, k, bias=bias, score=score, groups=G, top_groups=tg, group_top=gt,
                           renorm=renorm, scale=1.5)
        assert int(st) == status
        idx, gate = idx.cpu(), gate.cpu()
        assert torch.equal(idx, ri[rows])
        assert torch.equal(gate, gate[:n][rows])
        err = (gate[:n].double() - rw).abs()
        assert bool((err <= 128 * U * rw.abs() + 1e-37).all()), float(err.max())

    for renorm in (False, True):
        for bias in (None, b, bm):
            check(bias, renorm)
    x[11, E - 1], x[n - 1, 0] = math.nan, math.inf
    check(None, False, moe.STATUS_BAD_LOGIT)
    check(b, True, moe.STATUS_BAD_LOGIT)


def test_route_wide_ranges(moe):
    """Saturated sigmoids, peaked softmaxes and large biases: fp64 still decides rightly."""
    g = torch.Generator().manual_seed(2)
    x = 12.0 * torch.randn(300, 64, generator=g)
    b = torch.randn(64, generator=g)
    # without a bias the logits decide; with one, sums that fp64 rounds to the same value are
    # ties in the reference too
    for score in ("softmax", "sigmoid"):
        check_route(moe, x.clamp(-30, 30), 8, score=score)
        check_route(moe, x.clamp(-30, 30), 8, score=score, renorm=True)
        check_route(moe, x.clamp(-15, 15), 8, b, score=score)
        check_route(moe, x.clamp(-15, 15), 8, 1e4 * b, score=score)


def test_route_scores_that_saturate_are_ties(moe):
    """Where scores decide (a bias, or group values of two experts) what fp64 rounds to the same
    number is a tie; where they do not, the logits' order holds however far the scores saturate."""
    x = torch.full((3, 16), -5.0)
    x[0, 4:8] = torch.tensor([40.0, 39.0, 60.0, 50.0])     # sigmoids: all 1.0 in fp64
    x[1, 4:8] = torch.tensor([30.0, 29.0, 31.0, 30.5])     # told apart by fp64 only
    x[2, 8:12] = torch.tensor([-790.0, -780.0, -760.0, -770.0])   # sigmoids and softmax scores: 0
    x[2, :8] = -900.0
    x[2, 12:] = -800.0
    kw = dict(score="sigmoid", groups=4, top_groups=1)
    two, _ = check_route(moe, x, 4, group_top=2, **kw)
    one, _ = check_route(moe, x, 4, group_top=1, **kw)
    biased, _ = check_route(moe, x, 4, torch.full((16,), 0.125), group_top=1, **kw)
    assert two[0].tolist() == biased[0].tolist() == [4, 5, 6, 7] and one[0].tolist() == [6, 7, 4, 5]
    assert two[1].tolist() == biased[1].tolist() == one[1].tolist() == [6, 7, 4, 5]
    assert two[2].tolist() == biased[2].tolist() == [0, 1, 2, 3] and one[2].tolist() == [10, 11, 9, 8]
    x[2, 0] = 0.0                                          # the others' softmax scores underflow
    two, _ = check_route(moe, x[2:], 3, score="softmax", groups=4, top_groups=2, group_top=2)
    one, _ = check_route(moe, x[2:], 3, score="softmax", groups=4, top_groups=2, group_top=1)
    assert two[0].tolist() == [0, 1, 2] and one[0].tolist() == [0, 10, 11]


def test_route_empty_batch_and_refusals(moe):
    cfg = moe.make_route_config(0, 16, 4)
    idx, gate = moe.route(cfg, torch.empty(0, 16, device="cuda"))
    assert idx.shape == (0, 4) and gate.shape == (0, 4)
    cfg = moe.make_route_config(4, 16, 4)
    x = torch.zeros(4, 16, device="cuda")
    with pytest.raises(TypeError, match="logits"):
        moe.route(cfg, x.bfloat16())
    with pytest.raises(ValueError, match="shape"):
        moe.route(cfg, x[:3])
    with pytest.raises(ValueError, match="contiguous"):
        moe.route(cfg, torch.zeros(16, 4, device="cuda").t())
    with pytest.raises(TypeError, match="bias"):
        moe.route(cfg, x, torch.zeros(16, device="cuda", dtype=torch.float64))
    with pytest.raises(moe.MoEError, match="aligned"):
        moe.route(cfg, torch.zeros(65, device="cuda")[1:].view(4, 16))


def check_route_backward(moe, x, idx, dgate, want_status=0, **kw):
    T, E = x.shape
    k = idx.shape[1]
    cfg = moe.make_route_config(T, E, k, dtype=x.dtype, **kw)
    out = torch.full((T + 1, E), -77.0, dtype=x.dtype, device="cuda")
    st = status_word()
    moe.route_backward(cfg, x.cuda(), idx.cuda(), dgate.cuda(), dlogits=out[:T], status=st)
    assert int(st) == want_status
    assert bool((out[T] == -77).all())
    return out[:T].cpu().double()


def backward_bound(x, idx, dgate, want, **kw):
    s, _ = ref.scores(x, kw.get("score", "softmax"))
    a = (kw.get("scale", 1.0) * dgate.double()).abs()
    w = ref.gates(x.double(), idx, score=kw.get("score", "softmax"), renorm=kw.get("renorm", False))
    per = (a * w.abs()).sum(1, keepdim=True)
    if kw.get("renorm"):
        size = torch.zeros_like(s).scatter_add_(
            1, idx.clamp(min=0).long(), torch.where(idx >= 0, w.abs() * (a + per), 0.0))
    elif kw.get("score") == "sigmoid":
        size = torch.zeros_like(s).scatter_add_(
            1, idx.clamp(min=0).long(), torch.where(idx >= 0, w.abs() * a, 0.0))
    else:
        full = torch.zeros_like(s).scatter_add_(1, idx.clamp(min=0).long(),
                                                torch.where(idx >= 0, a, 0.0))
        size = s * (full + per)
    h = H if x.dtype == torch.bfloat16 else U
    # The reference's own rounding: autograd forms an entry that is exactly 0 (an expert that was
    # not chosen, renormalised) as s (ds - sum ds s) from terms of up to sum |a|, each off by a
    # few 2^-53, over at most 256 summands; 512 * 2^-53 of them covers it.
    own = 512 * 2.0 ** -53 * a.sum(1, keepdim=True)
    return 512 * U * size + h * want.abs() + own + 1e-37


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_backward(moe, score, renorm, dtype):
    for T, E, k in [(1, 1, 1), (5, 2, 2), (33, 60, 6), (130, 256, 8), (21, 255, 16), (700, 64, 5),
                    (9, 37, 3)]:
        g = torch.Generator().manual_seed(T + E)
        x = (1.5 * torch.randn(T, E, generator=g)).to(dtype)
        if T > 8:
            x[2] = -math.inf
            x[4, 1:] = torch.finfo(dtype).min
            x[5, ::2] = -math.inf
        kw = dict(score=score, renorm=renorm, scale=1.75)
        idx, _ = ref.route(x, k, **kw)
        dgate = torch.randn(T, k, generator=g)
        want = ref.route_backward(x, idx, dgate, **kw)
        got = check_route_backward(moe, x, idx, dgate, **kw)
        err = (got - want).abs()
        assert bool((err <= backward_bound(x, idx, dgate, want, **kw)).all()), float(err.max())


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_backward_against_differences(moe, score, renorm):
    """Central differences of the 64-bit weights: step 1e-5, truncation about 1e-10, and the
    fp32 kernel's own 512 u of values near 1."""
    g = torch.Generator().manual_seed(3)
    T, E, k, eps = 6, 12, 4, 1e-5
    x = torch.randn(T, E, generator=g)
    kw = dict(score=score, renorm=renorm, scale=1.25)
    idx, _ = ref.route(x, k, **kw)
    dgate = torch.randn(T, k, generator=g)
    got = check_route_backward(moe, x, idx, dgate, **kw)
    for e in range(E):
        d = torch.zeros(T, E, dtype=torch.float64)
        d[:, e] = eps
        up, down = (ref.gates(x.double() + f * d, idx, **kw) for f in (1, -1))
        diff = ((up - down) * dgate.double()).sum(1) / (2 * eps)
        assert bool(((got[:, e] - diff).abs() <= 1e-8 + 512 * U * 4).all())


def test_route_backward_repeated_and_bad_choices(moe):
    g = torch.Generator().manual_seed(5)
    T, E, k = 9, 20, 4
    x = torch.randn(T, E, generator=g)
    idx = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    idx[0] = 7                 # the same expert four times
    idx[1, 2] = -1             # not a choice
    idx[2, :2] = 3
    dgate = torch.randn(T, k, generator=g)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            kw = dict(score=score, renorm=renorm)
            want = ref.route_backward(x, idx, dgate, **kw)
            got = check_route_backward(moe, x, idx, dgate, **kw)
            assert bool(((got - want).abs() <= backward_bound(x, idx, dgate, want, **kw)).all())
    bad = idx.clone()
    bad[4, 1], bad[5, 0] = E, -5
    good = bad.clone()
    good[4, 1] = good[5, 0] = -1
    got = check_route_backward(moe, x, bad, dgate, want_status=moe.STATUS_BAD_INDEX)
    assert torch.equal(got, check_route_backward(moe, x, good, dgate))


# ---- the row exchange -------------------------------------------------------------


def choices(T, E, k, seed, share_missing=0.0):
    g = torch.Generator().manual_seed(seed)
    liking = torch.rand(T, E, generator=g) + 0.4 * torch.rand(E, generator=g)
    idx = liking.argsort(dim=1, descending=True)[:, :k].to(torch.int32).contiguous()
    if share_missing:
        idx[torch.rand(T, k, generator=g) < share_missing] = -1
    return idx


ROWS = [
    # T, E, k, C, d
    (1, 4, 3, 1, 64), (5, 128, 4, 5, 768), (37, 16, 8, 20, 128), (300, 9, 5, 100, 192),
    (64, 256, 16, 3, 64), (2000, 32, 3, 150, 64), (11, 3, 1, 4, 320), (50, 8, 2, 9, 2560),
    (400, 40, 9, 90, 64), (7, 16, 16, 0, 64), (333, 20, 16, 300, 128), (65, 12, 12, 60, 192),
    (6000, 64, 8, 800, 256), (9500, 32, 4, 1300, 64),
]


@pytest.mark.parametrize("case", ROWS, ids=[str(c) for c in ROWS])
def test_assign(moe, case):
    T, E, k, C, d = case
    idx = choices(T, E, k, T + E, 0.1)
    cfg = moe.make_config(T, d, 64, E, k, C)
    got = moe.assign(cfg, idx.cuda())
    want = ref.assign(idx, E, C)
    for name, v in want.items():
        assert torch.equal(got[name].cpu(), v), name


@pytest.mark.parametrize("T,E,k,C", [
    (128, 256, 8, 4), (1024, 9, 1, 200), (73, 16, 14, 30000), (40000, 64, 8, 4000), (4096, 256, 8, 100), (4095, 256, 8, 200), (8191, 200, 8, 300),
    (65536 + 31, 7, 1, 70000), (8200, 16, 16, 5000), (2051, 256, 16, 40), (300_000, 256, 8, 0),
    (50_001, 33, 5, 9000)])
def test_assign_many_choices(moe, T, E, k, C):
    """Long lists (several blocks, a last block of its own or merged into the one before)."""
    idx = choices(T, E, k, 1, 0.02)
    if T % 2:
        idx[T // 3:2 * T // 3] = idx[0]        # a long run of the same experts
        idx[5] = E
    got = moe.assign(moe.make_config(T, 64, 64, E, k, C), idx.cuda())
    e = idx.reshape(-1).long()
    there = (e >= 0) & (e < E)
    order = torch.argsort(torch.where(there, e, E), stable=True)
    arrivals = torch.bincount(e[there], minlength=E)
    first = torch.cat([torch.zeros(1, dtype=torch.long), arrivals.cumsum(0)[:-1]])
    slot = torch.full((T * k,), 2 ** 31 - 1)
    n = int(there.sum())
    slot[order[:n]] = torch.arange(n) - first[e[order[:n]]]
    kept = there & (slot < C)
    tok = torch.full((E * C,), -1)
    tok[(e * C + slot)[kept]] = (torch.arange(T * k) // k)[kept]
    assert torch.equal(got["slot"].cpu().view(-1).long(), slot)
    assert torch.equal(got["arrivals"].cpu().long(), arrivals)
    assert torch.equal(got["kept_cnt"].cpu().long(), arrivals.clamp(max=C))
    assert torch.equal(got["kept"].cpu().view(-1).bool(), kept)
    assert torch.equal(got["tok_of_row"].cpu().long(), tok)
    assert int(got["n_dropped"]) == int((arrivals - C).clamp(min=0).sum())


def exchange(case, dtype, seed=0):
    T, E, k, C, d = case
    g = torch.Generator().manual_seed(seed + T)
    idx = choices(T, E, k, T + E, 0.05)
    a = ref.assign(idx, E, C)
    x = torch.randn(T, d, generator=g).to(dtype)
    rows = torch.randn(E, C, d, generator=g).to(dtype)
    gate = torch.rand(T, k, generator=g)
    return idx, a["slot"], a["kept"], x, rows, gate


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("case", ROWS, ids=[str(c) for c in ROWS])
def test_row_exchange(moe, case, dtype):
    T, E, k, C, d = case
    idx, slot, kept, x, rows, gate = exchange(case, dtype)
    cfg = moe.make_config(T, d, 64, E, k, C, dtype=dtype)
    D = [t.cuda() for t in (idx, slot, kept)]
    h = half_step(dtype)
    P = 2
    # dispatch: the kept rows, canaries elsewhere
    big = torch.full((E * C + 2 * P, d), -7.0, dtype=dtype, device="cuda")
    moe.dispatch(cfg, x.cuda(), *D, xe=big[P:P + E * C].view(E, C, d))
    want = torch.full((E * C + 2 * P, d), -7.0, dtype=dtype)
    t, j, r = ref.rows_of(idx, slot, kept, C)
    want[P + r] = x[t]
    assert torch.equal(big.cpu(), want)
    # combine and dispatch's gradient
    out = torch.full((T + 1, d), -7.0, dtype=dtype, device="cuda")
    for w in (gate, None):
        if w is not None:
            moe.combine(cfg, rows.cuda(), D[0], w.cuda(), D[1], D[2], y=out[:T])
        else:
            moe.dispatch_backward(cfg, rows.cuda(), *D, dx=out[:T])
        exact = ref.gather(rows, idx, slot, kept, w)
        size = ref.gather(rows.abs(), idx, slot, kept, w)
        err = (out[:T].cpu().double() - exact).abs()
        assert bool((err <= k * U * size + h * (exact.abs() + k * U * size)).all()), float(err.max())
        assert bool((out[T] == -7).all())
    # combine's gradient
    dye = torch.full((E * C + 2 * P, d), -7.0, dtype=dtype, device="cuda")
    dgate = torch.full((T + 1, k), -7.0, device="cuda")
    moe.combine_backward(cfg, x.cuda(), rows.cuda(), D[0], gate.cuda(), D[1], D[2],
                         dye=dye[P:P + E * C].view(E, C, d), dgate=dgate[:T])
    rdye, rdg = ref.combine_backward(x, rows, idx, gate, slot, kept)
    got = dye.cpu().double()
    full = torch.full((E * C + 2 * P, d), -7.0, dtype=torch.float64)
    full[P + r] = rdye.view(-1, d)[r]
    # a product rounded to fp32, then to the type
    assert bool(((got - full).abs() <= (h + U) * full.abs()).all())
    _, mag = ref.combine_backward(x.abs(), rows.abs(), idx, gate, slot, kept)
    assert bool(((dgate[:T].cpu().double() - rdg).abs() <= (d / 32 + 16) * U * mag).all())
    assert bool((dgate[T] == -7).all())


def test_row_exchange_refusals(moe):
    case = (37, 16, 8, 20, 128)
    T, E, k, C, d = case
    idx, slot, kept, x, rows, gate = (t.cuda() for t in exchange(case, torch.bfloat16))
    cfg = moe.make_config(T, d, 64, E, k, C)
    with pytest.raises(ValueError, match="expert_idx"):
        moe.dispatch(cfg, x, idx[:, :2].contiguous(), slot, kept)
    with pytest.raises(ValueError, match="xe"):
        moe.dispatch(cfg, x, idx, slot, kept, xe=rows[:, :-1].contiguous())
    with pytest.raises(TypeError, match="kept"):
        moe.combine(cfg, rows, idx, gate, slot, kept.int())
    with pytest.raises(ValueError, match="ye"):
        moe.combine(cfg, rows[:-1], idx, gate, slot, kept)
    with pytest.raises(TypeError, match="dy"):
        moe.combine_backward(cfg, x.float(), rows, idx, gate, slot, kept)
    with pytest.raises(ValueError, match="dx"):
        moe.dispatch_backward(cfg, rows, idx, slot, kept, dx=x[:-1])
    with pytest.raises(moe.MoEError, match="k must be 1..16"):
        moe.assign(moe.make_config(4, 64, 64, 32, 17, 2),
                   torch.zeros(4, 17, dtype=torch.int32, device="cuda"))
    with pytest.raises(moe.MoEError, match="k must be 1 or 2"):
        moe.expert_ffn(cfg, rows, rows, rows, torch.zeros(E, dtype=torch.int32, device="cuda"),
                       workspace=torch.zeros(4096, dtype=torch.uint8, device="cuda"))


CHECKED = """
import sys
sys.path.insert(0, ROOT)
sys.path.insert(0, ROOT + "/tests")
import torch
import sparse_mixture_experts_fwd_b200 as moe
if moe.lib.moe_bounds_checked() != 1:
    sys.exit(3)
import routed_ref as ref
T, E, k, C, d = 50, 12, 5, 30, 64
g = torch.Generator().manual_seed(2)
idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
a = ref.assign(idx, E, C)
slot, kept = a["slot"].clone(), a["kept"].clone()
good = kept.clone()
bad = idx.clone()
for t, j, e, s in ((1, 0, E, 0), (7, 2, -1, 1), (9, 4, 3, C), (20, 1, 4, -1)):
    bad[t, j], slot[t, j] = e, s
    kept[t, j], good[t, j] = 1, 0
cfg = moe.make_config(T, d, 64, E, k, C, dtype=torch.float32)
x = torch.randn(T, d, generator=g)
rows = torch.randn(E, C, d, generator=g)
gate = torch.rand(T, k, generator=g)
st = torch.zeros(1, dtype=torch.int32, device="cuda")
dev = [v.cuda() for v in (bad, slot, kept)]
def reported():
    torch.cuda.synchronize()
    seen = int(st.item())
    st.zero_()
    return seen == moe.STATUS_BAD_INDEX
big = torch.full((E * C + 8, d), -7.0, device="cuda")
moe.dispatch(cfg, x.cuda(), *dev, xe=big[4:-4].view(E, C, d), status=st)
assert reported()
t, j, r = ref.rows_of(idx, slot, good, C)
want = torch.full((E * C + 8, d), -7.0)
want[4 + r] = x[t]
assert torch.equal(big.cpu(), want)
y = moe.combine(cfg, rows.cuda(), dev[0], gate.cuda(), dev[1], dev[2], status=st)
assert reported()
assert (y.cpu().double() - ref.gather(rows, idx, slot, good, gate)).abs().max() < 1e-5
dx = moe.dispatch_backward(cfg, rows.cuda(), *dev, status=st)
assert reported()
assert (dx.cpu().double() - ref.gather(rows, idx, slot, good)).abs().max() < 1e-5
dye, dg = moe.combine_backward(cfg, x.cuda(), rows.cuda(), dev[0], gate.cuda(), dev[1], dev[2], status=st)
assert reported()
rdye, rdg = ref.combine_backward(x, rows, idx, gate, slot, good)
assert (dye.cpu().double() - rdye).abs().max() < 1e-5
assert (dg.cpu().double() - rdg).abs().max() < 1e-4
print("CHECKED_OK")
"""


def test_bounds_checked_build_skips_bad_choices(cuda_device):
    """libmoe_b200_checked.so, in a process of its own that stops unless that build is loaded:
    planted indices and slots outside the buffer are tested before a row is touched."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", f"ROOT = {root!r}\n" + CHECKED], capture_output=True,
                       text=True, timeout=300, env={**os.environ, "MOE_B200_CHECK_BOUNDS": "1"})
    assert r.returncode == 0 and "CHECKED_OK" in r.stdout, r.stdout + r.stderr


def test_combine_backward_in_place(moe):
    case = (37, 16, 8, 20, 128)
    T, E, k, C, d = case
    idx, slot, kept, x, rows, gate = exchange(case, torch.bfloat16, 1)
    cfg = moe.make_config(T, d, 64, E, k, C)
    args = [t.cuda() for t in (idx, gate, slot, kept)]
    ye = rows.cuda()
    dye, dg = moe.combine_backward(cfg, x.cuda(), ye.clone(), *args, dye=ye.clone())
    same, dg2 = moe.combine_backward(cfg, x.cuda(), ye, *args, dye=ye)
    assert same is ye and torch.equal(same, dye) and torch.equal(dg, dg2)


def test_combine_gradients_against_differences(moe):
    """The loss <dy, combine(ye, gate)> is linear in both: its change along one weight and along
    one row equals the gradient's entry (fp32 rows, relative 1e-4 of the terms' size)."""
    case = (9, 5, 3, 4, 64)
    T, E, k, C, d = case
    idx, slot, kept, dy, ye, gate = exchange(case, torch.float32, 2)
    cfg = moe.make_config(T, d, 64, E, k, C, dtype=torch.float32)
    i, s, kp = idx.cuda(), slot.cuda(), kept.cuda()
    dye, dgate = moe.combine_backward(cfg, dy.cuda(), ye.cuda(), i, gate.cuda(), s, kp,
                                      dye=torch.zeros_like(ye).cuda())

    def loss(y_, g_):
        y = moe.combine(cfg, y_.cuda(), i, g_.cuda(), s, kp)
        return float((y.cpu().double() * dy.double()).sum())

    base = loss(ye, gate)
    t, j, r = ref.rows_of(idx, slot, kept, C)
    for n in range(0, len(t), 3):
        g2 = gate.clone()
        g2[t[n], j[n]] += 1.0
        assert abs(loss(ye, g2) - base - float(dgate[t[n], j[n]])) < 1e-4 * d
        y2 = ye.clone()
        y2.view(-1, d)[r[n], 5] += 1.0
        assert abs(loss(y2, gate) - base - float(dye.view(-1, d)[r[n], 5])) < 1e-4 * d


def test_whole_layer_with_eight_choices(moe):
    """Router logits, scored routing, slots, dispatch, the expert FFN, combine; then the gradients
    of the weights, of the expert rows, of the logits and of the dispatched rows."""
    g = torch.Generator().manual_seed(6)
    T, d, f, E, k, C = 260, 128, 192, 32, 8, 80
    x = torch.randn(T, d, generator=g).bfloat16()
    Wr = (torch.randn(E, d, generator=g) / math.sqrt(d)).bfloat16()
    W1 = (0.05 * torch.randn(E, f, d, generator=g)).bfloat16()
    W2 = (0.05 * torch.randn(E, d, f, generator=g)).bfloat16()
    b = 0.05 * torch.randn(E, generator=g)
    cfg = moe.make_config(T, d, f, E, k, C)
    ffn = moe.ep_ffn_config(cfg, 1)
    rcfg = moe.make_route_config(T, E, k, score="sigmoid", num_groups=4, top_groups=2, group_top=2,
                                 renorm=True, scale=2.5)
    st = status_word()
    logits = moe.router(ffn, x.cuda(), Wr.cuda(), status=st)
    idx, gate = moe.route(rcfg, logits, b.cuda(), status=st)
    a = moe.assign(cfg, idx, status=st)
    xe = moe.dispatch(cfg, x.cuda(), idx, a["slot"], a["kept"], status=st)
    _, ye = moe.expert_ffn(ffn, xe, W1.cuda(), W2.cuda(), a["kept_cnt"], status=st)
    y = moe.combine(cfg, ye, idx, gate, a["slot"], a["kept"], status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    # from the same logits, one expert after the other in 64 bits with H rounded to bf16
    ri, rw = ref.route(logits.cpu(), k, score="sigmoid", groups=4, top_groups=2, group_top=2,
                       renorm=True, scale=2.5, bias=b)
    assert torch.equal(idx.cpu(), ri)
    ra = ref.assign(ri, E, C)
    want = torch.zeros(T, d, dtype=torch.float64)
    for e in range(E):
        Hx = torch.relu(x.double() @ W1[e].double().t()).bfloat16().double()
        o = (Hx @ W2[e].double().t()).bfloat16().double()
        m = (ri == e) & (ra["kept"] != 0)
        want += (rw * m).sum(1, keepdim=True) * o
    err = (y.cpu().double() - want).abs()
    assert bool((err <= 2e-2 + 1e-2 * want.abs()).all()), float(err.max())
    # backward
    dy = torch.randn(T, d, generator=g).bfloat16()
    dye, dgate = moe.combine_backward(cfg, dy.cuda(), ye, idx, gate, a["slot"], a["kept"])
    dlogits = moe.route_backward(rcfg, logits, idx, dgate)
    dx = moe.dispatch_backward(cfg, dye, idx, a["slot"], a["kept"])
    filled = torch.zeros(E * C, dtype=torch.bool)
    filled[ref.rows_of(ri, ra["slot"], ra["kept"], C)[2]] = True
    yec = torch.where(filled.view(E, C, 1), ye.cpu(), torch.zeros((), dtype=torch.bfloat16))
    rdye, rdg = ref.combine_backward(dy, yec, ri, gate.cpu(), ra["slot"], ra["kept"])
    assert bool(((dye.cpu().double() - rdye).abs() <= (H + U) * rdye.abs()).all())
    _, mag = ref.combine_backward(dy.abs(), yec.abs(), ri, gate.cpu(), ra["slot"], ra["kept"])
    assert bool(((dgate.cpu().double() - rdg).abs() <= (d / 32 + 16) * U * mag).all())
    kw = dict(score="sigmoid", renorm=True, scale=2.5)
    dg = dgate.cpu()
    want = ref.route_backward(logits.cpu(), ri, dg, **kw)
    err = (dlogits.cpu().double() - want).abs()
    assert bool((err <= backward_bound(logits.cpu(), ri, dg, want, **kw)).all())
    dyc = dye.cpu()
    want = ref.gather(dyc, ri, ra["slot"], ra["kept"])
    size = ref.gather(dyc.abs(), ri, ra["slot"], ra["kept"])
    assert bool(((dx.cpu().double() - want).abs() <= k * U * size + H * (want.abs() + k * U * size)).all())


def test_streams_and_graph(moe):
    """The chain on a side stream, and captured and replayed with new contents, gives the eager
    call's bits."""
    g = torch.Generator().manual_seed(8)
    T, d, E, k, C = 90, 64, 32, 8, 40
    cfg = moe.make_config(T, d, 64, E, k, C)
    rcfg = moe.make_route_config(T, E, k, score="sigmoid", num_groups=4, top_groups=2, group_top=2,
                                 renorm=True)
    logits = torch.randn(T, E, generator=g).cuda()
    b = (0.1 * torch.randn(E, generator=g)).cuda()
    x = torch.randn(T, d, generator=g).bfloat16().cuda()
    dy = torch.randn(T, d, generator=g).bfloat16().cuda()
    o = dict(idx=torch.empty(T, k, dtype=torch.int32, device="cuda"),
             gate=torch.empty(T, k, device="cuda"), a={},
             xe=torch.zeros(E, C, d, dtype=torch.bfloat16, device="cuda"),
             y=torch.empty(T, d, dtype=torch.bfloat16, device="cuda"),
             dye=torch.zeros(E, C, d, dtype=torch.bfloat16, device="cuda"),
             dgate=torch.empty(T, k, device="cuda"), dl=torch.empty(T, E, device="cuda"),
             dx=torch.empty(T, d, dtype=torch.bfloat16, device="cuda"))

    def chain(stream):
        kw = dict(stream=stream)
        moe.route(rcfg, logits, b, expert_idx=o["idx"], gate=o["gate"], **kw)
        moe.assign(cfg, o["idx"], out=o["a"], **kw)
        s, kp = o["a"]["slot"], o["a"]["kept"]
        moe.dispatch(cfg, x, o["idx"], s, kp, xe=o["xe"], **kw)
        moe.combine(cfg, o["xe"], o["idx"], o["gate"], s, kp, y=o["y"], **kw)
        moe.combine_backward(cfg, dy, o["xe"], o["idx"], o["gate"], s, kp, dye=o["dye"],
                             dgate=o["dgate"], **kw)
        moe.route_backward(rcfg, logits, o["idx"], o["dgate"], dlogits=o["dl"], **kw)
        moe.dispatch_backward(cfg, o["dye"], o["idx"], s, kp, dx=o["dx"], **kw)

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in (o["idx"], o["gate"], o["y"], o["dgate"], o["dl"], o["dx"],
                                    o["a"]["slot"])]

    def clear():
        for n in ("gate", "y", "dgate", "dl", "dx"):
            o[n].fill_(float("nan"))
        torch.cuda.synchronize()

    chain(None)
    eager = results()
    side = torch.cuda.Stream()
    clear()
    chain(side)
    assert all(torch.equal(p, q) for p, q in zip(eager, results()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side, capture_error_mode="global"):
        chain(side)
    clear()
    graph.replay()
    assert all(torch.equal(p, q) for p, q in zip(eager, results()))
    logits.copy_(torch.randn(T, E, generator=g))
    x.copy_(torch.randn(T, d, generator=g))
    o["xe"].zero_()
    o["dye"].zero_()
    chain(None)
    eager2 = results()
    assert not torch.equal(eager[1], eager2[1])
    clear()
    graph.replay()
    assert all(torch.equal(p, q) for p, q in zip(eager2, results()))
    del graph


def test_two_streams_at_once(moe):
    """Calls in flight on two streams share nothing."""
    g = torch.Generator().manual_seed(10)
    T, E, k = 20000, 256, 8
    rcfg = moe.make_route_config(T, E, k, score="sigmoid", num_groups=8, top_groups=4, group_top=2)
    xs = [torch.randn(T, E, generator=g).cuda() for _ in range(2)]
    b = (0.1 * torch.randn(E, generator=g)).cuda()
    alone = [moe.route(rcfg, x, b) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(4):
        for n in range(2):
            got[n].append(moe.route(rcfg, xs[n], b, stream=streams[n]))
    torch.cuda.synchronize()
    for n in range(2):
        for idx, gate in got[n]:
            assert torch.equal(idx, alone[n][0]) and torch.equal(gate, alone[n][1])


def test_route_offsets_past_32_bits(moe):
    """Rows whose element offset passes 2^31: the last tokens come out as they do alone."""
    T, E, k = 2 ** 23 + 40, 256, 1
    x = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")  # 4.3 GB
    tail = torch.randn(64, E, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    x[-64:] = tail
    cfg = moe.make_route_config(T, E, k, dtype=torch.bfloat16)
    idx, gate = moe.route(cfg, x)
    one = moe.make_route_config(64, E, k, dtype=torch.bfloat16)
    ti, tg = moe.route(one, tail.contiguous())
    assert torch.equal(idx[-64:], ti) and torch.equal(gate[-64:], tg)
    assert int(idx[:-64].abs().max()) == 0
    d = moe.route_backward(cfg, x, idx, gate)
    assert torch.equal(d[-64:], moe.route_backward(one, tail, ti, tg))


def test_row_exchange_offsets_past_32_bits(moe):
    """Expert rows behind element 2^31 (4.4 GB of rows): the last experts' rows come and go as in
    a layer of those experts alone."""
    E, C, d, T, k, last = 256, 8400, 1024, 40, 3, 4
    g = torch.Generator().manual_seed(13)
    assert (E - last) * C * d > 2 ** 31
    few = torch.stack([torch.randperm(last, generator=g)[:k] for _ in range(T)]).int()
    a = ref.assign(few, last, C)
    slot = torch.where(a["kept"] != 0, a["slot"] + (C - T * k), a["slot"]).cuda()   # at the end
    kept, few = a["kept"].cuda(), few.cuda()
    idx = few + (E - last)
    x = torch.randn(T, d, generator=g).bfloat16().cuda()
    gate = torch.rand(T, k, generator=g).cuda()
    big = moe.make_config(T, d, 64, E, k, C)
    one = moe.make_config(T, d, 64, last, k, C)
    xe = torch.zeros(E, C, d, dtype=torch.bfloat16, device="cuda")
    xs = torch.zeros(last, C, d, dtype=torch.bfloat16, device="cuda")
    moe.dispatch(big, x, idx, slot, kept, xe=xe)
    moe.dispatch(one, x, few, slot, kept, xe=xs)
    assert torch.equal(xe[-last:], xs) and int(torch.count_nonzero(xe[:-last])) == 0
    assert torch.equal(moe.combine(big, xe, idx, gate, slot, kept),
                       moe.combine(one, xs, few, gate, slot, kept))
    assert torch.equal(moe.dispatch_backward(big, xe, idx, slot, kept),
                       moe.dispatch_backward(one, xs, few, slot, kept))
    _, dg = moe.combine_backward(big, x, xe, idx, gate, slot, kept, dye=xe)
    _, ds = moe.combine_backward(one, x, xs, few, gate, slot, kept, dye=xs)
    assert torch.equal(dg, ds) and torch.equal(xe[-last:], xs)
    assert int(torch.count_nonzero(xe[:-last])) == 0


CHECKED_ROUTE = """
import math, sys
sys.path.insert(0, ROOT)
sys.path.insert(0, ROOT + "/tests")
import torch
import sparse_mixture_experts_fwd_b200 as moe
if moe.lib.moe_bounds_checked() != 1:
    sys.exit(3)
import routed_ref as ref
g = torch.Generator().manual_seed(31)
T = 24
for E, k, G, tg, gt in ((48, 6, 1, 1, 1), (48, 6, 4, 2, 2), (48, 6, 4, 2, 1), (7, 7, 1, 1, 1),
                        (255, 16, 5, 2, 2), (33, 4, 1, 1, 1), (2, 1, 1, 1, 1)):
    x = torch.randn(T, E, generator=g)
    x[torch.rand(T, E, generator=g) < 0.5] = -math.inf
    x[4::5] = -math.inf                      # nothing left
    x[5::7, 1:] = torch.finfo(torch.bfloat16).min
    x[T - 2:] = -math.inf                    # the last rows of the buffer too
    near = x.clone()                         # candidates that only fp64 can order
    near[:T // 2] = torch.where(x[:T // 2] > -1, 0.5 + 2.0 ** -20 * torch.arange(E), x[:T // 2])
    b = 0.1 * torch.randn(E, generator=g)
    bm = b.clone()
    bm[E // 3:] = -math.inf                  # masked for every token
    for dt in (torch.float32, torch.bfloat16):
        for logits in (x.to(dt), near.to(dt)):
            for bias in (None, b, bm):
                for score in ("softmax", "sigmoid"):
                    kw = dict(score=score, top_groups=tg, group_top=gt)
                    cfg = moe.make_route_config(T, E, k, num_groups=G, dtype=dt, **kw)
                    st = torch.zeros(1, dtype=torch.int32, device="cuda")
                    idx, gate = moe.route(cfg, logits.cuda(), None if bias is None else bias.cuda(),
                                          status=st)
                    ri, rw = ref.route(logits, k, bias=bias, groups=G, **kw)
                    assert int(st) == 0, (E, score, dt, int(st))
                    assert torch.equal(idx.cpu(), ri)
                    assert bool((ri == -1).any()) or k == 1
                    assert bool(((gate.cpu().double() - rw).abs() <= 2.0 ** -17 * rw + 1e-37).all())
print("CHECKED_OK")
"""


def test_route_stays_inside_its_rows(cuda_device):
    """Rows with fewer experts left than choices, in the bounds-checked build: no expert index
    outside the row is formed for a read of the logits or of the bias (the status stays 0)."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", f"ROOT = {root!r}\n" + CHECKED_ROUTE],
                       capture_output=True, text=True, timeout=300,
                       env={**os.environ, "MOE_B200_CHECK_BOUNDS": "1"})
    assert r.returncode == 0 and "CHECKED_OK" in r.stdout, r.stdout + r.stderr
