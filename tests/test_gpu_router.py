"""GPU: routing against the float64 definition: experts and places exactly, weights and the
logits' gradient within a bound.

Tolerance of a weight: an exponential (2 ulp: 4 u with u = 2^-24) of an argument whose rounding
gives |z - top| u, a sum of at most 32 chosen (or 1024 row) terms by lanes (12 roundings), a
sigmoid's quotient (2 ulp) and one more quotient: with |z - top| <= 40 under 70 u relative,
taken as 2^-17 (128 u).  A gradient is a weight's product with the difference of terms of size
sum |dw w|: 2^-17 times |w| (|dw| + sum |dw w|) and the 32-term sum's own 12 u; 2^-16 of it, and
half a step of the logits' type.
"""

import numpy as np
import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import FusedRouter
from oracle import router as RO

from _support import assert_guards_intact, empty, guarded_empty

pytestmark = pytest.mark.gpu
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126}
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def wide(t):
    return t.detach().double().cpu().numpy()


def rows_of(a, dtype, pad=0, shift=0):
    r, c = a.shape
    t = guarded_empty(r * (c + pad), dtype, shift).view(r, c + pad)
    t.fill_(7.0)
    t = t[:, :c]
    t.copy_(torch.from_numpy(a.astype(np.float32)))
    return t


def check(z, bias, k, score="softmax", groups=1, top=1, group_score="max", renorm=True, scale=1.0, dtype=torch.float32,
          pad=0, shift=0, seed=3):
    tokens, experts = z.shape
    logits = rows_of(z, dtype, pad, shift)
    zz = wide(logits)
    b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda()
    bb = None if bias is None else wide(b)
    router = FusedRouter(tokens, experts, k, score=score, groups=groups, top_groups=top, group_score=group_score,
                         renormalise=renorm, scale=scale)
    out = [empty(tokens * k).view(tokens, k)] + [empty(tokens * k, torch.int32).view(tokens, k) for _ in range(2)]
    starts = empty(experts + 1, torch.int32)
    router.route(logits, b, weights=out[0], ids=out[1], slots=out[2], starts=starts)
    scale = float(np.float32(scale))
    w, ids, slots, want_starts = RO.route(zz, bb, k, score, groups, top, group_score, renorm, scale)
    assert np.array_equal(out[1].cpu().numpy(), ids)
    assert np.array_equal(starts.cpu().numpy(), want_starts)
    assert np.array_equal(out[2].cpu().numpy(), slots)
    assert (np.abs(wide(out[0]) - w) <= 2.0 ** -17 * w + 2.0 ** -126).all()
    dw = np.random.default_rng(seed).normal(size=(tokens, k)).astype(np.float32)
    dlogits = rows_of(np.zeros(z.shape), dtype, pad, shift)
    router.backward(torch.from_numpy(dw).cuda(), logits, out[1], dlogits=dlogits)
    want = RO.backward(dw.astype(np.float64), zz, ids, score, renorm, scale)
    # |w| (|dw| + sum |dw w|) per chosen entry, p sum |dw w| elsewhere
    load = (np.abs(dw) * w).sum(1, keepdims=True)
    size = np.zeros(z.shape)
    for t in range(tokens):
        live = ids[t] >= 0
        if score == "softmax" and not renorm:
            size[t] = RO.scores(zz[t], score) * load[t]
        size[t, ids[t][live]] += w[t][live] * (np.abs(dw[t][live]) + load[t] / scale)
    err = np.abs(wide(dlogits) - want)
    bound = 2.0 ** -16 * size + HALF[dtype] * (np.abs(want) + 2.0 ** -16 * size) + TINY[dtype]
    assert (err <= bound).all(), (float((err - bound).max()), float(err.max()))
    assert_guards_intact()
    return ids


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,experts,k", [(1, 1, 1), (1, 4, 4), (7, 8, 2), (32, 33, 5), (33, 64, 6), (70, 60, 8), (90, 128, 8),
                                              (50, 256, 8), (40, 384, 16), (20, 512, 32), (9, 1000, 7), (5, 1024, 32)])
def test_without_a_bias(tokens, experts, k, dtype):
    rng = np.random.default_rng(tokens + experts)
    z = rng.normal(0, 2, (tokens, experts))
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            check(z, None, k, score, renorm=renorm, dtype=dtype, scale=2.5 if renorm else 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("experts,groups,top,k", [(64, 8, 3, 6), (256, 8, 4, 8), (96, 32, 5, 9), (40, 4, 4, 8), (60, 5, 2, 7),
                                                 (12, 12, 3, 3), (1024, 16, 2, 32), (480, 20, 4, 8), (289, 17, 8, 3)])
def test_groups_and_biases(experts, groups, top, k, group_score, score):
    rng = np.random.default_rng(experts + groups)
    z = rng.normal(0, 1.5, (60, experts))
    steps = 0.001 * rng.integers(-30, 31, experts)
    for bias in (None, np.zeros(experts), steps, rng.normal(0, 0.3, experts), 4.0 + steps):
        for dtype in (torch.float32, torch.bfloat16):
            check(z, bias, k, score, groups, top, group_score, dtype=dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("experts,pad,shift", [(32, 1, 0), (64, 8, 0), (128, 0, 1), (256, 3, 0), (256, 8, 8), (100, 4, 2)])
def test_strides_and_places_off_the_grid(experts, pad, shift, dtype):
    z = np.random.default_rng(experts).normal(0, 2, (37, experts))
    check(z, None, 4, "softmax", renorm=False, dtype=dtype, pad=pad, shift=shift)
    check(z, np.linspace(-0.1, 0.1, experts), 4, "sigmoid", dtype=dtype, pad=pad, shift=shift)


def test_equal_scores_go_to_the_lowest():
    z = np.zeros((5, 64))
    assert (check(z, None, 4) == np.arange(4)).all()
    assert (check(z, np.full(64, 0.25), 4, "sigmoid") == np.arange(4)).all()
    assert (check(z, None, 4, groups=8, top=2, group_score="top2") == np.arange(4)).all()
    assert (check(z, np.full(64, 0.25), 10, groups=8, top=2, group_score="top2") == np.arange(10)).all()
    z[:, 1::2] = -0.0
    assert (check(z, None, 4, "sigmoid") == np.arange(4)).all()
    few = np.random.default_rng(0).integers(-2, 3, (200, 96)).astype(float)    # many ties
    for score in ("softmax", "sigmoid"):
        check(few, None, 8, score)
        check(few, 0.5 * np.random.default_rng(1).integers(0, 2, 96), 8, score, 8, 3, "top2")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top,group_score", [(1, 1, "max"), (8, 3, "max"), (8, 3, "top2")])
def test_keys_closer_than_float32_tells(score, groups, top, group_score):
    """Biases that make one row's keys equal but for their rounding: the order is the 64-bit one."""
    rng = np.random.default_rng(8)
    for seed in range(6):
        z = rng.normal(0, 1, (20, 64)).astype(np.float32)
        s = RO.scores(z[0].astype(np.float64), score)
        bias = (0.75 - s).astype(np.float32)
        check(z, bias, 8, score, groups, top, group_score)


def test_logits_past_where_scores_differ():
    rng = np.random.default_rng(4)
    z = rng.normal(0, 1, (30, 64)) * np.repeat([1e-6, 1.0, 30.0, 3e4, 1e30], 6)[:, None]
    for score in ("softmax", "sigmoid"):
        check(z, None, 6, score)
    low = -200 + rng.normal(0, 3, (9, 64))          # sigmoids below float32's range: their ratios are not
    check(low, None, 6, "sigmoid")
    check(np.vstack([low, 200 + low]), None, 6, "softmax", renorm=False)
    for dtype in DTYPES:
        z = rng.normal(0, 1, (9, 64))
        z[:, 5:] = float(torch.finfo(dtype).min)
        check(z, None, 8, "softmax", dtype=dtype)


@pytest.mark.parametrize("bias", [None, "steps"])
@pytest.mark.parametrize("groups,top", [(1, 1), (4, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_experts_that_are_not_there(score, groups, top, bias):
    rng = np.random.default_rng(6)
    z = rng.normal(0, 1, (50, 32))
    z[rng.random(z.shape) < 0.7] = -np.inf
    z[10] = -np.inf                                 # a padded token
    z[11, 1:] = -np.inf
    z[-5:] = -np.inf
    b = None if bias is None else 0.01 * rng.integers(-9, 10, 32)
    if b is not None:
        b[3] = -np.inf
    for renorm in (True, False):
        ids = check(z, b, 6, score, groups, top, "top2", renorm)
        assert (ids[10] == -1).all() and (ids[-5:] == -1).all() and (ids == -1).sum() > 7 * 6
    check(np.full((40, 32), -np.inf), b, 6, score, groups, top, "max")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_numbers_that_are_none(score):
    z = torch.randn(12, 48, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7))
    z[3, 40] = float("nan")
    z[4, :] = float("nan")
    z[5, 7] = float("inf")
    bias = 0.001 * torch.arange(48, device="cuda") + 1
    bias[9] = float("nan")                          # expert 9 is taken by none
    router = FusedRouter(12, 48, 4, score=score, groups=4, top_groups=2, group_score="top2", renormalise=False)
    w, ids, slots, starts = router.route(z, bias)
    w, ids = w.cpu(), ids.cpu()
    nan = [3, 4] + ([5] if score == "softmax" else [])
    assert w[nan].isnan().all() and w[[t for t in range(12) if t not in nan]].isfinite().all()
    assert (ids[4] == -1).all() and 40 not in ids[3] and not (ids == 9).any()
    # the row with an infinite logit: by its logits under softmax, by scores and bias (whose groups may be others) else
    zz = wide(z[5])
    zz[9] = -np.inf
    if score == "softmax":
        infinite = RO.choose(zz, None, 4, "sigmoid", 4, 2, "max")
    else:
        infinite = RO.choose(zz, np.nan_to_num(wide(bias), nan=-np.inf), 4, "sigmoid", 4, 2, "top2")
    assert ids[5].tolist() == infinite and (score == "sigmoid" or ids[5, 0] == 7)
    assert (ids[[t for t in range(12) if t != 4]] >= 0).all()
    assert int(starts[-1]) == 11 * 4
    d = router.backward(torch.ones(12, 4, device="cuda"), z, ids.cuda())
    rest = [t for t in range(12) if t not in (3, 4, 5)]
    assert d[rest].isfinite().all() and (score == "sigmoid" or d[3].isnan().any())


@pytest.mark.parametrize("tokens,experts,k", [(1000, 16, 2), (5000, 256, 8), (20_001, 64, 6), (3000, 1024, 32), (33, 8, 8), (40_000, 5, 1)])
def test_places_of_many_tokens(tokens, experts, k):
    """Places by a stable sort; the experts of a few rows by the definition."""
    g = torch.Generator(device="cuda").manual_seed(tokens)
    z = torch.randn(tokens, experts, device="cuda", generator=g)
    z[:, 0] += 2
    z[torch.rand(tokens, device="cuda", generator=g) < 0.1] = -np.inf
    router = FusedRouter(tokens, experts, k)
    w, ids, slots, starts = router.route(z)
    for t in range(0, tokens, max(1, tokens // 40)):
        c = RO.choose(wide(z[t]), None, k, "softmax")
        assert ids[t].tolist() == c + [-1] * (k - len(c))
    flat = torch.where(ids < 0, experts, ids).flatten().cpu().long()
    order = torch.sort(flat, stable=True).indices
    want = torch.empty_like(order)
    want[order] = torch.arange(order.numel())
    want[flat == experts] = -1
    assert torch.equal(slots.flatten().cpu().long(), want)
    counts = torch.bincount(flat, minlength=experts + 1)[:experts]
    assert torch.equal(starts.cpu().long(), torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]))
    assert torch.equal(router.route(z)[2], slots)   # and again


def test_no_tokens_and_fewer_than_the_plan():
    router = FusedRouter(100, 16, 2)
    z = torch.randn(100, 16, device="cuda")
    w, ids, slots, starts = router.route(z[:0])
    assert w.shape == (0, 2) and not starts.any()
    assert router.backward(w, z[:0], ids).shape == (0, 16)
    whole, part = router.route(z), router.route(z[:50])
    assert torch.equal(whole[1][:50], part[1]) and int(part[3][-1]) == 100
    from adamw_optimizer_step_tensor_gb300 import AdamWError
    with pytest.raises(AdamWError, match="101 tokens"):
        router.route(torch.randn(101, 16, device="cuda"))


def test_gradient_by_differences():
    z = np.random.default_rng(2).normal(0, 1, (3, 16))
    dw = np.random.default_rng(5).normal(size=(3, 4)).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            router = FusedRouter(3, 16, 4, score=score, renormalise=renorm, scale=1.5)
            zt = torch.from_numpy(z.astype(np.float32)).cuda()
            w, ids, _, _ = router.route(zt)
            got = wide(router.backward(torch.from_numpy(dw).cuda(), zt, ids))
            zz, chosen, h = wide(zt), ids.cpu().numpy(), 1e-6
            loss = lambda a: sum((RO.weights(a[t], chosen[t], score, renorm, 1.5) * dw[t]).sum() for t in range(3))  # noqa: E731
            want = np.zeros_like(zz)
            for i in np.ndindex(zz.shape):
                up, down = zz.copy(), zz.copy()
                up[i] += h
                down[i] -= h
                want[i] = (loss(up) - loss(down)) / (2 * h)
            assert np.abs(got - want).max() < 1e-6   # differences: 1e-9; float32: 2^-17 of terms below 0.1


def test_gradient_in_place_and_ids_out_of_range():
    z = torch.randn(50, 64, device="cuda")
    for renorm in (True, False):
        router = FusedRouter(50, 64, 4, renormalise=renorm)
        w, ids, _, _ = router.route(z)
        dw = torch.randn(50, 4, device="cuda")
        want = router.backward(dw, z, ids)
        own = z.clone()
        assert torch.equal(router.backward(dw, own, ids, dlogits=own), want)
        bad = ids.clone()
        bad[::2] = torch.tensor([64, -1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
        got = router.backward(dw, z, bad)
        assert torch.equal(got[1::2], want[1::2]) and not got[::2].any()


def test_balance():
    starts = torch.tensor([0, 10, 13, 13, 16], dtype=torch.int32, device="cuda")
    bias = torch.tensor([0.5, 0.0, -0.25, 1.0], device="cuda")
    router = FusedRouter(8, 4, 2)
    router.balance(bias, starts, 0.125)
    assert bias.tolist() == [0.375, 0.125, -0.125, 1.125]
    router.balance(bias, torch.tensor([0, 4, 8, 12, 16], dtype=torch.int32, device="cuda"), 0.125)
    assert bias.tolist() == [0.375, 0.125, -0.125, 1.125]          # all at the mean
    far = torch.tensor([0, 2 ** 30, 2 ** 31 - 3, 2 ** 31 - 2, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    router.balance(bias, far, 1.0)
    assert bias.tolist() == [-0.625, -0.875, 0.875, 2.125]
    # a load that is off is pulled towards the mean
    z = torch.randn(4096, 16, device="cuda") + torch.linspace(-1, 1, 16, device="cuda")
    router, b = FusedRouter(4096, 16, 2, score="sigmoid"), torch.zeros(16, device="cuda")
    first = router.route(z, b)[3].diff().float().std()
    for _ in range(60):
        router.balance(b, router.route(z, b)[3], 0.01)
    assert router.route(z, b)[3].diff().float().std() < 0.5 * first


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,top,k", [(64, 8, 3, 6), (256, 8, 4, 8), (60, 5, 2, 7), (1000, 8, 2, 9), (16, 1, 1, 3)])
def test_a_bias_that_is_infinite(experts, groups, top, k, score):
    rng = np.random.default_rng(experts)
    z, bias = rng.normal(0, 1, (50, experts)), 0.01 * rng.integers(-5, 6, experts)
    bias[3] = bias[7] = np.inf
    bias[5] = -np.inf
    for group_score in ("max", "top2"):
        ids = check(z, bias, k, score, groups, top, group_score)
        assert (ids == 3).any(1).all() and (ids == 7).any(1).all() and not (ids == 5).any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("experts,k", [(3, 3), (32, 8), (48, 9), (64, 17), (120, 5), (200, 8), (256, 17), (300, 6), (512, 20), (513, 2)])
def test_teams_of_every_size(experts, k, dtype):
    rng = np.random.default_rng(experts * k)
    z = rng.normal(0, 1.5, (75, experts))
    z[5] = -np.inf
    bias = 0.001 * rng.integers(-30, 31, experts)
    for b, score in ((None, "softmax"), (bias, "sigmoid"), (bias, "softmax")):
        check(z, b, k, score, dtype=dtype)
    z[10] = np.sort(z[10])                      # a lane holds all that is chosen
    check(z, None, k, "sigmoid", renorm=False, dtype=dtype)
