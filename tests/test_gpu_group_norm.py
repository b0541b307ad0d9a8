"""GPU: group norm with an activation against the float64 definition.

Tolerances (u = 2^-24).  The mean is off by a few u of the largest value's distance from the
first one and of itself; rstd by the spread's error: a run of n <= 64 values loses at most 2 n u
of it, joins by counts a few u: 160 u.  xhat then is off by under 200 u (1 + |xhat|) + 4 u
|mean| rstd: 2^-16 (1 + |xhat|) while |mean| rstd < 10.  The activation's slope is below 1.1 and
its fast exponential off by (|z| + 4) u: 2^-15 of (1 + |z|) covers both.  A group's or a column's
sum of n terms, over runs, threads and CTAs, is off by at most 400 u of its magnitudes (the
longest chain of additions here) plus the terms' own 2^-15: 2^-14.  16-bit outputs add half a
step.
"""

import numpy as np
import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import AdamWError, FusedGroupNorm
from oracle import group_norm as GN

from _support import assert_guards_intact, empty, guarded_empty

pytestmark = pytest.mark.gpu
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126}
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def wide(t):
    return t.detach().double().cpu().numpy()


def tensor_of(a, dtype, pad=0, shift=0, swap=False):
    """A guarded device tensor of a's values: `pad` elements behind each position's channels; samples inside
    positions with `swap`."""
    n, length, c = a.shape
    t = guarded_empty(n * length * (c + pad), dtype, shift)
    t = t.view(length, n, c + pad).transpose(0, 1) if swap else t.view(n, length, c + pad)
    t.fill_(7.0)
    t = t[:, :, :c]
    t.copy_(torch.from_numpy(a.astype(np.float32)))
    return t


def vec_of(a, dtype):
    t = empty(a.size, dtype)
    t.copy_(torch.from_numpy(a.astype(np.float32)))
    return t


def near(got, want, size, rel, dtype):
    err = np.abs(wide(got) - want)
    bound = rel * size + HALF[dtype] * (np.abs(want) + rel * size) + TINY[dtype]
    assert (err <= bound).all(), (float((err - bound).max()), float(err.max()))


def check(shape, groups, dtype=torch.float32, wdtype=torch.float32, silu=False, pad=0, shift=0, swap=False, offset=0.5, none=False):
    n, length, c = shape
    rng = np.random.default_rng(n * 7 + length * 3 + c)
    x = tensor_of(rng.normal(offset, 1.5, shape) * (1 + 0.3 * np.arange(c) / c), dtype, pad, shift, swap)
    dy = tensor_of(rng.normal(0, 1, shape), dtype, pad, shift, swap)
    w = None if none else vec_of(rng.normal(1, 0.2, c), wdtype)
    b = None if none else vec_of(rng.normal(0, 0.2, c), wdtype)
    y, dx = (tensor_of(np.zeros(shape), dtype, pad, shift, swap) for _ in range(2))
    odt = dtype if none else wdtype
    dw, db = empty(c, odt), empty(c, odt)
    mean, rstd = (empty(n * groups).view(n, groups) for _ in range(2))
    norm = FusedGroupNorm(c, groups, n, activation="silu" if silu else "none")
    norm.forward(x, w, b, y=y, mean=mean, rstd=rstd)
    norm.backward(dy, x, w, b, mean, rstd, dx=dx, dweight=dw, dbias=db)
    assert_guards_intact()
    xx, ww, bb = wide(x), None if none else wide(w), None if none else wide(b)
    want, m, r = GN.forward(xx, groups, ww, bb, silu=silu)
    span = np.abs(xx.reshape(n, length, groups, -1)).max((1, 3))
    assert (np.abs(wide(mean) - m) <= 2.0 ** -20 * span).all()
    assert (np.abs(wide(rstd) - r) <= 2.0 ** -16 * r).all()
    xhat = GN.forward(xx, groups)[0]
    wabs = 1 if none else np.abs(ww)
    z = np.abs(xhat * (1 if none else ww)) + (0 if none else np.abs(bb))
    size = wabs * (1 + np.abs(xhat)) + z
    near(y, want, size, 2.0 ** -15, dtype)
    mm, rr = wide(mean), wide(rstd)
    gx, gw, gb = GN.backward(wide(dy), xx, groups, ww, bb, mm, rr, silu)
    term = np.abs(wide(dy)) * 1.1 * (2 + z) * (1 + np.abs(xhat))      # of dz and dz xhat
    spread = lambda t: np.repeat(t.reshape(n, length, groups, -1).mean((1, 3)), c // groups, 1)[:, None, :]  # noqa: E731
    size = np.repeat(rr, c // groups, 1)[:, None, :] * (term * wabs + spread(term * wabs) * (1 + np.abs(xhat)))
    near(dx, gx, size, 2.0 ** -14, dtype)
    near(dw, gw, term.sum((0, 1)), 2.0 ** -14, odt)
    near(db, gb, term.sum((0, 1)), 2.0 ** -14, odt)
    return norm, x, w, b, y, mean, rstd


SHAPES = [((1, 1, 1), 1), ((2, 3, 4), 2), ((3, 1, 64), 8), ((1, 257, 8), 1), ((2, 100, 40), 5), ((5, 33, 96), 32), ((2, 70, 330), 30),
          ((1, 1000, 128), 4), ((3, 17, 2056), 8), ((2, 9, 5000), 10), ((300, 1, 512), 16), ((40, 2, 264), 33), ((1, 5, 20_000), 1),
          ((2, 4096, 32), 32), ((7, 64, 7), 7), ((2, 3, 600), 2)]


@pytest.mark.parametrize("dtype,wdtype", [(torch.float32, torch.float32), (torch.float16, torch.float32), (torch.float16, torch.float16),
                                          (torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16)])
@pytest.mark.parametrize("shape,groups", SHAPES)
def test_matches_the_definition(shape, groups, dtype, wdtype):
    check(shape, groups, dtype, wdtype, silu=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape,groups", SHAPES[:8])
def test_without_activation_or_weights(shape, groups, dtype):
    check(shape, groups, dtype)
    check(shape, groups, dtype, none=True, silu=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,shift,swap", [(8, 0, False), (1, 0, False), (0, 1, False), (0, 0, True), (3, 1, True), (8, 8, True)])
def test_strides(pad, shift, swap, dtype):
    check((3, 40, 96), 4, dtype, silu=True, pad=pad, shift=shift, swap=swap)
    check((1, 300, 40), 5, dtype, silu=True, pad=pad, shift=shift, swap=swap)


def test_means_far_from_zero():
    """xhat is off by 4 u |mean| rstd more: 700 / 1.5 of them are 1.2e-4."""
    x = torch.randn(2, 500, 64, dtype=torch.float64).mul(1.5).add(700).float()
    norm = FusedGroupNorm(64, 4, 2)
    y, mean, rstd = norm.forward(x.cuda())
    want, m, r = GN.forward(x.double().numpy(), 4)
    assert np.abs(wide(mean) - m).max() < 700 * 2.0 ** -22
    assert (np.abs(wide(rstd) - r) < 2.0 ** -16 * r).all()
    assert np.abs(wide(y) - want).max() < 700 / 1.5 * 2.0 ** -21 + 2.0 ** -16 * 6


def test_a_first_value_far_from_the_rest():
    """The sums' own shift is then the value that the spread is made of."""
    x = torch.randn(1, 4000, 8, generator=torch.Generator().manual_seed(0))
    x[0, 0] = 3e4
    norm = FusedGroupNorm(8, 2, 1)
    y, mean, rstd = norm.forward(x.cuda())
    want, m, r = GN.forward(x.double().numpy(), 2)
    assert (np.abs(wide(mean) - m) < 2.0 ** -20 * 3e4).all() and (np.abs(wide(rstd) - r) < 2.0 ** -16 * r).all()


def test_constant_groups_and_values_that_are_no_numbers():
    x = torch.full((2, 50, 16), 3.25, device="cuda")
    norm = FusedGroupNorm(16, 4, 2, eps=1e-5)
    y, mean, rstd = norm.forward(x)
    assert not y.any() and (mean == 3.25).all() and ((rstd - 1e5 ** 0.5).abs() < 1e-4).all()
    x.normal_()
    for bad in (float("nan"), float("inf"), float("-inf")):
        for at in ((0, 0, 0), (0, 49, 5), (1, 20, 10)):
            z = x.clone()
            z[at] = bad
            y, mean, rstd = norm.forward(z)
            hit = torch.zeros(2, 4, dtype=torch.bool, device="cuda")
            hit[at[0], at[2] // 4] = True
            assert rstd[hit].isnan().all() and rstd[~hit].isfinite().all()
            per = y.view(2, 50, 4, 4).transpose(1, 2)
            assert per[hit].isnan().all() and per[~hit].isfinite().all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_in_place(dtype):
    norm, x, w, b, y, mean, rstd = check((3, 50, 64), 8, dtype, silu=True)
    dy = torch.randn(3, 50, 64, device="cuda").to(dtype)
    want = norm.backward(dy, x, w, b, mean, rstd)
    for into in ("dy", "x"):
        t = {"dy": dy.clone(), "x": x.clone()}
        got = norm.backward(t["dy"], t["x"], w, b, mean, rstd, dx=t[into])
        assert all(torch.equal(a, c) for a, c in zip(got, want))
    z = x.clone()
    norm.forward(z, w, b, y=z)
    assert torch.equal(z, y)


def test_no_samples_and_refusals():
    norm = FusedGroupNorm(8, 2, 3)
    x = torch.randn(3, 5, 8, device="cuda")
    y, mean, rstd = norm.forward(x[:0])
    assert y.shape == (0, 5, 8) and mean.shape == (0, 2)
    dx, dw, db = norm.backward(x[:0], x[:0], None, None, mean, rstd)
    assert not dw.any() and not db.any()
    with pytest.raises(AdamWError, match="4 samples"):
        norm.forward(torch.randn(4, 5, 8, device="cuda"))
    with pytest.raises(AdamWError, match="no elements"):
        norm.forward(torch.randn(3, 0, 8, device="cuda"))
    with pytest.raises(AdamWError, match="strides"):
        norm.forward(x, y=x.as_strided((3, 5, 8), (8, 24, 1)))
    with pytest.raises(AdamWError, match="overlapping"):
        norm.forward(x, y=torch.empty(100, device="cuda").as_strided((3, 5, 8), (8, 8, 1)))


def test_gradient_by_differences():
    rng = np.random.default_rng(12)
    x, dy = rng.normal(size=(2, 6, 8)).astype(np.float32), rng.normal(size=(2, 6, 8)).astype(np.float32)
    w, b = rng.normal(1, 0.2, 8).astype(np.float32), rng.normal(0, 0.2, 8).astype(np.float32)
    put = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    norm = FusedGroupNorm(8, 2, 2, activation="silu")
    _, mean, rstd = norm.forward(put(x), put(w), put(b))
    got = norm.backward(put(dy), put(x), put(w), put(b), mean, rstd)
    args = [a.astype(np.float64) for a in (x, w, b)]
    loss = lambda x, w, b: (GN.forward(x, 2, w, b, silu=True)[0] * dy).sum()  # noqa: E731
    for i, g in enumerate(got):
        want = np.zeros_like(args[i])
        for at in np.ndindex(want.shape):
            up, down = [a.copy() for a in args], [a.copy() for a in args]
            up[i][at] += 1e-6
            down[i][at] -= 1e-6
            want[at] = (loss(*up) - loss(*down)) / 2e-6
        assert np.abs(wide(g) - want).max() < 2e-5   # differences 1e-8; float32 2^-15 of terms of a few units


@pytest.mark.parametrize("shape,groups", [((1, 60_000, 64), 4), ((40, 3000, 40), 5), ((3, 20_000, 264), 33), ((700, 90, 264), 3), ((2, 3000, 4104), 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_samples_in_many_parts(shape, groups, dtype):
    check(shape, groups, dtype, silu=True)


def test_a_wait_that_gives_up_is_reported_and_the_plan_is_fit_again():
    from adamw_optimizer_step_tensor_gb300 import _capi
    x = torch.randn(2, 100_000, 64, device="cuda")
    norm = FusedGroupNorm(64, 4, 2)
    want = norm.forward(x)
    back = norm.backward(x, x, None, None, *want[1:])
    assert norm.status() == 0
    for _ in range(3):
        _capi.adamw_group_norm_plan_set_wait_limit(norm.plan, 0)
        norm.forward(x)
        with pytest.raises(AdamWError) as e:
            norm.status()
        assert e.value.status == _capi.ETIMEOUT
        assert norm.status() == 0
        norm.backward(x, x, None, None, *want[1:])
        with pytest.raises(AdamWError):
            norm.status()
        _capi.adamw_group_norm_plan_set_wait_limit(norm.plan, 2_000_000)
        assert all(torch.equal(a, b) for a, b in zip(norm.forward(x), want))
        assert all(torch.equal(a, b) for a, b in zip(norm.backward(x, x, None, None, *want[1:]), back))
        assert norm.status() == 0


@pytest.mark.parametrize("shape,groups", [((9, 28, 16), 2), ((112, 359, 58), 2), ((1500, 20, 96), 3), ((1, 3, 40), 5), ((700, 1, 2056), 257),
                                          ((3, 600, 1032), 8), ((1, 400, 8), 8), ((2500, 1, 256), 8), ((1300, 1, 4096), 64), ((7, 1, 16), 16), ((900, 1, 96), 12), ((5, 77, 65536), 64), ((1, 9, 129 * 400), 400)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_cuts_of_every_kind(shape, groups, dtype):
    check(shape, groups, dtype, silu=True)


def test_positions_at_the_limit():
    """2^31 - 1 positions, elements past 2^31 and 2^32.  A thread merges its 2^31 / (304 256) / 8 =
    3450 runs one after another, each merge off by 3 u of a run's mean, below 6 for normal numbers:
    4e-3 at most of a mean, a spread and, relative to 1, of the means of the gradient."""
    n, length = 2, 2 ** 31 - 1
    x = torch.empty(n, length, 1, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(5))
    norm = FusedGroupNorm(1, 1, n)
    y, mean, rstd = norm.forward(x)
    step = 1 << 27
    for s in range(n):
        sums = torch.zeros(2, dtype=torch.float64, device="cuda")
        for at in range(0, length, step):
            part = x[s, at:at + step].double()
            sums += torch.stack([part.sum(), (part * part).sum()])
        m = sums[0] / length
        r = 1 / torch.sqrt(sums[1] / length - m * m + 1e-5)
        assert abs(mean[s, 0] - m) <= 4e-3 and abs(rstd[s, 0] - r) <= 4e-3 * r
        for at in (0, 1 << 30, length - 4096):
            want = (x[s, at:at + 4096].double() - m) * r
            assert ((y[s, at:at + 4096].double() - want).abs() <= 2.0 ** -8 * want.abs() + 4e-3 * (1 + want.abs())).all()
    # of dy = 1 nothing is left: one mean off by 4e-3, the other, with the forward pass's, by 8e-3 of xhat < 6.3
    dx, _, _ = norm.backward(torch.ones((), dtype=torch.bfloat16, device="cuda").expand(n, length, 1).contiguous(), x, None, None, mean, rstd, dx=y)
    assert dx[:, :: 1 << 20].abs().max() <= 6e-2 and dx[:, -4096:].abs().max() <= 6e-2
    assert norm.status() == 0


def test_strides_past_32_bits():
    """Every position lies more than 2^31 elements behind the one before."""
    n, length, c = 2, 3, 64
    pace = 2 ** 31 + 64
    room = torch.empty(n * length * pace, dtype=torch.bfloat16, device="cuda")
    x = room.as_strided((n, length, c), (length * pace, pace, 1))
    dense = torch.randn(n, length, c, device="cuda").to(torch.bfloat16)
    dy = torch.randn(n, length, c, device="cuda").to(torch.bfloat16)
    norm = FusedGroupNorm(c, 4, n, activation="silu")
    want = norm.forward(dense)
    want_dx = norm.backward(dy, dense, None, None, *want[1:])
    x.copy_(dense)
    assert all(torch.equal(a, b) for a, b in zip(want_dx, norm.backward(dy, x, None, None, *want[1:])))
    got = norm.forward(x, y=x)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape,groups", [((900, 1, 256), 8), ((40, 6, 96), 4), ((2, 33, 2280), 3), ((7, 39, 3584), 14), ((2, 40_000, 96), 4),
                                          ((2, 314, 3662), 2), ((3, 1, 3364), 2)])
def test_a_mean_near_zero_keeps_its_bits(shape, groups, dtype):
    """Whole numbers of at most 8: every sum of them is exact, so a mean is off by the rounding of a
    quotient, or of a reciprocal and a product: 2 u of itself, whatever the kernel."""
    n, length, c = shape
    x = np.random.default_rng(c).integers(-8, 9, shape).astype(np.float64)
    _, mean, rstd = FusedGroupNorm(c, groups, n).forward(tensor_of(x, dtype))
    want = x.reshape(n, length, groups, -1).mean((1, 3))
    assert (np.abs(wide(mean) - want) <= 2.0 ** -23 * np.abs(want)).all()
    assert (np.abs(wide(rstd) - GN.forward(x, groups)[2]) <= 2.0 ** -16).all()
