"""GPU: dropout against the float64 definition, whose mask is the generator's, word by word.

Tolerance: y = fma(x, scale, r) with scale rounded once: 2^-24 |x scale| for the scale and
2^-24 |y| for the sum, then half a step of the type.  Which elements are dropped is exact.
"""

import numpy as np
import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import FusedDropout
from oracle import dropout as DR

from _support import assert_guards_intact, dev, guarded_empty

pytestmark = pytest.mark.gpu
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
SEED = 0x1234_5678_9ABC_DEF0


def wide(t):
    return t.detach().double().cpu().numpy()


def rows_of(a, dtype, pad=0, shift=0):
    r, c = a.shape
    t = guarded_empty(r * (c + pad), dtype, shift).view(r, c + pad)
    t.fill_(7.0)
    t = t[:, :c]
    t.copy_(torch.from_numpy(a.astype(np.float32)))
    return t


def close(got, x, r, want, p, dtype):
    part = np.abs(want - (0 if r is None else r))
    bound = 2.0 ** -24 * (part + np.abs(want)) * 1.01 + HALF[dtype] * np.abs(want) * 1.01 + TINY[dtype]
    err = np.abs(wide(got) - want)
    assert (err <= bound).all(), (float(err.max()), np.argwhere(err > bound)[:3])


def step_of(t):
    return dev(np.array([t], np.int32))


# dense and on the grid, odd ends, off the grid, padded rows, rows of one element
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,width,pad,shift", [
    (1, 1, 0, 0), (1, 3, 0, 0), (1, 4, 0, 0), (3, 5, 0, 0), (2, 1024, 0, 0), (1, 8191, 0, 0), (33, 257, 0, 0), (17, 96, 8, 0),
    (17, 96, 3, 0), (5, 129, 1, 1), (9, 64, 0, 1), (300, 264, 16, 0), (1000, 1, 2, 0), (7, 4096, 0, 0)])
def test_matches_the_definition(rows, width, pad, shift, dtype):
    rng = np.random.default_rng(rows * 31 + width)
    x, r, dy = (rows_of(rng.normal(0, 1.5, (rows, width)), dtype, pad, shift) for _ in range(3))
    for p, step, site in ((0.1, 0, 0), (0.5, 12345, 3), (0.013, -7, 2 ** 32 - 1)):
        drop = FusedDropout(p, SEED, site)
        for res in (None, r):
            y = rows_of(np.zeros((rows, width)), dtype, pad, shift)
            drop.forward(x, step_of(step), res, y=y)
            want = DR.forward(wide(x), None if res is None else wide(res), p, SEED, step, site)
            close(y, wide(x), None if res is None else wide(res), want, p, dtype)
            kept = DR.keep((rows, width), p, SEED, step, site)
            if res is None:
                assert np.array_equal(wide(y) != 0, kept & (wide(x) != 0))
        dx = drop.backward(dy, step_of(step))
        close(dx, wide(dy), None, DR.forward(wide(dy), None, p, SEED, step, site), p, dtype)
        assert_guards_intact()


@pytest.mark.parametrize("dtype", DTYPES)
def test_the_mask_is_the_element_s_wherever_it_lies(dtype):
    x = torch.rand(40, 130, device="cuda").add(1).to(dtype)
    drop = FusedDropout(0.3, 5, 1)
    want = drop.forward(x)
    apart = torch.zeros(40, 200, dtype=dtype, device="cuda")[:, 3:133]
    apart.copy_(x)
    assert torch.equal(drop.forward(apart), want)
    assert torch.equal(drop.forward(x.view(-1)).view_as(x), want)
    assert torch.equal(drop.forward(x.view(4, 10, 130)).view_as(x), want)
    for y in (x.clone(), apart):
        drop.forward(y, y=y)
        assert torch.equal(y, want)
    other = [FusedDropout(0.3, 6, 1).forward(x), FusedDropout(0.3, 5, 2).forward(x), drop.forward(x, step_of(1)),
             FusedDropout(0.3, 5 + 2 ** 32, 1).forward(x)]
    assert all(((o == 0) != (want == 0)).any() for o in other)


@pytest.mark.parametrize("dtype", DTYPES)
def test_dropped_values_are_not_used(dtype):
    kept = torch.from_numpy(DR.keep((64, 64), 0.4, 9)).cuda()
    for bad in (float("nan"), float("inf"), float("-inf")):
        x = torch.where(kept, 1.0, bad).to(dtype)
        r = torch.full((64, 64), 2.0, dtype=dtype, device="cuda")
        y = FusedDropout(0.4, 9).forward(x, None, r)
        assert torch.isfinite(y).all() and (y[~kept] == 2).all()
        r[0, :8] = bad                              # the residual's own values stay
        y = FusedDropout(0.4, 9).forward(x, None, r)
        assert not torch.isfinite(y[0, :8]).any() and torch.isfinite(y[1:]).all()


@pytest.mark.parametrize("shift", [0, 1])
def test_the_ends_of_p(shift):
    x = torch.randn(257 + shift, device="cuda")[shift:]
    r = torch.randn(257 + shift, device="cuda")[shift:]
    assert torch.equal(FusedDropout(0.0, 1).forward(x), x)
    assert torch.equal(FusedDropout(0.0, 1).forward(x, None, r), x + r)
    bad = torch.full_like(x, float("nan"))
    assert torch.equal(FusedDropout(1.0, 1).forward(bad, None, r), r)
    assert not FusedDropout(1.0, 1).forward(bad).any()
    last = 1 - 2.0 ** -24                           # the largest p below 1
    y = FusedDropout(last, 1).forward(torch.ones(1 << 20, device="cuda"))
    kept = DR.keep((1 << 20,), last, 1)
    assert np.array_equal(y.cpu().numpy() != 0, kept)


def test_the_residual_in_place_and_nothing_at_all():
    x, r = torch.randn(9, 40, device="cuda"), torch.randn(9, 40, device="cuda")
    drop = FusedDropout(0.2, 3)
    want = drop.forward(x, None, r)
    drop.forward(x, None, r, y=r)
    assert torch.equal(r, want)
    for shape in ((0, 5), (5, 0), (0,)):
        assert drop.forward(torch.empty(shape, device="cuda")).shape == shape


def test_far_elements_have_words_of_their_own():
    """Element numbers past 2^32 go into the counter whole: a row of 2^32 + 40 bytes of bf16 zeros and ones."""
    n = (1 << 34) + 24
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    drop = FusedDropout(0.5, 77)
    drop.forward(x, y=x)
    for at in (0, (1 << 32) - 8, 1 << 32, (1 << 34) - 8, 1 << 34):
        got = x[at:at + 24].float().cpu().numpy() != 0
        m = len(got)
        assert np.array_equal(got, DR.words(at, m, 77).astype(np.int64) >= 2 ** 31), at
