"""GPU: rows to their experts and back against the float64 definition.

Tolerance: the combine is k float32 fused steps, at most k u (u = 2^-24) of the sum of
magnitudes, and half a step of the type; its backward's product is rounded to float32 and
to the type; a dot product over a row is at most (width / 32 + 10) u of its magnitudes.
"""

import numpy as np
import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import FusedRouter
from oracle import router as RO

from _support import assert_guards_intact, empty, guarded_empty

pytestmark = pytest.mark.gpu
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
U = 2.0 ** -24


def wide(t):
    return t.detach().double().cpu().numpy()


def rows_of(a, dtype, pad=0, shift=0):
    r, c = a.shape
    t = guarded_empty(r * (c + pad), dtype, shift).view(r, c + pad)
    t.fill_(7.0)
    t = t[:, :c]
    t.copy_(torch.from_numpy(a.astype(np.float32)))
    return t


def near(got, want, size, dtype):
    named = ~np.isnan(want)
    err = np.abs(wide(got) - want)[named]
    bound = (size + HALF[dtype] * (np.abs(want) + size) + TINY[dtype])[named]
    assert (err <= bound).all(), (float((err - bound).max()), float(err.max()))
    assert (wide(got)[~named] == 3.0).all()         # rows that no slot names


def slots_of(tokens, k, experts, rng, gone=0.2):
    ids = np.array([rng.permutation(experts)[:k] for _ in range(tokens)]).reshape(tokens, k)
    ids[rng.random(ids.shape) < gone] = -1
    if tokens > 2:
        ids[1] = -1
    return RO.places(ids, experts)[0]


def check(tokens, width, k, dtype, pad=0, shift=0, experts=None):
    rng = np.random.default_rng(tokens + width)
    slots = slots_of(tokens, k, experts or 2 * k, rng)
    n = tokens * k
    x, dy = (rows_of(rng.normal(size=(tokens, width)), dtype, pad, shift) for _ in range(2))
    ys = rows_of(rng.normal(size=(n, width)), dtype, pad, shift)
    at = torch.from_numpy(slots.astype(np.int32)).cuda()
    w = rng.uniform(0, 1, (tokens, k)).astype(np.float32)
    wt, ww = torch.from_numpy(w).cuda(), w.astype(np.float64)
    router = FusedRouter(tokens, experts or 2 * k, k)
    xs, dys = (rows_of(np.full((n, width), 3.0), dtype, pad, shift) for _ in range(2))
    y = rows_of(np.zeros((tokens, width)), dtype, pad, shift)
    dw = empty(n).view(tokens, k)
    router.dispatch(x, at, xs=xs)
    near(xs, RO.dispatch(wide(x), slots, n), 0.0 * RO.dispatch(wide(x), slots, n), dtype)
    for weights, oracle in ((wt, ww), (None, None)):
        router.combine(ys, at, weights, y=y)
        size = RO.combine(np.abs(wide(ys)), slots, oracle)
        near(y, RO.combine(wide(ys), slots, oracle), k * U * size, dtype)
    router.combine_backward(dy, ys, at, wt, dys=dys, dweights=dw)
    want, want_w = RO.combine_backward(wide(dy), wide(ys), slots, ww)
    near(dys, want, U * np.abs(want), dtype)
    size = RO.combine_backward(np.abs(wide(dy)), np.abs(wide(ys)), slots, ww)[1]
    assert (np.abs(wide(dw) - want_w) <= (width / 32 + 10) * U * size).all()
    assert_guards_intact()
    router.combine_backward(dy, ys, at, wt, dys=ys, dweights=dw)       # in place
    live = ~np.isnan(want[:, 0])
    assert torch.equal(ys[torch.from_numpy(live).cuda()], dys[torch.from_numpy(live).cuda()])
    assert (np.abs(wide(dw) - want_w) <= (width / 32 + 10) * U * size).all()
    assert_guards_intact()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,width,k,pad,shift", [
    (1, 1, 1, 0, 0), (3, 7, 2, 0, 0), (5, 4096, 4, 0, 0), (40, 256, 8, 0, 0), (33, 129, 3, 0, 0), (20, 64, 6, 8, 0),
    (20, 64, 6, 1, 0), (20, 64, 5, 0, 1), (301, 24, 3, 0, 0), (100, 40, 32, 0, 0), (57, 3, 2, 0, 0), (65, 130, 2, 2, 0), (9, 1601, 2, 0, 0), (7, 520, 32, 0, 0), (200, 8, 1, 0, 0), (11, 6000, 2, 0, 0)])
def test_matches_the_definition(tokens, width, k, pad, shift, dtype):
    check(tokens, width, k, dtype, pad, shift)


@pytest.mark.parametrize("dtype", DTYPES)
def test_slots_that_name_no_row(dtype):
    """Slots past the rows, or below 0, move nothing and add nothing."""
    router = FusedRouter(4, 8, 2)
    x = torch.randn(4, 96, device="cuda").to(dtype)
    slots = torch.tensor([[0, 5], [-1, 4], [2 ** 31 - 1, 1], [-2 ** 31, 3]], dtype=torch.int32, device="cuda")
    xs = rows_of(np.full((4, 96), 3.0), dtype)
    router.dispatch(x, slots, xs=xs)
    assert torch.equal(xs[0], x[0]) and torch.equal(xs[1], x[2]) and torch.equal(xs[3], x[3]) and (xs[2] == 3).all()
    y = router.combine(xs, slots)
    assert torch.equal(y[0], x[0]) and not y[1].any() and torch.equal(y[2], x[2])
    dys, dw = router.combine_backward(x, xs, slots, torch.ones(4, 2, device="cuda"), dys=torch.full_like(xs, 3.0))
    assert (dys[2] == 3).all() and torch.equal(dys[0], x[0]) and not dw[1].any() and dw[0, 1] == 0 and dw[0, 0] > 0
    none = torch.full_like(slots, -1)
    assert not router.combine(xs, none).any() and not router.combine(torch.empty(0, 96, dtype=dtype, device="cuda"), none).any()


def test_no_tokens_and_refusals():
    router = FusedRouter(4, 8, 2)
    x, slots = torch.randn(4, 8, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    assert router.dispatch(x[:0], slots[:0]).shape == (0, 8)
    assert router.combine(x, slots[:0]).shape == (0, 8)
    from adamw_optimizer_step_tensor_gb300 import AdamWError
    with pytest.raises(AdamWError, match="may not be ys"):
        router.combine(x, slots, y=x)
    with pytest.raises(AdamWError, match="may not be x"):
        router.dispatch(x, slots, xs=x)
    with pytest.raises(AdamWError, match="may not be dy"):
        router.combine_backward(x, x.clone(), slots, torch.ones(4, 2, device="cuda"), dys=x)
    with pytest.raises(AdamWError, match="5 tokens"):
        router.dispatch(torch.randn(5, 8, device="cuda"), torch.zeros(5, 2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        router.dispatch(x, slots[:, :1].contiguous())


def test_offsets_past_32_bits():
    """Rows whose elements lie past 2^31 and 2^32 of their matrix."""
    width, n = 1 << 20, 4200
    ys = torch.zeros(n, width, dtype=torch.bfloat16, device="cuda")
    router = FusedRouter(2, 4, 2)
    x = torch.randn(2, width, device="cuda").to(torch.bfloat16)
    slots = torch.tensor([[n - 1, 0], [2048, 4096]], dtype=torch.int32, device="cuda")
    router.dispatch(x, slots, xs=ys)
    for t in range(2):
        for j in range(2):
            assert torch.equal(ys[int(slots[t, j])], x[t])
    assert int((ys[1:2048].abs().amax() + ys[2049:4096].abs().amax()).item()) == 0
    y = router.combine(ys, slots, torch.tensor([[0.25, 0.75], [1.0, 0.0]], device="cuda"))
    assert torch.equal(y, x)
    dys, dw = router.combine_backward(x, ys, slots, torch.ones(2, 2, device="cuda"), dys=ys)
    assert torch.equal(ys[n - 1], x[0])
    want = (x.double() ** 2).sum(1)
    assert ((dw.double() - want[:, None]).abs() <= (width / 32 + 10) * U * want[:, None]).all()
