"""GPU: a padded batch through the experts' rows.  Rows that no slot names are 0 in what the calls make, whatever
the memory held before, so that products over all rows have the definition's gradients."""

import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import FusedRouter

pytestmark = pytest.mark.gpu
TOKENS, EXPERTS, K, WIDTH = 100, 8, 2, 72


def routed(dtype):
    g = torch.Generator("cuda").manual_seed(3)
    z = torch.randn(TOKENS, EXPERTS, device="cuda", generator=g)
    z[80:] = float("-inf")                       # padded
    z[3, 1:] = float("-inf")                     # one expert where two are asked for
    router = FusedRouter(TOKENS, EXPERTS, K)
    w, ids, slots, starts = router.route(z)
    x, dy = (torch.randn(TOKENS, WIDTH, device="cuda", generator=g).to(dtype) for _ in range(2))
    return router, w, slots, int(starts[-1]), x, dy


def spoil(dtype):
    """Leaves NaN in the memory that the next tensor of that size gets."""
    t = [torch.full((TOKENS * K, WIDTH), float("nan"), dtype=dtype, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del t


@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_rows_behind_the_last_are_zeros(dtype, stream):
    router, w, slots, live, x, dy = routed(dtype)
    s = torch.cuda.Stream() if stream else torch.cuda.current_stream()
    s.wait_stream(torch.cuda.current_stream())
    assert live == 80 * K - 1
    with torch.cuda.stream(s):
        spoil(dtype)
    xs = router.dispatch(x, slots, stream=s)
    s.synchronize()
    assert not xs[live:].any() and xs[:live].any(1).all()
    ys = torch.randn(TOKENS * K, WIDTH, device="cuda").to(dtype)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        spoil(dtype)
    dys, dw = router.combine_backward(dy, ys, slots, w, stream=s)
    s.synchronize()
    assert not dys[live:].any() and dys[:live].any(1).all() and not dw[80:].any() and dw[3, 1] == 0
    given = torch.full_like(ys, 3.0)             # left as they were
    assert router.combine_backward(dy, ys, slots, w, dys=given)[0] is given
    assert (given[live:] == 3).all() and torch.equal(given[:live], dys[:live])
    given = torch.full_like(xs, 3.0)
    assert (router.dispatch(x, slots, xs=given)[live:] == 3).all() and torch.equal(given[:live], xs[:live])


def test_the_experts_gradients_over_all_rows():
    """One product over every row: its weight's gradient is that of the live rows alone, by the definition."""
    router, w, slots, live, x, dy = routed(torch.float32)
    up = torch.randn(WIDTH, WIDTH, device="cuda") / 8
    spoil(torch.float32)
    xs = router.dispatch(x, slots)
    ys = (xs.double() @ up.double()).float()
    spoil(torch.float32)
    dys, _ = router.combine_backward(dy, ys, slots, w)
    got = xs.double().t() @ dys.double()
    want = sum(x[t].double()[:, None] * (w[t, j].double() * dy[t].double()) for t in range(TOKENS) for j in range(K) if slots[t, j] >= 0)
    # dys is rounded to float32: 2^-24 of each of the terms
    size = sum(x[t].double().abs()[:, None] * (w[t, j].double() * dy[t].double()).abs() for t in range(TOKENS) for j in range(K) if slots[t, j] >= 0)
    assert ((got - want).abs() <= 2.0 ** -23 * size).all()
