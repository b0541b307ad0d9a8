"""GPU: a block's operators where counts and offsets pass 32 bits: dropout of rows at strides and off the grid past
2^31 words and elements, rows of as many tokens as a plan takes, more than 2^31 samples of a group norm."""

import numpy as np
import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import FusedDropout, FusedGroupNorm, FusedRouter
from oracle import dropout as DR

pytestmark = pytest.mark.gpu
STEP = 1 << 27


@pytest.fixture(autouse=True)
def give_the_memory_back():
    """The library's plans take memory that torch's cache holds otherwise."""
    yield
    torch.cuda.empty_cache()


def windows(n):
    return [at for at in (0, (1 << 31) - 8, (1 << 32) - 8, (1 << 33) + 4, (1 << 34) - 8, n - 48) if at + 48 <= n]


@pytest.mark.parametrize("width,pad,shift,rows", [(1 << 12, 8, 0, (1 << 22) + 5), (4099, 0, 1, (1 << 21) + 3), (4099, 3, 0, (1 << 20) + 3)])
def test_dropout_past_32_bits(width, pad, shift, rows):
    """16-byte words at strides (2^31 of them), one run off the grid, and rows off the grid at strides."""
    room = torch.ones(rows * (width + pad) + shift, dtype=torch.bfloat16, device="cuda")
    x = room[shift:].view(rows, width + pad)[:, :width]
    FusedDropout(0.5, 77, 2).forward(x, y=x)
    n = rows * width
    assert n > 1 << 32 and (pad != 8 or n > 1 << 34)
    for at in windows(n):
        i = torch.arange(at, at + 48, device="cuda")
        got = x[i // width, i % width].float().cpu().numpy()
        assert np.array_equal(got != 0, DR.words(at // 4 * 4, 48 + at % 4, 77, 0, 2)[at % 4:].astype(np.int64) >= 2 ** 31), at
        assert set(np.unique(got)) <= {0.0, 2.0}
    for r in (0, rows // 2, rows - 1):           # what lies between the rows is as it was
        assert (room[shift:].view(rows, width + pad)[r, width:] == 1).all()


def test_rows_of_as_many_tokens_as_a_plan_takes():
    n = 2 ** 31 - 1
    router = FusedRouter(n, 1, 1)
    slots = torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda")[:, None]
    x = torch.empty(n, 1, dtype=torch.bfloat16, device="cuda")
    for at in range(0, n, STEP):
        x[at:at + STEP, 0] = (torch.arange(at, min(n, at + STEP), device="cuda") % 251).to(torch.bfloat16)
    xs = router.dispatch(x, slots, xs=torch.empty_like(x))
    assert torch.equal(xs.flip(0), x)
    weights = torch.full((n, 1), 2.0, device="cuda")
    assert torch.equal(router.combine(xs, slots, weights), x + x)
    dys, dw = router.combine_backward(x, xs, slots, weights, dys=torch.empty_like(xs))
    assert torch.equal(dys, xs + xs)
    for at in range(0, n, STEP):
        assert torch.equal(dw[at:at + STEP], x[at:at + STEP].float() ** 2)


def test_more_samples_than_32_bits_count():
    n = 2 ** 31 + 12345
    x = torch.empty(n, 1, 2, dtype=torch.bfloat16, device="cuda")
    for at in range(0, n, STEP):                 # pairs a, a + 2: mean a + 1, deviation 1
        a = (torch.arange(at, min(n, at + STEP), device="cuda") % 61 - 30).to(torch.bfloat16)
        x[at:at + STEP, 0] = torch.stack([a, a + 2], 1)
    norm = FusedGroupNorm(2, 1, n, eps=0.0)
    y, mean, rstd = norm.forward(x)
    dy = x                                       # of which nothing is left but the mean of two
    dx, dw, db = norm.backward(dy, x, None, None, mean, rstd)
    total = torch.zeros(2, dtype=torch.float64, device="cuda")
    for at in range(0, n, STEP):
        part = x[at:at + STEP, 0].float()
        assert torch.equal(mean[at:at + STEP, 0], part[:, 0] + 1) and (rstd[at:at + STEP] == 1).all()
        assert (y[at:at + STEP, 0, 0] == -1).all() and (y[at:at + STEP, 0, 1] == 1).all()
        assert not dx[at:at + STEP].any()
        total += (part * torch.tensor([-1.0, 1.0], device="cuda")).double().sum(0)
    # sums of whole numbers over 608 CTAs' threads, each of 2^31 / (608 256) = 13 800 samples: 64 at a time, then 216
    # flushes: under 512 u of the sum of 2^31 magnitudes below 32
    assert ((dw.double() - total).abs() <= 2.0 ** -15 * n * 32 + 2.0 ** -8 * total.abs()).all()
    assert norm.status() == 0
