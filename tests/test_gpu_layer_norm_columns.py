"""GPU: column sums over many rows, with the bound of test_gpu_layer_norm.py.

dy = 1 + 2^-k everywhere, a term that a float32 sum of 2^(23 - k) or more rounds down
every time: one long sum of such terms is off by up to 2^-k of its size.
"""

import numpy as np
import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import FusedLayerNorm
from test_gpu_layer_norm import close, wide

pytestmark = pytest.mark.gpu


def check(rows, width, k):
    x = torch.empty(rows, width, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(rows))
    dy = torch.full((rows, width), 1 + 2.0 ** -k, device="cuda")
    norm = FusedLayerNorm(width)
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")     # xhat = x
    _, dw, db = norm.backward(dy, x, None, mean, rstd, dx=dy)
    want, size = np.zeros(width), np.zeros(width)
    for at in range(0, rows, 1 << 16):
        part = x[at:at + (1 << 16)].double()
        want += wide(part.sum(0)) * (1 + 2.0 ** -k)
        size += wide(part.abs().sum(0)) * (1 + 2.0 ** -k)
    close(dw, want, size, torch.float32, 2e-5)
    close(db, np.full(width, rows * (1 + 2.0 ** -k)), rows, torch.float32, 2e-5)


@pytest.mark.parametrize("rows,width,k", [(20_000, 20_003, 13), (8000, 40_960, 13), (3000, 160_001, 13)])
def test_rows_wider_than_registers(rows, width, k):
    check(rows, width, k)


def test_many_rows_in_registers():
    check(4_900_000, 64, 14)


@pytest.mark.parametrize("rows,width,dtype", [(1_300_001, 33, torch.float32), (400_003, 1001, torch.bfloat16),
                                              (90_001, 4096, torch.bfloat16), (700_003, 1001, torch.bfloat16),
                                              (180_001, 2050, torch.bfloat16)])
def test_rows_of_several_launches(rows, width, dtype):
    """Odd rows, and in place; rows give the same bits in a call of their own that lies the same way."""
    g = torch.Generator(device="cuda").manual_seed(width)
    x, dy = (torch.randn(rows, width, device="cuda", generator=g).to(dtype) for _ in range(2))
    norm = FusedLayerNorm(width)
    _, mean, rstd = norm.forward(x)
    dx, dw, db = norm.backward(dy, x, None, mean, rstd)
    for at in (0, rows // 2, rows - 301):
        at = at // 8 * 8                           # on the 16-byte grid
        part = slice(at, at + 301)
        one, _, _ = norm.backward(*(t[part].clone() if t is not None else None for t in (dy, x, None, mean, rstd)))
        assert torch.equal(one, dx[part])
    xhat = ((x.double() - mean.double()[:, None]) * rstd.double()[:, None])
    size = wide((dy.double() * xhat).abs().sum(0)) + rows
    close(dw, wide((dy.double() * xhat).sum(0)), size, dtype, 2e-5)
    close(db, wide(dy.double().sum(0)), wide(dy.double().abs().sum(0)), dtype, 2e-5)
    again = norm.backward(dy, x, None, mean, rstd, dx=dy)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw) and torch.equal(again[2], db)
