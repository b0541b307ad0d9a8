"""GPU: values at float32's edges, kernel by kernel: spreads past its range have rstd 0 and leave the bias, as the
header says; just inside it, and far below 1, the definition holds (test_gpu_group_norm's bounds)."""

import numpy as np
import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import FusedGroupNorm
from oracle import group_norm as GN

from test_gpu_group_norm_no_numbers import SHAPES

pytestmark = pytest.mark.gpu
FEW = [s for s in SHAPES if np.prod(s[0]) < 6_000_000]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape,groups", SHAPES)
def test_spreads_past_the_range(shape, groups, dtype):
    n, length, c = shape
    x = (1e25 * torch.randn(shape, device="cuda", generator=torch.Generator("cuda").manual_seed(1))).to(dtype)
    b = torch.randn(c, device="cuda")
    y, mean, rstd = FusedGroupNorm(c, groups, n).forward(x, None, b)
    assert not rstd.any() and mean.isfinite().all()
    assert torch.equal(y, b.to(dtype).expand(shape))


@pytest.mark.parametrize("scale", [1e15, 1e-15])
@pytest.mark.parametrize("shape,groups", FEW)
def test_spreads_inside_the_range(shape, groups, scale):
    n, _, c = shape
    x = (scale * torch.randn(shape, device="cuda", generator=torch.Generator("cuda").manual_seed(2)))
    y, mean, rstd = FusedGroupNorm(c, groups, n, eps=0.0 if scale > 1 else 1e-30).forward(x)
    want, m, r = GN.forward(x.double().cpu().numpy(), groups, eps=0.0 if scale > 1 else float(np.float32(1e-30)))
    wide = lambda t: t.double().cpu().numpy()  # noqa: E731
    assert (np.abs(wide(mean) - m) <= 2.0 ** -20 * float(x.abs().max())).all()
    assert (np.abs(wide(rstd) - r) <= 2.0 ** -16 * r).all()
    assert (np.abs(wide(y) - want) <= 2.0 ** -15 * (1 + np.abs(want))).all()
