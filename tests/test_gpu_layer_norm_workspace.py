"""GPU: what a layer norm plan holds on the device."""

import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import FusedLayerNorm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width,most", [(768, 64), (8192, 64), (8193, 32), (65_537, 32), (1_000_000, 32)])
def test_workspace(width, most):
    """Column sums of the parts in use: MB, not a row of them per CTA that fits the GPU."""
    FusedLayerNorm(8).close()                    # what the context and the kernels themselves take
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    norm = FusedLayerNorm(width)
    assert before - torch.cuda.mem_get_info()[0] <= most << 20
    norm.close()
