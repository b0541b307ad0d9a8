"""GPU: the bounded waits of the layer norm's row kernels.

A limit of 0 makes waits give up on rows that are merely on their way: the call
ends, the plan reports it unless every row was there and the results are right,
nothing is left behind in flight, and the context and the plan (with its limit
back) go on to give right results.
"""

import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import AdamWError, FusedLayerNorm, _capi

pytestmark = pytest.mark.gpu


def _matrix(rows, width, dtype, pad, shift):
    t = torch.empty(rows * (width + pad) + shift, dtype=dtype, device="cuda")
    t.normal_(generator=torch.Generator(device="cuda").manual_seed(rows + width))
    return t[shift:].view(rows, width + pad)[:, :width]


def _reported(rows, width, pad=0, shift=0, other=0):
    """How many of a forward and a backward call without patience the plan reports; checks the rest."""
    x = _matrix(rows, width, torch.bfloat16, pad, shift)
    dy = _matrix(rows, width, torch.bfloat16, pad + other, shift)
    norm = FusedLayerNorm(width)
    y, mean, rstd = norm.forward(x)
    want = (y, mean, rstd, *norm.backward(dy, x, None, mean, rstd))
    assert norm.status() == 0
    reported = 0
    for backward in (False, True):
        norm = FusedLayerNorm(width)
        _capi.adamw_layer_norm_plan_set_wait_limit(norm.plan, 0)
        got = norm.backward(dy, x, None, mean, rstd) if backward else norm.forward(x)
        try:
            norm.status()                          # healthy: no row had to be waited for, all are right
            assert all(torch.equal(a, b) for a, b in zip(want[3:] if backward else want[:3], got))
        except AdamWError as e:
            assert e.status == _capi.ETIMEOUT
            reported += 1
        _capi.adamw_layer_norm_plan_set_wait_limit(norm.plan, 2_000_000)
        got = (*norm.forward(x), *norm.backward(dy, x, None, mean, rstd))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    return reported


# rows on the 16-byte grid, off it by one shift, and each matrix in its own way; every group size
@pytest.mark.parametrize("pad,shift,other", [(0, 0, 0), (1, 3, 0), (1, 3, 1)])
@pytest.mark.parametrize("width", [64, 1000, 2000, 4096, 8192, 16_000])
def test_waits_that_give_up(width, pad, shift, other):
    _reported(3000, width, pad, shift, other)      # rows may be in L2, and there at once


def test_rows_from_memory_cannot_be_there_at_once():
    assert _reported(60_000, 4096) == 2            # 490 MB


def test_the_limit_is_checked():
    norm = FusedLayerNorm(8)
    for plan, limit in ((norm.plan, -1), (None, 5)):
        with pytest.raises(AdamWError) as e:
            _capi.adamw_layer_norm_plan_set_wait_limit(plan, limit)
        assert e.value.status == _capi.EINVAL
