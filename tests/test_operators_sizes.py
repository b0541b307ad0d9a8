"""Plan sizes past what the entry points count in are refused before any device work."""

import pytest

from adamw_optimizer_step_tensor_gb300 import _capi as C


@pytest.mark.parametrize("rows", [2 ** 40 + 1, 2 ** 61, 2 ** 62, 2 ** 62 + 5, 2 ** 63 - 1])
def test_loss_plans(rows):
    with pytest.raises(C.AdamWError) as e:
        C.adamw_loss_plan_create(rows, 0)
    assert e.value.status == C.EUNSUPPORTED


@pytest.mark.parametrize("width", [2 ** 30 + 1, 2 ** 31 - 1])
def test_layer_norm_plans(width):
    with pytest.raises(C.AdamWError) as e:
        C.adamw_layer_norm_plan_create(width, 1e-5)
    assert e.value.status == C.EUNSUPPORTED
