"""GPU: an operator's failure stays its own: the calls after it succeed."""

import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import AdamWError, FusedAdamW, FusedLayerNorm, FusedTokenLoss, _capi

pytestmark = pytest.mark.gpu


def test_calls_after_a_plan_that_did_not_fit():
    x = torch.randn(8, 64, device="cuda")
    y = torch.zeros(8, dtype=torch.int64, device="cuda")
    norm, loss = FusedLayerNorm(64), FusedTokenLoss(8)
    tensors = [torch.ones(100, device="cuda") for _ in range(4)]
    opt = FusedAdamW(*[[t] for t in tensors], [0.0])
    total = torch.zeros(1, device="cuda")
    want = norm.forward(x)
    calls = [lambda: norm.forward(x), lambda: norm.backward(x, x, None, want[1], want[2]), lambda: loss.logps(x, y),
             lambda: opt.grad_norm(total), lambda: opt.clip_grads(total)]
    for call in calls:
        with pytest.raises(AdamWError) as e:
            FusedTokenLoss(2 ** 40)                # 8 TB
        assert e.value.status == _capi.ENOMEM
        call()
    assert total.item() == 10.0
    assert all(torch.equal(a, b) for a, b in zip(want, norm.forward(x)))
