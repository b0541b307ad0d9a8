"""GPU: rows of advantage 0 add nothing to the policy part, whatever their ratio.

exp(logp - old) passes float32 from a difference of 88.7 on; times 0 it is 0 in the
definition.  A ratio that is no number stays one.
"""

import numpy as np
import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import FusedTokenLoss
from oracle import token_loss as TL
from test_gpu_token_loss import REL, Batch, check_grad, wide

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [300, 50_257])
@pytest.mark.parametrize("clip", [(0.2, 0.28), (0.2, float("inf"))])
def test_a_ratio_past_float32(vocab, dtype, clip):
    b = Batch(6, vocab, dtype, masked=0.0)
    adv, old, ref = b.policy_inputs()
    adv[1] = adv[2] = 0.0
    adv[3] = -0.0
    old[1] -= 100.0
    old[3] -= 90.0
    want = TL.policy(b.Z, b.y, wide(b.w), wide(adv), wide(old), wide(ref),
                     tuple(float(np.float32(c)) for c in clip), float(np.float32(0.05)))
    stats, _, _ = FusedTokenLoss(6).policy(b.logits, b.labels, b.w, adv, old, ref, clip=clip, kl_coef=0.05,
                                           dlogits=b.dz)
    torch.cuda.synchronize()
    assert np.isfinite(want["stats"]).all()
    assert np.all(np.abs(wide(stats) - want["stats"]) <= REL * (want["size"] + np.abs(want["stats"])))
    check_grad(b, b.dz, want["slopes"], want["live"], want["terms"])


def test_a_ratio_that_is_no_number_stays_one():
    b = Batch(4, 300, torch.float32, masked=0.0)
    adv, old, ref = b.policy_inputs()
    adv[2] = 0.0
    old[2] = float("nan")
    stats, _, dz = FusedTokenLoss(4).policy(b.logits, b.labels, b.w, adv, old, ref, kl_coef=0.05)
    assert torch.isnan(stats[:2]).all() and torch.isnan(dz[2]).all()
    assert torch.isfinite(dz[[0, 1, 3]]).all()
