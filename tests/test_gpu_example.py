"""GPU: the example runs the operators together and the model learns; the same
updates with torch's own autograd give the same parameters."""

import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_example_learns():
    import tune_policy as E
    reward, ahead, loss, policy = E.main()
    assert sum(reward[-5:]) > 3 * sum(reward[:5])
    assert loss[0] == pytest.approx(0.6931, abs=1e-3) and loss[-1] < 0.35 and ahead[-1] > 0.95
    assert int(policy.steps) == 40 and policy.opt.status() == 0
    assert policy.loss.status() == 0 and policy.norm.status() == 0


def test_update_equals_autograd():
    """One preference update by hand-written operators against torch autograd and torch AdamW."""
    import tune_policy as E
    policy, twin = E.Policy(3, 64, 2), E.Policy(3, 64, 2)
    g = torch.Generator(device="cuda").manual_seed(5)
    tokens = torch.randint(0, E.VOCAB, (40,), device="cuda", generator=g)
    taken = torch.randint(0, E.VOCAB, (40,), device="cuda", generator=g)
    starts = torch.tensor([0, 7, 20, 33, 40], dtype=torch.int32, device="cuda")
    ref, _ = policy.loss.logps(policy.logits(tokens)[0], taken)
    ref = ref + 0.1 * torch.randn(40, device="cuda", generator=g)
    logits, saved = policy.logits(tokens)
    stats, _, _, dlogits = policy.loss.preference(logits, taken, None, ref, starts, beta=0.5)
    policy.update(dlogits, saved, max_norm=0.05)

    ps = [p.double().requires_grad_() for p in (twin.emb, twin.out, twin.weight, twin.bias)]
    opt = torch.optim.AdamW([{"params": ps[:2], "weight_decay": 0.01}, {"params": ps[2:], "weight_decay": 0.0}],
                            lr=float(twin.lr), betas=(0.9, 0.999), eps=1e-8)
    y = torch.nn.functional.layer_norm(ps[0][tokens], (E.WIDTH,), ps[2], ps[3], 1e-5)
    lp = torch.log_softmax(y @ ps[1].t(), 1).gather(1, taken[:, None])[:, 0] - ref.double()
    at = starts.tolist()
    sums = torch.stack([0.5 * lp[i:j].sum() for i, j in zip(at, at[1:])])
    loss = torch.nn.functional.softplus(sums[2:] - sums[:2]).mean()
    loss.backward()
    norm = torch.nn.utils.clip_grad_norm_(ps, 0.05)
    opt.step()
    assert float(stats[0]) == pytest.approx(float(loss), rel=1e-5)
    assert float(policy.grad_norm) == pytest.approx(float(norm), rel=1e-4) and float(norm) > 0.05
    # a first AdamW step is lr * sign-like: compare where the clipped grad is well above eps
    for p, q, grad in zip((policy.emb, policy.out, policy.weight, policy.bias), ps, policy.grads):
        sure = grad.abs() > 1e-5
        assert torch.allclose(p.double()[sure], q.detach()[sure], rtol=0, atol=2e-5)
