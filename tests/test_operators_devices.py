"""The operators refuse tensors of another device than their plan's, without a GPU."""

import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import FusedLayerNorm, FusedTokenLoss
from adamw_optimizer_step_tensor_gb300 import operators as O


class _Fake:
    """A torch tensor's face over a CPU tensor that says on which GPU it is."""

    is_cuda = True

    def __init__(self, t, device=0):
        self._t, self._device = t, device

    def __getattr__(self, name):
        return getattr(self._t, name)

    def get_device(self):
        return self._device


@pytest.fixture
def launches(monkeypatch):
    count = []
    for name in ("adamw_token_logps", "adamw_policy_loss", "adamw_preference_loss",
                 "adamw_layer_norm_forward", "adamw_layer_norm_backward"):
        monkeypatch.setattr(O._capi, name, lambda *args: count.append(args))
    for name in ("adamw_loss_plan", "adamw_layer_norm_plan"):
        monkeypatch.setattr(O._capi, name + "_create", lambda *args: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(O, "_stream", lambda s: 1)
    return count


def _calls():
    """Every call with its tensors by name."""
    f = lambda *s, dtype=torch.float32: _Fake(torch.zeros(*s, dtype=dtype))  # noqa: E731
    z, v = (lambda: f(4, 8)), (lambda: f(4))
    y = lambda: f(4, dtype=torch.int64)  # noqa: E731
    loss, norm = FusedTokenLoss(4, 1), FusedLayerNorm(8)
    grad = dict(grad_scale=f(1), stats=f(4), logps=v(), dlogits=z())
    return [
        (loss.logps, dict(logits=z(), labels=y(), logps=v(), lse=v())),
        (loss.policy, dict(logits=z(), labels=y(), weights=v(), advantages=v(), old_logps=v(), ref_logps=v(), **grad)),
        (loss.preference, dict(logits=z(), labels=y(), weights=v(), ref_logps=v(),
                               seq_starts=f(3, dtype=torch.int32), rewards=f(2), **grad)),
        (norm.forward, dict(x=z(), weight=f(8), bias=f(8), y=z(), mean=v(), rstd=v())),
        (norm.backward, dict(dy=z(), x=z(), weight=f(8), mean=v(), rstd=v(), dx=z(), dweight=f(8), dbias=f(8))),
    ]


def test_every_tensor_is_checked(launches):
    for call, tensors in _calls():
        call(**tensors)
        assert len(launches) == 1
        for name, t in tensors.items():
            elsewhere = _Fake(t._t, 1)
            with pytest.raises(ValueError, match=f"^{name} is on device 1, the plan on device 0"):
                call(**{**tensors, name: elsewhere})
        assert len(launches) == 1
        launches.clear()
