"""The operators' outputs belong to the stream of the launch, without a GPU: what
the binding allocates is made with that stream as the current one."""

from contextlib import contextmanager

import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import FusedLayerNorm, FusedTokenLoss
from adamw_optimizer_step_tensor_gb300 import operators as O


class _Fake:
    """A torch tensor's face over a CPU tensor that says it is on the GPU."""

    is_cuda = True

    def __init__(self, t):
        self._t = t

    def __getattr__(self, name):
        return getattr(self._t, name)

    def get_device(self):
        return 0


@pytest.fixture
def streams(monkeypatch):
    """Lists of the stream current at every allocation and every launch."""
    current, made, launched = [None], [], []

    @contextmanager
    def as_current(s):
        current.append(s)
        yield
        current.pop()

    def empty_like(t):
        made.append(current[-1])
        return _Fake(torch.zeros(t.shape, dtype=t.dtype))

    def empty(n, like, dtype=torch.float32):
        made.append(current[-1])
        return _Fake(torch.zeros(n, dtype=dtype))

    monkeypatch.setattr(torch.cuda, "stream", as_current)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: handle)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: "default")
    monkeypatch.setattr(torch, "empty_like", empty_like)
    monkeypatch.setattr(O, "_empty", empty)
    monkeypatch.setattr(O, "_stream", lambda s: current[-1] if s is None else s)
    for name in ("adamw_token_logps", "adamw_policy_loss", "adamw_preference_loss",
                 "adamw_layer_norm_forward", "adamw_layer_norm_backward"):
        monkeypatch.setattr(O._capi, name, lambda *args: launched.append(args[-1]))
    for name in ("adamw_loss_plan", "adamw_layer_norm_plan"):
        monkeypatch.setattr(O._capi, name + "_create", lambda *args: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return made, launched


def _calls():
    z, y, v = _Fake(torch.zeros(4, 8)), _Fake(torch.zeros(4, dtype=torch.int64)), _Fake(torch.zeros(4))
    starts = _Fake(torch.zeros(3, dtype=torch.int32))
    loss, norm = FusedTokenLoss(4, 1), FusedLayerNorm(8)
    return [(2, lambda **kw: loss.logps(z, y, **kw)), (3, lambda **kw: loss.policy(z, y, v, v, **kw)),
            (4, lambda **kw: loss.preference(z, y, v, v, starts, **kw)), (3, lambda **kw: norm.forward(z, **kw)),
            (3, lambda **kw: norm.backward(z, z, None, v, v, **kw))]


@pytest.mark.parametrize("stream,want", [(None, None), (123, 123), (0, "default"), (1, "default")])
def test_outputs_belong_to_the_launch_stream(streams, stream, want):
    made, launched = streams
    for outputs, call in _calls():
        del made[:], launched[:]
        call(stream=stream)
        assert made == [want] * outputs and launched == [want]
