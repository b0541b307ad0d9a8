"""GPU: calls on a stream other than the current one."""

import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import FusedLayerNorm, FusedTokenLoss

pytestmark = pytest.mark.gpu


def _cases():
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    z, v = rand(64, 20_011), rand(64)
    y = torch.randint(0, 20_011, (64,), device="cuda", generator=g)
    starts = torch.tensor([0, 30, 64], dtype=torch.int32, device="cuda")
    loss, norm = FusedTokenLoss(64, 1), FusedLayerNorm(20_011)
    mean, rstd = norm.forward(z)[1:]
    return [lambda **kw: loss.logps(z, y, **kw), lambda **kw: loss.policy(z, y, v, v, **kw),
            lambda **kw: loss.preference(z, y, v, v, starts, **kw), lambda **kw: norm.forward(z, **kw),
            lambda **kw: norm.backward(z, z, None, mean, rstd, **kw)]


@pytest.mark.parametrize("raw", [False, True])
def test_outputs_do_not_share_memory_with_work_on_the_current_stream(raw):
    """Blocks freed here are still written by what is queued here; outputs of another stream stay clear of them."""
    s = torch.cuda.Stream()
    for call in _cases():
        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        blocks = [torch.empty_like(t) for t in want]
        at = {b.data_ptr() for b in blocks}
        torch.cuda._sleep(20_000_000)           # about 10 ms, far longer than the call
        for b in blocks:
            b.fill_(float("nan"))
        del b, blocks
        got = call(stream=s.cuda_stream if raw else s)
        assert not at & {t.data_ptr() for t in got}
        s.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        current = torch.cuda.current_stream()
        for t in got:
            t.record_stream(current)


def test_the_default_stream_by_its_handle():
    call = _cases()[0]
    want = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = call(stream=0)
        assert torch.cuda.current_stream() == s
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
