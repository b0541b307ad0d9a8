"""GPU: layer norm in place: the same row stride, or a refusal (a row's output would
land on rows that others still read)."""

import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import AdamWError, FusedLayerNorm, _capi

pytestmark = pytest.mark.gpu


def _refused(fn):
    with pytest.raises(AdamWError, match="row stride") as e:
        fn()
    assert e.value.status == _capi.EINVAL


def test_another_row_stride_is_refused():
    norm = FusedLayerNorm(64)
    buf = torch.randn(8 * 80, device="cuda")
    wide, dense = buf.view(8, 80)[:, :64], buf[: 8 * 64].view(8, 64)
    other = torch.randn(8, 64, device="cuda")
    _, mean, rstd = norm.forward(other)
    before = buf.clone()
    for a, b in ((wide, dense), (dense, wide)):
        _refused(lambda: norm.forward(a, y=b))
        _refused(lambda: norm.backward(a, other, None, mean, rstd, dx=b))
        _refused(lambda: norm.backward(other, a, None, mean, rstd, dx=b))
    assert torch.equal(buf, before)
    norm.forward(wide[:1], y=dense[:1])             # one row has no stride


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("width", [96, 1601, 9001, 16_400])
def test_dx_in_the_place_of_x(width, dtype):
    g = torch.Generator(device="cuda").manual_seed(width)
    x, dy = (torch.randn(500, width, device="cuda", generator=g).to(dtype) for _ in range(2))
    norm = FusedLayerNorm(width)
    _, mean, rstd = norm.forward(x)
    want = norm.backward(dy, x, None, mean, rstd)
    got = norm.backward(dy, x, None, mean, rstd, dx=x)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
