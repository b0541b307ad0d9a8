"""GPU: gradient norm, clip and layer norm captured and replayed give the bits of plain calls,
with inputs that change between replays and launches that overlap at their ends."""

import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import FusedAdamW, FusedLayerNorm

pytestmark = pytest.mark.gpu


def _captured(run):
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            run()
    return g


# one launch, a column kernel beside the rows', rows wider than registers, several launches
@pytest.mark.parametrize("rows,width", [(700, 96), (700, 1601), (300, 4096), (200, 9001), (100, 20_003), (620_000, 5), (1_300_000, 5)])
def test_layer_norm(rows, width):
    x, dy = torch.empty(rows, width, device="cuda"), torch.empty(rows, width, device="cuda")
    w, b = torch.rand(width, device="cuda"), torch.rand(width, device="cuda")
    norm = FusedLayerNorm(width)
    out = [torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"),
           torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)]

    def run():
        norm.forward(x, w, b, y=out[0], mean=out[1], rstd=out[2])
        norm.backward(dy, x, w, out[1], out[2], dx=out[3], dweight=out[4], dbias=out[5])

    x.normal_(), dy.normal_()
    g = _captured(run)
    for _ in range(3):
        x.normal_(), dy.normal_()
        run()
        want = [t.clone() for t in out]
        for t in out:
            t.fill_(-1.0)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, out))
    assert norm.status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_gradient_norm_and_clip(dtype):
    sizes = [100_003, 1, 17, 4096]
    zeros = lambda: [torch.zeros(n, device="cuda") for n in sizes]  # noqa: E731
    grads, source = ([torch.zeros(n, dtype=dtype, device="cuda") for n in sizes] for _ in range(2))
    opt = FusedAdamW(zeros(), grads, zeros(), zeros(), [0.0] * 4)
    norm, scale, found = (torch.zeros(1, device="cuda") for _ in range(3))

    def run():
        for a, c in zip(grads, source):
            a.copy_(c)
        opt.grad_norm(norm, max_norm=1.0, clip_scale=scale, found_inf=found)
        opt.clip_grads(scale)

    g = _captured(run)
    for size in (1.0, 0.01, 1e-6):
        for t in source:
            t.normal_().mul_(size)
        run()
        want = [t.clone() for t in (norm, scale, found, *grads)]
        norm.fill_(-1.0), scale.fill_(-1.0), found.fill_(-1.0)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, (norm, scale, found, *grads)))
