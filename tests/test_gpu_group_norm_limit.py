"""GPU: group norm over 2^31 - 1 positions, every output against sums in 64 bits.

A thread has 2^31 / (304 256) < 27 700 positions, u = 2^-24.
Forward: values are added in runs of 64 (64 u of their magnitudes), runs without rounding errors, then 8 + 5
threads' sums and 10 + 5 parts': under 128 u of the mean magnitude for the mean.  A run's spread loses at most
128 u of itself; 433 runs join one after another, each off by u, and by the running mean's 3 u a run, 1300 u,
times twice the distance of a run's mean from it (below 2^-1 standard deviations): under 2000 u for the spread,
1000 u = 2^-14 for rstd.
Backward: a thread adds its positions one after another: 27 700 u = 1.7e-3 of the mean magnitudes, and 2^-14
for the terms.
"""

import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import FusedGroupNorm

pytestmark = pytest.mark.gpu
STEP = 1 << 27


@pytest.fixture(autouse=True)
def give_the_memory_back():
    """The library's plans take memory that torch's cache holds otherwise."""
    yield
    torch.cuda.empty_cache()


def test_every_position_of_the_longest_samples():
    n, length = 2, 2 ** 31 - 1
    g = torch.Generator("cuda").manual_seed(31)
    x, dy = (torch.empty(n, length, 1, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for s in range(n):                           # means of 1 and 2, and a dy that x has a part in
        for at in range(0, length, STEP):
            part = x[s, at:at + STEP].normal_(1.0 + s, 1.5, generator=g)
            dy[s, at:at + STEP].normal_(0.5, 0.4, generator=g).add_(part, alpha=0.25)
    w, b = torch.tensor([1.5], device="cuda"), torch.tensor([-0.25], device="cuda")
    norm = FusedGroupNorm(1, 1, n)
    y, mean, rstd = norm.forward(x, w, b)
    dx, dw, db = norm.backward(dy, x, w, b, mean, rstd)
    assert norm.status() == 0
    sums = torch.zeros(n, 3, dtype=torch.float64, device="cuda")
    pieces = [(s, at) for s in range(n) for at in range(0, length, STEP)]
    for s, at in pieces:
        part = x[s, at:at + STEP].double()
        sums[s] += torch.stack([part.sum(), part.abs().sum(), (part - 1 - s).square().sum()])
    m = sums[:, 0] / length
    r = 1 / torch.sqrt(sums[:, 2] / length - (m - torch.tensor([1.0, 2.0], device="cuda").double()) ** 2 + 1e-5)
    assert ((mean[:, 0] - m).abs() <= 128 * 2.0 ** -24 * sums[:, 1] / length).all() and (m > 0.9).all()
    assert ((rstd[:, 0] - r).abs() <= 2.0 ** -14 * r).all()
    back = torch.zeros(n, 4, dtype=torch.float64, device="cuda")
    m32, r32 = mean[:, 0].double(), rstd[:, 0].double()
    for s, at in pieces:
        want = (x[s, at:at + STEP].double() - m[s]) * r[s] * 1.5 - 0.25
        off = (y[s, at:at + STEP].double() - want).abs() - 2.0 ** -8 * want.abs()
        assert (off <= 2.0 ** -13 * (1 + want.abs())).all(), (s, at)
        xhat, d = (x[s, at:at + STEP].double() - m32[s]) * r32[s], dy[s, at:at + STEP].double()
        back[s] += torch.stack([d.sum(), (d * xhat).sum(), d.abs().sum(), (d * xhat).abs().sum()])
    a, q, a_size, q_size = (1.5 * back / length).unbind(1)
    assert (a > 0.5).all() and (q > 0.25).all()  # what a pass without them would miss
    near = 1.7e-3 + 2.0 ** -14
    for s, at in pieces:
        xhat, d = (x[s, at:at + STEP].double() - m32[s]) * r32[s], dy[s, at:at + STEP].double()
        want = r32[s] * (1.5 * d - a[s] - xhat * q[s])
        size = r32[s] * (near * (a_size[s] + xhat.abs() * q_size[s]) + 2.0 ** -20 * (1.5 * d).abs())
        off = (dx[s, at:at + STEP].double() - want).abs() - 2.0 ** -8 * want.abs()
        assert (off <= 1.01 * size).all(), (s, at)
    assert abs(dw[0] - back[:, 1].sum()) <= near * back[:, 3].sum()
    assert abs(db[0] - back[:, 0].sum()) <= near * back[:, 2].sum()
