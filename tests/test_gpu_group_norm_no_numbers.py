"""GPU: infinities and NaN in group norm, kernel by kernel.  By the definition an infinity makes its group's
mean infinite (of both signs, or a NaN: NaN) and its spread, rstd and outputs NaN; other groups and samples
keep what they have."""

import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import FusedGroupNorm

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
# sizes by the kernel that they get: lone positions; a CTA's registers; clusters of 1, 1, 2, 8 (and 8 backward)
# CTAs; parts of samples, with tiles of whole groups and without; one wide group
SHAPES = [((900, 1, 256), 8), ((2, 3, 24), 3), ((2, 50, 16), 4), ((32, 300, 64), 4), ((64, 64, 1280), 32), ((1, 1058, 14), 2),
          ((5, 5781, 24), 1), ((2, 5972, 40), 1), ((2, 60_000, 64), 4), ((2, 3000, 4104), 2), ((3, 5, 20_000), 1)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("shape,groups", SHAPES)
def test_values_that_are_no_numbers_stay_in_their_group(shape, groups, silu, dtype):
    n, length, c = shape
    g = torch.Generator("cuda").manual_seed(length)
    x, dy = (torch.randn(shape, device="cuda", generator=g).to(dtype) for _ in range(2))
    w = 1 + 0.1 * torch.randn(c, device="cuda", generator=g)
    norm = FusedGroupNorm(c, groups, n, activation="silu" if silu else "none")
    plain = norm.forward(x, w)
    plain_dx = norm.backward(dy, x, w, None, *plain[1:])[0]
    per = c // groups
    split = lambda t: t.view(n, length, groups, per).transpose(1, 2)  # noqa: E731
    places = [(0, 0, 0), (n - 1, length - 1, c - 1), (n // 2, length // 2, c // 2)]
    for values, mean_is in (((INF,), INF), ((-INF,), -INF), ((NAN,), NAN), ((INF, INF), INF), ((INF, -INF), NAN), ((NAN, INF), NAN)):
        for s, at, ch in places:
            bad = x.clone()
            bad[s, at, ch] = values[0]
            if len(values) == 2:                 # another of the group's values, at the other end
                first = ch // per * per
                bad[s, length - 1 - at, first + per - 1 - (ch - first)] = values[1]
                if (bad[s, :, first:first + per].isfinite().logical_not().sum()) < 2:
                    continue                     # the group's only middle value
            y, mean, rstd = norm.forward(bad, w)
            hit = torch.zeros(n, groups, dtype=torch.bool, device="cuda")
            hit[s, ch // per] = True
            got = float(mean[s, ch // per])
            assert got != got if mean_is != mean_is else got == mean_is
            assert rstd[hit].isnan().all() and split(y)[hit].isnan().all()
            assert torch.equal(mean[~hit], plain[1][~hit]) and torch.equal(rstd[~hit], plain[2][~hit])
            assert torch.equal(split(y)[~hit], split(plain[0])[~hit])
            dx, dw, db = norm.backward(dy, bad, w, None, mean, rstd)
            assert split(dx)[hit].isnan().all() and torch.equal(split(dx)[~hit], split(plain_dx)[~hit])
            of_group = torch.arange(c, device="cuda") // per == ch // per
            assert dw[of_group].isnan().all() and dw[~of_group].isfinite().all() and db[~of_group].isfinite().all()
    assert norm.status() == 0
