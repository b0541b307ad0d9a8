"""The float64 definitions of the operators around the step, pinned on the CPU:
gradients against central differences of the definitions' own losses, the
layer norm against torch's, closed forms of the losses."""

import numpy as np
import pytest
import torch

from oracle import grad_norm as GN
from oracle import layer_norm as LN
from oracle import token_loss as TL

RNG = np.random.default_rng(11)


def _case(rows=6, vocab=9):
    z = RNG.normal(0, 2, (rows, vocab))
    y = RNG.integers(0, vocab, rows)
    y[2] = -100
    w = RNG.uniform(0.1, 1, rows)
    w[4] = 0.0
    return z, y, w


def _differences(loss, z, h=1e-5):
    g = np.zeros_like(z)
    for i in np.ndindex(z.shape):
        up, down = z.copy(), z.copy()
        up[i] += h
        down[i] -= h
        g[i] = (loss(up) - loss(down)) / (2 * h)
    return g


@pytest.mark.parametrize("temperature", [1.0, 0.7])
def test_policy_gradient_is_the_difference_quotient(temperature):
    z, y, w = _case()
    a = RNG.normal(size=6)
    lp, _ = TL.logps(z, y, temperature)
    old, ref = lp + RNG.normal(0, 0.3, 6), lp + RNG.normal(0, 0.3, 6)
    run = lambda x: TL.policy(x, y, w, a, old, ref, (0.2, 0.28), 0.05, temperature)  # noqa: E731
    out = run(z)
    got = TL.dlogits(z, y, out["slopes"], out["live"], temperature)
    assert np.allclose(got, _differences(lambda x: run(x)["stats"][0], z), atol=1e-8)
    assert not got[2].any() and not got[4].any()


def test_preference_gradient_is_the_difference_quotient():
    z, y, w = _case(rows=9)
    ref = TL.logps(z, y)[0] + RNG.normal(0, 0.5, 9)
    starts = np.array([0, 2, 5, 5, 8])          # an empty sequence, and row 8 outside all of them
    run = lambda x: TL.preference(x, y, w, ref, starts, 0.3, 0.1)  # noqa: E731
    out = run(z)
    got = TL.dlogits(z, y, out["slopes"], out["live"])
    assert np.allclose(got, _differences(lambda x: run(x)["stats"][0], z), atol=1e-8)
    assert out["rewards"][2] == 0.0 and not got[8].any()


def test_logps_are_log_softmax():
    z, y, _ = _case()
    want = torch.log_softmax(torch.from_numpy(z), 1).numpy()
    lp, lse = TL.logps(z, y)
    for t in range(6):
        if y[t] >= 0:
            assert lp[t] == pytest.approx(want[t, y[t]], rel=1e-13)
            assert lse[t] == pytest.approx(z[t, 0] - want[t, 0], rel=1e-13)
        else:
            assert lp[t] == 0.0


def test_on_policy_loss_is_minus_the_mean_advantage():
    z, y, _ = _case()
    live = y >= 0
    w, a = live / live.sum(), RNG.normal(size=6)
    out = TL.policy(z, y, w, a)
    assert out["stats"][0] == pytest.approx(-a[live].mean())
    assert out["stats"][3] == 0.0
    assert np.allclose(out["slopes"][live], -a[live] / live.sum())


def test_layer_norm_is_torchs():
    x, w, b, dy = (RNG.normal(size=s) for s in ((5, 12), 12, 12, (5, 12)))
    tx, tw, tb = (torch.from_numpy(v).requires_grad_() for v in (x, w, b))
    y = torch.nn.functional.layer_norm(tx, (12,), tw, tb, 1e-5)
    y.backward(torch.from_numpy(dy))
    got, mean, rstd = LN.forward(x, w, b, 1e-5)
    assert np.allclose(got, y.detach().numpy())
    for mine, theirs in zip(LN.backward(dy, x, w, mean, rstd), (tx.grad, tw.grad, tb.grad)):
        assert np.allclose(mine, theirs.numpy())


def test_norm_and_clip():
    g = [np.array([3.0, 0.0]), np.array([4.0])]
    assert GN.norm_and_clip(g) == (5.0, 1.0, 0.0)
    norm, scale, found = GN.norm_and_clip(g, scale=2.0, max_norm=1.0)
    assert norm == 2.5 and found == 0.0 and scale == pytest.approx(2.0 * 2.500001)
    assert GN.norm_and_clip([np.array([np.inf])], max_norm=1.0)[1:] == (np.inf, 1.0)
