"""The float64 definitions of a block's operators, pinned on the CPU: Philox against its
published test vectors, gradients against central differences, group norm against torch's."""

import numpy as np
import pytest
import torch

from oracle import dropout as DR
from oracle import group_norm as GN
from oracle import router as RO

RNG = np.random.default_rng(21)


# the generator's own known answers: counter, key, words
@pytest.mark.parametrize("counter,key,want", [
    ((0,) * 4, (0,) * 2, (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))])
def test_philox_known_answers(counter, key, want):
    assert tuple(DR.philox(counter, key)) == want


def test_words_are_the_generator_element_by_element():
    seed, step, site = 0x299f31d0a4093822, -5, 7
    for first in (0, 3, 2 ** 34 - 6):
        got = DR.words(first, 11, seed, step, site)
        want = [DR.philox((i // 4 & DR.M32, i // 4 >> 32, step & DR.M32, site), (seed & DR.M32, seed >> 32))[i % 4]
                for i in range(first, first + 11)]
        assert got.tolist() == want


def test_dropout_keeps_the_mean():
    x = np.ones(200_000)
    y = DR.forward(x, None, 0.25, 99)
    assert set(np.unique(y)) == {0.0, 1 / 0.75}
    assert abs(y.mean() - 1) < 5 * np.sqrt(0.25 / 0.75 / x.size)
    assert not DR.forward(x, None, 1.0, 99).any() and (DR.forward(x, None, 0.0, 99) == 1).all()


def _differences(loss, z, h=1e-6):
    g = np.zeros_like(z)
    for i in np.ndindex(z.shape):
        up, down = z.copy(), z.copy()
        up[i] += h
        down[i] -= h
        g[i] = (loss(up) - loss(down)) / (2 * h)
    return g


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_router_gradient_is_the_difference_quotient(score, renormalise):
    z = RNG.normal(0, 1.5, (4, 12))
    z[1, 3:] = -np.inf
    z[2] = -np.inf
    dw = RNG.normal(size=(4, 4))
    _, ids, _, _ = RO.route(z, None, 4, score)

    def loss(z):
        return sum((RO.weights(z[t], ids[t][ids[t] >= 0], score, renormalise, 2.5) * dw[t][ids[t] >= 0]).sum() for t in range(4))

    got = RO.backward(dw, z, ids, score, renormalise, 2.5)
    with np.errstate(invalid="ignore"):
        want = np.where(z > -np.inf, _differences(loss, z), 0.0)
    assert np.allclose(got, want, atol=1e-7)


def test_routing_by_hand():
    z = np.log(np.array([[0.1, 0.4, 0.1, 0.4], [0.3, 0.2, 0.4, 0.1]]))
    w, ids, slots, starts = RO.route(z, None, 2)
    assert ids.tolist() == [[1, 3], [2, 0]]            # equal scores: the lowest first
    assert np.allclose(w, [[0.5, 0.5], [4 / 7, 3 / 7]])
    assert starts.tolist() == [0, 1, 2, 3, 4] and slots.tolist() == [[1, 3], [2, 0]]
    _, ids, _, _ = RO.route(z, np.array([0.0, -0.5, 0.0, 0.0]), 1)
    assert ids.tolist() == [[3], [2]]
    # groups {0, 1} and {2, 3}: by the largest, and by the sum of two
    _, ids, _, _ = RO.route(z[1:], None, 2, groups=2, top_groups=1)
    assert ids.tolist() == [[2, 3]]
    _, ids, _, _ = RO.route(np.log([[0.3, 0.25, 0.4, 0.05]]), None, 2, groups=2, top_groups=1, group_score="top2")
    assert ids.tolist() == [[0, 1]]


def test_moves_are_each_other_s_gradients():
    ids = np.array([[0, 2], [1, 0], [-1, -1], [2, 1]])
    slots, starts = RO.places(ids, 3)
    assert starts.tolist() == [0, 2, 4, 6] and slots.tolist() == [[0, 4], [2, 1], [-1, -1], [5, 3]]
    x, ys, dy, w = RNG.normal(size=(4, 3)), RNG.normal(size=(6, 3)), RNG.normal(size=(4, 3)), RNG.uniform(size=(4, 2))
    dxs = RNG.normal(size=(6, 3))
    assert np.allclose(RO.combine(dxs, slots), _differences(lambda x: (RO.dispatch(x, slots, 6) * dxs).sum(), x), atol=1e-7)
    dys, dw = RO.combine_backward(dy, ys, slots, w)
    assert np.allclose(dys, _differences(lambda ys: (RO.combine(ys, slots, w) * dy).sum(), ys), atol=1e-7)
    assert np.allclose(dw, _differences(lambda w: (RO.combine(ys, slots, w) * dy).sum(), w), atol=1e-7)


@pytest.mark.parametrize("silu", [False, True])
def test_group_norm_is_torch_s(silu):
    x = torch.randn(3, 7, 12, dtype=torch.float64, generator=torch.Generator().manual_seed(1)).requires_grad_()
    w, b = (torch.randn(12, dtype=torch.float64, generator=torch.Generator().manual_seed(s)).requires_grad_() for s in (2, 3))
    dy = torch.randn(3, 7, 12, dtype=torch.float64, generator=torch.Generator().manual_seed(4))
    y = torch.nn.functional.group_norm(x.transpose(1, 2), 4, w, b, 1e-5).transpose(1, 2)
    y = torch.nn.functional.silu(y) if silu else y
    want = torch.autograd.grad(y, (x, w, b), dy)
    n = lambda t: t.detach().numpy()  # noqa: E731
    got, mean, rstd = GN.forward(n(x), 4, n(w), n(b), silu=silu)
    assert np.allclose(got, n(y), atol=1e-12)
    for g, t in zip(GN.backward(n(dy), n(x), 4, n(w), n(b), mean, rstd, silu), want):
        assert np.allclose(g, n(t), atol=1e-11)
