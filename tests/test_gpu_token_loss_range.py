"""GPU: the token losses over the whole range of finite logits -- masks of large
finite values, rows of nothing else, tokens behind a mask, large positive rows --
against the float64 definitions, with the bounds of test_gpu_token_loss.py.

A log-probability beyond float32 rounds to -inf; one of a token far below its row
is its logit over the temperature but for two roundings, which `lp_tol`'s
6 u |logp| covers.
"""

import numpy as np
import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import FusedTokenLoss
from oracle import token_loss as TL
from test_gpu_token_loss import Batch, check_grad, check_policy, check_preference, f32, lp_tol, starts_of, wide

from _support import dev

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
VALUES = [-1e9, -1e10, -1e12, -1e20, -1e30, "lowest"]


def values_of(dtype):
    """The mask values that dtype holds as finite numbers."""
    low = float(torch.finfo(dtype).min)
    return [low if v == "lowest" else v for v in VALUES if v == "lowest" or v >= low]


def fill(b, z, temperature):
    """Puts z into the batch; returns float64 log-probabilities and log sums."""
    b.logits.copy_(torch.from_numpy(z.astype(f32)))
    b.Z = wide(b.logits)
    return TL.logps(b.Z, b.y, temperature)


def near(got, want, tol):
    with np.errstate(over="ignore", invalid="ignore"):
        want32 = want.astype(f32).astype(np.float64)
        ok = (got == want32) | (np.abs(got - want) <= tol)
    assert ok.all(), (got[~ok][:5], want[~ok][:5])


def check_rows(b, temperature):
    """Log-probabilities, and the gradient of a policy loss without a sampler's or a reference's log-probabilities."""
    want, lse = TL.logps(b.Z, b.y, temperature)
    loss = FusedTokenLoss(b.rows)
    lp, got_lse = loss.logps(b.logits, b.labels, temperature=temperature)
    near(wide(lp), want, lp_tol(want, b.vocab))
    near(wide(got_lse), lse, lp_tol(lse, b.vocab))
    adv = b.vec(b.rng.normal(0.3, 1, b.rows))
    stats, _, _ = loss.policy(b.logits, b.labels, b.w, adv, temperature=temperature, dlogits=b.dz)
    size = wide(b.w) * np.abs(wide(adv))
    check_grad(b, b.dz, -wide(b.w) * wide(adv), TL.live_rows(b.y, b.vocab, wide(b.w)), size, temperature)
    s = -np.sum(wide(b.w) * wide(adv))
    assert abs(float(stats[0]) - s) <= 2e-5 * size.sum()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [300, 9001, 50_257, 128_256])
def test_finite_masks(vocab, dtype):
    """Masked columns, whole stretches of them among the rest, have probability 0."""
    b = Batch(4, vocab, dtype, masked=0.0)
    base, at = b.Z.copy(), np.arange(4)
    hit = b.rng.random(base.shape) < 0.4
    hit[0] = True                               # only the token is left
    hit[1, : vocab // 2] = True                 # a whole stretch
    hit[3] = np.arange(vocab) % 512 < 256       # whole threads
    hit[at, b.y] = False
    for value in values_of(dtype):
        for temperature in (0.5, 1.0, 2.0, 4.0):
            fill(b, np.where(hit, value, base), temperature)
            check_rows(b, temperature)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [1, 7, 300, 9001, 50_257])
def test_rows_of_one_finite_value(vocab, dtype):
    """A mask that leaves nothing: every token is as likely; so it is at the other end."""
    b = Batch(3, vocab, dtype, masked=0.0)
    for value in values_of(dtype) + [-v for v in values_of(dtype)]:
        for temperature in (0.1, 1.0, 4.0):
            fill(b, np.full((3, vocab), value), temperature)
            check_rows(b, temperature)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [300, 9001, 50_257])
def test_rows_far_from_zero(vocab, dtype):
    """Rows that lie far out as a whole, some steps of the type apart."""
    b = Batch(4, vocab, dtype, masked=0.0)
    eps = 2.0 ** -23 if dtype == torch.float32 else 2.0 ** -7
    for at in (2.0 ** 23, 2.0 ** 24, 2.0 ** 25, 1e9, 1e30, 1.5e38):
        steps = b.rng.integers(0, 3, (4, vocab)) * eps
        for sign in (-1.0, 1.0):
            for temperature in (1.0, 3.0, 1e5):
                fill(b, sign * at * (1 + steps), temperature)
                b.y[:] = b.Z.argmax(1)
                b.labels.copy_(torch.from_numpy(b.y))
                check_rows(b, temperature)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [300, 50_257])
def test_a_token_behind_a_finite_mask(vocab, dtype):
    """Its log-probability is finite where float32 holds it."""
    b = Batch(4, vocab, dtype, masked=0.0)
    base = b.Z.copy()
    for value in values_of(dtype):
        for temperature in (0.5, 1.0, 2.0):
            z = base.copy()
            z[1, b.y[1]] = value
            z[2, :] = value
            z[2, b.y[2]] = 1.0
            z[3, b.y[3]] = value
            z[3, (b.y[3] + 1) % vocab] = 60000.0 if dtype == torch.float16 else 2.0 ** 127
            fill(b, z, temperature)
            check_rows(b, temperature)


@pytest.mark.parametrize("vocab,dtype", [(300, torch.bfloat16), (20_011, torch.float32), (50_257, torch.bfloat16),
                                         (860_003, torch.bfloat16)])
def test_losses_and_layouts_of_far_rows(vocab, dtype):
    """Every pass that sums or differentiates: in place, in another layout, the preference loss, large vocabularies."""
    low = float(torch.finfo(dtype).min)

    def edit(z, y, w, rng):
        hit = rng.random(z.shape) < 0.5
        hit[np.arange(len(y)), y] = False
        z[hit] = -1e30
        z[1], z[2], z[4, :] = low, -1e20, 1e30
    b = Batch(6, vocab, dtype, masked=0.0, edit=edit)
    check_policy(b)
    check_policy(b, temperature=2.0)
    check_preference(b, np.array([0, 2, 6], np.int32))
    check_preference(b, np.array([0, 4, 6], np.int32), temperature=4.0)
    if vocab < 100_000:
        other = Batch(6, vocab, dtype, pad=3, shift=1, masked=0.0, edit=edit)
        check_policy(other)
        check_policy(b, in_place=True)


@pytest.mark.parametrize("vocab", [3000, 50_257])
def test_far_rows_among_many(vocab):
    """Several rows per CTA, far ones next to ordinary ones and to rows without a token."""
    def edit(z, y, w, rng):
        at = np.arange(len(y))[1::7]
        token = z[at, y[at]]
        z[1::7, : z.shape[1] // 3] = -1e10
        z[at, y[at]] = token
        z[::3] = -1e12
        y[::11] = -100
    b = Batch(400, vocab, torch.bfloat16, edit=edit)
    check_policy(b)
    check_preference(b, starts_of(400, 5, b.rng))
