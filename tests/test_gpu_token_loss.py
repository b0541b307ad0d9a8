"""GPU: token log-probabilities, the clipped policy loss and the preference loss
against the float64 definitions.

Tolerances (u = 2^-24).  In base 2 a token's log-probability is
fma(z, k, -c) - log2 S: k, the fma and c's use round by u of a value of at most
|logp| + log S over ln 2, S (exponentials good to 2^-22, short sums) by about
2^-21 relative, log2 and the last product by an ulp or two: together under
2^-20 + 3 u (|logp| + log V) in natural units, doubled below as `lp_tol`.
A probability is exp of that argument: relative error lp_tol + 2^-21.  A row's
slope adds a ratio (lp_tol again) and the KL factor: `REL` = 2e-5 of the
gradient's terms covers |logp| up to 60.  16-bit gradients add half an ulp.
"""

import numpy as np
import pytest
import torch

from adamw_optimizer_step_tensor_gb300 import AdamWError, FusedTokenLoss, _capi
from oracle import token_loss as TL

from _support import assert_guards_intact, dev, empty, guarded_empty, scalar_f32

pytestmark = pytest.mark.gpu
HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126}
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
REL = 2e-5
f32 = np.float32


def wide(t):
    return t.detach().double().cpu().numpy()


def lp_tol(logp, vocab):
    return 2.0 ** -19 + 6 * 2.0 ** -24 * (np.abs(logp) + np.log(vocab) + 1)


def rows_of(a, dtype, pad=0, shift=0):
    r, c = a.shape
    t = guarded_empty(r * (c + pad), dtype, shift).view(r, c + pad)
    t.fill_(3.0)
    t = t[:, :c]
    t.copy_(torch.from_numpy(a.astype(f32)))
    return t


def grad_rows(z, pad, shift):
    r, c = z.shape
    t = guarded_empty(r * (c + pad), z.dtype, shift).view(r, c + pad)
    t.fill_(3.0)
    return t[:, :c], t[:, c:]


class Batch:
    """Logits with a likely token per row, labels, weights and per-row inputs."""

    def __init__(self, rows, vocab, dtype, seed=0, pad=0, shift=0, masked=0.3, labels=torch.int64, spread=2.0,
                 edit=None):
        rng = self.rng = np.random.default_rng(seed + 1000 * rows + vocab)
        z = rng.normal(0, spread, (rows, vocab))
        y = rng.integers(0, vocab, rows)
        z[np.arange(rows), y] += rng.uniform(0, 8, rows)
        w = np.where(rng.random(rows) < masked, 0.0, rng.uniform(0.2, 1, rows)) / max(1, rows)
        if edit is not None:
            edit(z, y, w, rng)
        self.logits = rows_of(z, dtype, pad, shift)
        self.Z = wide(self.logits)
        self.y, self.labels = y, dev(y.astype(np.int64 if labels == torch.int64 else np.int32))
        self.w = self.vec(w)
        self.rows, self.vocab, self.dtype = rows, vocab, dtype
        self.dz, self.gap = grad_rows(self.logits, pad, shift)

    def vec(self, a):
        return dev(np.asarray(a, f32))

    def policy_inputs(self, temperature=1.0, clip=(0.2, 0.28)):
        rng = self.rng
        lp, _ = TL.logps(self.Z, self.y, temperature)
        lp = np.where(np.isfinite(lp), lp, 0.0)
        delta = rng.normal(0, 0.2, self.rows)
        for edge in (np.log(1 - clip[0]), np.log(1 + clip[1])):      # no ratio right at a bound
            near = np.abs(delta - edge) < 1e-3
            delta[near] = edge + 2e-3
        return self.vec(rng.normal(0.3, 1, self.rows)), self.vec(lp - delta), self.vec(lp + rng.normal(0, 0.3, self.rows))


def check_grad(b, dz, slopes, live, sizes, temperature=1.0, scale=1.0):
    """dz against the definition; sizes[t] bounds the magnitude of the terms of slope t."""
    want = scale * TL.dlogits(b.Z, b.y, slopes, live, temperature)
    lsm, _ = TL.log_softmax(b.Z, temperature)
    with np.errstate(invalid="ignore"):
        p = np.where(live[:, None], np.exp(lsm), 0.0)
    t = np.nonzero(live)[0]
    p[t, b.y[t]] += 1
    size = scale / temperature * p * np.maximum(sizes, np.abs(slopes))[:, None]
    got = wide(dz)
    bound = REL * size + HALF_ULP[b.dtype] * (np.abs(want) + REL * size) + TINY[b.dtype]
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])
    assert not got[~live].any()
    assert (b.gap == 3.0).all()
    assert_guards_intact()


def check_policy(b, temperature=1.0, kl=0.05, old=True, ref=True, scale=None, clip=(0.2, 0.28), in_place=False):
    adv, old_lp, ref_lp = b.policy_inputs(temperature, clip)
    old_lp, ref_lp = old_lp if old else None, ref_lp if ref else None
    stats, lp = empty(4), empty(b.rows)
    want = TL.policy(b.Z, b.y, wide(b.w), wide(adv), wide(old_lp) if old else None, wide(ref_lp) if ref else None,
                     tuple(map(float, map(f32, clip))), float(f32(kl)), temperature)
    dz = b.logits if in_place else b.dz
    FusedTokenLoss(b.rows).policy(
        b.logits, b.labels, b.w, adv, old_lp, ref_lp, clip=clip, kl_coef=kl if ref else 0.0, temperature=temperature,
        grad_scale=None if scale is None else scalar_f32(scale), stats=stats, logps=lp, dlogits=dz)
    torch.cuda.synchronize()
    assert np.all(np.abs(wide(lp) - want["logps"]) <= lp_tol(want["logps"], b.vocab))
    s = want["stats"]
    if not ref:
        s = np.array([s[1], s[1], 0.0, s[3]])
    assert np.all(np.abs(wide(stats) - s) <= REL * (want["size"] + np.abs(s))), (wide(stats), s)
    check_grad(b, dz, want["slopes"], want["live"], want["terms"], temperature, scale or 1.0)


VOCABS = [1, 2, 7, 8, 33, 500, 1003, 2048, 4096, 5001, 8192, 16_411, 32_000, 50_257, 131_075]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", VOCABS)
def test_policy_vocabularies(vocab, dtype):
    check_policy(Batch(11, vocab, dtype))


@pytest.mark.parametrize("rows", [1, 2, 3, 37, 153, 400])
@pytest.mark.parametrize("vocab", [129, 3001, 20_000])
def test_policy_rows(rows, vocab):
    check_policy(Batch(rows, vocab, torch.bfloat16, masked=0.0 if rows < 3 else 0.3))


@pytest.mark.parametrize("vocab", [3, 100, 1000, 20_011])
def test_policy_many_rows(vocab):
    check_policy(Batch(5000 if vocab < 2000 else 700, vocab, torch.float32, masked=0.5))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [77, 1000, 8200, 40_003])
@pytest.mark.parametrize("pad,shift", [(1, 0), (8, 0), (0, 1), (5, 3)])
def test_policy_strides_and_alignment(vocab, dtype, pad, shift):
    check_policy(Batch(7, vocab, dtype, pad=pad, shift=shift))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [77, 8200, 40_003])
def test_gradient_with_another_layout_than_the_logits(vocab, dtype):
    b = Batch(6, vocab, dtype, pad=3)
    b.dz, b.gap = grad_rows(b.logits, 6, 1)
    check_policy(b)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [77, 8200, 40_003, 131_075])
def test_policy_in_place(vocab, dtype):
    check_policy(Batch(9, vocab, dtype), in_place=True)


@pytest.mark.parametrize("kw", [dict(old=False), dict(ref=False), dict(old=False, ref=False), dict(kl=0.0),
                                dict(temperature=0.6), dict(temperature=1.7), dict(scale=512.0),
                                dict(clip=(0.0, 0.0)), dict(clip=(1.0, 9.0))])
def test_policy_options(kw):
    for vocab in (700, 24_001):
        check_policy(Batch(21, vocab, torch.float32), **kw)


def test_int32_labels_and_labels_outside():
    def edit(z, y, w, rng):
        y[1], y[4], y[7] = -100, z.shape[1], -1
    for vocab in (90, 20_011):
        check_policy(Batch(12, vocab, torch.bfloat16, labels=torch.int32, edit=edit))
        check_policy(Batch(12, vocab, torch.bfloat16, edit=edit))


def test_every_row_masked():
    for vocab in (90, 20_011):
        b = Batch(5, vocab, torch.float32, masked=1.0)
        check_policy(b)
        assert not wide(b.dz).any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("low", ["inf", "lowest"])
def test_masked_columns(low, dtype):
    """Columns of -inf or of the type's lowest value have probability 0 and gradient 0."""
    value = -np.inf if low == "inf" else float(torch.finfo(dtype).min)

    def edit(z, y, w, rng):
        hit = rng.random(z.shape) < 0.4
        hit[0] = True                       # only the token is left
        hit[np.arange(len(y)), y] = False
        z[hit] = value
        z[3, : z.shape[1] // 2] = value     # a whole stretch, from the row's start
        z[3, y[3]] = 1.0
    for vocab in (300, 9001, 50_257):
        check_policy(Batch(8, vocab, dtype, edit=edit, masked=0.0))


def test_nan_in_masked_rows_stays_out():
    def edit(z, y, w, rng):
        w[2], y[5] = 0.0, -100
    for vocab in (300, 50_257):
        b = Batch(8, vocab, torch.float32, edit=edit, masked=0.0)
        b.logits[2] = float("nan")
        b.logits[5, 7] = float("inf")
        check_policy(b)


def test_undefined_rows_are_nan_and_alone():
    """A NaN or +inf logit, or nothing but -inf, makes its own row NaN and no other."""
    for vocab in (300, 50_257):
        b = Batch(6, vocab, torch.float32, masked=0.0)
        loss = FusedTokenLoss(6)
        clean, _ = loss.logps(b.logits, b.labels)
        b.logits[1, 4], b.logits[3, 9], b.logits[4] = float("nan"), float("inf"), -float("inf")
        lp, lse = loss.logps(b.logits, b.labels)
        bad = torch.tensor([0, 1, 0, 1, 1, 0], dtype=torch.bool, device="cuda")
        assert torch.isnan(lp[bad]).all() and torch.equal(lp[~bad], clean[~bad])


def test_a_token_of_probability_zero():
    def edit(z, y, w, rng):
        z[2, y[2]] = -np.inf
    for vocab in (300, 50_257):
        b = Batch(4, vocab, torch.float32, edit=edit, masked=0.0)
        lp, _ = FusedTokenLoss(4).logps(b.logits, b.labels)
        want, _ = TL.logps(b.Z, b.y)
        assert lp[2].item() == -np.inf and want[2] == -np.inf
        assert np.all(np.abs(np.delete(wide(lp) - want, 2)) <= lp_tol(np.delete(want, 2), vocab))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab", [(1, 1), (1, 128_256), (3, 50_257), (7, 17_000), (500, 100), (64, 4097)])
def test_logps(rows, vocab, dtype):
    b = Batch(rows, vocab, dtype, pad=2)
    lp, lse = empty(rows), empty(rows)
    FusedTokenLoss(rows).logps(b.logits, b.labels, temperature=0.8, logps=lp, lse=lse)
    want, wl = TL.logps(b.Z, b.y, float(f32(0.8)))
    assert_guards_intact()
    assert np.all(np.abs(wide(lp) - want) <= lp_tol(want, vocab))
    assert np.all(np.abs(wide(lse) - wl) <= lp_tol(wl, vocab))


def test_probability_zero_at_any_temperature():
    """-inf stays probability 0 whatever the sign of the rounding of 1 / temperature."""
    def edit(z, y, w, rng):
        hit = rng.random(z.shape) < 0.3
        hit[np.arange(len(y)), y] = False
        z[hit] = -np.inf
    for vocab in (300, 20_011):
        for temperature in (0.3, 0.5, 0.7, 0.9, 1.1, 1.3, 2.0, 3.0):
            b = Batch(4, vocab, torch.float32, edit=edit, masked=0.0)
            check_policy(b, temperature=float(f32(temperature)))


def test_plan_status_is_clear():
    b = Batch(30, 40_003, torch.bfloat16)
    adv, old, ref = b.policy_inputs()
    loss = FusedTokenLoss(30, 1)
    loss.policy(b.logits, b.labels, b.w, adv, old, ref)
    loss.preference(b.logits, b.labels, None, ref, dev(np.array([0, 9, 30], np.int32)))
    assert loss.status() == 0


@pytest.mark.parametrize("dtype,vocab", [(torch.bfloat16, 300_007), (torch.float32, 430_001), (torch.bfloat16, 860_003)])
def test_very_large_vocabularies(dtype, vocab):
    """Rows of more slots than one CTA's, and rows that do not fit a cluster's shared memory."""
    b = Batch(5, vocab, dtype, masked=0.2)
    check_policy(b)
    check_preference(b, np.array([0, 2, 5], np.int32))


def test_losses_of_a_token_of_probability_zero():
    """An infinite log ratio stays in its pair's numbers: no NaN where the definition has none."""
    def edit(z, y, w, rng):
        z[1, y[1]] = -np.inf
    for vocab in (300, 40_003):
        b = Batch(8, vocab, torch.float32, edit=edit, masked=0.0)
        ref = b.vec(np.full(8, -5.0))
        loss = FusedTokenLoss(8, 2)
        inf, one = float("inf"), torch.ones(8, device="cuda")
        # row 1 in the first chosen sequence
        stats, rewards, _, dz = loss.preference(b.logits, b.labels, None, ref, dev(np.array([0, 2, 4, 6, 8], np.int32)))
        assert float(rewards[0]) == -inf and torch.isfinite(rewards[1:]).all()
        assert float(stats[0]) == inf and float(stats[2]) == -inf and torch.isfinite(dz[2:]).all()
        # and in the first rejected one: the pair is won
        stats, rewards, _, dz = loss.preference(b.logits, b.labels, None, ref, dev(np.array([2, 4, 6, 6, 8], np.int32)))
        stats2, rewards2, _, dz2 = loss.preference(
            b.logits.roll(6, 0), b.labels.roll(6, 0), None, ref, dev(np.array([0, 2, 4, 8, 8], np.int32)))
        assert torch.isfinite(stats).all() and torch.isfinite(dz).all()
        assert float(rewards2[2]) == -inf and torch.isfinite(stats2[:3]).all() and torch.isfinite(dz2).all()
        # the policy's KL is infinite, its clipped part is not; without a coefficient nothing is
        stats, _, _ = loss.policy(b.logits, b.labels, one, one, ref, ref, kl_coef=0.1, backward=False)
        assert torch.isfinite(stats[1]) and float(stats[2]) == inf and float(stats[0]) == inf
        stats, _, dz = loss.policy(b.logits, b.labels, one, one, ref, ref, kl_coef=0.0)
        assert torch.isfinite(stats[:2]).all() and torch.isfinite(dz).all()


def test_large_logits():
    """Logits of several hundred: the softmax depends on differences alone."""
    for vocab in (500, 30_000):
        b = Batch(6, vocab, torch.float32, spread=1.0, edit=lambda z, y, w, rng: z.__iadd__(400.0), masked=0.0)
        lp, _ = FusedTokenLoss(6).logps(b.logits, b.labels)
        want, _ = TL.logps(b.Z, b.y)
        assert np.all(np.abs(wide(lp) - want) <= lp_tol(want, vocab) + 2.0 ** -24 * 400)


def starts_of(rows, pairs, rng, tail=0):
    cut = np.sort(rng.integers(0, rows - tail + 1, 2 * pairs - 1))
    return np.concatenate([[0], cut, [rows - tail]]).astype(np.int32)


def check_preference(b, starts, beta=0.1, smoothing=0.05, temperature=1.0, scale=None, weights=True):
    pairs = (len(starts) - 1) // 2
    w = b.w * b.rows if weights else None
    lp, _ = TL.logps(b.Z, b.y, temperature)
    ref = b.vec(np.where(np.isfinite(lp), lp, 0) + b.rng.normal(0, 0.3, b.rows))
    want = TL.preference(b.Z, b.y, wide(w) if weights else None, wide(ref), starts, float(f32(beta)),
                         float(f32(smoothing)), temperature)
    stats, rewards, got_lp = empty(4), empty(2 * pairs), empty(b.rows)
    FusedTokenLoss(b.rows, pairs).preference(
        b.logits, b.labels, w, ref, dev(starts), beta=beta, label_smoothing=smoothing, temperature=temperature,
        grad_scale=None if scale is None else scalar_f32(scale), stats=stats, rewards=rewards, logps=got_lp,
        dlogits=b.dz)
    torch.cuda.synchronize()
    assert np.all(np.abs(wide(got_lp) - want["logps"]) <= lp_tol(want["logps"], b.vocab))
    # a reward is off by at most its rows' errors
    each = np.array([lp_tol(want["logps"][s:e], b.vocab).sum() for s, e in zip(starts, starts[1:])])
    tol = beta * each + 2.0 ** -23 * np.abs(want["rewards"])
    assert np.all(np.abs(wide(rewards) - want["rewards"]) <= tol)
    assert np.all(np.abs(wide(stats) - want["stats"]) <= 2 * tol.max() + 2.0 ** -23 * (1 + np.abs(want["stats"])))
    # the slope's error is at most a quarter of the margin's, times beta / pairs
    sizes = np.abs(want["slopes"]) + (0.25 * 2 * tol.max() * beta / pairs * (wide(w) if weights else 1.0)) / REL
    check_grad(b, b.dz, want["slopes"], want["live"], sizes, temperature, scale or 1.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [1, 9, 500, 4099, 20_000, 50_257])
def test_preference_vocabularies(vocab, dtype):
    b = Batch(23, vocab, dtype)
    check_preference(b, starts_of(23, 2, b.rng, 1))


@pytest.mark.parametrize("rows,pairs", [(2, 1), (5, 4), (600, 1), (600, 37), (1500, 160)])
def test_preference_pairs(rows, pairs):
    for vocab in (65, 17_001):
        b = Batch(rows if vocab < 1000 else min(rows, 160), vocab, torch.bfloat16)
        check_preference(b, starts_of(b.rows, pairs, b.rng))


@pytest.mark.parametrize("kw", [dict(weights=False), dict(beta=1.3), dict(smoothing=0.0), dict(temperature=0.7),
                                dict(scale=256.0)])
def test_preference_options(kw):
    for vocab in (700, 24_001):
        b = Batch(40, vocab, torch.float32)
        check_preference(b, starts_of(40, 3, b.rng, 2), **kw)


def test_preference_of_empty_sequences():
    b = Batch(6, 100, torch.float32)
    check_preference(b, np.array([0, 0, 6, 6, 6], np.int32))
    b = Batch(4, 100, torch.float32)
    stats, rewards, lp, dz = FusedTokenLoss(4, 1).preference(b.logits, b.labels, None, b.w, dev(np.zeros(3, np.int32)))
    assert stats[0].item() == pytest.approx(np.log(2)) and not rewards.any() and not dz.any()


def test_sequence_starts_outside_the_rows_touch_nothing_else():
    """Starts are device data nobody can check beforehand: they are clamped to the rows."""
    b = Batch(8, 64, torch.float32, masked=0.0)
    for starts in ([-5, 3, 900], [8, 4, 2], [3, 1000, -7]):
        out = FusedTokenLoss(8, 1).preference(b.logits, b.labels, None, b.w, dev(np.array(starts, np.int32)),
                                              dlogits=b.dz)
        torch.cuda.synchronize()
        assert all(torch.isfinite(t).all() for t in out)
        assert_guards_intact()


def test_forward_alone():
    for vocab in (300, 20_011):
        b = Batch(12, vocab, torch.bfloat16)
        adv, old, ref = b.policy_inputs()
        loss = FusedTokenLoss(12, 2)
        full = loss.policy(b.logits, b.labels, b.w, adv, old, ref, kl_coef=0.1)
        part = loss.policy(b.logits, b.labels, b.w, adv, old, ref, kl_coef=0.1, backward=False)
        assert part[2] is None and torch.equal(full[0], part[0]) and torch.equal(full[1], part[1])
        starts = dev(np.array([0, 3, 6, 9, 12], np.int32))
        full = loss.preference(b.logits, b.labels, None, ref, starts)
        part = loss.preference(b.logits, b.labels, None, ref, starts, backward=False)
        assert part[3] is None and all(torch.equal(a, c) for a, c in zip(full[:3], part[:3]))


def test_no_rows():
    loss = FusedTokenLoss(4, 1)
    z, y, v = torch.empty(0, 50, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    assert loss.logps(z, y)[0].numel() == 0
    stats, _, dz = loss.policy(z, y, v, v)
    assert not stats.any() and dz.shape == (0, 50)
    stats, rewards, _, _ = loss.preference(z, y, None, v, torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert stats[0].item() == pytest.approx(np.log(2)) and not rewards.any()


@pytest.mark.parametrize("vocab", [200, 5000, 40_000])
def test_results_are_the_same_bits_every_time(vocab):
    b = Batch(300, vocab, torch.bfloat16)
    adv, old, ref = b.policy_inputs()
    loss = FusedTokenLoss(300, 3)
    starts = dev(starts_of(300, 3, b.rng))
    first = [t.clone() for t in (*loss.policy(b.logits, b.labels, b.w, adv, old, ref, kl_coef=0.1),
                                 *loss.preference(b.logits, b.labels, b.w, ref, starts))]
    for _ in range(5):
        again = (*loss.policy(b.logits, b.labels, b.w, adv, old, ref, kl_coef=0.1),
                 *loss.preference(b.logits, b.labels, b.w, ref, starts))
        assert all(torch.equal(a, c) for a, c in zip(first, again))


def test_one_plan_serves_other_shapes_and_streams():
    loss = FusedTokenLoss(400, 2)
    s = torch.cuda.Stream()
    for rows, vocab in ((400, 50), (3, 60_000), (120, 9000), (1, 7)):
        b = Batch(rows, vocab, torch.float32)
        s.wait_stream(torch.cuda.current_stream())
        lp, lse = loss.logps(b.logits, b.labels, stream=s)
        s.synchronize()
        want, _ = TL.logps(b.Z, b.y)
        assert np.all(np.abs(wide(lp) - want) <= lp_tol(want, vocab))


def test_graph_replay():
    b = Batch(64, 20_000, torch.bfloat16)
    adv, old, ref = b.policy_inputs()
    loss = FusedTokenLoss(64)
    want = [t.clone() for t in loss.policy(b.logits, b.labels, b.w, adv, old, ref, kl_coef=0.1)]
    out = [torch.zeros_like(t) for t in want]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss.policy(b.logits, b.labels, b.w, adv, old, ref, kl_coef=0.1, stats=out[0], logps=out[1], dlogits=out[2])
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(want, out))


@pytest.mark.parametrize("vocab", [3000, 40_000])
def test_preference_graph_replay(vocab):
    """The three launches overlap at their ends; replayed back to back they give the same bits."""
    b = Batch(400, vocab, torch.bfloat16)
    ref = b.policy_inputs()[2]
    loss = FusedTokenLoss(400, 7)
    starts = dev(starts_of(400, 7, b.rng))
    want = [t.clone() for t in loss.preference(b.logits, b.labels, b.w, ref, starts)]
    out = [torch.zeros_like(t) for t in want]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            loss.preference(b.logits, b.labels, b.w, ref, starts, stats=out[0], rewards=out[1], logps=out[2],
                            dlogits=out[3])
    for _ in range(5):
        for t in out:
            t.fill_(-1.0)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, out))


def test_offsets_past_32_bits():
    rows, vocab = 17_000, 128_256           # 2.18e9 logits
    logits = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    labels = torch.full((rows,), -100, dtype=torch.int64, device="cuda")
    some = [0, 16_743, 16_744, rows - 1]    # on both sides of element 2^31
    g = torch.Generator(device="cuda").manual_seed(2)
    for t in some:
        logits[t] = torch.randn(vocab, device="cuda", generator=g).to(torch.bfloat16)
        labels[t] = 100 + t % 1000
    w = torch.ones(rows, device="cuda")
    loss = FusedTokenLoss(rows, 1)
    stats, lp, dz = loss.policy(logits, labels, w, w)
    sub = FusedTokenLoss(4, 1)
    s2, lp2, dz2 = sub.policy(logits[some].contiguous(), labels[some], w[:4].contiguous(), w[:4].contiguous())
    assert torch.equal(lp[some], lp2) and torch.equal(dz[some], dz2)
    assert stats[0].item() == pytest.approx(s2[0].item())
    assert int(torch.count_nonzero(dz.view(torch.int16).any(1))) == 4
    starts = torch.tensor([0, 16_744, rows], dtype=torch.int32, device="cuda")
    ref = torch.zeros(rows, device="cuda")
    _, rewards, _, dz3 = loss.preference(logits, labels, w, ref, starts, dlogits=dz)
    starts2 = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    _, rewards2, _, dz4 = sub.preference(logits[some].contiguous(), labels[some], w[:4].contiguous(),
                                         ref[:4].contiguous(), starts2)
    assert torch.equal(rewards, rewards2) and torch.equal(dz3[some], dz4)


def test_differences():
    """dlogits against central differences of the library's own loss."""
    for vocab in (40, 20_011):
        b = Batch(5, vocab, torch.float32, masked=0.0)
        b.w.fill_(0.2)
        adv, old, ref = b.policy_inputs()
        loss = FusedTokenLoss(5)
        run = lambda z: loss.policy(z, b.labels, b.w, adv, old, ref, kl_coef=0.5)  # noqa: E731
        _, _, dz = run(b.logits)
        h = 2.0 ** -4      # the loss is good to about 1e-6, so a quotient to 1e-6 / h + O(h^2)
        for t in range(5):
            c = int(b.labels[t])
            up, down = b.logits.clone(), b.logits.clone()
            up[t, c] += h
            down[t, c] -= h
            su, sd = run(up)[0], run(down)[0]
            if su[3] != sd[3]:
                continue        # the step crossed a clip bound
            assert abs(float(su[0].double() - sd[0].double()) / (2 * h) - float(dz[t, c])) < 2e-3


def test_refusals():
    z, y = torch.zeros(4, 50, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    v, starts = torch.zeros(4, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    loss = FusedTokenLoss(4, 1)

    def status(fn):
        with pytest.raises(AdamWError) as e:
            fn()
        return e.value.status

    assert status(lambda: FusedTokenLoss(3).logps(z, y)) == _capi.EINVAL
    for t in (0.0, -1.0, float("nan"), float("inf")):
        assert status(lambda: loss.logps(z, y, temperature=t)) == _capi.EINVAL
    for clip in ((-0.1, 0.2), (1.1, 0.2), (0.2, -0.1), (float("nan"), 0.2)):
        assert status(lambda: loss.policy(z, y, v, v, clip=clip)) == _capi.EINVAL
    assert status(lambda: loss.policy(z, y, v, v, kl_coef=0.1)) == _capi.EINVAL      # no ref_logps
    assert status(lambda: loss.policy(z, y, v, v, v, v, kl_coef=-0.1)) == _capi.EINVAL
    assert status(lambda: FusedTokenLoss(4).preference(z, y, v, v, starts)) == _capi.EINVAL
    for kw in (dict(beta=0.0), dict(beta=float("nan")), dict(label_smoothing=0.5), dict(label_smoothing=-0.1)):
        assert status(lambda: loss.preference(z, y, v, v, starts, **kw)) == _capi.EINVAL
    with pytest.raises(TypeError, match="logits dtype"):
        loss.logps(z.double(), y)
    with pytest.raises(TypeError, match="int32 or int64"):
        loss.logps(z, v)
    with pytest.raises(TypeError, match="weights"):
        loss.policy(z, y, v.half(), v)
    with pytest.raises(ValueError, match="4 elements"):
        loss.policy(z, y, v[:3], v)
    with pytest.raises(ValueError, match="shape"):
        loss.policy(z, y, v, v, dlogits=torch.zeros(4, 49, device="cuda"))
    with pytest.raises(TypeError, match="dlogits"):
        loss.policy(z, y, v, v, dlogits=torch.zeros(4, 50, device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError, match="last axis"):
        loss.logps(torch.zeros(50, 4, device="cuda").t(), y)
    with pytest.raises(ValueError, match="elements"):
        loss.preference(z, y, v, v, torch.zeros(4, dtype=torch.int32, device="cuda"))
    rec = _capi.adamw_logits(z.data_ptr(), y.data_ptr(), 4, 49, 50, 8, 0, 1.0)
    assert status(lambda: _capi.adamw_token_logps(loss.plan, rec, v.data_ptr(), None, None)) == _capi.EINVAL
    rec = _capi.adamw_logits(z.data_ptr(), y.data_ptr(), 4, 50, 50, 2, 0, 1.0)
    assert status(lambda: _capi.adamw_token_logps(loss.plan, rec, v.data_ptr(), None, None)) == _capi.EDTYPE
    rec = _capi.adamw_logits(z.data_ptr(), y.data_ptr(), 4, 50, 50, 8, 7, 1.0)
    assert status(lambda: _capi.adamw_token_logps(loss.plan, rec, v.data_ptr(), None, None)) == _capi.EDTYPE
    rec = _capi.adamw_logits(z.data_ptr() + 2, y.data_ptr(), 4, 50, 50, 8, 0, 1.0)
    assert status(lambda: _capi.adamw_token_logps(loss.plan, rec, v.data_ptr(), None, None)) == _capi.EALIGN
