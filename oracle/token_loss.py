"""Float64 definitions of the token losses and their gradients (numpy).

Inputs are float64 arrays holding the exact values of the library's inputs;
``labels`` outside [0, vocab) and rows of weight 0 count for nothing.
"""

from __future__ import annotations

import numpy as np


def log_softmax(logits, temperature=1.0):
    """(log softmax, log sum exp) per row; -inf logits have probability 0.  The log
    softmax is a sum of differences, which rows far from zero do not round away."""
    z = np.asarray(logits, np.float64)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        top = z.max(1, keepdims=True)
        below = (z - top) / temperature
        log_sum = np.log(np.exp(below).sum(1, keepdims=True))
        return below - log_sum, (top / temperature + log_sum)[:, 0]


def live_rows(labels, vocab, weights=None):
    live = (labels >= 0) & (labels < vocab)
    return live if weights is None else live & (weights != 0)


def logps(logits, labels, temperature=1.0, weights=None):
    lsm, lse = log_softmax(logits, temperature)
    live = live_rows(labels, logits.shape[1], weights)
    at = np.where(live, labels, 0)
    lp = np.where(live, lsm[np.arange(len(labels)), at], 0.0)
    return lp, np.where(live, lse, 0.0)


def dlogits(logits, labels, slopes, live, temperature=1.0):
    """slopes[t] = d loss / d logp[t]."""
    lsm, _ = log_softmax(logits, temperature)
    g = np.zeros(logits.shape)
    t = np.nonzero(live)[0]
    g[t] = -np.exp(lsm[t]) * slopes[t, None]
    g[t, labels[t]] += slopes[t]
    return g / temperature


def policy(logits, labels, weights, advantages, old=None, ref=None, clip=(0.2, 0.2), kl_coef=0.0,
           temperature=1.0):
    """dict(stats, logps, slopes, live, size): size = sum of the terms' magnitudes."""
    live = live_rows(labels, logits.shape[1], weights)
    lp, _ = logps(logits, labels, temperature, weights)
    w, a = np.where(live, weights, 0.0), np.where(live, advantages, 0.0)
    r = np.exp(lp - old) if old is not None else np.ones_like(lp)
    r = np.where(live, r, 1.0)
    plain, bounded = r * a, np.clip(r, 1 - clip[0], 1 + clip[1]) * a
    cut = bounded < plain
    term = -np.where(cut, bounded, plain)
    slope = np.where(cut, 0.0, -plain)
    kl = np.zeros_like(lp)
    if ref is not None:
        x = np.where(live, ref - lp, 0.0)
        kl = np.expm1(x) - x
        slope = slope - kl_coef * np.expm1(x)
    sums = [float(np.sum(w * v)) for v in (term, kl, cut)]
    return dict(stats=np.array([sums[0] + kl_coef * sums[1], *sums]), logps=lp, slopes=w * slope, live=live,
                size=float(np.sum(np.abs(w) * (np.abs(term) + kl + 1))),
                terms=np.abs(w) * (np.abs(plain) + kl_coef * (kl + 1)))


def preference(logits, labels, weights, ref, starts, beta=0.1, smoothing=0.0, temperature=1.0):
    pairs = (len(starts) - 1) // 2
    w = np.ones(len(labels)) if weights is None else weights
    live = live_rows(labels, logits.shape[1], w)
    lp, _ = logps(logits, labels, temperature, w)
    gap = np.where(live, w * (lp - ref), 0.0)
    rewards = np.array([beta * gap[starts[s]:starts[s + 1]].sum() for s in range(2 * pairs)])
    d = rewards[:pairs] - rewards[pairs:]
    softplus = lambda x: np.logaddexp(0.0, x)  # noqa: E731
    losses = (1 - smoothing) * softplus(-d) + smoothing * softplus(d)
    slope = (smoothing - 1 / (1 + np.exp(d))) * beta / pairs
    slopes, inside = np.zeros(len(labels)), np.zeros(len(labels), bool)
    for s in range(2 * pairs):
        rows = slice(starts[s], starts[s + 1])
        slopes[rows] = w[rows] * (slope[s] if s < pairs else -slope[s - pairs])
        inside[rows] = True
    live_grad = live & inside
    stats = np.array([losses.mean(), (d > 0).mean(), rewards[:pairs].mean(), rewards[pairs:].mean()])
    return dict(stats=stats, rewards=rewards, logps=lp, slopes=np.where(live_grad, slopes, 0.0), live=live_grad)
