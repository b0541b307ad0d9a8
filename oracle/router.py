"""Float64 definition of routing to experts and of the rows' moves (numpy, token by token)."""

from __future__ import annotations

import numpy as np


def scores(z, score):
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1 / (1 + np.exp(-z))
    top = z.max()
    e = np.exp(z - top) if top > -np.inf else np.zeros_like(z)
    return e / e.sum() if e.sum() else e


def choose(z, bias, k, score, groups=1, top_groups=1, group_score="max"):
    """The experts of one token's logits, best first (fewer than k where fewer are there)."""
    s = scores(z, score)
    there = z > -np.inf
    if bias is not None:
        there = there & (bias > -np.inf)
    by_logit = bias is None or not bias.any()
    key = np.where(there, s if bias is None else s + bias, -np.inf)
    per = len(z) // groups
    allowed = np.ones(len(z), bool)
    if groups > 1 and top_groups < groups:
        of = np.full(groups, -np.inf)
        for g in range(groups):
            best = sorted(key[g * per:(g + 1) * per][there[g * per:(g + 1) * per]], reverse=True)
            if best:
                of[g] = best[0] if group_score == "max" else sum(best[:2])
        kept = [g for g in sorted(range(groups), key=lambda g: (-of[g], g))[:top_groups] if of[g] > -np.inf]
        allowed = np.repeat(np.isin(np.arange(groups), kept), per)
    order = z if by_logit else key
    ids = [e for e in sorted(range(len(z)), key=lambda e: (-order[e], e)) if there[e] and allowed[e]]
    return ids[:k]


def falling(z):
    """1 - sigmoid(z)"""
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(z))


def weights(z, ids, score, renormalise, scale=1.0):
    """Of the chosen experts, by logarithms where scores are small."""
    zc = z[ids]
    if not len(ids):
        return zc
    if renormalise:
        log = zc if score == "softmax" else -np.logaddexp(0, -zc)
        e = np.exp(log - log.max())
        return scale * e / e.sum()
    return scale * scores(z, score)[ids]


def route(z, bias, k, score="softmax", groups=1, top_groups=1, group_score="max", renormalise=True, scale=1.0):
    """(weights, ids, slots, starts) over the rows of z; -1 and 0 where there is no expert."""
    tokens, experts = z.shape
    w, ids = np.zeros((tokens, k)), np.full((tokens, k), -1)
    for t in range(tokens):
        c = choose(z[t], bias, k, score, groups, top_groups, group_score)
        ids[t, :len(c)] = c
        w[t, :len(c)] = weights(z[t], c, score, renormalise, scale)
    return (w, ids, *places(ids, experts))


def places(ids, experts):
    """(slots, starts): every assignment's place, ordered by expert and then by token."""
    slots, starts, n = np.full(ids.shape, -1), [0], 0
    for e in range(experts):
        for t, j in np.argwhere(ids == e):
            slots[t, j] = n
            n += 1
        starts.append(n)
    return slots, np.array(starts)


def backward(dw, z, ids, score="softmax", renormalise=True, scale=1.0):
    """The gradient of the logits with the choice held."""
    dz = np.zeros_like(z)
    for t in range(len(z)):
        live = ids[t] >= 0
        c, d = ids[t][live], dw[t][live]
        if not len(c):
            continue
        s = scores(z[t], score)
        if renormalise:
            w = weights(z[t], c, score, True)
            part = scale * w * (d - (d * w).sum())
            if score == "sigmoid":
                part = part * falling(z[t][c])
            np.add.at(dz[t], c, part)
        elif score == "sigmoid":
            np.add.at(dz[t], c, scale * d * s[c] * falling(z[t][c]))
        else:
            dz[t] = -s * scale * (d * s[c]).sum()
            np.add.at(dz[t], c, scale * d * s[c])
    return dz


def dispatch(x, slots, rows):
    xs = np.full((rows, x.shape[1]), np.nan)
    for t, j in np.argwhere((slots >= 0) & (slots < rows)):
        xs[slots[t, j]] = x[t]
    return xs


def combine(ys, slots, w=None):
    y = np.zeros((len(slots), ys.shape[1]))
    for t, j in np.argwhere((slots >= 0) & (slots < len(ys))):
        y[t] += ys[slots[t, j]] * (1 if w is None else w[t, j])
    return y


def combine_backward(dy, ys, slots, w):
    dys, dw = np.full(ys.shape, np.nan), np.zeros(slots.shape)
    for t, j in np.argwhere((slots >= 0) & (slots < len(ys))):
        dys[slots[t, j]] = w[t, j] * dy[t]
        dw[t, j] = dy[t] @ ys[slots[t, j]]
    return dys, dw
