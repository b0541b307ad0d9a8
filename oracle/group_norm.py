"""Float64 definition of group norm with an activation, channels last (numpy)."""

from __future__ import annotations

import numpy as np


def _sigmoid(z):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-z))


def _spread(t, channels):
    """Per group to per channel: [samples, groups] -> [samples, 1, channels]."""
    return np.repeat(t, channels // t.shape[1], 1)[:, None, :]


def forward(x, groups, weight=None, bias=None, eps=1e-5, silu=False):
    """(y, mean, rstd) of x [samples, positions, channels]"""
    n, length, c = x.shape
    split = x.reshape(n, length, groups, c // groups)
    mean = split.mean((1, 3))
    rstd = 1 / np.sqrt(((split - mean[:, None, :, None]) ** 2).mean((1, 3)) + eps)
    z = (x - _spread(mean, c)) * _spread(rstd, c)
    if weight is not None:
        z = z * weight
    if bias is not None:
        z = z + bias
    return (z * _sigmoid(z) if silu else z), mean, rstd


def backward(dy, x, groups, weight, bias, mean, rstd, silu=False):
    """(dx, dweight, dbias)"""
    n, length, c = x.shape
    xhat = (x - _spread(mean, c)) * _spread(rstd, c)
    w = np.ones(c) if weight is None else weight
    dz = dy
    if silu:
        z = xhat * w + (0 if bias is None else bias)
        s = _sigmoid(z)
        dz = dy * s * (1 + z * (1 - s))
    per = lambda t: _spread(t.reshape(n, length, groups, c // groups).mean((1, 3)), c)  # noqa: E731
    dx = _spread(rstd, c) * (dz * w - per(dz * w) - xhat * per(dz * w * xhat))
    return dx, (dz * xhat).sum((0, 1)), dz.sum((0, 1))
