"""Float64 definition of layer norm, forward and backward (numpy)."""

from __future__ import annotations

import numpy as np


def forward(x, weight=None, bias=None, eps=1e-5):
    """(y, mean, rstd)"""
    mean = x.mean(1)
    rstd = 1 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def backward(dy, x, weight, mean, rstd):
    """(dx, dweight, dbias)"""
    xhat = (x - mean[:, None]) * rstd[:, None]
    g = dy if weight is None else dy * weight
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - xhat * (g * xhat).mean(1, keepdims=True))
    return dx, (dy * xhat).sum(0), dy.sum(0)
