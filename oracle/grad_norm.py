"""Float64 definition of the global gradient norm and the scale that clips (numpy)."""

from __future__ import annotations

import numpy as np


def norm_and_clip(grads, scale=1.0, max_norm=np.inf):
    """(norm, clip_scale, found_inf) over a list of float64 arrays."""
    with np.errstate(over="ignore", invalid="ignore"):
        norm = float(np.sqrt(sum(float(np.sum(g * g)) for g in grads)) / abs(scale))
        coef = min(1.0, max_norm / (norm + 1e-6)) if np.isfinite(max_norm) else 1.0
    found = not np.isfinite(norm) or norm > float(np.finfo(np.float32).max)
    return norm, (scale if coef == 1.0 else (scale / coef if coef else np.inf)), float(found)
