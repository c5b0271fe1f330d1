"""fp64 oracle of layer norm and RMS norm over the last axis and of their
gradients."""

from __future__ import annotations

from typing import Optional, Tuple

import numpy as np


def norm_forward(x, weight, bias, kind: str, eps: float) -> Tuple[np.ndarray, Optional[np.ndarray], np.ndarray]:
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(axis=1) if kind == "layer" else None
    d = x - mean[:, None] if kind == "layer" else x
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    y = d * rstd[:, None] * weight
    return (y if bias is None else y + bias), mean, rstd


def norm_backward(dy, x, weight, mean, rstd, kind: str):
    """(dx, dweight, dbias) from given statistics."""
    x, dy = np.asarray(x, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    h = (x - mean[:, None] if kind == "layer" else x) * rstd[:, None]
    g = dy * weight
    dx = g - h * (g * h).mean(axis=1, keepdims=True)
    if kind == "layer":
        dx = dx - g.mean(axis=1, keepdims=True)
    return dx * rstd[:, None], (dy * h).sum(axis=0), dy.sum(axis=0)
