"""fp64 oracle of the embedding lookup with scaling and of its gradient."""

from __future__ import annotations

import numpy as np


def embedding_forward(tokens, table, scale: float) -> np.ndarray:
    table = np.asarray(table, dtype=np.float64)
    out = np.zeros((len(tokens), table.shape[1]))
    for i, t in enumerate(tokens):
        if 0 <= t < len(table):
            out[i] = scale * table[t]
    return out


def embedding_backward(tokens, dout, rows: int, scale: float) -> np.ndarray:
    dout = np.asarray(dout, dtype=np.float64)
    grad = np.zeros((rows, dout.shape[1]))
    tokens = np.asarray(tokens)
    known = (tokens >= 0) & (tokens < rows)
    np.add.at(grad, tokens[known], dout[known])
    return scale * grad
