"""fp64 oracle of causal attention over packed sequences with grouped heads, and
of its gradients: one sequence and head at a time."""

from __future__ import annotations

import numpy as np


def _blocks(cu, tokens, heads):
    """(rows, head) of every sequence and head; ends are taken into [0, tokens]."""
    ends = [min(max(int(c), 0), tokens) for c in cu]
    for s, e in zip(ends[:-1], ends[1:]):
        if e > s:
            for h in range(heads):
                yield slice(s, e), h


def probabilities(q, k, scale):
    """(S, lse, P) of one sequence and head; S is -inf above the diagonal."""
    n = len(q)
    s = np.where(np.tril(np.ones((n, n), dtype=bool)), scale * (q @ k.T), -np.inf)
    top = s.max(axis=1)
    lse = top + np.log(np.exp(s - top[:, None]).sum(axis=1))
    return s, lse, np.exp(s - lse[:, None])


def attention_forward(q, k, v, cu, scale):
    """(out, lse) with NaN in the rows that no sequence holds."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    tokens, heads, _ = q.shape
    group = heads // k.shape[1]
    out, lse = np.full(q.shape, np.nan), np.full((heads, tokens), np.nan)
    for rows, h in _blocks(cu, tokens, heads):
        _, lse[h, rows], p = probabilities(q[rows, h], k[rows, h // group], scale)
        out[rows, h] = p @ v[rows, h // group]
    return out, lse


def attention_backward(dout, q, k, v, out, lse, cu, scale):
    """(dq, dk, dv) from given forward results, NaN as above."""
    dout, q, k, v, out, lse = (np.asarray(t, dtype=np.float64) for t in (dout, q, k, v, out, lse))
    tokens, heads, _ = q.shape
    group = heads // k.shape[1]
    dq, dk, dv = np.full(q.shape, np.nan), np.full(k.shape, np.nan), np.full(v.shape, np.nan)
    for rows, h in _blocks(cu, tokens, heads):
        g = h // group
        if h % group == 0:
            dk[rows, g] = dv[rows, g] = 0.0
        s = probabilities(q[rows, h], k[rows, g], scale)[0]
        p = np.exp(s - lse[h, rows][:, None])
        delta = (dout[rows, h] * out[rows, h]).sum(axis=1, keepdims=True)
        ds = scale * p * (dout[rows, h] @ v[rows, g].T - delta)
        dq[rows, h] = ds @ k[rows, g]
        dk[rows, g] += ds.T @ q[rows, h]
        dv[rows, g] += p.T @ dout[rows, h]
    return dq, dk, dv
