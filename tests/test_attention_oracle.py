"""Pins of the attention's oracle on something other than itself (CPU only):
closed forms, torch's own attention, finite differences."""

import numpy as np
import torch

from oracle import attention


def _inputs(seed, lens, heads, kv, dim):
    rng = np.random.default_rng(seed)
    n = sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    return rng.standard_normal((n, heads, dim)), rng.standard_normal((n, kv, dim)), rng.standard_normal((n, kv, dim)), cu


def test_closed_forms():
    """A token alone returns its value; equal keys average the values seen."""
    q, k, v, cu = _inputs(0, [1, 7], 2, 1, 8)
    out, lse = attention.attention_forward(q, k, v, cu, 0.5)
    assert np.allclose(out[0], np.broadcast_to(v[0], (2, 8)), rtol=1e-15)
    assert np.allclose(lse[:, 0], 0.5 * (q[0] @ k[0, 0]), rtol=1e-14)
    k[1:] = k[1]
    out, lse = attention.attention_forward(q, k, v, cu, 0.5)
    for i in range(7):
        assert np.allclose(out[1 + i], v[1:2 + i].mean(axis=0), rtol=1e-12)
        assert np.allclose(lse[:, 1 + i], 0.5 * (q[1 + i] @ k[1, 0]) + np.log(i + 1), rtol=1e-12)


def test_agrees_with_torch():
    q, k, v, cu = _inputs(1, [9, 0, 5], 4, 2, 16)
    out, _ = attention.attention_forward(q, k, v, cu, 0.25)
    for s, e in ((0, 9), (9, 14)):
        a, b, c = (torch.from_numpy(t[s:e]).transpose(0, 1) for t in (q, k, v))
        want = torch.nn.functional.scaled_dot_product_attention(a, b.repeat_interleave(2, 0), c.repeat_interleave(2, 0),
                                                                is_causal=True, scale=0.25)
        assert np.allclose(out[s:e], want.transpose(0, 1).numpy(), rtol=1e-12, atol=1e-12)


def test_rows_of_no_sequence_and_ends_outside():
    q, k, v, _ = _inputs(2, [8], 2, 2, 8)
    out, lse = attention.attention_forward(q, k, v, [2, 5, 4, 99], 1.0)
    assert np.isnan(out[:2]).all() and np.isnan(lse[:, :2]).all() and np.isfinite(out[2:]).all()
    whole, _ = attention.attention_forward(q, k, v, [2, 4, 8], 1.0)
    assert np.array_equal(out[5:], whole[5:])


def test_gradients_by_differences():
    q, k, v, cu = _inputs(3, [4, 3], 4, 2, 8)
    dout = np.random.default_rng(4).standard_normal(q.shape)

    def loss():
        return float((attention.attention_forward(q, k, v, cu, 0.3)[0] * dout).sum())

    out, lse = attention.attention_forward(q, k, v, cu, 0.3)
    h = 1e-5
    for arr, grad in zip((q, k, v), attention.attention_backward(dout, q, k, v, out, lse, cu, 0.3)):
        for i in np.ndindex(arr.shape):
            keep = arr[i]
            arr[i] = keep + h
            up = loss()
            arr[i] = keep - h
            down = loss()
            arr[i] = keep
            # central differences: h^2 times a third derivative of order one, and cancellation
            assert abs((up - down) / (2 * h) - grad[i]) < 1e-7
