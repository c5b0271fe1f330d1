"""Pins of the operators' oracle on something other than itself (CPU only):
the E4M3 grid by enumeration and by torch's own conversion, block scales by
their defining inequality, the norms' gradients by finite differences."""

import numpy as np
import pytest
import torch

from oracle import block_fp8, norm


def test_e4m3_round_is_the_nearest_encoding():
    """Against the list of the 256 encodings: nearest value, ties to an even
    fraction (neighbouring encodings alternate)."""
    grid = block_fp8.e4m3_values()
    pos = np.sort(grid[:127])
    assert pos[-1] == 448.0 and pos[1] == 2.0 ** -9
    mids = (pos[:-1] + pos[1:]) / 2
    v = np.concatenate([pos, mids, np.nextafter(mids, 0), np.nextafter(mids, 1e9),
                        np.random.default_rng(0).uniform(0, 448, 2000)])
    got = block_fp8.e4m3_round(v)
    near = np.abs(v[:, None] - pos[None, :])
    assert np.array_equal(np.abs(got - v), near.min(axis=1))
    idx = np.searchsorted(pos, got)
    ties = np.isin(v, mids)
    assert np.all(idx[ties] % 2 == 0)
    assert np.array_equal(block_fp8.e4m3_round(-v), -got)


def test_e4m3_round_agrees_with_torch():
    v = torch.cat([torch.randn(4000) * 10 ** torch.empty(4000).uniform_(-4, 1.5), torch.tensor([0.0, 448.0])])
    v = v.clamp(-448, 448)
    assert np.array_equal(v.to(torch.float8_e4m3fn).double().numpy(), block_fp8.e4m3_round(v.double().numpy()))


@pytest.mark.parametrize("block_rows", [1, 128])
def test_block_scales(block_rows):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((131, 300)) * np.exp(8 * rng.standard_normal((131, 1)))
    x[5] = 0.0
    x[7, 9] = np.inf
    q = block_fp8.quantize(x, block_rows)
    for i in range(q.exponents.shape[0]):
        for j in range(3):
            b = x[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128]
            amax = np.abs(b[np.isfinite(b)]).max()
            e = int(q.exponents[i, j])
            if amax == 0:
                assert e == 0
            else:
                assert amax <= 448 * 2.0 ** e and amax > 448 * 2.0 ** (e - 1)
    d = q.dequantize()
    assert np.isnan(d[7, 9]) and np.isnan(d).sum() == 1
    # half a step of 2^-3 relative, or of 2^-9 scales near zero
    ok = np.isfinite(x)
    e = np.repeat(np.repeat(q.exponents, block_rows, 0)[:131], 128, 1)[:, :300]
    assert np.all(np.abs(d - x)[ok] <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** (e - 10.0))[ok])


def test_least_exponent():
    assert block_fp8.block_exponent(1e-45) == -127 and block_fp8.block_exponent(448.0) == 0
    assert block_fp8.block_exponent(np.nextafter(448.0, 1e9)) == 1
    assert block_fp8.block_exponent(float(np.finfo(np.float32).max)) == 120


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_gradients_by_differences(kind):
    rng = np.random.default_rng(5)
    x, w, b, dy = rng.standard_normal((4, 9)), rng.standard_normal(9), rng.standard_normal(9), rng.standard_normal((4, 9))

    def loss(x_, w_, b_):
        return float((norm.norm_forward(x_, w_, b_, kind, 1e-3)[0] * dy).sum())

    _, mean, rstd = norm.norm_forward(x, w, b, kind, 1e-3)
    dx, dw, db = norm.norm_backward(dy, x, w, mean, rstd, kind)
    h = 1e-5
    for arr, grad in ((x, dx), (w, dw), (b, db)):
        for i in np.ndindex(arr.shape):
            keep = arr[i]
            arr[i] = keep + h
            up = loss(x, w, b)
            arr[i] = keep - h
            down = loss(x, w, b)
            arr[i] = keep
            # central differences: h^2 times a third derivative of order one, and cancellation
            assert abs((up - down) / (2 * h) - grad[i]) < 1e-7


def test_norm_agrees_with_torch():
    x, w, b = torch.randn(5, 33, dtype=torch.float64), torch.randn(33, dtype=torch.float64), torch.randn(33, dtype=torch.float64)
    y = norm.norm_forward(x.numpy(), w.numpy(), b.numpy(), "layer", 1e-5)[0]
    assert np.allclose(y, torch.nn.functional.layer_norm(x, (33,), w, b, 1e-5).numpy(), rtol=1e-12, atol=1e-12)
    y = norm.norm_forward(x.numpy(), w.numpy(), None, "rms", 1e-5)[0]
    assert np.allclose(y, torch.nn.functional.rms_norm(x, (33,), w, 1e-5).numpy(), rtol=1e-12, atol=1e-12)
