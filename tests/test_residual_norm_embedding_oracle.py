"""Pins of the oracles of the residual norm's gradient and of the embedding on
something other than themselves (CPU only)."""

import numpy as np
import torch

from oracle import embedding, norm


def test_add_norm_gradients_by_differences():
    rng = np.random.default_rng(6)
    x, r, w, dy, dh = (rng.standard_normal(s) for s in ((4, 9), (4, 9), (9,), (4, 9), (4, 9)))

    def loss():
        h = x + r
        return float((norm.norm_forward(h, w, None, "rms", 1e-3)[0] * dy).sum() + (h * dh).sum())

    h = x + r
    rstd = norm.norm_forward(h, w, None, "rms", 1e-3)[2]
    dx, dw = norm.add_norm_backward(dy, dh, h, w, rstd)
    e = 1e-5
    for arr, grad in ((x, dx), (r, dx), (w, dw)):
        for i in np.ndindex(arr.shape):
            keep = arr[i]
            arr[i] = keep + e
            up = loss()
            arr[i] = keep - e
            down = loss()
            arr[i] = keep
            # central differences: e^2 times a third derivative of order one, and cancellation
            assert abs((up - down) / (2 * e) - grad[i]) < 1e-7


def test_embedding_agrees_with_torch():
    gen = torch.Generator().manual_seed(1)
    table = torch.randn((11, 5), dtype=torch.float64, generator=gen, requires_grad=True)
    tokens = torch.randint(0, 11, (40,), generator=gen)
    dout = torch.randn((40, 5), dtype=torch.float64, generator=gen)
    y = 2.5 * torch.nn.functional.embedding(tokens, table)
    y.backward(dout)
    assert np.allclose(embedding.embedding_forward(tokens.numpy(), table.detach().numpy(), 2.5), y.detach().numpy(), rtol=1e-14)
    assert np.allclose(embedding.embedding_backward(tokens.numpy(), dout.numpy(), 11, 2.5), table.grad.numpy(), rtol=1e-12)
    tokens[::3] = torch.tensor([-1, 11, 1 << 40] * 5)[:14]
    out = embedding.embedding_forward(tokens.numpy(), table.detach().numpy(), 1.0)
    assert (out[::3] == 0).all() and (out[1::3] != 0).all()
    keep = torch.ones(40, dtype=torch.bool)
    keep[::3] = False
    assert np.array_equal(embedding.embedding_backward(tokens.numpy(), dout.numpy(), 11, 1.0),
                          embedding.embedding_backward(tokens[keep].numpy(), dout[keep].numpy(), 11, 1.0))
