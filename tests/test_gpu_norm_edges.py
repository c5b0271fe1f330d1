"""Rows at which the norms' kernels can go wrong by their layout, on an MI355X
against the fp64 oracle: columns behind a row's end, very long rows,
several long rows per workgroup, more rows than a launch takes at once."""

import numpy as np
import pytest
import torch

import pretraining_optimizer_amd as pm
from oracle import norm
from parity import announce
from test_gpu_norm import DTYPES, HALF, KINDS, U, _check_backward, _check_forward, _inputs, _np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [1, 3, 32, 100, 200, 300, 777, 1500, 2500, 5001, 9000, 17000])
def test_columns_behind_a_row_add_nothing(cols, dtype, bias):
    """Rows that are constant at 2^119 with a deviation of 2^-10: mean * rstd is
    beyond fp32, and no column of the row has that product.

    x - mean is zero, so h = 0, dw = 0 and dx = r (g - mean g): g off by u |g|, the
    mean by 70 u mean|g| (64 additions, the terms and the division), the difference
    and the product by u each; half a step of dx's type.  db: as dw of the other
    tests (rows / 512 + 80 additions)."""
    announce(f"norm far constant rows {cols} {dtype} bias {bias}")
    rows = 5
    gen = torch.Generator().manual_seed(cols)
    dy = torch.randn((rows, cols), generator=gen).to(dtype).cuda()
    w = (1.0 + 0.2 * torch.randn(cols, generator=gen)).cuda()
    x = torch.full((rows, cols), 2.0 ** 119, dtype=dtype, device="cuda")
    mean, rstd = torch.full((rows,), 2.0 ** 119, device="cuda"), torch.full((rows,), 2.0 ** 10, device="cuda")
    dx, dw, db = pm.norm_backward(dy, x, w, mean, rstd, kind="layer", bias=bias)
    ref, _, rdb = norm.norm_backward(_np(dy), _np(x), _np(w), _np(mean), _np(rstd), "layer")
    g = np.abs(_np(dy) * _np(w))
    off = 2.0 ** 10 * (4 * U * g + 72 * U * g.mean(1, keepdims=True))
    assert np.all(np.abs(_np(dx) - ref) <= off + HALF[dtype] * (np.abs(ref) + off))
    assert not dw.any()
    if bias:
        assert np.all(np.abs(_np(db) - rdb) <= (rows / 512 + 80) * U * np.abs(_np(dy)).sum(0))


def test_constant_far_rows_through_both_passes():
    """The same through the forward pass: 32 values of 2^119, whose sum is exact, and
    eps = 1e-6, so rstd = 1000 and mean * rstd is 6.6e38."""
    x = torch.full((3, 32), 2.0 ** 119, device="cuda")
    w, b = torch.ones(32, device="cuda"), torch.full((32,), 0.25, device="cuda")
    y, mean, rstd = pm.norm_forward(x, w, b, kind="layer", eps=1e-6)
    assert torch.equal(y, b.expand(3, 32)) and torch.all(mean == 2.0 ** 119)
    dy = torch.randn((3, 32), generator=torch.Generator().manual_seed(1)).cuda()
    dx, dw, _ = pm.norm_backward(dy, x, w, mean, rstd, kind="layer")
    g = _np(dy)
    ref = _np(rstd)[:, None] * (g - g.mean(1, keepdims=True))
    off = _np(rstd)[:, None] * (4 * U * np.abs(g) + 72 * U * np.abs(g).mean(1, keepdims=True))
    assert np.all(np.abs(_np(dx) - ref) <= off + U * (np.abs(ref) + off)) and not dw.any()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_very_long_rows(dtype, kind):
    """Rows of 2^22 + 3 columns, 4097 per thread, to the same 64 u: a sum of one
    sign (a constant row, whose partial sums outgrow the terms) and a mixed one."""
    announce(f"norm very long rows {dtype} {kind}")
    cols = (1 << 22) + 3
    gen = torch.Generator().manual_seed(11)
    x = torch.randn((2, cols), generator=gen)
    x[0] = 141 / 128
    x[1] += 0.3
    x = x.to(dtype).cuda()
    dy = torch.randn((2, cols), generator=gen)
    dy[0] = 0.1015625
    dy = dy.to(dtype).cuda()
    w = (1.0 + 0.2 * torch.randn(cols, generator=gen)).cuda()
    got = pm.norm_forward(x, w, None, kind=kind, eps=1e-5)
    _check_forward(got, x, w, None, kind, 1e-5, dtype, "forward")
    _, mean, rstd = got
    _check_backward(pm.norm_backward(dy, x, w, mean, rstd, kind=kind, bias=True), dy, x, w, mean, rstd, kind, dtype, "backward")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols,dtype", [(133, 5001, torch.float32), (133, 9000, torch.bfloat16), (133, 17000, torch.float32),
                                             (600, 9000, torch.float32), (600, 5001, torch.bfloat16), (600, 17000, torch.bfloat16),
                                             (1100, 3001, torch.float32)])
def test_several_long_rows_per_workgroup(rows, cols, dtype, kind):
    """Two and three rows per workgroup of the backward pass for the row lengths of
    512 and 1024 threads and for those beyond the registers, into new and into given
    gradients."""
    announce(f"norm {rows}x{cols} {dtype} {kind}")
    x, dy, w, b = (t.cuda() for t in _inputs(rows, cols, dtype))
    for bias in (None, b):
        got = pm.norm_forward(x, w, bias, kind=kind, eps=1e-5)
        _check_forward(got, x, w, bias, kind, 1e-5, dtype, "forward")
        _, mean, rstd = got
        got = pm.norm_backward(dy, x, w, mean, rstd, kind=kind, bias=bias is not None)
        _check_backward(got, dy, x, w, mean, rstd, kind, dtype, "backward")
        given = [torch.randn(cols, generator=torch.Generator().manual_seed(5 + i)).cuda() for i in range(2)]
        before = {"dw": _np(given[0]), "db": _np(given[1])}
        got = pm.norm_backward(dy, x, w, mean, rstd, kind=kind, dweight=given[0], dbias=given[1] if bias is not None else None, accumulate=True)
        _check_backward(got, dy, x, w, mean, rstd, kind, dtype, "accumulate", before)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols,dtype", [((1 << 25) + 5, 1, torch.float32), ((1 << 21) + 5, 1025, torch.bfloat16)])
def test_more_rows_than_one_trip_of_a_forward_launch(rows, cols, dtype, kind):
    """2^20 workgroups take 2^25 rows of one column or 2^21 of 1025 (whose groups of
    two wavefronts add through LDS); the rows of the next trip, and windows around
    its start, equal the same rows alone."""
    announce(f"norm forward {rows}x{cols} {kind}")
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty((rows, cols), dtype=dtype, device="cuda").normal_(generator=gen)
    w = torch.randn(cols, generator=gen, device="cuda")
    b = torch.randn(cols, generator=gen, device="cuda")
    y, mean, rstd = pm.norm_forward(x, w, b, kind=kind, eps=1e-5)
    for r0, r1 in ((0, 100), (rows // 2, rows // 2 + 77), (rows - 45, rows)):
        alone = pm.norm_forward(x[r0:r1], w, b, kind=kind, eps=1e-5)
        _check_forward(alone, x[r0:r1], w, b, kind, 1e-5, dtype, "window")
        assert torch.equal(y[r0:r1], alone[0]) and torch.equal(rstd[r0:r1], alone[2])
        assert mean is None or torch.equal(mean[r0:r1], alone[1])
    assert bool(torch.isfinite(y).all()) and bool(torch.isfinite(rstd).all())


@pytest.mark.parametrize("cols", [700, 20000])
def test_squares_beyond_fp32(cols):
    """A row whose sum of squares is beyond fp32 gets rstd 0 and y = 0, and its
    neighbours are as without it."""
    announce(f"norm squares beyond fp32 {cols}")
    x, _, w, _ = (t.cuda() for t in _inputs(3, cols, torch.float32))
    want = pm.norm_forward(x, w, kind="rms")
    x[1] = 1e20
    y, _, rstd = pm.norm_forward(x, w, kind="rms")
    assert rstd[1] == 0 and not y[1].any()
    for i in (0, 2):
        assert torch.equal(y[i], want[0][i]) and rstd[i] == want[2][i]
