"""Layer norm and RMS norm, forward and backward, on an MI355X against the fp64
oracle.

Tolerances (u = 2^-24).  A row's sum runs through at most 64 additions one
after another (32 per thread, then a tree over the threads; the longest rows
here leave fewer per thread), so a sum of terms t is off by at most
64 u sum|t|, with each term off by a few u of its own:
  mean:  64 u mean|x|;  rstd: half of the sum of squares' 66 u, plus the shift
         of the mean, plus 4 u of its own operations: 40 u
  h:     dh = r (dmean + u (|x| + |mean|)) + 42 u |h|
  y:     |w| dh + 2 u (|h w| + |b|), and half a step of y's type
In the backward pass mean and rstd are inputs, so dh = 3 u r (|x| + |mean|):
  mean(g): 70 u mean|g|;  mean(g h): 70 u mean|g h| + mean(|g| dh)
  dx:    r (4 u |g| + |h| (70 u mean|g h| + mean(|g| dh)) + dh |mean(g h)|
            + 70 u mean|g| + 6 u (|g| + |h mean(g h)| + |mean g|)), and half a step
  dw:    rows / 512 + 80 additions one after another at most:
         (rows / 512 + 80) u sum|dy h| + sum(|dy| dh);  db likewise
"""

import numpy as np
import pytest
import torch

import pretraining_optimizer_amd as pm
from oracle import norm
from parity import announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
DTYPES = [torch.float32, torch.bfloat16]
KINDS = ["layer", "rms"]


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _inputs(rows, cols, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed + 31 * rows + cols)
    x = (torch.randn((rows, cols), generator=gen) * torch.exp(torch.randn((rows, 1), generator=gen)) + 0.3).to(dtype)
    dy = (0.1 * torch.randn((rows, cols), generator=gen)).to(dtype)
    w = 1.0 + 0.2 * torch.randn(cols, generator=gen)
    b = 0.2 * torch.randn(cols, generator=gen)
    return x, dy, w, b


def _check_forward(got, x, w, b, kind, eps, dtype, what):
    y, mean, rstd = got
    ry, rm, rr = norm.norm_forward(_np(x), _np(w), _np(b), kind, eps)
    ax = np.abs(_np(x))
    dm = 64 * U * ax.mean(1) if kind == "layer" else np.zeros(len(ax))
    if kind == "layer":
        assert np.all(np.abs(_np(mean) - rm) <= dm + U * np.abs(rm)), what
    else:
        assert mean is None
    assert np.all(np.abs(_np(rstd) - rr) <= 40 * U * rr + rr * rr * dm), what
    m = rm[:, None] if kind == "layer" else 0.0
    h = (_np(x) - m) * rr[:, None]
    dh = rr[:, None] * (dm[:, None] + U * (ax + np.abs(m))) + 42 * U * np.abs(h) + np.abs(h) * (rr * dm)[:, None]
    tol = np.abs(_np(w)) * dh + 2 * U * (np.abs(h * _np(w)) + (0 if b is None else np.abs(_np(b))))
    tol = tol + HALF[dtype] * (np.abs(ry) + tol)
    err = np.abs(_np(y) - ry)
    assert np.all(err <= tol), (what, float((err - tol).max()))


def _check_backward(got, dy, x, w, mean, rstd, kind, dtype, what, before=None):
    dx, dw, db = got
    X, D, W, M, R = _np(x), _np(dy), _np(w), _np(mean), _np(rstd)
    rdx, rdw, rdb = norm.norm_backward(D, X, W, M, R, kind)
    m = M[:, None] if kind == "layer" else 0.0
    r = R[:, None]
    h, g = (X - m) * r, D * W
    dh = 3 * U * r * (np.abs(X) + np.abs(m))
    c1 = np.abs((g * h).mean(1, keepdims=True))
    ec1 = 70 * U * np.abs(g * h).mean(1, keepdims=True) + (np.abs(g) * dh).mean(1, keepdims=True)
    c0 = np.abs(g.mean(1, keepdims=True)) if kind == "layer" else 0.0
    ec0 = 70 * U * np.abs(g).mean(1, keepdims=True) if kind == "layer" else 0.0
    tol = r * (4 * U * np.abs(g) + np.abs(h) * ec1 + dh * c1 + ec0 + 6 * U * (np.abs(g) + np.abs(h) * c1 + c0))
    tol = tol + HALF[dtype] * (np.abs(rdx) + tol)
    err = np.abs(_np(dx) - rdx)
    assert np.all(err <= tol), (what, "dx", float((err - tol).max()))
    n = len(X) / 512 + 80
    for name, a, ref, terms, slack in (("dw", dw, rdw, np.abs(D * h), (np.abs(D) * dh).sum(0)), ("db", db, rdb, np.abs(D), 0.0)):
        if a is None:
            continue
        old = 0.0 if before is None else before[name]
        tol = n * U * terms.sum(0) + slack + (0.0 if before is None else 2 * U * (np.abs(old) + np.abs(ref)))
        err = np.abs(_np(a) - ref - old)
        assert np.all(err <= tol), (what, name, float((err - tol).max()))


SHAPES = [(1, 1), (1, 128), (3, 5), (37, 777), (130, 128), (257, 129), (33, 256), (19, 300), (21, 512), (9, 1000),
          (70, 1024), (11, 1500), (600, 2048), (13, 2049), (5, 4096), (6, 5001), (3, 8192), (4, 9000), (2, 16384),
          (3, 16385), (2, 40000), (5000, 64), (2100, 40)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_shapes(rows, cols, dtype, kind):
    announce(f"norm {rows}x{cols} {dtype} {kind}")
    x, dy, w, b = (t.cuda() for t in _inputs(rows, cols, dtype))
    for bias in (None, b):
        y, mean, rstd = got = pm.norm_forward(x, w, bias, kind=kind, eps=1e-5)
        _check_forward(got, x, w, bias, kind, 1e-5, dtype, "forward")
        got = pm.norm_backward(dy, x, w, mean, rstd, kind=kind, bias=bias is not None)
        assert (got[2] is None) == (bias is None)
        _check_backward(got, dy, x, w, mean, rstd, kind, dtype, "backward")
        again = pm.norm_backward(dy, x, w, mean, rstd, kind=kind, bias=bias is not None)
        for p, q in zip(got, again):
            assert p is None or torch.equal(p, q)


def test_many_rows():
    """More rows than one trip of every workgroup takes."""
    for rows, cols, kind in ((40000, 128, "rms"), (9000, 200, "layer"), (5001, 600, "layer"), (1500, 2500, "rms")):
        announce(f"norm {rows}x{cols}")
        x, dy, w, b = (t.cuda() for t in _inputs(rows, cols, torch.bfloat16))
        got = pm.norm_forward(x, w, b, kind=kind)
        _check_forward(got, x, w, b, kind, 1e-6, torch.bfloat16, "forward")
        _check_backward(pm.norm_backward(dy, x, w, got[1], got[2], kind=kind, bias=True), dy, x, w, got[1], got[2], kind,
                        torch.bfloat16, "backward")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [100, 2051, 17000])
def test_pitch_in_place_and_neighbours(cols, dtype, kind):
    """Windows of larger matrices with odd pitches and offsets, whose other
    elements stay; y over x, dx over dy and dx over x; neighbouring windows of
    one matrix as input and output."""
    announce(f"norm windows {cols} {dtype} {kind}")
    rows = 7
    x, dy, w, b = (t.cuda() for t in _inputs(rows, cols, dtype))
    want = pm.norm_forward(x, w, b, kind=kind)
    wantg = pm.norm_backward(dy, x, w, want[1], want[2], kind=kind, bias=True)
    two = torch.full((rows + 2, 2 * cols + 5), 3.0, dtype=dtype, device="cuda")
    left, right = two[1:-1, 1:1 + cols], two[1:-1, 3 + cols:3 + 2 * cols]
    left.copy_(x)
    got = pm.norm_forward(left, w, b, kind=kind, out=right)
    assert got[0] is right and torch.equal(right, want[0])
    assert torch.equal(left, x)
    mask = torch.ones_like(two, dtype=torch.bool)
    mask[1:-1, 1:1 + cols] = False
    mask[1:-1, 3 + cols:3 + 2 * cols] = False
    assert torch.all(two[mask] == 3)
    right.copy_(dy)
    got = pm.norm_backward(right, left, w, want[1], want[2], kind=kind, bias=True, dx=right)
    assert torch.equal(right, wantg[0]) and torch.equal(got[1], wantg[1]) and torch.equal(got[2], wantg[2])
    right.copy_(dy)
    pm.norm_backward(right, left, w, want[1], want[2], kind=kind, dx=left)
    assert torch.equal(left, wantg[0]) and torch.equal(right, dy)
    z = x.clone()
    pm.norm_forward(z, w, b, kind=kind, out=z)
    assert torch.equal(z, want[0]) and torch.all(two[mask] == 3)


def test_accumulate():
    for rows, cols in ((50, 300), (3, 20000), (0, 64)):
        x, dy, w, b = (t.cuda() for t in _inputs(rows, cols, torch.float32))
        y, mean, rstd = pm.norm_forward(x, w, b, kind="layer")
        dw, db = torch.randn(cols, device="cuda"), torch.randn(cols, device="cuda")
        before = {"dw": _np(dw), "db": _np(db)}
        got = pm.norm_backward(dy, x, w, mean, rstd, kind="layer", dweight=dw, dbias=db, accumulate=True)
        assert got[1] is dw and got[2] is db
        if rows:
            _check_backward(got, dy, x, w, mean, rstd, "layer", torch.float32, "accumulate", before)
        else:
            assert np.array_equal(_np(dw), before["dw"]) and np.array_equal(_np(db), before["db"])
            dw2 = pm.norm_backward(dy, x, w, mean, rstd, kind="layer")[1]
            assert torch.all(dw2 == 0)


@pytest.mark.parametrize("kind", KINDS)
def test_far_from_zero_and_non_finite(kind):
    """A mean of 1000 spreads (a difference of moments would lose the variance);
    rows with NaN or Inf keep to themselves; rows of zeros."""
    announce(f"norm special rows {kind}")
    x, dy, w, b = (t.cuda() for t in _inputs(64, 700, torch.float32))
    x = torch.randn((64, 700), device="cuda") + 1000.0
    got = pm.norm_forward(x, w, b, kind=kind)
    _check_forward(got, x, w, b, kind, 1e-6, torch.float32, "offset")
    x[3, 5], x[9, 699] = float("nan"), float("inf")
    x[20] = 0.0
    y, mean, rstd = pm.norm_forward(x, w, b, kind=kind)
    ok = torch.ones(64, dtype=torch.bool)
    ok[3] = ok[9] = False
    assert torch.isnan(y[3]).all() and not torch.isfinite(y[9]).all() and torch.isfinite(y[ok.cuda()]).all()
    assert torch.equal(y[20], b)
    dx = pm.norm_backward(dy, x, w, mean, rstd, kind=kind)[0]
    assert torch.isfinite(dx[ok.cuda()]).all() and not torch.isfinite(dx[3]).any()


def test_gradient_by_differences():
    """The fp32 kernels' own differences: a step s in one input moves the loss
    sum(y dy) by s times its gradient, to the fp32 rounding of y (u |y| per
    element, divided by s) and the second derivative (s times a value of order
    |x|^-2 |dy|; rows here have unit spread)."""
    x, dy, w, b = (t.cuda() for t in _inputs(2, 48, torch.float32, seed=4))
    x = (x - x.mean(1, keepdim=True)) / x.std(1, keepdim=True)
    for kind in KINDS:
        y, mean, rstd = pm.norm_forward(x, w, b, kind=kind)
        dx, dw, db = pm.norm_backward(dy, x, w, mean, rstd, kind=kind, bias=True)
        s = 2.0 ** -8

        def loss(x_, w_, b_):
            return (pm.norm_forward(x_, w_, b_, kind=kind)[0].double() * dy.double()).sum().item()

        tol = 2 * 50 * U * (y.abs() * dy.abs()).sum().item() / (2 * s) + 8 * s * s * dy.abs().sum().item()
        for t, grad in ((x, dx), (w, dw), (b, db)):
            for i in (0, 7, 47):
                flat = t.view(-1)
                keep = flat[i].item()
                flat[i] = keep + s
                hi, up = flat[i].item(), loss(x, w, b)
                flat[i] = keep - s
                lo, down = flat[i].item(), loss(x, w, b)
                flat[i] = keep
                assert abs((up - down) / (hi - lo) - grad.view(-1)[i].item()) <= tol, (kind, i)


def test_streams_and_graph():
    announce("norm streams and graph")
    x, dy, w, b = (t.cuda() for t in _inputs(300, 700, torch.bfloat16))
    want = pm.norm_forward(x, w, b, kind="layer")
    wantg = pm.norm_backward(dy, x, w, want[1], want[2], kind="layer", bias=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = pm.norm_forward(x, w, b, kind="layer", stream=s)
    gotg = pm.norm_backward(dy, x, w, got[1], got[2], kind="layer", bias=True, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for p, q in zip(got + gotg, want + wantg):
        assert torch.equal(p, q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = pm.norm_forward(x, w, b, kind="layer")
        capg = pm.norm_backward(dy, x, w, cap[1], cap[2], kind="layer", bias=True)
    for k in range(4):
        x.mul_(0.9).add_(0.05 * k)
        g.replay()
        torch.cuda.synchronize()
        e = pm.norm_forward(x, w, b, kind="layer")
        eg = pm.norm_backward(dy, x, w, e[1], e[2], kind="layer", bias=True)
        for p, q in zip(cap + capg, e + eg):
            assert torch.equal(p, q), k


def test_python_refusals():
    x, dy, w, b = (t.cuda() for t in _inputs(4, 96, torch.float32))
    y, mean, rstd = pm.norm_forward(x, w, b, kind="layer")
    with pytest.raises(ValueError):
        pm.norm_forward(x, w, kind="batch")
    with pytest.raises(ValueError):
        pm.norm_forward(x, w[:95])
    with pytest.raises(ValueError):
        pm.norm_forward(x, w.bfloat16())
    with pytest.raises(ValueError):
        pm.norm_forward(x.t(), w)
    with pytest.raises(TypeError):
        pm.norm_forward(x.double(), w)
    with pytest.raises(ValueError):
        pm.norm_forward(x, w, out=torch.empty((4, 95), device="cuda"))
    with pytest.raises(ValueError):
        pm.norm_forward(x, w.cpu())
    with pytest.raises(pm.MuonHError):
        pm.norm_forward(x, w, eps=-1.0)
    big = torch.zeros(800, device="cuda")
    with pytest.raises(pm.MuonHError):
        pm.norm_forward(big[:384].view(4, 96), w, out=big[96:480].view(4, 96))
    with pytest.raises(ValueError):
        pm.norm_backward(dy, x, w, None, rstd, kind="layer")
    with pytest.raises(ValueError):
        pm.norm_backward(dy, x, w, mean, rstd, kind="rms")
    with pytest.raises(ValueError):
        pm.norm_backward(dy.bfloat16(), x, w, mean, rstd, kind="layer")
    with pytest.raises(ValueError):
        pm.norm_backward(dy, x, w, mean, rstd, kind="layer", accumulate=True)
