"""Residual addition with RMS norm and FP8 output, and its gradient, on an MI355X.

The sum is exact to its rounding, so h equals the fp32 sum rounded, bit for bit.
rstd is within 40 u of the formula's on that h (u = 2^-24; as for norm_forward).
From h and rstd on everything is elementwise: y = (h rstd) weight in fp32 and
the quantiser's rounding, so the forms equal the oracle's of those y bit for bit, and
are within 2^-4 (half a step) of the formula's y, or half of the scale's smallest step,
beside y's own error of 42 u.
Backward: norm_backward's tolerances, and the addition of dh before the rounding.
"""

import numpy as np
import pytest
import torch

import pretraining_optimizer_amd as pm
from oracle import block_fp8, norm
from parity import announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
DTYPES = [torch.float32, torch.bfloat16]


def _np(t):
    return t.detach().double().cpu().numpy()


def _inputs(rows, cols, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed + 17 * rows + cols)
    spread = torch.exp(torch.randn((1, cols), generator=gen))
    x, r = ((torch.randn((rows, cols), generator=gen) * spread).to(dtype).cuda() for _ in range(2))
    dy, dh = ((0.1 * torch.randn((rows, cols), generator=gen)).to(dtype).cuda() for _ in range(2))
    return x, r, (1.0 + 0.2 * torch.randn(cols, generator=gen)).cuda(), dy, dh


def _same_form(m, ref):
    """An Fp8Matrix against the oracle's, padding included."""
    data, scale = m.data.float().cpu().numpy(), m.scale.cpu().numpy().astype(int)
    q = ref.dequantize()
    rows, cols = q.shape
    e = ref.exponents
    kb = e.shape[1]
    assert np.array_equal(scale[:, :kb], e + 127) and (scale[:, kb:] == 0).all()
    assert (data[:, cols:] == 0).all()
    value = data[:, :cols].astype(np.float64) * 2.0 ** np.repeat(e, 128, axis=1)[:, :cols]
    return np.array_equal(value, q, equal_nan=True)


def _check_forward(x, r, w, eps, got, form, what):
    h, rstd, q = got
    if r is None:
        assert h is x
    else:
        assert torch.equal(h, (x.float() + r.float()).to(x.dtype)), what
    H, W = _np(h), _np(w)
    ref = 1.0 / np.sqrt((H * H).mean(axis=1) + eps)
    assert np.all(np.abs(_np(rstd) - ref) <= 40 * U * ref), what
    y = (h.float() * rstd[:, None]) * w
    forms = q if form == "both" else (q,)
    exact = H * ref[:, None] * W
    for m, kind in zip(forms, ("row", "col") if form == "both" else (form,)):
        side, full = (_np(y), exact) if kind == "row" else (_np(y).T, exact.T)
        # all of it as the quantiser gives it, and the first rows as the oracle does
        whole = pm.fp8_quantize(y, form=kind)
        assert torch.equal(m.scale, whole.scale) and torch.equal(m.data.view(torch.uint8), whole.data.view(torch.uint8)), what
        n = max(1, min(len(side), 400000 // side.shape[1], 300))
        quantised = block_fp8.quantize(side[:n])
        assert _same_form(pm.Fp8Matrix(m.data[:n], m.scale[:n], m.cols), quantised), (what, kind)
        e = np.repeat(quantised.exponents, 128, axis=1)[:, :side.shape[1]]
        err = np.abs(quantised.dequantize() - full[:n])
        assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(full[:n]), 2.0 ** (e - 10.0)) + 45 * U * np.abs(full[:n])), what


def _check_backward(got, dy, dh, h, w, rstd, dtype, what, before=None):
    """norm_backward's bounds (rms), one more addition in dx."""
    dx, dw = got
    X, D, W, R, E = _np(h), _np(dy), _np(w), _np(rstd), _np(dh)
    rdx, rdw = norm.add_norm_backward(D, E, X, W, R)
    r = R[:, None]
    n, g = X * r, D * W
    dn = 3 * U * r * np.abs(X)
    c1 = np.abs((g * n).mean(1, keepdims=True))
    ec1 = 70 * U * np.abs(g * n).mean(1, keepdims=True) + (np.abs(g) * dn).mean(1, keepdims=True)
    tol = r * (4 * U * np.abs(g) + np.abs(n) * ec1 + dn * c1 + 6 * U * (np.abs(g) + np.abs(n) * c1))
    tol = tol + 2 * U * (np.abs(E) + np.abs(rdx))
    tol = tol + HALF[dtype] * (np.abs(rdx) + tol)
    err = np.abs(_np(dx) - rdx)
    assert np.all(err <= tol), (what, "dx", float((err - tol).max()))
    old = 0.0 if before is None else before
    tol = (len(X) / 512 + 80) * U * np.abs(D * n).sum(0) + (np.abs(D) * dn).sum(0)
    tol = tol + (0.0 if before is None else 2 * U * (np.abs(old) + np.abs(rdw)))
    err = np.abs(_np(dw) - rdw - old)
    assert np.all(err <= tol), (what, "dw", float((err - tol).max()))


SHAPES = [(1, 1), (1, 128), (3, 5), (37, 777), (130, 128), (257, 129), (33, 256), (19, 300), (70, 1024), (11, 1500),
          (300, 2048), (13, 2049), (6, 5001), (4, 9000), (2, 16384), (3, 16385), (2, 40000), (1500, 64)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_shapes(rows, cols, dtype):
    announce(f"add norm {rows}x{cols} {dtype}")
    x, r, w, dy, dh = _inputs(rows, cols, dtype)
    for res, form in ((r, "both"), (None, "both"), (r, "row"), (None, "row"), (r, "col"), (None, "col")):
        got = pm.add_norm_quantize(x, res, w, eps=1e-5, form=form)
        _check_forward(x, res, w, 1e-5, got, form, (res is None, form))
    h, rstd, _ = pm.add_norm_quantize(x, r, w, eps=1e-5)
    grads = pm.add_norm_backward(dy, dh, h, w, rstd)
    _check_backward(grads, dy, dh, h, w, rstd, dtype, "backward")
    again = pm.add_norm_backward(dy, dh, h, w, rstd)
    assert torch.equal(grads[0], again[0]) and torch.equal(grads[1], again[1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("base", [8, 1016])
def test_every_row_end(base, dtype):
    """Rows that end after each number of elements of a vector."""
    for cols in range(base, base + 9):
        announce(f"add norm 9x{cols} {dtype}")
        x, r, w, dy, dh = _inputs(9, cols, dtype)
        for res in (r, None):
            _check_forward(x, res, w, 1e-5, pm.add_norm_quantize(x, res, w, eps=1e-5, form="both"), "both", cols)
        h, rstd, _ = pm.add_norm_quantize(x, r, w, eps=1e-5)
        _check_backward(pm.add_norm_backward(dy, dh, h, w, rstd), dy, dh, h, w, rstd, dtype, cols)


@pytest.mark.parametrize("dtype", DTYPES)
def test_forms_are_the_quantisers(dtype):
    """Bit for bit what quantising the fp32 norm gives, also where values are special,
    zero or far apart."""
    announce(f"add norm forms {dtype}")
    x, r, w, _, _ = _inputs(300, 700, dtype)
    x[3], r[3] = 0.0, 0.0
    x[5, 7] = float("inf")
    x[9, 600] = float("nan")
    x[11] *= 1e-18
    r[11] *= 1e-18
    x[12] *= 1e15
    w[40] = 1e30
    w[41] = 0.0
    w[42] = float("inf")
    h, rstd, (q, qt) = pm.add_norm_quantize(x, r, w, form="both", eps=0.0)
    y = (h.float() * rstd[:, None]) * w
    a, b = pm.fp8_quantize(y, form="both")
    for m, ref in ((q, a), (qt, b)):
        assert torch.equal(m.scale, ref.scale) and torch.equal(m.data.view(torch.uint8), ref.data.view(torch.uint8))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [100, 2051, 17000])
def test_pitch_in_place_and_neighbours(cols, dtype):
    """Windows with odd pitches and offsets, whose other elements stay; h over x and over
    the residual; dx over each of its inputs."""
    announce(f"add norm windows {cols} {dtype}")
    rows = 7
    x, r, w, dy, dh = _inputs(rows, cols, dtype)
    want = pm.add_norm_quantize(x, r, w, form="both")

    def window(t):
        wide = torch.full((rows + 2, cols + 5), 3.0, dtype=dtype, device="cuda")
        wide[1:-1, 3:3 + cols] = t
        return wide, wide[1:-1, 3:3 + cols]

    def untouched(wide, inner):
        keep = inner.clone()
        inner.fill_(3.0)
        ok = (wide == 3).all()
        inner.copy_(keep)
        return bool(ok)

    def same(got):
        return torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and all(
            torch.equal(a.scale, b.scale) and torch.equal(a.data.view(torch.uint8), b.data.view(torch.uint8))
            for a, b in zip(got[2], want[2]))

    (wx, vx), (wr, vr), (wh, vh) = window(x), window(r), window(x)
    got = pm.add_norm_quantize(vx, vr, w, form="both", h=vh)
    assert got[0] is vh and same(got) and untouched(wh, vh)
    for t, (wide, v) in (("x", window(x)), ("residual", window(r))):
        a, b = (v, r) if t == "x" else (x, v)
        got = pm.add_norm_quantize(a, b, w, form="both", h=v)
        assert same(got) and untouched(wide, v), t
    h, rstd, _ = want
    base = pm.add_norm_backward(dy, dh, h, w, rstd)
    for i in range(3):
        args = [window(t) for t in (dy, dh, h)]
        dx, dw = pm.add_norm_backward(*(v for _, v in args), w, rstd, dx=args[i][1])
        assert dx is args[i][1] and torch.equal(dx, base[0]) and torch.equal(dw, base[1]) and untouched(*args[i])


def test_many_rows_accumulate_and_norm_backward():
    """More rows than one trip of every workgroup takes; dweight added to; without a
    stream's gradient the result is norm_backward's."""
    for rows, cols, dtype in ((20000, 128, torch.bfloat16), (5001, 600, torch.float32), (1500, 2500, torch.bfloat16)):
        announce(f"add norm {rows}x{cols}")
        x, r, w, dy, dh = _inputs(rows, cols, dtype)
        h, rstd, _ = pm.add_norm_quantize(x, r, w)
        before = torch.linspace(-1, 1, cols, device="cuda")
        dw = before.clone()
        got = pm.add_norm_backward(dy, dh, h, w, rstd, dweight=dw, accumulate=True)
        assert got[1] is dw
        _check_backward(got, dy, dh, h, w, rstd, dtype, "accumulate", _np(before))
        plain = pm.norm_backward(dy, h, w, None, rstd)
        zero = pm.add_norm_backward(dy, torch.zeros_like(dh), h, w, rstd)
        assert torch.equal(zero[0].float() + 0.0, plain[0].float() + 0.0) and torch.equal(zero[1], plain[1])


def test_given_operands_empty_and_streams():
    announce("add norm operands, empty, streams")
    x, r, w, dy, dh = _inputs(150, 300, torch.bfloat16)
    want = pm.add_norm_quantize(x, r, w, form="both")
    q, qt = pm.Fp8Matrix.empty(150, 300), pm.Fp8Matrix.empty(300, 150)
    got = pm.add_norm_quantize(x, r, w, form="both", out=q, out_t=qt)
    assert got[2][0] is q and got[2][1] is qt
    assert torch.equal(q.data.view(torch.uint8), want[2][0].data.view(torch.uint8))
    none = torch.empty((0, 300), dtype=torch.bfloat16, device="cuda")
    h, rstd, m = pm.add_norm_quantize(none, none, w)
    assert h.shape == (0, 300) and rstd.shape == (0,) and m.rows == 0
    dx, dw = pm.add_norm_backward(none, none, none, w, rstd)
    assert dx.shape == (0, 300) and (dw == 0).all()
    base = pm.add_norm_backward(dy, dh, want[0], w, want[1])
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        h, rstd, (a, b) = pm.add_norm_quantize(x, r, w, form="both", stream=st)
        dx, dw = pm.add_norm_backward(dy, dh, h, w, rstd, stream=st)
        torch.cuda.synchronize()
        assert torch.equal(h, want[0]) and torch.equal(dx, base[0]) and torch.equal(dw, base[1])
        assert torch.equal(b.data.view(torch.uint8), want[2][1].data.view(torch.uint8))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, rstd, (a, b) = pm.add_norm_quantize(x, r, w, form="both")
        dx, dw = pm.add_norm_backward(dy, dh, h, w, rstd)
    for _ in range(4):
        for t in (h, rstd, dx, dw):
            t.fill_(5.0)
        graph.replay()
        pm.add_norm_quantize(x, r, w, form="both")
        torch.cuda.synchronize()
        assert torch.equal(h, want[0]) and torch.equal(dx, base[0]) and torch.equal(dw, base[1])
        assert torch.equal(a.data.view(torch.uint8), want[2][0].data.view(torch.uint8))


def test_python_refusals():
    announce("add norm refusals")
    x, r, w, dy, dh = _inputs(8, 96, torch.bfloat16)
    h, rstd, q = pm.add_norm_quantize(x, r, w)
    bad = [lambda: pm.add_norm_quantize(x, r, w, form="rows"), lambda: pm.add_norm_quantize(x, r.float(), w),
           lambda: pm.add_norm_quantize(x, r[:4], w), lambda: pm.add_norm_quantize(x, r, w[:95]),
           lambda: pm.add_norm_quantize(x, None, w, h=r), lambda: pm.add_norm_quantize(x, r, w, form="col", out=q),
           lambda: pm.add_norm_quantize(x, r, w, out=pm.Fp8Matrix.empty(8, 97)), lambda: pm.add_norm_quantize(x.cpu(), r, w),
           lambda: pm.add_norm_quantize(x, r, w, out=pm.Fp8Matrix.empty(8, 96, 128)),
           lambda: pm.add_norm_quantize(x[0], r, w), lambda: pm.add_norm_quantize(x.t(), r.t(), w),
           lambda: pm.add_norm_backward(dy.float(), dh, h, w, rstd), lambda: pm.add_norm_backward(dy, dh[:4], h, w, rstd),
           lambda: pm.add_norm_backward(dy, dh, h, w, rstd[:4]), lambda: pm.add_norm_backward(dy, dh, h, w, rstd, accumulate=True)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        pm.add_norm_quantize(x.half(), r.half(), w)
    with pytest.raises(pm.MuonHError):
        pm.add_norm_quantize(x, r, w, eps=-1.0)
    shifted = torch.empty(9 * 96, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pm.MuonHError):
        pm.add_norm_quantize(shifted[:768].view(8, 96), r, w, h=shifted[32:800].view(8, 96))
