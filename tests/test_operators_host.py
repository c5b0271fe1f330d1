"""Argument checks of the FP8 operators' and the norms' C entry points (CPU
only): every refused call returns its status before any device work."""

import ctypes

import pytest

import pretraining_optimizer_amd as pm
from pretraining_optimizer_amd import muonh as mb

BASE = 1 << 40     # never dereferenced: the calls below are refused, or have nothing to do


def _mat(rows=256, cols=256, ld=None, lds=None, block=1, data=BASE, scale=BASE + (1 << 32), reserved=0):
    ld = -(-cols // 128) * 128 if ld is None else ld
    lds = -(-ld // 512) * 4 if lds is None else lds
    return mb.muonh_fp8_matrix(data, scale, rows, cols, ld, lds, block, reserved)


def _refused(rc, status, text):
    assert rc == status, (rc, pm.load_library().muonh_last_error())
    assert text in pm.load_library().muonh_last_error().decode()


BAD_MATRIX = [
    (dict(rows=-1), "rows"), (dict(cols=-1, ld=128, lds=4), "cols"), (dict(block=64), "block_rows"), (dict(reserved=1), "reserved"),
    (dict(ld=128), "ld"), (dict(ld=300), "multiple of 128"), (dict(lds=3), "multiple of 4"), (dict(lds=0), "ld_scale"),
    (dict(data=None), "null"), (dict(scale=None), "null"), (dict(data=BASE + 8), "aligned"), (dict(scale=BASE + 1), "aligned"),
    (dict(rows=(1 << 30) + 1), "rows"),
]


@pytest.mark.parametrize("kw,text", BAD_MATRIX)
def test_matmul_refuses_bad_operands(kw, text):
    lib = pm.load_library()
    bad, good = _mat(**kw), _mat(cols=kw.get("cols", 256) if kw.get("cols", 256) > 0 else 256)
    for a, b in ((bad, good), (good, bad)):
        rc = lib.muonh_block_matmul(ctypes.byref(a), ctypes.byref(b), BASE * 2, pm.MUONH_F32, 1 << 31, 0, None, 0, None)
        _refused(rc, mb.MUONH_EINVAL, text)


def test_matmul_refusals():
    lib = pm.load_library()

    def call(a=None, b=None, c=BASE * 2, dtype=pm.MUONH_F32, ldc=256, acc=0):
        a, b = _mat() if a is None else a, _mat(data=BASE * 4, scale=BASE * 5) if b is None else b
        return lib.muonh_block_matmul(ctypes.byref(a), ctypes.byref(b), c, dtype, ldc, acc, None, 0, None)

    _refused(call(b=_mat(cols=128)), mb.MUONH_EINVAL, "a.cols differs")
    _refused(call(c=None), mb.MUONH_EINVAL, "null c")
    _refused(call(c=BASE * 2 + 2), mb.MUONH_EINVAL, "misaligned c")
    _refused(call(dtype=2), mb.MUONH_EINVAL, "dtype")
    _refused(call(ldc=255), mb.MUONH_EINVAL, "ldc")
    _refused(call(acc=2), mb.MUONH_EINVAL, "accumulate")
    _refused(call(c=BASE + 1024), mb.MUONH_EINVAL, "overlaps")
    _refused(call(c=BASE + (1 << 32) - 256), mb.MUONH_EINVAL, "overlaps")
    _refused(call(a=_mat(rows=1 << 26), b=_mat(rows=1 << 26, data=BASE * 4, scale=BASE * 5), c=BASE << 12, ldc=1 << 26),
             mb.MUONH_EINVAL, "too large")
    _refused(lib.muonh_block_matmul(None, None, BASE, 0, 1, 0, None, 0, None), mb.MUONH_EINVAL, "null operand")
    # nothing to compute: no pointer is needed
    empty = _mat(rows=0, data=None, scale=None)
    assert call(a=empty, c=None) == mb.MUONH_OK and call(b=empty, c=None, ldc=0) == mb.MUONH_OK
    need = ctypes.c_size_t(7)
    assert lib.muonh_block_matmul_workspace(ctypes.byref(_mat()), ctypes.byref(_mat()), pm.MUONH_BF16, ctypes.byref(need)) == mb.MUONH_OK
    _refused(lib.muonh_block_matmul_workspace(ctypes.byref(_mat()), ctypes.byref(_mat()), pm.MUONH_BF16, None), mb.MUONH_EINVAL, "null")


def test_quantize_refusals():
    lib = pm.load_library()

    def call(x=BASE * 2, dtype=pm.MUONH_BF16, rows=256, cols=384, ldx=384, q="q", qt="qt"):
        q = _mat(rows, cols) if q == "q" else q
        qt = _mat(cols, rows, data=BASE * 4, scale=BASE * 5) if qt == "qt" else qt
        return lib.muonh_block_quantize(x, dtype, rows, cols, ldx, q and ctypes.byref(q), qt and ctypes.byref(qt), None)

    _refused(call(q=None, qt=None), mb.MUONH_EINVAL, "neither form")
    _refused(call(dtype=7), mb.MUONH_EINVAL, "dtype")
    _refused(call(ldx=383), mb.MUONH_EINVAL, "ldx")
    _refused(call(x=None), mb.MUONH_EINVAL, "null x")
    _refused(call(x=BASE * 2 + 1), mb.MUONH_EINVAL, "misaligned")
    _refused(call(q=_mat(255, 384)), mb.MUONH_EINVAL, "q: shape")
    _refused(call(qt=_mat(384, 255, data=BASE * 4, scale=BASE * 5)), mb.MUONH_EINVAL, "qt: shape")
    _refused(call(q=_mat(256, 384, block=128)), mb.MUONH_EINVAL, "block_rows differ")
    _refused(call(q=_mat(256, 384, data=BASE * 2 + 4096)), mb.MUONH_EINVAL, "overlap")
    _refused(call(q=_mat(256, 384, scale=BASE + 16)), mb.MUONH_EINVAL, "overlap")
    _refused(call(qt=_mat(384, 256, data=BASE + 128, scale=BASE * 5)), mb.MUONH_EINVAL, "overlap")
    _refused(call(rows=1 << 28, cols=1 << 28, ldx=1 << 28, q=_mat(1 << 28, 1 << 28, lds=1 << 21, scale=BASE << 22),
                  qt=None, x=BASE << 20), mb.MUONH_EINVAL, "too large")
    # empty matrices need no pointer
    assert call(x=None, rows=0, q=_mat(0, 384, data=None, scale=None), qt=_mat(384, 0, data=None, scale=None, ld=0, lds=0)) == mb.MUONH_OK


def _norm(**kw):
    f = dict(x=BASE, weight=BASE * 2, bias=None, y=BASE * 3, mean=None, rstd=BASE * 4, rows=8, cols=96, ldx=96, ldy=96,
             dtype=pm.MUONH_F32, kind=1, eps=1e-6, reserved=0)
    f.update(kw)
    return mb.muonh_norm_args(**f)


NORM_BAD = [
    (dict(dtype=3), "dtype"), (dict(kind=2), "kind"), (dict(reserved=1), "reserved"), (dict(eps=-1.0), "eps"),
    (dict(eps=float("nan")), "eps"), (dict(rows=-1), "rows"), (dict(cols=0), "cols"), (dict(ldx=95), "ldx"),
    (dict(cols=(1 << 26) + 1, ldx=1 << 27, ldy=1 << 27), "cols"),
    (dict(ldy=95), "ldy"), (dict(mean=BASE * 5), "mean must be NULL"), (dict(kind=0), "null"), (dict(x=None), "null"),
    (dict(weight=None), "null"), (dict(y=None), "null"), (dict(rstd=None), "null"), (dict(x=BASE + 2), "misaligned"),
    (dict(weight=BASE * 2 + 2), "misaligned"), (dict(y=BASE + 4), "overlaps"), (dict(y=BASE, ldy=128), "overlaps"),
    (dict(ldx=192, ldy=192, y=BASE + 95 * 4), "overlaps"),
]


@pytest.mark.parametrize("kw,text", NORM_BAD)
def test_norm_forward_refusals(kw, text):
    _refused(pm.load_library().muonh_norm_forward(ctypes.byref(_norm(**kw)), None), mb.MUONH_EINVAL, text)


def _grad(**kw):
    f = dict(dy=BASE, x=BASE * 2, weight=BASE * 3, mean=None, rstd=BASE * 4, dx=BASE * 5, dweight=BASE * 6, dbias=None,
             rows=8, cols=96, ld_dy=96, ldx=96, ld_dx=96, dtype=pm.MUONH_BF16, kind=1, accumulate=0, reserved=0,
             workspace=BASE * 7, workspace_bytes=1 << 30)
    f.update(kw)
    return mb.muonh_norm_grad_args(**f)


GRAD_BAD = [
    (dict(dtype=3), "dtype"), (dict(kind=-1), "kind"), (dict(reserved=1), "reserved"), (dict(accumulate=2), "accumulate"),
    (dict(rows=-1), "rows"), (dict(cols=0), "cols"), (dict(ldx=95), "ldx"), (dict(ld_dy=95), "ld_dy"),
    (dict(ld_dx=95), "ld_dx"), (dict(mean=BASE * 8), "mean must be NULL"), (dict(kind=0), "null"), (dict(dy=None), "null"),
    (dict(x=None), "null"), (dict(dx=None), "null"), (dict(rstd=None), "null"), (dict(weight=None), "null"),
    (dict(dweight=None), "null"), (dict(x=BASE * 2 + 1), "misaligned"), (dict(dweight=BASE * 6 + 2), "misaligned"),
    (dict(dx=BASE + 2), "overlaps"), (dict(dx=BASE * 2, ld_dx=128), "overlaps"), (dict(workspace=BASE * 7 + 16), "256-byte"),
]


@pytest.mark.parametrize("kw,text", GRAD_BAD)
def test_norm_backward_refusals(kw, text):
    _refused(pm.load_library().muonh_norm_backward(ctypes.byref(_grad(**kw)), None), mb.MUONH_EINVAL, text)


def test_norm_backward_workspace():
    lib = pm.load_library()
    need = ctypes.c_size_t()
    assert lib.muonh_norm_backward_workspace(8192, 2048, ctypes.byref(need)) == mb.MUONH_OK and need.value > 0
    small = _grad(rows=8192, cols=2048, ld_dy=2048, ldx=2048, ld_dx=2048, workspace_bytes=need.value - 1)
    _refused(lib.muonh_norm_backward(ctypes.byref(small), None), mb.MUONH_ENOMEM, str(need.value))
    _refused(lib.muonh_norm_backward(ctypes.byref(_grad(workspace=None)), None), mb.MUONH_ENOMEM, "workspace")
    _refused(lib.muonh_norm_backward_workspace(1, 0, ctypes.byref(need)), mb.MUONH_EINVAL, "cols")
    assert lib.muonh_norm_backward_workspace(0, 64, ctypes.byref(need)) == mb.MUONH_OK and need.value == 0


def test_empty_norm_needs_no_rows():
    lib = pm.load_library()
    assert lib.muonh_norm_forward(ctypes.byref(_norm(rows=0, x=None, y=None, rstd=None)), None) == mb.MUONH_OK
    _refused(lib.muonh_norm_forward(None, None), mb.MUONH_EINVAL, "null")
    _refused(lib.muonh_norm_backward(None, None), mb.MUONH_EINVAL, "null")


def test_quantized_step_refusals():
    lib = pm.load_library()
    mats = mb.shape_descs([(256, 128)])
    args = mb.muonh_step_args()
    q = _mat(256, 128, block=128)
    for call in ((None, mats, 1, ctypes.byref(q), None, ctypes.byref(args)),):
        _refused(lib.muonh_step_quantized(*call, None), mb.MUONH_EINVAL, "null")


VECTORS = dict(weight=BASE * 2, bias=BASE * 6, mean=BASE * 7, rstd=BASE * 4, kind=0)


@pytest.mark.parametrize("kw", [
    dict(y=BASE * 2), dict(y=BASE * 6 - 96 * 4), dict(rstd=BASE + 32), dict(mean=BASE + 95 * 4), dict(rstd=BASE * 2),
    dict(mean=BASE * 6), dict(mean=BASE * 4 + 28), dict(mean=BASE * 3 + 4),
])
def test_norm_forward_refuses_overlapping_vectors(kw):
    a = _norm(**{**VECTORS, **kw})
    _refused(pm.load_library().muonh_norm_forward(ctypes.byref(a), None), mb.MUONH_EINVAL, "overlap")


@pytest.mark.parametrize("kw", [
    dict(dweight=BASE * 3), dict(dbias=BASE * 6), dict(dbias=BASE * 6 + 95 * 4), dict(dbias=BASE * 5), dict(dweight=BASE),
    dict(dweight=BASE * 2 + 64), dict(dx=BASE * 3), dict(dx=BASE * 4 - 64), dict(dweight=BASE * 8), dict(workspace=BASE * 3),
    dict(workspace=BASE), dict(workspace=BASE * 5), dict(workspace=BASE * 6), dict(workspace=BASE * 8),
])
def test_norm_backward_refuses_overlapping_vectors(kw):
    a = _grad(**{**dict(kind=0, mean=BASE * 8, dbias=BASE * 9), **kw})
    _refused(pm.load_library().muonh_norm_backward(ctypes.byref(a), None), mb.MUONH_EINVAL, "overlap")


def test_matmul_refuses_overlapping_workspace():
    lib = pm.load_library()
    a, b = _mat(rows=400, cols=9216), _mat(rows=700, cols=9216, data=BASE * 4, scale=BASE * 5)
    need = ctypes.c_size_t()
    assert lib.muonh_block_matmul_workspace(ctypes.byref(a), ctypes.byref(b), pm.MUONH_F32, ctypes.byref(need)) == mb.MUONH_OK
    assert need.value > 0
    for ws in (BASE, BASE + (1 << 32), BASE * 4 + 256, BASE * 5, BASE * 2):
        rc = lib.muonh_block_matmul(ctypes.byref(a), ctypes.byref(b), BASE * 2, pm.MUONH_F32, 700, 0, ws, need.value, None)
        _refused(rc, mb.MUONH_EINVAL, "workspace overlaps")


def test_pitches_beyond_64_bits_are_refused():
    """rows * pitch, in bytes, has to stay below 2^63."""
    lib = pm.load_library()
    rows, ld = 1 << 30, 1 << 40
    text = "pitch"
    _refused(lib.muonh_norm_forward(ctypes.byref(_norm(rows=rows, ldx=ld)), None), mb.MUONH_EINVAL, text)
    _refused(lib.muonh_norm_forward(ctypes.byref(_norm(rows=rows, ldy=ld)), None), mb.MUONH_EINVAL, text)
    for name in ("ld_dy", "ldx", "ld_dx"):
        _refused(lib.muonh_norm_backward(ctypes.byref(_grad(rows=rows, **{name: ld})), None), mb.MUONH_EINVAL, text)
    for m in (_mat(rows=rows, ld=ld), _mat(rows=rows, lds=ld)):
        rc = lib.muonh_block_matmul(ctypes.byref(m), ctypes.byref(_mat()), BASE * 8, 0, 256, 0, None, 0, None)
        _refused(rc, mb.MUONH_EINVAL, text)
        rc = lib.muonh_block_quantize(BASE * 8, 0, rows, 256, 256, ctypes.byref(m), None, None)
        _refused(rc, mb.MUONH_EINVAL, text)
    rc = lib.muonh_block_matmul(ctypes.byref(_mat(rows=rows)), ctypes.byref(_mat()), BASE * 8, 0, ld, 0, None, 0, None)
    _refused(rc, mb.MUONH_EINVAL, text)
    rc = lib.muonh_block_quantize(BASE * 8, 0, rows, 256, ld, ctypes.byref(_mat(rows=rows)), None, None)
    _refused(rc, mb.MUONH_EINVAL, text)
