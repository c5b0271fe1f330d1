"""Argument checks of the residual norm's and the embedding's C entry points (CPU
only): every refused call returns its status before any device work."""

import ctypes

import pytest

import pretraining_optimizer_amd as pm
from pretraining_optimizer_amd import muonh as mb

BASE = 1 << 40     # never dereferenced: the calls below are refused, or have nothing to do


def _refused(rc, status, text):
    assert rc == status, (rc, pm.load_library().muonh_last_error())
    assert text in pm.load_library().muonh_last_error().decode()


def _mat(rows, cols, data, block=1, ld=None, lds=None):
    ld = -(-cols // 128) * 128 if ld is None else ld
    return mb.muonh_fp8_matrix(data, data + (1 << 36), rows, cols, ld, -(-ld // 512) * 4 if lds is None else lds, block, 0)


def _add_norm(q="q", qt="qt", **kw):
    f = dict(x=BASE, residual=BASE * 2, weight=BASE * 3, h=BASE * 4, rstd=BASE * 5, rows=40, cols=300, ldx=300, ld_residual=300,
             ldh=300, dtype=pm.MUONH_BF16, eps=1e-6)
    f.update(kw)
    q = _mat(40, 300, BASE * 6) if q == "q" else q
    qt = _mat(300, 40, BASE * 7) if qt == "qt" else qt
    args = mb.muonh_add_norm_args(**f)
    return pm.load_library().muonh_add_norm_quantize(ctypes.byref(args), q and ctypes.byref(q), qt and ctypes.byref(qt), None)


ADD_NORM = [
    (dict(q=None, qt=None), "neither form"), (dict(dtype=2), "dtype"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"),
    (dict(rows=-1), "rows"), (dict(cols=0), "cols"), (dict(cols=(1 << 26) + 1), "cols"), (dict(ldx=299), "ldx"),
    (dict(ld_residual=299), "ld_residual"), (dict(ldh=1), "ldh"), (dict(residual=None), "h must be NULL"), (dict(h=None), "null"),
    (dict(x=None), "null"), (dict(weight=None), "null"), (dict(rstd=None), "null"), (dict(x=BASE + 1), "misaligned"),
    (dict(weight=BASE * 3 + 2), "misaligned"), (dict(rstd=BASE * 5 + 2), "misaligned"), (dict(h=BASE + 4), "h overlaps"),
    (dict(h=BASE * 2, ldh=301), "h overlaps"), (dict(rstd=BASE), "overlaps"), (dict(rstd=BASE * 3), "overlaps"),
    (dict(h=BASE * 3), "overlaps"), (dict(rstd=BASE * 4 + 16), "overlaps"),
    (dict(q=_mat(39, 300, BASE * 6)), "q: shape"), (dict(qt=_mat(40, 300, BASE * 7)), "qt: shape"),
    (dict(q=_mat(40, 300, BASE * 6, block=128)), "block_rows must be 1"), (dict(q=_mat(40, 300, BASE)), "FP8 output overlaps"),
    (dict(q=_mat(40, 300, BASE * 4 + 16)), "FP8 output overlaps"), (dict(qt=_mat(300, 40, BASE * 6 + 128)), "FP8 output overlaps"),
    (dict(qt=_mat(300, 40, BASE * 5)), "FP8 output overlaps"), (dict(q=_mat(40, 300, BASE * 6 + 8)), "16-byte"),
]


@pytest.mark.parametrize("kw,text", ADD_NORM)
def test_add_norm_refusals(kw, text):
    _refused(_add_norm(**kw), mb.MUONH_EINVAL, text)


def test_add_norm_too_large_and_empty():
    rows, cols = 1 << 30, 1 << 26
    big = _mat(rows, cols, 1 << 59, lds=1 << 19)
    _refused(_add_norm(q=big, qt=None, rows=rows, cols=cols, ldx=cols, residual=None, h=None), mb.MUONH_EINVAL, "")
    none = dict(x=None, residual=None, weight=None, h=None, rstd=None, rows=0)
    empty = mb.muonh_fp8_matrix(None, None, 0, 300, 384, 4, 1, 0)
    assert _add_norm(q=empty, qt=None, **none) == mb.MUONH_OK
    _refused(pm.load_library().muonh_add_norm_quantize(None, None, None, None), mb.MUONH_EINVAL, "null")


def _grad(**kw):
    f = dict(dy=BASE, x=BASE * 2, weight=BASE * 3, mean=None, rstd=BASE * 4, dx=BASE * 5, dweight=BASE * 6, dbias=None,
             rows=8, cols=96, ld_dy=96, ldx=96, ld_dx=96, dtype=pm.MUONH_BF16, kind=1, accumulate=0, reserved=0,
             workspace=BASE * 7, workspace_bytes=1 << 30)
    own = dict(dh=BASE * 8, ld_dh=96)
    own.update({k: kw.pop(k) for k in list(kw) if k in own})
    f.update(kw)
    args = mb.muonh_add_norm_grad_args(g=mb.muonh_norm_grad_args(**f), **own)
    return pm.load_library().muonh_add_norm_backward(ctypes.byref(args), None)


GRAD = [
    (dict(dtype=3), "dtype"), (dict(kind=0), "kind"), (dict(reserved=1), "reserved"), (dict(accumulate=2), "accumulate"),
    (dict(rows=-1), "rows"), (dict(cols=0), "cols"), (dict(ldx=95), "ldx"), (dict(ld_dy=95), "ld_dy"), (dict(ld_dx=95), "ld_dx"),
    (dict(ld_dh=95), "ld_dh"), (dict(mean=BASE * 9), "must be NULL"), (dict(dbias=BASE * 9), "must be NULL"),
    (dict(dy=None), "null"), (dict(dh=None), "null"), (dict(dx=None), "null"), (dict(weight=None), "null"), (dict(dweight=None), "null"),
    (dict(dh=BASE * 8 + 1), "misaligned"), (dict(dweight=BASE * 6 + 2), "misaligned"), (dict(dx=BASE * 8 + 2), "dx overlaps"),
    (dict(dx=BASE * 8, ld_dx=128), "dx overlaps"), (dict(dweight=BASE * 8), "overlaps"), (dict(workspace=BASE * 8), "overlaps"),
    (dict(workspace=BASE * 7 + 16), "256-byte"),
]


@pytest.mark.parametrize("kw,text", GRAD)
def test_add_norm_backward_refusals(kw, text):
    _refused(_grad(**kw), mb.MUONH_EINVAL, text)


def test_add_norm_backward_workspace():
    _refused(_grad(workspace=None), mb.MUONH_ENOMEM, "workspace")
    _refused(_grad(workspace_bytes=8), mb.MUONH_ENOMEM, "workspace")
    _refused(pm.load_library().muonh_add_norm_backward(None, None), mb.MUONH_EINVAL, "null")


def _embed(**kw):
    f = dict(tokens=BASE, table=BASE * 2, out=BASE * 3, count=50, rows=100, cols=64, ld_table=64, ld_out=64, token_bytes=8,
             table_dtype=pm.MUONH_F32, out_dtype=pm.MUONH_BF16, scale=1.0)
    f.update(kw)
    return pm.load_library().muonh_embedding_forward(ctypes.byref(mb.muonh_embedding_args(**f)), None)


SIZES = [
    (dict(count=-1), "count"), (dict(count=(1 << 30) + 1), "count"), (dict(rows=-1), "rows"), (dict(rows=(1 << 30) + 1), "rows"),
    (dict(cols=0), "cols"), (dict(cols=(1 << 20) + 1), "cols"), (dict(count=1 << 24), "too large"), (dict(token_bytes=2), "token_bytes"),
    (dict(table_dtype=2), "dtype"), (dict(ld_table=63), "ld_table"), (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"),
    (dict(tokens=None), "null"), (dict(tokens=BASE + 4), "misaligned"),
]
EMBED = SIZES + [(dict(out_dtype=-1), "dtype"), (dict(ld_out=63), "ld_out"), (dict(table=None), "null"), (dict(out=None), "null"),
                 (dict(table=BASE * 2 + 2), "misaligned"), (dict(out=BASE * 3 + 1), "misaligned"), (dict(out=BASE * 2 + 64), "overlaps"),
                 (dict(out=BASE + 8), "overlaps")]


@pytest.mark.parametrize("kw,text", EMBED)
def test_embedding_refusals(kw, text):
    _refused(_embed(**kw), mb.MUONH_EINVAL, text)


def _embed_grad(**kw):
    f = dict(tokens=BASE, dout=BASE * 2, dtable=BASE * 3, count=50, rows=100, cols=64, ld_dout=64, ld_table=64, token_bytes=8,
             dout_dtype=pm.MUONH_BF16, table_dtype=pm.MUONH_F32, accumulate=0, scale=1.0, reserved=0, workspace=BASE * 4,
             workspace_bytes=1 << 40)
    f.update(kw)
    return pm.load_library().muonh_embedding_backward(ctypes.byref(mb.muonh_embedding_grad_args(**f)), None)


EMBED_GRAD = SIZES + [(dict(dout_dtype=2), "dtype"), (dict(ld_dout=63), "ld_dout"), (dict(accumulate=2), "accumulate"),
                      (dict(reserved=1), "reserved"), (dict(dout=None), "null"), (dict(dtable=None), "null"),
                      (dict(dout=BASE * 2 + 1), "misaligned"), (dict(dtable=BASE * 3 + 2), "misaligned"),
                      (dict(workspace=BASE * 4 + 128), "256-byte"), (dict(dtable=BASE * 2), "overlaps"),
                      (dict(workspace=BASE), "overlaps"), (dict(workspace=BASE * 3), "overlaps")]


@pytest.mark.parametrize("kw,text", EMBED_GRAD)
def test_embedding_backward_refusals(kw, text):
    _refused(_embed_grad(**kw), mb.MUONH_EINVAL, text)


def test_embedding_workspace_and_empty():
    lib = pm.load_library()
    need = ctypes.c_size_t()
    for count, rows in ((1, 10), (16, 10), (17, 10), (8192, 151936), (8193, 151936), (70000, 3)):
        assert lib.muonh_embedding_backward_workspace(count, rows, 64, ctypes.byref(need)) == mb.MUONH_OK
        assert need.value >= 16 * count and need.value % 256 == 0
        _refused(_embed_grad(count=count, rows=rows, workspace_bytes=need.value - 1), mb.MUONH_ENOMEM, str(need.value))
    _refused(_embed_grad(workspace=None), mb.MUONH_ENOMEM, "workspace")
    assert lib.muonh_embedding_backward_workspace(0, 5, 64, ctypes.byref(need)) == mb.MUONH_OK and need.value == 0
    _refused(lib.muonh_embedding_backward_workspace(5, 5, 64, None), mb.MUONH_EINVAL, "null")
    _refused(lib.muonh_embedding_backward_workspace(5, 5, 0, ctypes.byref(need)), mb.MUONH_EINVAL, "cols")
    assert _embed(count=0, tokens=None, table=None, out=None) == mb.MUONH_OK
    none = dict(tokens=None, dout=None, dtable=None, workspace=None)
    assert _embed_grad(count=0, accumulate=1, **none) == mb.MUONH_OK
    assert _embed_grad(rows=0, **none) == mb.MUONH_OK
    _refused(lib.muonh_embedding_forward(None, None), mb.MUONH_EINVAL, "null")
    _refused(lib.muonh_embedding_backward(None, None), mb.MUONH_EINVAL, "null")


def test_embedding_counts():
    """The most tokens do not depend on the columns."""
    lib = pm.load_library()
    need = ctypes.c_size_t()
    most = (1 << 24) - 1
    for cols in (1, 64, 4096, 1 << 20):
        assert lib.muonh_embedding_backward_workspace(most, 300, cols, ctypes.byref(need)) == mb.MUONH_OK
        _refused(lib.muonh_embedding_backward_workspace(most + 1, 300, cols, ctypes.byref(need)), mb.MUONH_EINVAL, "count")
        wide = dict(cols=cols, ld_table=cols, count=most)
        # past the sizes, to the next check
        _refused(_embed(**wide, ld_out=cols, tokens=None), mb.MUONH_EINVAL, "null")
        _refused(_embed_grad(**wide, ld_dout=cols, tokens=None), mb.MUONH_EINVAL, "null")
