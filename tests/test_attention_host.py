"""Argument checks of the attention's C entry points (CPU only): every refused call
returns its status before any device work."""

import ctypes
import os

import pytest

import pretraining_optimizer_amd as pm
from pretraining_optimizer_amd import muonh as mb

BASE = 1 << 40     # never dereferenced: the calls below are refused, or have nothing to do


def _args(**kw):
    f = dict(q=BASE, k=BASE * 2, v=BASE * 3, out=BASE * 4, lse=BASE * 5, cu_seqlens=BASE * 6, tokens=300, sequences=2,
             ld_q=1024, ld_k=512, ld_v=512, ld_out=1024, heads=8, kv_heads=4, dim=128, scale=0.1)
    f.update(kw)
    return mb.muonh_attention_args(**f)


def _grad(**kw):
    own = dict(dout=BASE * 7, dq=BASE * 8, dk=BASE * 9, dv=BASE * 10, ld_dout=1024, ld_dq=1024, ld_dk=512, ld_dv=512,
               workspace=BASE * 11, workspace_bytes=1 << 30)
    for name in list(kw):
        if name in own:
            own[name] = kw.pop(name)
    return mb.muonh_attention_grad_args(a=_args(**kw), **own)


def _refused(rc, status, text):
    assert rc == status, (rc, pm.load_library().muonh_last_error())
    assert text in pm.load_library().muonh_last_error().decode()


SHAPES = [
    (dict(tokens=-1), "tokens"), (dict(tokens=(1 << 30) + 1), "tokens"), (dict(sequences=-1), "sequences"),
    (dict(heads=6), "multiple of kv_heads"), (dict(heads=0), "heads"), (dict(kv_heads=0), "heads"), (dict(heads=-8), "heads"),
    (dict(kv_heads=-4), "heads"), (dict(dim=0), "dim"), (dict(dim=136), "dim"), (dict(dim=20), "dim"),
    (dict(scale=0.0), "scale"), (dict(scale=-1.0), "scale"), (dict(scale=float("inf")), "scale"),
    (dict(scale=float("nan")), "scale"), (dict(tokens=1 << 30, sequences=1 << 30), "too many"),
    (dict(tokens=1 << 27, heads=1 << 16, kv_heads=1 << 16, dim=8, ld_q=1 << 19, ld_k=1 << 19, ld_v=1 << 19, ld_out=1 << 19), "too many"),
]
FORWARD = SHAPES + [
    (dict(ld_q=1016), "q: the pitch"), (dict(ld_k=511), "k: the pitch"), (dict(ld_v=515), "v: the pitch"),
    (dict(ld_out=1 << 23), "out: the pitch"), (dict(q=None), "null pointer: q"), (dict(out=None), "null pointer: out"),
    (dict(lse=None), "null pointer"), (dict(cu_seqlens=None), "null pointer"), (dict(k=BASE * 2 + 8), "k must be 16-byte"),
    (dict(out=BASE * 4 + 2), "out must be 16-byte"), (dict(lse=BASE * 5 + 2), "misaligned"), (dict(cu_seqlens=BASE * 6 + 1), "misaligned"),
    (dict(out=BASE), "out overlaps q"), (dict(out=BASE * 2 + 16), "out overlaps k"), (dict(lse=BASE * 4 + 64), "out overlaps lse"),
    (dict(lse=BASE * 3 + 64), "overlaps v"), (dict(lse=BASE * 6), "overlap"),
    # slices of one fused buffer that share a column
    (dict(q=BASE, out=BASE + 2 * 1016, ld_q=2048, ld_out=2048), "out overlaps q"),
]


@pytest.mark.parametrize("kw,text", FORWARD)
def test_forward_refusals(kw, text):
    _refused(pm.load_library().muonh_attention_forward(ctypes.byref(_args(**kw)), None), mb.MUONH_EINVAL, text)


BACKWARD = SHAPES + [
    (dict(ld_dq=1000), "dq: the pitch"), (dict(ld_dk=508), "dk: the pitch"), (dict(ld_dv=520 - 4), "dv: the pitch"),
    (dict(ld_dout=1025), "dout: the pitch"), (dict(dout=None), "null pointer: dout"), (dict(dk=None), "null pointer: dk"),
    (dict(out=None), "null pointer: out"), (dict(lse=None), "null pointer"), (dict(dv=BASE * 10 + 8), "dv must be 16-byte"),
    (dict(dq=BASE * 7), "dq overlaps dout"), (dict(dk=BASE * 2), "dk overlaps k"), (dict(dv=BASE * 9 + 256), "dk overlaps dv"),
    (dict(dq=BASE * 5), "dq overlaps lse"), (dict(workspace=BASE * 11 + 16), "256-byte"), (dict(workspace=BASE * 7), "overlaps dout"),
    (dict(workspace=BASE * 8), "overlaps"), (dict(workspace=BASE * 5), "overlap"),
]


@pytest.mark.parametrize("kw,text", BACKWARD)
def test_backward_refusals(kw, text):
    _refused(pm.load_library().muonh_attention_backward(ctypes.byref(_grad(**kw)), None), mb.MUONH_EINVAL, text)


def test_workspace_and_null():
    lib = pm.load_library()
    need = ctypes.c_size_t()
    assert lib.muonh_attention_backward_workspace(ctypes.byref(_args()), ctypes.byref(need)) == mb.MUONH_OK
    assert need.value >= 2 * 8 * 300 * 4
    _refused(lib.muonh_attention_backward(ctypes.byref(_grad(workspace_bytes=need.value - 1)), None), mb.MUONH_ENOMEM, str(need.value))
    _refused(lib.muonh_attention_backward(ctypes.byref(_grad(workspace=None)), None), mb.MUONH_ENOMEM, "workspace")
    _refused(lib.muonh_attention_backward_workspace(ctypes.byref(_args()), None), mb.MUONH_EINVAL, "null")
    _refused(lib.muonh_attention_backward_workspace(ctypes.byref(_args(dim=4)), ctypes.byref(need)), mb.MUONH_EINVAL, "dim")
    _refused(lib.muonh_attention_forward(None, None), mb.MUONH_EINVAL, "null")
    _refused(lib.muonh_attention_backward(None, None), mb.MUONH_EINVAL, "null")


def test_nothing_to_do_needs_no_pointer():
    lib = pm.load_library()
    none = dict(q=None, k=None, v=None, out=None, lse=None, cu_seqlens=None)
    for kw in (dict(tokens=0), dict(sequences=0)):
        assert lib.muonh_attention_forward(ctypes.byref(_args(**none, **kw)), None) == mb.MUONH_OK
        assert lib.muonh_attention_backward(ctypes.byref(_grad(**none, **kw, dout=None, dq=None, dk=None, dv=None,
                                                               workspace=None)), None) == mb.MUONH_OK
        need = ctypes.c_size_t(7)
        assert lib.muonh_attention_backward_workspace(ctypes.byref(_args(**kw)), ctypes.byref(need)) == mb.MUONH_OK
        assert need.value == 0


def test_zero_rest_is_checked():
    """Unknown bits are refused; with a bit of the call's own results there is something to do
    without sequences, too, so pointers are required."""
    lib = pm.load_library()
    forward = lambda **kw: lib.muonh_attention_forward(ctypes.byref(_args(**kw)), None)  # noqa: E731
    backward = lambda **kw: lib.muonh_attention_backward(ctypes.byref(_grad(**kw)), None)  # noqa: E731
    own = {forward: mb.MUONH_ZERO_OUT | mb.MUONH_ZERO_LSE, backward: mb.MUONH_ZERO_DQ | mb.MUONH_ZERO_DK | mb.MUONH_ZERO_DV}
    for call in (forward, backward):
        for bad in (32, -1, 64 + 1):
            _refused(call(zero_rest=bad), mb.MUONH_EINVAL, "zero_rest")
        _refused(call(reserved=1), mb.MUONH_EINVAL, "reserved")
        for bit in (1, 2, 4, 8, 16):
            rc = call(sequences=0, zero_rest=bit, q=None)
            if bit & own[call]:
                _refused(rc, mb.MUONH_EINVAL, "null pointer: q")
            else:
                assert rc == mb.MUONH_OK
        assert call(tokens=0, zero_rest=31, q=None) == mb.MUONH_OK


def test_zero_bits_are_the_headers():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "muonh.h")).read()
    for name in ("OUT", "LSE", "DQ", "DK", "DV"):
        assert f"#define MUONH_ZERO_{name} {getattr(mb, 'MUONH_ZERO_' + name)}\n" in text
