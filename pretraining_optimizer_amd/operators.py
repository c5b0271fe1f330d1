"""ctypes binding of the block-scaled FP8 operators and the norms (argument
marshalling only; the work runs in the library's HIP kernels).

One linear layer y = x W^T, its gradients and the step of its weight:

    xr, xc = fp8_quantize(x, form="both")                  # [tokens, in]
    wr, wc = fp8_quantize(w, form="both", block_rows=128)  # [out, in], fp32 master weight
    y = fp8_matmul(xr, wr)                                 # [tokens, out]
    gr, gc = fp8_quantize(dy, form="both")
    dx = fp8_matmul(gr, wc)                                # [tokens, in]
    dw = fp8_matmul(gc, xc, out_dtype=torch.float32)       # [out, in], the gradient MuonH.step takes

All tensors are on the current device.  Work is enqueued on `stream`, or on
torch's current stream.
"""

from __future__ import annotations

import ctypes
from typing import Optional

from .muonh import (MUONH_BF16, MUONH_F32, _check, _record, _stream_ptr, load_library, muonh_fp8_matrix,
                    muonh_norm_args, muonh_norm_grad_args)

NORM_KINDS = {"layer": 0, "rms": 1}
_CODES = {}


def _code(t, what: str) -> int:
    if not _CODES:
        import torch
        _CODES.update({torch.float32: MUONH_F32, torch.bfloat16: MUONH_BF16})
    try:
        return _CODES[t.dtype]
    except KeyError:
        raise TypeError(f"{what}: dtype must be float32 or bfloat16, got {t.dtype}") from None


def _here(*tensors):
    """Every tensor is on the current device."""
    import torch
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and (not t.is_cuda or t.device.index != dev):
            raise ValueError("all tensors must be CUDA tensors of the current device")


def _rows2d(t, what: str) -> int:
    """The row pitch of a matrix whose rows are contiguous."""
    if t.dim() != 2:
        raise ValueError(f"{what}: a 2-D tensor is required")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}: the elements of a row must be contiguous")
    if rows <= 1:
        return max(cols, t.stride(0))
    if t.stride(0) < cols:
        raise ValueError(f"{what}: rows overlap")
    return t.stride(0)


def _vector(t, n: int, what: str):
    import torch
    if t.dtype != torch.float32 or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous float32 vector of {n} elements is required")


def _empty(shape, dtype, device, stream):
    """A new tensor that work on `stream` may write at once: memory of that
    stream's pool, so no earlier work of another stream still uses it."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


class Fp8Matrix:
    """A block-scaled FP8 operand [rows, cols]: value = data * 2^(scale - 127).

    data       : float8_e4m3fn [rows, ld], ld a multiple of 128 >= cols, zeros
                 behind the columns
    scale      : uint8 exponents [rows or ceil(rows / 128), ld_scale], ld_scale a
                 multiple of 4 >= ceil(cols / 128)
    block_rows : 1 (a scale per row and 128 columns) or 128 (per 128 x 128)
    """

    __slots__ = ("data", "scale", "rows", "cols", "block_rows", "_desc")

    def __init__(self, data, scale, cols: int, block_rows: int = 1):
        import torch
        if data.dtype != torch.float8_e4m3fn or scale.dtype != torch.uint8:
            raise TypeError("data must be float8_e4m3fn and scale uint8")
        if data.dim() != 2 or scale.dim() != 2 or not data.is_contiguous() or not scale.is_contiguous():
            raise ValueError("data and scale must be contiguous 2-D tensors")
        if block_rows not in (1, 128):
            raise ValueError("block_rows must be 1 or 128")
        _here(data, scale)
        self.data, self.scale = data, scale
        self.rows, self.cols, self.block_rows = data.shape[0], int(cols), block_rows
        ld, lds = data.shape[1], scale.shape[1]
        if not 0 <= self.cols <= ld or ld % 128:
            raise ValueError("data: its columns must be a multiple of 128 that holds cols")
        if lds % 4 or lds * 128 < self.cols or scale.shape[0] != -(-self.rows // block_rows):
            raise ValueError("scale: shape does not fit the data's blocks")
        self._desc = muonh_fp8_matrix(data.data_ptr(), scale.data_ptr(), self.rows, self.cols, ld, lds,
                                      block_rows, 0)

    @classmethod
    def empty(cls, rows: int, cols: int, block_rows: int = 1, device=None, stream=None):
        """An operand of this shape to quantise into (uninitialised)."""
        import torch
        blocks = -(-cols // 128)
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        return cls(_empty((rows, blocks * 128), torch.float8_e4m3fn, device, stream),
                   _empty((-(-rows // block_rows), -(-blocks // 4) * 4), torch.uint8, device, stream),
                   cols, block_rows)


def fp8_quantize(x, form: str = "row", block_rows: int = 1, out: Optional[Fp8Matrix] = None,
                 out_t: Optional[Fp8Matrix] = None, stream=None):
    """Quantise x [rows, cols] (float32 or bfloat16, contiguous rows of any pitch).

    form       : "row" returns x's Fp8Matrix (contracted along its columns), "col"
                 that of x transposed (along its rows), "both" the pair
    block_rows : 1 for activations and gradients, 128 for weights
    out, out_t : operands to write instead of new ones (row form, column form)
    """
    if form not in ("row", "col", "both"):
        raise ValueError("form must be 'row', 'col' or 'both'")
    code, ldx = _code(x, "x"), _rows2d(x, "x")
    _here(x)
    rows, cols = x.shape
    q = qt = None
    if form != "col":
        q = Fp8Matrix.empty(rows, cols, block_rows, x.device, stream) if out is None else out
        if (q.rows, q.cols, q.block_rows) != (rows, cols, block_rows):
            raise ValueError("out: shape or block_rows differs")
    elif out is not None:
        raise ValueError("out is the row form, which form='col' does not write")
    if form != "row":
        qt = Fp8Matrix.empty(cols, rows, block_rows, x.device, stream) if out_t is None else out_t
        if (qt.rows, qt.cols, qt.block_rows) != (cols, rows, block_rows):
            raise ValueError("out_t: shape or block_rows differs")
    elif out_t is not None:
        raise ValueError("out_t is the column form, which form='row' does not write")
    if stream is not None:
        _record(stream, [x] + [t for m in (q, qt) if m is not None for t in (m.data, m.scale)])
    _check(load_library().muonh_block_quantize(
        x.data_ptr(), code, rows, cols, ldx, None if q is None else ctypes.byref(q._desc),
        None if qt is None else ctypes.byref(qt._desc), _stream_ptr(stream)), "muonh_block_quantize")
    return (q, qt) if form == "both" else q if qt is None else qt


def fp8_matmul(a: Fp8Matrix, b: Fp8Matrix, out=None, out_dtype=None, accumulate: bool = False, stream=None):
    """a b^T: [a.rows, b.rows], contracted over a.cols == b.cols.

    out        : matrix to write (float32 or bfloat16, contiguous rows of any
                 pitch); a new one of out_dtype (bfloat16 if None) if not given
    accumulate : add the product to what out holds
    """
    import torch
    if a.cols != b.cols:
        raise ValueError(f"the operands contract {a.cols} and {b.cols} columns")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = _empty((a.rows, b.rows), out_dtype or torch.bfloat16, a.data.device, stream)
    elif tuple(out.shape) != (a.rows, b.rows) or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError(f"out: a matrix of shape {(a.rows, b.rows)} and the asked dtype is required")
    code, ldc = _code(out, "out"), _rows2d(out, "out")
    _here(a.data, b.data, out)
    lib = load_library()
    ra, rb = ctypes.byref(a._desc), ctypes.byref(b._desc)
    need = ctypes.c_size_t()
    _check(lib.muonh_block_matmul_workspace(ra, rb, ctypes.byref(need)), "muonh_block_matmul_workspace")
    ws = _empty(need.value, torch.uint8, out.device, stream) if need.value else None
    if stream is not None:
        _record(stream, [a.data, a.scale, b.data, b.scale, out] + ([] if ws is None else [ws]))
    _check(lib.muonh_block_matmul(ra, rb, out.data_ptr(), code, ldc, 1 if accumulate else 0,
                                  None if ws is None else ws.data_ptr(), need.value, _stream_ptr(stream)),
           "muonh_block_matmul")
    return out


def _kind(kind: str) -> int:
    try:
        return NORM_KINDS[kind]
    except KeyError:
        raise ValueError("kind must be 'layer' or 'rms'") from None


def _like(out, x, what: str, stream):
    if out is None:
        return _empty(x.shape, x.dtype, x.device, stream)
    if out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError(f"{what}: shape or dtype differs from x")
    return out


def norm_forward(x, weight, bias=None, kind: str = "rms", eps: float = 1e-6, out=None, stream=None):
    """(y, mean, rstd) of the layer norm or RMS norm of x's rows.

    x            : float32 or bfloat16 [rows, cols], contiguous rows of any pitch
    weight, bias : float32 [cols]; bias may be None
    out          : y's memory; may be x itself
    mean is None for kind "rms".
    """
    import torch
    kind_code, code, ldx = _kind(kind), _code(x, "x"), _rows2d(x, "x")
    rows, cols = x.shape
    _vector(weight, cols, "weight")
    if bias is not None:
        _vector(bias, cols, "bias")
    y = _like(out, x, "out", stream)
    stats = _empty((2 if kind_code == 0 else 1, rows), torch.float32, x.device, stream)
    rstd = stats[0]
    mean = stats[1] if kind_code == 0 else None
    _here(x, weight, bias, y)
    args = muonh_norm_args(x.data_ptr(), weight.data_ptr(), None if bias is None else bias.data_ptr(),
                           y.data_ptr(), None if mean is None else mean.data_ptr(), rstd.data_ptr(), rows, cols,
                           ldx, _rows2d(y, "out"), code, kind_code, eps, 0)
    if stream is not None:
        _record(stream, [x, weight, y, stats] + ([] if bias is None else [bias]))
    _check(load_library().muonh_norm_forward(ctypes.byref(args), _stream_ptr(stream)), "muonh_norm_forward")
    return y, mean, rstd


def norm_backward(dy, x, weight, mean, rstd, kind: str = "rms", bias: bool = False, dx=None, dweight=None,
                  dbias=None, accumulate: bool = False, stream=None):
    """(dx, dweight, dbias) from the output's gradient and the forward pass's
    input and statistics; dbias is None unless bias (or dbias) is given.

    dx             : memory of dx; may be dy or x itself
    dweight, dbias : float32 [cols] to write, or with accumulate to add to
    """
    import torch
    kind_code, code, ldx = _kind(kind), _code(x, "x"), _rows2d(x, "x")
    rows, cols = x.shape
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError("dy: shape or dtype differs from x")
    _vector(weight, cols, "weight")
    _vector(rstd, rows, "rstd")
    if (mean is None) != (kind_code == 1):
        raise ValueError("mean is the layer norm's, and None for kind 'rms'")
    if mean is not None:
        _vector(mean, rows, "mean")
    dx = _like(dx, x, "dx", stream)
    if accumulate and (dweight is None or (bias and dbias is None)):
        raise ValueError("accumulate needs dweight (and dbias)")
    if dweight is None:
        dweight = _empty(cols, torch.float32, x.device, stream)
    if bias and dbias is None:
        dbias = _empty(cols, torch.float32, x.device, stream)
    _vector(dweight, cols, "dweight")
    if dbias is not None:
        _vector(dbias, cols, "dbias")
    _here(dy, x, weight, mean, rstd, dx, dweight, dbias)
    lib = load_library()
    need = ctypes.c_size_t()
    _check(lib.muonh_norm_backward_workspace(rows, cols, ctypes.byref(need)), "muonh_norm_backward_workspace")
    ws = _empty(max(need.value, 1), torch.uint8, x.device, stream)
    args = muonh_norm_grad_args(
        dy.data_ptr(), x.data_ptr(), weight.data_ptr(), None if mean is None else mean.data_ptr(), rstd.data_ptr(),
        dx.data_ptr(), dweight.data_ptr(), None if dbias is None else dbias.data_ptr(), rows, cols,
        _rows2d(dy, "dy"), ldx, _rows2d(dx, "dx"), code, kind_code, 1 if accumulate else 0, 0, ws.data_ptr(),
        need.value)
    if stream is not None:
        _record(stream, [t for t in (dy, x, weight, mean, rstd, dx, dweight, dbias, ws) if t is not None])
    _check(lib.muonh_norm_backward(ctypes.byref(args), _stream_ptr(stream)), "muonh_norm_backward")
    return dx, dweight, dbias
