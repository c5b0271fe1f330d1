"""ctypes binding of the block-scaled FP8 operators, the norms, the attention and
the embedding (argument marshalling only; the work runs in the library's HIP kernels).

One linear layer y = x W^T, its gradients and the step of its weight:

    xr, xc = fp8_quantize(x, form="both")                  # [tokens, in]
    wr, wc = fp8_quantize(w, form="both", block_rows=128)  # [out, in], fp32 master weight
    y = fp8_matmul(xr, wr)                                 # [tokens, out]
    gr, gc = fp8_quantize(dy, form="both")
    dx = fp8_matmul(gr, wc)                                # [tokens, in]
    dw = fp8_matmul(gc, xc, out_dtype=torch.float32)       # [out, in], the gradient MuonH.step takes (or .bfloat16())

Between such layers, each with its gradient:

    x = embedding_forward(tokens, table)                   # the residual stream
    h, rstd, (nr, nc) = add_norm_quantize(y, x, gamma, form="both")   # h = y + x, its norm in FP8
    out, lse = attention_forward(q, k, v, cu_seqlens)      # heads of a product's output

All tensors are on the current device.  Work is enqueued on `stream`, or on
torch's current stream.
"""

from __future__ import annotations

import ctypes
from typing import Optional

from .muonh import (MUONH_BF16, MUONH_F32, MUONH_ZERO_DK, MUONH_ZERO_DQ, MUONH_ZERO_DV, MUONH_ZERO_LSE,
                    MUONH_ZERO_OUT, _check, _record, load_library, muonh_add_norm_args, muonh_add_norm_grad_args,
                    muonh_attention_args, muonh_attention_grad_args, muonh_embedding_args, muonh_embedding_grad_args,
                    muonh_fp8_matrix, muonh_norm_args, muonh_norm_grad_args)

# The smallest calls are bound by this module: a launch takes about 3.5 us,
# a tensor 1.5 us, torch.cuda.current_stream() 2.8 us.  So the library and
# torch are looked up once, and the current stream is read as a raw pointer.
NORM_KINDS = {"layer": 0, "rms": 1}
_torch = None
_lib = None
_CODES = {}


def _setup():
    global _torch, _lib
    import torch
    _lib = load_library()
    _CODES.update({torch.float32: MUONH_F32, torch.bfloat16: MUONH_BF16})
    _torch = torch


def _code(t, what: str) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{what}: dtype must be float32 or bfloat16, got {t.dtype}")
    return code


def _here(first, *rest) -> int:
    """Every tensor is on the current device, whose index is returned."""
    dev = first.get_device()
    for t in rest:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors must be CUDA tensors of the current device")
    if dev < 0 or dev != _torch.cuda.current_device():
        raise ValueError("all tensors must be CUDA tensors of the current device")
    return dev


def _stream(stream, dev: int) -> int:
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(dev)
    if stream.device.index != dev:
        raise ValueError("stream: of another device than the tensors")
    return stream.cuda_stream


def _pitch(t, rows: int, cols: int, what: str) -> int:
    """The row pitch of a matrix whose rows are contiguous."""
    s0, s1 = t.stride()
    if cols > 1 and s1 != 1:
        raise ValueError(f"{what}: the elements of a row must be contiguous")
    if rows <= 1:
        return max(cols, s0)
    if s0 < cols:
        raise ValueError(f"{what}: rows overlap")
    return s0


def _matrix(t, what: str):
    """(rows, cols, row pitch) of a 2-D tensor."""
    if t.dim() != 2:
        raise ValueError(f"{what}: a 2-D tensor is required")
    rows, cols = t.shape
    return rows, cols, _pitch(t, rows, cols, what)


def _vector(t, n: int, what: str):
    if t.dtype is not _torch.float32 or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous float32 vector of {n} elements is required")


def _on(stream, make, result=True):
    """A new tensor that work on `stream` may write at once: memory of that
    stream's pool, so no earlier work of another stream still uses it.  A result is
    used on torch's current stream afterwards (behind a wait), so its memory returns
    to the pool only behind that stream's work."""
    user = _torch.cuda.current_stream()
    with _torch.cuda.stream(stream):
        t = make()
    if result and user != stream:
        t.record_stream(user)
    return t


def _empty(shape, dtype, device, stream):
    """A new tensor for work on `stream`, or on torch's current stream."""
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=device)
    return _on(stream, lambda: _torch.empty(shape, dtype=dtype, device=device))


def _like(t, shape, stream, result=True):
    """_empty of t's dtype and device (the quicker call)."""
    if stream is None:
        return t.new_empty(shape)
    return _on(stream, lambda: t.new_empty(shape), result)


class Fp8Matrix:
    """A block-scaled FP8 operand [rows, cols]: value = data * 2^(scale - 127).

    data       : float8_e4m3fn [rows, ld], ld a multiple of 128 >= cols, zeros
                 behind the columns
    scale      : uint8 exponents [rows or ceil(rows / 128), ld_scale], ld_scale a
                 multiple of 4 >= ceil(cols / 128)
    block_rows : 1 (a scale per row and 128 columns) or 128 (per 128 x 128)

    The tensors' contents may change, the tensors themselves not (they are
    read-only attributes, and the library is given their addresses).
    """

    __slots__ = ("_data", "_scale", "_rows", "_cols", "_block_rows", "_desc")

    data = property(lambda self: self._data)
    scale = property(lambda self: self._scale)
    rows = property(lambda self: self._rows)
    cols = property(lambda self: self._cols)
    block_rows = property(lambda self: self._block_rows)

    def __init__(self, data, scale, cols: int, block_rows: int = 1):
        if _torch is None:
            _setup()
        if data.dtype is not _torch.float8_e4m3fn or scale.dtype is not _torch.uint8:
            raise TypeError("data must be float8_e4m3fn and scale uint8")
        if data.dim() != 2 or scale.dim() != 2 or not data.is_contiguous() or not scale.is_contiguous():
            raise ValueError("data and scale must be contiguous 2-D tensors")
        if block_rows != 1 and block_rows != 128:
            raise ValueError("block_rows must be 1 or 128")
        _here(data, scale)
        rows, ld = data.shape
        srows, lds = scale.shape
        cols = int(cols)
        if not 0 <= cols <= ld or ld % 128:
            raise ValueError("data: its columns must be a multiple of 128 that holds cols")
        if lds % 4 or lds * 128 < cols or srows != (rows + block_rows - 1) // block_rows:
            raise ValueError("scale: shape does not fit the data's blocks")
        self._data, self._scale = data, scale
        self._rows, self._cols, self._block_rows = rows, cols, block_rows
        self._desc = muonh_fp8_matrix(data.data_ptr(), scale.data_ptr(), rows, cols, ld, lds, block_rows, 0)

    @classmethod
    def empty(cls, rows: int, cols: int, block_rows: int = 1, device=None, stream=None):
        """An operand of this shape to quantise into (uninitialised)."""
        if _torch is None:
            _setup()
        if block_rows not in (1, 128):
            raise ValueError("block_rows must be 1 or 128")
        device = _torch.device("cuda", _torch.cuda.current_device()) if device is None else device
        ld = (cols + 127) // 128 * 128
        lds = (ld + 511) // 512 * 4
        m = cls.__new__(cls)
        m._rows, m._cols, m._block_rows = rows, cols, block_rows
        m._data = _empty((rows, ld), _torch.float8_e4m3fn, device, stream)
        m._scale = _empty(((rows + block_rows - 1) // block_rows, lds), _torch.uint8, device, stream)
        m._desc = muonh_fp8_matrix(m._data.data_ptr(), m._scale.data_ptr(), rows, cols, ld, lds, block_rows, 0)
        return m


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
    if _torch is None:
        _setup()
    code = _code(x, "x")
    rows, cols, ldx = _matrix(x, "x")
    q = qt = None
    dev = _here(x, None if out is None else out.data, None if out_t is None else out_t.data)
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
    rc = _lib.muonh_block_quantize(x.data_ptr(), code, rows, cols, ldx, None if q is None else ctypes.byref(q._desc),
                                   None if qt is None else ctypes.byref(qt._desc), _stream(stream, dev))
    if rc:
        _check(rc, "muonh_block_quantize")
    return (q, qt) if form == "both" else q if qt is None else qt


def fp8_matmul(a: Fp8Matrix, b: Fp8Matrix, out=None, out_dtype=None, accumulate: bool = False, stream=None):
    """a b^T: [a.rows, b.rows], contracted over a.cols == b.cols.

    out        : matrix to write (float32 or bfloat16, contiguous rows of any
                 pitch); a new one of out_dtype (bfloat16 if None) if not given
    accumulate : add the product to what out holds

    The result's type chooses the arithmetic.  bfloat16: the FP8 matrix unit, off
    by at most 7 2^-13 of the sum of |a_k b_k| (2e-5 of the result on operands of
    random signs, far below bfloat16's own rounding, but not where products
    cancel).  float32: float32 sums, at half the rate; round them for a bfloat16
    result with such sums, as for a weight gradient.
    """
    if a._cols != b._cols:
        raise ValueError(f"the operands contract {a.cols} and {b.cols} columns")
    m, n = a._rows, b._rows
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = _empty((m, n), out_dtype or _torch.bfloat16, a.data.device, stream)
        ldc = n
    else:
        if out.dim() != 2 or out.shape[0] != m or out.shape[1] != n or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError(f"out: a matrix of shape {(m, n)} and the asked dtype is required")
        ldc = _pitch(out, m, n, "out")
    code = _code(out, "out")
    dev = _here(a.data, b.data, out)
    ra, rb = ctypes.byref(a._desc), ctypes.byref(b._desc)
    need = ctypes.c_size_t()
    rc = _lib.muonh_block_matmul_workspace(ra, rb, code, ctypes.byref(need))
    if rc:
        _check(rc, "muonh_block_matmul_workspace")
    need = need.value
    ws = _like(a.scale, need, stream, result=False) if need else None
    if stream is not None:
        _record(stream, [a.data, a.scale, b.data, b.scale, out] + ([] if ws is None else [ws]))
    rc = _lib.muonh_block_matmul(ra, rb, out.data_ptr(), code, ldc, 1 if accumulate else 0,
                                 None if ws is None else ws.data_ptr(), need, _stream(stream, dev))
    if rc:
        _check(rc, "muonh_block_matmul")
    return out


def _kind(kind: str) -> int:
    code = NORM_KINDS.get(kind)
    if code is None:
        raise ValueError("kind must be 'layer' or 'rms'")
    return code


def _result(out, x, rows: int, cols: int, what: str, stream):
    """(out, its pitch): x's shape and dtype, new if out is None."""
    if out is None:
        return _like(x, (rows, cols), stream), cols
    if out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError(f"{what}: shape or dtype differs from x")
    return out, _pitch(out, rows, cols, what)


def norm_forward(x, weight, bias=None, kind: str = "rms", eps: float = 1e-6, out=None, stream=None):
    """(y, mean, rstd) of the layer norm or RMS norm of x's rows.

    x            : float32 or bfloat16 [rows, cols], contiguous rows of any pitch
    weight, bias : float32 [cols]; bias may be None
    out          : y's memory; may be x itself
    mean is None for kind "rms".
    """
    if _torch is None:
        _setup()
    kind_code, code = _kind(kind), _code(x, "x")
    rows, cols, ldx = _matrix(x, "x")
    _vector(weight, cols, "weight")
    if bias is not None:
        _vector(bias, cols, "bias")
    dev = _here(x, weight, bias, out)
    y, ldy = _result(out, x, rows, cols, "out", stream)
    rstd = _like(weight, rows, stream)
    mean = None if kind_code else _like(weight, rows, stream)
    args = muonh_norm_args(x.data_ptr(), weight.data_ptr(), None if bias is None else bias.data_ptr(),
                           y.data_ptr(), None if mean is None else mean.data_ptr(), rstd.data_ptr(), rows, cols,
                           ldx, ldy, code, kind_code, eps, 0)
    if stream is not None:
        _record(stream, [t for t in (x, weight, bias, y, mean, rstd) if t is not None])
    rc = _lib.muonh_norm_forward(ctypes.byref(args), _stream(stream, dev))
    if rc:
        _check(rc, "muonh_norm_forward")
    return y, mean, rstd


def norm_backward(dy, x, weight, mean, rstd, kind: str = "rms", bias: bool = False, dx=None, dweight=None,
                  dbias=None, accumulate: bool = False, stream=None):
    """(dx, dweight, dbias) from the output's gradient and the forward pass's
    input and statistics; dbias is None unless bias (or dbias) is given.

    dx             : memory of dx; may be dy or x itself
    dweight, dbias : float32 [cols] to write, or with accumulate to add to
    """
    if _torch is None:
        _setup()
    kind_code, code = _kind(kind), _code(x, "x")
    rows, cols, ldx = _matrix(x, "x")
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError("dy: shape or dtype differs from x")
    ld_dy = _pitch(dy, rows, cols, "dy")
    _vector(weight, cols, "weight")
    _vector(rstd, rows, "rstd")
    if (mean is None) != (kind_code == 1):
        raise ValueError("mean is the layer norm's, and None for kind 'rms'")
    if mean is not None:
        _vector(mean, rows, "mean")
    if accumulate and (dweight is None or (bias and dbias is None)):
        raise ValueError("accumulate needs dweight (and dbias)")
    if dweight is not None:
        _vector(dweight, cols, "dweight")
    if dbias is not None:
        _vector(dbias, cols, "dbias")
    dev = _here(dy, x, weight, mean, rstd, dx, dweight, dbias)
    dx, ld_dx = _result(dx, x, rows, cols, "dx", stream)
    if dweight is None:
        dweight = _like(weight, cols, stream)
    if bias and dbias is None:
        dbias = _like(weight, cols, stream)
    need = ctypes.c_size_t()
    rc = _lib.muonh_norm_backward_workspace(rows, cols, ctypes.byref(need))
    if rc:
        _check(rc, "muonh_norm_backward_workspace")
    need = need.value
    ws = _like(weight, need // 4, stream, result=False) if need else None
    args = muonh_norm_grad_args(
        dy.data_ptr(), x.data_ptr(), weight.data_ptr(), None if mean is None else mean.data_ptr(), rstd.data_ptr(),
        dx.data_ptr(), dweight.data_ptr(), None if dbias is None else dbias.data_ptr(), rows, cols,
        ld_dy, ldx, ld_dx, code, kind_code, 1 if accumulate else 0, 0, None if ws is None else ws.data_ptr(), need)
    if stream is not None:
        _record(stream, [t for t in (dy, x, weight, mean, rstd, dx, dweight, dbias, ws) if t is not None])
    rc = _lib.muonh_norm_backward(ctypes.byref(args), _stream(stream, dev))
    if rc:
        _check(rc, "muonh_norm_backward")
    return dx, dweight, dbias


def add_norm_quantize(x, residual, weight, eps: float = 1e-6, form: str = "row", h=None, out: Optional[Fp8Matrix] = None,
                      out_t: Optional[Fp8Matrix] = None, stream=None):
    """(h, rstd, q): h = x + residual, and the RMS norm of h in block-scaled FP8.

    x, residual : float32 or bfloat16 [rows, cols], contiguous rows of any pitch;
                  residual may be None, h is then x itself
    weight      : float32 [cols]
    form        : "row", "col" or "both", as fp8_quantize takes it; q is what that returns
    h           : memory of the sum (x's type); may be x or residual
    out, out_t  : operands to write instead of new ones (row form, column form)
    The norm is not rounded before it is quantised, and h is (to x's type) before it is
    normalised.  h and rstd are what add_norm_backward needs.
    """
    if form not in ("row", "col", "both"):
        raise ValueError("form must be 'row', 'col' or 'both'")
    if _torch is None:
        _setup()
    code = _code(x, "x")
    rows, cols, ldx = _matrix(x, "x")
    ldr = ldh = cols
    if residual is not None:
        if residual.shape != x.shape or residual.dtype != x.dtype:
            raise ValueError("residual: shape or dtype differs from x")
        ldr = _pitch(residual, rows, cols, "residual")
    elif h is not None:
        raise ValueError("h is x where there is no residual")
    _vector(weight, cols, "weight")
    if (out is not None and form == "col") or (out_t is not None and form == "row"):
        raise ValueError("out is the row form and out_t the column form")
    dev = _here(x, residual, weight, h, None if out is None else out.data, None if out_t is None else out_t.data)
    q = qt = None
    if form != "col":
        q = Fp8Matrix.empty(rows, cols, 1, x.device, stream) if out is None else out
        if (q.rows, q.cols, q.block_rows) != (rows, cols, 1):
            raise ValueError("out: shape or block_rows differs")
    if form != "row":
        qt = Fp8Matrix.empty(cols, rows, 1, x.device, stream) if out_t is None else out_t
        if (qt.rows, qt.cols, qt.block_rows) != (cols, rows, 1):
            raise ValueError("out_t: shape or block_rows differs")
    if residual is not None:
        h, ldh = _result(h, x, rows, cols, "h", stream)
    rstd = _like(weight, rows, stream)
    args = muonh_add_norm_args(x.data_ptr(), None if residual is None else residual.data_ptr(), weight.data_ptr(),
                               None if residual is None else h.data_ptr(), rstd.data_ptr(), rows, cols, ldx, ldr, ldh,
                               code, eps)
    if stream is not None:
        _record(stream, [t for t in (x, residual, weight, h, rstd) if t is not None] +
                [t for m in (q, qt) if m is not None for t in (m.data, m.scale)])
    rc = _lib.muonh_add_norm_quantize(ctypes.byref(args), None if q is None else ctypes.byref(q._desc),
                                      None if qt is None else ctypes.byref(qt._desc), _stream(stream, dev))
    if rc:
        _check(rc, "muonh_add_norm_quantize")
    return x if residual is None else h, rstd, (q, qt) if form == "both" else q if qt is None else qt


def add_norm_backward(dy, dh, h, weight, rstd, dx=None, dweight=None, accumulate: bool = False, stream=None):
    """(dx, dweight) of add_norm_quantize: dx, the gradient of x and of residual, is
    that of the norm plus dh, the gradient which reaches h by the residual stream.

    dy      : the gradient of the norm's output, in h's type
    h, rstd : the forward pass's results
    dx      : memory of dx; may be dh, dy or h itself
    dweight : float32 [cols] to write, or with accumulate to add to
    """
    if _torch is None:
        _setup()
    code = _code(h, "h")
    rows, cols, ldh = _matrix(h, "h")
    for t, what in ((dy, "dy"), (dh, "dh")):
        if t.shape != h.shape or t.dtype != h.dtype:
            raise ValueError(f"{what}: shape or dtype differs from h")
    ld_dy, ld_dh = _pitch(dy, rows, cols, "dy"), _pitch(dh, rows, cols, "dh")
    _vector(weight, cols, "weight")
    _vector(rstd, rows, "rstd")
    if accumulate and dweight is None:
        raise ValueError("accumulate needs dweight")
    if dweight is not None:
        _vector(dweight, cols, "dweight")
    dev = _here(dy, dh, h, weight, rstd, dx, dweight)
    dx, ld_dx = _result(dx, h, rows, cols, "dx", stream)
    if dweight is None:
        dweight = _like(weight, cols, stream)
    need = ctypes.c_size_t()
    rc = _lib.muonh_norm_backward_workspace(rows, cols, ctypes.byref(need))
    if rc:
        _check(rc, "muonh_norm_backward_workspace")
    need = need.value
    ws = _like(weight, need // 4, stream, result=False) if need else None
    args = muonh_add_norm_grad_args(muonh_norm_grad_args(
        dy.data_ptr(), h.data_ptr(), weight.data_ptr(), None, rstd.data_ptr(), dx.data_ptr(), dweight.data_ptr(), None,
        rows, cols, ld_dy, ldh, ld_dx, code, NORM_KINDS["rms"], 1 if accumulate else 0, 0,
        None if ws is None else ws.data_ptr(), need), dh.data_ptr(), ld_dh)
    if stream is not None:
        _record(stream, [t for t in (dy, dh, h, weight, rstd, dx, dweight, ws) if t is not None])
    rc = _lib.muonh_add_norm_backward(ctypes.byref(args), _stream(stream, dev))
    if rc:
        _check(rc, "muonh_add_norm_backward")
    return dx, dweight


def _tokens(tokens) -> int:
    """Bytes of a token."""
    if tokens.dtype is not _torch.int64 and tokens.dtype is not _torch.int32:
        raise TypeError(f"tokens: dtype must be int32 or int64, got {tokens.dtype}")
    if tokens.dim() != 1 or not tokens.is_contiguous():
        raise ValueError("tokens: a contiguous vector is required")
    return tokens.element_size()


def embedding_forward(tokens, table, scale: float = 1.0, out=None, out_dtype=None, stream=None):
    """scale * table[tokens]: [tokens, cols].

    tokens : int32 or int64 vector; one outside the table (padding, such as -1) gives zeros
    table  : float32 or bfloat16 [rows, cols], contiguous rows of any pitch
    out    : memory of the result (float32 or bfloat16); a new one of out_dtype (bfloat16
             if None) if not given
    """
    if _torch is None:
        _setup()
    size = _tokens(tokens)
    code = _code(table, "table")
    rows, cols, ld = _matrix(table, "table")
    n = tokens.numel()
    if out is None:
        out = _empty((n, cols), out_dtype or _torch.bfloat16, table.device, stream)
        ld_out = cols
    else:
        if out.shape != (n, cols) or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError(f"out: a matrix of shape {(n, cols)} and the asked dtype is required")
        ld_out = _pitch(out, n, cols, "out")
    out_code = _code(out, "out")
    dev = _here(tokens, table, out)
    args = muonh_embedding_args(tokens.data_ptr(), table.data_ptr(), out.data_ptr(), n, rows, cols, ld, ld_out, size,
                                code, out_code, scale)
    if stream is not None:
        _record(stream, [tokens, table, out])
    rc = _lib.muonh_embedding_forward(ctypes.byref(args), _stream(stream, dev))
    if rc:
        _check(rc, "muonh_embedding_forward")
    return out


def embedding_backward(tokens, dout, rows: int, scale: float = 1.0, dtable=None, out_dtype=None, accumulate: bool = False,
                       stream=None):
    """The table's gradient [rows, cols] from that of the lookup's output, dense:
    scale times the sum of dout's rows over each token's places.

    rows       : of the table; a token outside it (padding) adds nothing
    dout       : float32 or bfloat16 [tokens, cols], contiguous rows of any pitch
    dtable     : memory of the gradient (float32 or bfloat16), which AdamW.step takes;
                 a new one of out_dtype (float32 if None) if not given
    accumulate : add to what dtable holds
    """
    if _torch is None:
        _setup()
    size = _tokens(tokens)
    code = _code(dout, "dout")
    n, cols, ld = _matrix(dout, "dout")
    if n != tokens.numel():
        raise ValueError(f"dout: {tokens.numel()} rows are required")
    if dtable is None:
        if accumulate:
            raise ValueError("accumulate needs dtable")
        dtable = _empty((rows, cols), out_dtype or _torch.float32, dout.device, stream)
        ld_table = cols
    else:
        if dtable.shape != (rows, cols) or (out_dtype is not None and dtable.dtype != out_dtype):
            raise ValueError(f"dtable: a matrix of shape {(rows, cols)} and the asked dtype is required")
        ld_table = _pitch(dtable, rows, cols, "dtable")
    table_code = _code(dtable, "dtable")
    dev = _here(tokens, dout, dtable)
    need = ctypes.c_size_t()
    rc = _lib.muonh_embedding_backward_workspace(n, rows, cols, ctypes.byref(need))
    if rc:
        _check(rc, "muonh_embedding_backward_workspace")
    need = need.value
    ws = None
    if need:
        make = lambda: _torch.empty(need, dtype=_torch.uint8, device=dout.device)  # noqa: E731
        ws = make() if stream is None else _on(stream, make, False)
    args = muonh_embedding_grad_args(tokens.data_ptr(), dout.data_ptr(), dtable.data_ptr(), n, rows, cols, ld, ld_table,
                                     size, code, table_code, 1 if accumulate else 0, scale, 0,
                                     None if ws is None else ws.data_ptr(), need)
    if stream is not None:
        _record(stream, [t for t in (tokens, dout, dtable, ws) if t is not None])
    rc = _lib.muonh_embedding_backward(ctypes.byref(args), _stream(stream, dev))
    if rc:
        _check(rc, "muonh_embedding_backward")
    return dtable


def _heads(t, tokens: int, heads: int, dim: int, what: str) -> int:
    """The token pitch of a bfloat16 tensor [tokens, heads, dim] with contiguous heads."""
    if t.dtype is not _torch.bfloat16:
        raise TypeError(f"{what}: dtype must be bfloat16, got {t.dtype}")
    if t.shape != (tokens, heads, dim):
        raise ValueError(f"{what}: shape {(tokens, heads, dim)} is required")
    s0, s1, s2 = t.stride()
    if (dim > 1 and s2 != 1) or (heads > 1 and s1 != dim):
        raise ValueError(f"{what}: the heads of a token must be contiguous")
    return heads * dim if tokens <= 1 else s0


def _attention(q, k, v, cu_seqlens, scale, out, lse, stream):
    """muonh_attention_args, with new results where none are given: (args, out, lse, device)."""
    if _torch is None:
        _setup()
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k: tensors [tokens, heads, dim] are required")
    tokens, heads, dim = q.shape
    kv_heads = k.shape[1]
    ld_q, ld_k = _heads(q, tokens, heads, dim, "q"), _heads(k, tokens, kv_heads, dim, "k")
    ld_v = _heads(v, tokens, kv_heads, dim, "v")
    ends = cu_seqlens.numel()
    if cu_seqlens.dtype is not _torch.int32 or cu_seqlens.dim() != 1 or ends < 1 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens: a contiguous int32 vector of sequences + 1 elements is required")
    dev = _here(q, k, v, cu_seqlens, out, lse)
    zero = 0
    if out is None:
        out, ld_out = _like(q, (tokens, heads, dim), stream), heads * dim
        zero |= MUONH_ZERO_OUT
    else:
        ld_out = _heads(out, tokens, heads, dim, "out")
    if lse is None:
        lse = _empty((heads, tokens), _torch.float32, q.device, stream)
        zero |= MUONH_ZERO_LSE
    elif lse.dtype is not _torch.float32 or lse.shape != (heads, tokens) or not lse.is_contiguous():
        raise ValueError(f"lse: a contiguous float32 tensor of shape {(heads, tokens)} is required")
    args = muonh_attention_args(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                cu_seqlens.data_ptr(), tokens, ends - 1, ld_q, ld_k, ld_v, ld_out, heads,
                                kv_heads, dim, max(dim, 1) ** -0.5 if scale is None else scale, zero)
    return args, out, lse, dev


def attention_forward(q, k, v, cu_seqlens, scale: Optional[float] = None, out=None, lse=None, stream=None):
    """(out, lse) of causal attention over packed sequences with grouped heads.

    q          : bfloat16 [tokens, heads, dim], dim 8, 16, .. 128, heads contiguous
                 (so a slice of a fused projection's output will do)
    k, v       : [tokens, kv_heads, dim]; heads is a multiple of kv_heads
    cu_seqlens : int32 [sequences + 1]; sequence b is tokens cu_seqlens[b] ..
                 cu_seqlens[b + 1] - 1, each of which sees those up to itself.  It must not
                 decrease; repeat its last element to pad it
    scale      : of the scores, > 0; dim^-1/2 if None
    out, lse   : memory of the results; lse is float32 [heads, tokens], the log of
                 each row's sum of exponentials, which the backward pass reads
    Rows of tokens that no sequence holds (padding behind the last one) are zeros in new
    results and stay as they were in memory that is passed in.
    """
    args, out, lse, dev = _attention(q, k, v, cu_seqlens, scale, out, lse, stream)
    if stream is not None:
        _record(stream, [q, k, v, cu_seqlens, out, lse])
    rc = _lib.muonh_attention_forward(ctypes.byref(args), _stream(stream, dev))
    if rc:
        _check(rc, "muonh_attention_forward")
    return out, lse


def attention_backward(dout, q, k, v, out, lse, cu_seqlens, scale: Optional[float] = None, dq=None, dk=None, dv=None,
                       stream=None):
    """(dq, dk, dv) from the output's gradient and the forward pass's arguments and
    results.

    dq, dk, dv : their memory (slices of one fused gradient will do)
    Rows of tokens that no sequence holds: as attention_forward has them.
    """
    if out is None or lse is None:
        raise ValueError("out and lse are the forward pass's results")
    args, out, lse, dev = _attention(q, k, v, cu_seqlens, scale, out, lse, stream)
    tokens, heads, dim = q.shape
    kv_heads = k.shape[1]
    ld_dout = _heads(dout, tokens, heads, dim, "dout")
    _here(q, dout, dq, dk, dv)
    lds = []
    grads = []
    for t, like, n, what, zero in ((dq, q, heads, "dq", MUONH_ZERO_DQ), (dk, k, kv_heads, "dk", MUONH_ZERO_DK),
                                   (dv, v, kv_heads, "dv", MUONH_ZERO_DV)):
        lds.append(n * dim if t is None else _heads(t, tokens, n, dim, what))
        if t is None:
            t = _like(like, (tokens, n, dim), stream)
            args.zero_rest |= zero
        grads.append(t)
    dq, dk, dv = grads
    need = ctypes.c_size_t()
    rc = _lib.muonh_attention_backward_workspace(ctypes.byref(args), ctypes.byref(need))
    if rc:
        _check(rc, "muonh_attention_backward_workspace")
    need = need.value
    ws = _like(lse, need // 4, stream, result=False) if need else None
    grad = muonh_attention_grad_args(args, dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ld_dout, *lds,
                                     None if ws is None else ws.data_ptr(), need)
    if stream is not None:
        _record(stream, [t for t in (dout, q, k, v, out, lse, cu_seqlens, dq, dk, dv, ws) if t is not None])
    rc = _lib.muonh_attention_backward(ctypes.byref(grad), _stream(stream, dev))
    if rc:
        _check(rc, "muonh_attention_backward")
    return dq, dk, dv
