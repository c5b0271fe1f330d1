"""fp64 oracle of the block-scaled FP8 operators: the quantiser and the product
of two quantised operands, written from their definitions.

E4M3 (the OCP type without infinities): 1 sign, 4 exponent bits (bias 7), 3
fraction bits; largest value 448, least step 2^-9.
"""

from __future__ import annotations

import dataclasses

import numpy as np

E4M3_MAX = 448.0


def e4m3_round(v: np.ndarray) -> np.ndarray:
    """The nearest E4M3 value of each |v| <= 448, ties to the even fraction."""
    v = np.asarray(v, dtype=np.float64)
    mag = np.abs(v)
    with np.errstate(divide="ignore"):
        exp = np.floor(np.log2(np.where(mag > 0, mag, 1.0)))
    # log2 next to a power of two may round up to it
    exp = np.where(np.ldexp(1.0, exp.astype(np.int64)) > np.where(mag > 0, mag, 1.0), exp - 1, exp)
    step = np.ldexp(1.0, (np.maximum(exp, -6) - 3).astype(np.int64))
    return np.rint(v / step) * step


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 encodings, from the definition of the type."""
    out = np.empty(256)
    for code in range(256):
        sign = -1.0 if code & 0x80 else 1.0
        exp, frac = (code >> 3) & 15, code & 7
        if exp == 15 and frac == 7:
            out[code] = np.nan
        elif exp == 0:
            out[code] = sign * frac * 2.0 ** -9
        else:
            out[code] = sign * (1.0 + frac / 8.0) * 2.0 ** (exp - 7)
    return out


def block_exponent(amax: float) -> int:
    """The least e >= -127 with amax <= 448 2^e; 0 for a block of zeros."""
    if amax == 0.0:
        return 0
    e = -127
    while amax > E4M3_MAX * 2.0 ** e:
        e += 1
    return e


@dataclasses.dataclass
class Quantized:
    values: np.ndarray      # [rows, cols] E4M3 values (unscaled), NaN where x was not finite
    exponents: np.ndarray   # [ceil(rows / block_rows), ceil(cols / 128)]
    block_rows: int

    def dequantize(self) -> np.ndarray:
        rows, cols = self.values.shape
        e = np.repeat(np.repeat(self.exponents, self.block_rows, 0)[:rows], 128, 1)[:, :cols]
        return self.values * np.ldexp(1.0, e)


def quantize(x: np.ndarray, block_rows: int = 1) -> Quantized:
    """x's row form; the column form is quantize(x.T)."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    nr, nc = -(-rows // block_rows), -(-cols // 128)
    finite = np.isfinite(x)
    mag = np.where(finite, np.abs(x), 0.0)
    values = np.full(x.shape, np.nan)
    exponents = np.zeros((nr, nc), dtype=np.int64)
    for i in range(nr):
        rs = slice(i * block_rows, min((i + 1) * block_rows, rows))
        for j in range(nc):
            cs = slice(j * 128, min((j + 1) * 128, cols))
            e = block_exponent(float(mag[rs, cs].max()))
            exponents[i, j] = e
            scaled = np.where(finite[rs, cs], x[rs, cs], 0.0) * 2.0 ** -e
            values[rs, cs] = np.where(finite[rs, cs], e4m3_round(scaled), np.nan)
    return Quantized(values, exponents, block_rows)


def matmul(a: Quantized, b: Quantized) -> np.ndarray:
    return a.dequantize() @ b.dequantize().T
