"""8-bit forms (e4m3 codes, one power-of-two scale per block) -- CPU oracle.

TEST INFRASTRUCTURE ONLY (see ``oracle``): never imported by the product path.

The form of a matrix M [R][C], blocks of ``block_rows`` x 128:
  m = largest finite |x| of a block,
  e = smallest whole number in 1 .. 254 with m <= 448 * 2^(e - 127),
  code = the e4m3 value nearest to x * 2^(127 - e), ties to the even code; NaN where x is not finite.
Scales fill rows of 4 ceil(C / 512) bytes, those past the last block holding 127.

e4m3 is built from its definition (sign, 4 exponent bits with bias 7, 3
mantissa bits, exponent field 0 subnormal, code 0x7F NaN), and rounding is a
search among the 127 non-negative values.

Pins (``tests/test_oracle_fp8.py``): torch's own float8_e4m3fn cast and
float8_e8m0fnu view on the CPU, brute-force nearest value, the scale rule by
direct trial of every byte.
"""

import numpy as np

BLOCK = 128


def e4m3_values() -> np.ndarray:
    """The 256 codes' values, float64 (0x7F and 0xFF NaN)."""
    out = np.empty(256)
    for code in range(256):
        field, mant = (code >> 3) & 15, code & 7
        if field == 15 and mant == 7:
            v = np.nan
        elif field == 0:
            v = mant / 8.0 * 2.0 ** -6
        else:
            v = (1.0 + mant / 8.0) * 2.0 ** (field - 7)
        out[code] = -v if code & 128 else v
    return out


def round_e4m3(v) -> np.ndarray:
    """uint8 codes of float64 values of at most 448 in size: nearest, ties to the even code, the sign of zero kept."""
    v = np.asarray(v, np.float64)
    table = e4m3_values()[:127]
    a = np.abs(v)
    up = np.clip(np.searchsorted(table, a, side="left"), 1, 126)
    down = up - 1
    below, above = a - table[down], table[up] - a
    code = np.where(below < above, down, np.where(above < below, up, np.where(down % 2 == 0, down, up)))
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def scale_byte(m: float) -> int:
    """Smallest byte e in 1 .. 254 with m <= 448 * 2^(e - 127)."""
    for e in range(1, 255):
        if m <= 448.0 * 2.0 ** (e - 127):
            return e
    return 254


def scale_ld(cols: int) -> int:
    return -(-cols // 512) * 4


def quantize(M, block_rows: int = 1):
    """(codes uint8 [R][C], scales uint8 [ceil(R / block_rows)][scale_ld(C)])."""
    M = np.asarray(M, np.float64)
    R, C = M.shape
    codes = np.empty((R, C), np.uint8)
    scales = np.full((-(-R // block_rows), scale_ld(C)), 127, np.uint8)
    for i in range(scales.shape[0]):
        for b in range(-(-C // BLOCK)):
            at = np.s_[i * block_rows:(i + 1) * block_rows, b * BLOCK:(b + 1) * BLOCK]
            x = M[at]
            fine = np.isfinite(x)
            e = scale_byte(np.max(np.abs(x), where=fine, initial=0.0))
            scales[i, b] = e
            q = round_e4m3(np.where(fine, x, 0.0) * 2.0 ** (127 - e))
            codes[at] = np.where(fine, q, 0x7F)
    return codes, scales


def dequantize(codes, scales, block_rows: int = 1) -> np.ndarray:
    """The values the form stands for, float64."""
    R, C = codes.shape
    k = 2.0 ** (np.asarray(scales, np.float64) - 127.0)
    return e4m3_values()[codes] * k[np.arange(R) // block_rows][:, np.arange(C) // BLOCK]


def forward(W_hat, X_hat, A, B, alpha: float, r: int):
    """Y = X_hat W_hat^T + s (X_hat A^T) B^T and U, float64: the plain layer on the forms' values."""
    from . import lora
    return lora.forward(W_hat, X_hat, A, B, alpha, r)


def backward(W_hat, X_hat, A, B, dY, alpha: float, r: int):
    """(dX, dA, dB), float64: as the plain layer's, the base share of dX from the 8-bit form of dY."""
    from . import lora
    dX, dA, dB = lora.backward(W_hat, X_hat, A, B, dY, alpha, r)
    dY = np.asarray(dY, np.float64)
    dY_hat = dequantize(*quantize(dY, 1), 1)
    return dX + (dY_hat - dY) @ np.asarray(W_hat, np.float64), dA, dB
