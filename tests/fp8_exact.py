"""Layers whose every product and every sum is a whole number of halves that
32-bit sums hold exactly, whatever their order, so that outputs of the 8-bit
layer are known to the last bit.

Codes stand for whole numbers of at most 7 times 1, 2 or 4 (chosen by block),
which the 8-bit form keeps exactly; A and B are whole numbers of at most 7
(or 1), most of them zero; s = 1/2.  In a group of eight products the least (1) is
2^-6 of the largest (49) or more, far above what the matrix units drop.  U and
G stay below 2^16, so a hi/lo pair of bf16 holds them, and the sums of
absolute values below 2^23, so every partial sum of halves fits 24 bits; both
are checked where a layer is made.
"""

import numpy as np

from oracle.bf16 import bits_to_float, float_to_bits

S = 0.5


def _whole(rng, rows, cols, block_rows):
    """Whole numbers of at most 7, times 1, 2 or 4 by block."""
    m = rng.integers(-7, 8, (rows, cols))
    k = 1 << rng.integers(0, 3, (-(-rows // block_rows), -(-cols // 128)))
    return (m * np.repeat(np.repeat(k, block_rows, 0)[:rows], 128, 1)[:, :cols]).astype(np.float32)


def _sparse(rng, rows, cols, most):
    """Whole numbers of at most `most`, seven eighths of them zero."""
    return (rng.integers(-most, most + 1, (rows, cols)) * (rng.random((rows, cols)) < 0.125)).astype(np.float32)


def layer(N, K, T, r, seed):
    """{W, X, A, B, dY} in float32 (whole numbers) and alpha = r / 2, the scale being 1/2."""
    rng = np.random.default_rng(seed)
    most = 7 if T * max(N, K) ** 0.5 < 2 ** 16 else 1     # long sums of long sums, in dA and dB
    return {"W": _whole(rng, N, K, 128), "X": _whole(rng, T, K, 1), "A": _sparse(rng, r, K, most),
            "B": _sparse(rng, N, r, most),
            "dY": _whole(rng, T, N, 1), "alpha": r * S if r else 1.0}


def rounded(v):
    """Float64 values that fit float32, rounded to bf16: as float32."""
    f = v.astype(np.float32)
    assert np.array_equal(f, v)
    return bits_to_float(float_to_bits(f))


def pair(v):
    """(hi, lo): v to 8 significant bits, and what is left, which fits 8 as well."""
    hi = rounded(v)
    lo = v - hi
    assert np.array_equal(rounded(lo), lo)
    return hi, lo


def _small(*sums):
    """Every sum of absolute values (in 32 bits, far closer than a hundredth) leaves 24 bits to its halves."""
    assert all(np.max(m, initial=0.0) < 0.99 * 2.0 ** 23 for m in sums)


def outputs(p):
    """{Y, U, dX, dA, dB}, float64: exact, Y and dX before their rounding."""
    W, X, A, B, dY = (p[k].astype(np.float64) for k in ("W", "X", "A", "B", "dY"))
    U, G = X @ A.T, dY @ B
    pair(S * U)
    pair(S * G)
    aW, aX, aA, aB, aD, aU, aG = (np.abs(v).astype(np.float32) for v in (W, X, A, B, dY, U, G))
    _small(aX @ aW.T + aU @ aB.T, aD @ aW + aG @ aA, aX @ aA.T, aD @ aB, aG.T @ aX, aD.T @ aU)
    return {"Y": X @ W.T + S * (U @ B.T), "U": U, "dX": dY @ W + S * (G @ A), "dA": S * (G.T @ X), "dB": S * (dY.T @ U)}
