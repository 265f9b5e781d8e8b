"""The layers of fp8_exact keep every bit in the 8-bit form, and a mistake in
the adapter's term or in the contraction changes their rounded outputs."""

import numpy as np
import pytest

import fp8_exact as fe
from oracle import fp8 as of8
from oracle.bf16 import bits_to_float, float_to_bits

SIZES = [(192, 320, 7, 3), (576, 448, 100, 128), (1024, 1024, 40, 64), (256, 1088, 129, 12)]


@pytest.mark.parametrize("N,K,T,r", SIZES)
def test_the_forms_are_exact(N, K, T, r):
    p = fe.layer(N, K, T, r, seed=N + T)
    np.testing.assert_array_equal(of8.dequantize(*of8.quantize(p["W"], 128), 128), p["W"])
    np.testing.assert_array_equal(of8.dequantize(*of8.quantize(p["X"])), p["X"])
    np.testing.assert_array_equal(of8.dequantize(*of8.quantize(p["dY"])), p["dY"])
    for k in "AB":
        np.testing.assert_array_equal(bits_to_float(float_to_bits(p[k])), p[k])
    o = fe.outputs(p)
    Y, U = of8.forward(p["W"].astype(np.float64), p["X"], p["A"], p["B"], p["alpha"], r)
    dX, dA, dB = of8.backward(p["W"].astype(np.float64), p["X"], p["A"], p["B"], p["dY"], p["alpha"], r)
    for got, want in ((Y, o["Y"]), (U, o["U"]), (dX, o["dX"]), (dA, o["dA"]), (dB, o["dB"])):
        np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("N,K,T,r", SIZES)
def test_mistakes_change_the_outputs(N, K, T, r):
    """The whole rank-r term, its last column, the low half of its pair, one product of the contraction, the scale of
    one block: without any of them bits of Y or of dX are others."""
    p = fe.layer(N, K, T, r, seed=N + T)
    W, X, A, B, dY = (p[k].astype(np.float64) for k in ("W", "X", "A", "B", "dY"))
    o = fe.outputs(p)
    U, G = X @ A.T, dY @ B
    for right, base, V, M in ((o["Y"], X @ W.T, fe.S * U, B.T), (o["dX"], dY @ W, fe.S * G, A)):
        hi, lo = fe.pair(V)
        assert lo.any() or max(N, K) < 512     # short sums fit the high half
        last = np.flatnonzero(M.any(1))[-1]
        L, R = (X, W.T) if M.shape[1] == N else (dY, W)
        at = next(k for k in range(L.shape[1] - 1, -1, -1) if L[:, k].any() and R[k].any())
        doubled = R.copy()
        doubled[-64:, :64] *= 2
        wrong = {"no term": base, "last column": base + V @ M - np.outer(V[:, last], M[last]),
                 "low half": base + (hi if lo.any() else 0 * hi) @ M, "one product": right - np.outer(L[:, at], R[at]),
                 "a scale": right + L @ (doubled - R)}
        for what, bad in wrong.items():
            assert not np.array_equal(fe.rounded(bad), fe.rounded(right)), what
