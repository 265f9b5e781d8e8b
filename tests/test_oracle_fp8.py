"""The 8-bit form's oracle against torch's own e4m3 and e8m0 types, against
brute force, and the gradients of its layer against differences."""

import numpy as np
import pytest
import torch

from oracle import fp8 as of8
from oracle import lora as olora


def test_e4m3_values_are_torchs():
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(of8.e4m3_values(), t)


def test_rounding_is_torchs_on_every_bf16_within_range():
    bits = np.arange(65536, dtype=np.uint32) << np.uint32(16)
    v = bits.view(np.float32)
    v = v[np.abs(v) <= 448]
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(of8.round_e4m3(v), want)


def test_rounding_is_the_nearest_value():
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-448, 448, 500), rng.normal(size=500) * 2.0 ** -7])
    table = of8.e4m3_values()
    table = table[np.isfinite(table)]
    got = of8.e4m3_values()[of8.round_e4m3(v)]
    best = np.min(np.abs(v[:, None] - table[None, :]), axis=1)
    np.testing.assert_array_equal(np.abs(v - got), best)


@pytest.mark.parametrize("m", [0.0, 1e-45, 2.0 ** -118, 448.0, np.nextafter(np.float32(448), np.float32(500)), 1.0,
                               1.75, np.nextafter(np.float32(1.75), np.float32(2)), 3.3895e38])
def test_scale_byte_is_the_smallest_that_holds(m):
    m = float(np.float32(m))
    e = of8.scale_byte(m)
    assert 1 <= e <= 254 and m <= 448.0 * 2.0 ** (e - 127)
    assert e == 1 or m > 448.0 * 2.0 ** (e - 128)
    # the value of the byte is torch's e8m0
    assert float(torch.tensor([e], dtype=torch.uint8).view(torch.float8_e8m0fnu).double()) == 2.0 ** (e - 127)


@pytest.mark.parametrize("rows,cols,br", [(5, 192, 1), (130, 320, 128), (1, 64, 1), (129, 64, 128)])
def test_values_are_within_half_a_step(rows, cols, br):
    M = np.random.default_rng(1).normal(size=(rows, cols)).astype(np.float32)
    codes, scales = of8.quantize(M, br)
    assert scales.shape == (-(-rows // br), -(-cols // 512) * 4)
    assert (scales[:, -(-cols // 128):] == 127).all()
    v = of8.dequantize(codes, scales, br)
    k = 2.0 ** (scales.astype(float) - 127)
    k = k[np.arange(rows) // br][:, np.arange(cols) // 128]
    # half a step: 2^-4 of the value, or half of 2^-9 in units of the scale for the smallest
    assert (np.abs(v - M) <= np.maximum(2.0 ** -4 * np.abs(M), 2.0 ** -10 * k)).all()
    # a form of a form is itself
    c2, s2 = of8.quantize(v, br)
    np.testing.assert_array_equal(of8.dequantize(c2, s2, br), v)


def test_non_finite_elements_are_nan_and_leave_the_rest():
    M = np.random.default_rng(2).normal(size=(3, 128))
    ref = of8.dequantize(*of8.quantize(np.where(np.arange(128) < 3, 0.0, M)))
    M[:, 0], M[:, 1], M[:, 2] = np.nan, np.inf, -np.inf
    v = of8.dequantize(*of8.quantize(M))
    assert np.isnan(v[:, :3]).all()
    np.testing.assert_array_equal(v[:, 3:], ref[:, 3:])


def test_backward_is_the_formulas_and_differences():
    rng = np.random.default_rng(3)
    N, K, T, r, alpha = 64, 128, 5, 3, 6.0
    W = of8.dequantize(*of8.quantize(rng.normal(size=(N, K)) * 0.02, 128), 128)
    X = of8.dequantize(*of8.quantize(rng.normal(size=(T, K))))
    A, B = rng.normal(size=(r, K)), rng.normal(size=(N, r))
    dY = of8.dequantize(*of8.quantize(rng.normal(size=(T, N))))      # already a form: dX is the plain one
    dX, dA, dB = of8.backward(W, X, A, B, dY, alpha, r)
    loss = lambda X, A, B: float(np.sum(of8.forward(W, X, A, B, alpha, r)[0] * dY))  # noqa: E731
    for M, g, at in ((X, dX, (2, 77)), (A, dA, (1, 5)), (B, dB, (40, 2))):
        d = np.zeros_like(M)
        d[at] = 1e-4
        args = [(m + d, m - d) if m is M else (m, m) for m in (X, A, B)]
        diff = (loss(*[a[0] for a in args]) - loss(*[a[1] for a in args])) / 2e-4
        assert abs(diff - g[at]) <= 1e-6 * max(1.0, abs(g[at]))
    # and with a dY that is not a form, only the base share of dX changes
    dY2 = dY + rng.normal(size=dY.shape) * 1e-3
    dX2, dA2, dB2 = of8.backward(W, X, A, B, dY2, alpha, r)
    p = olora.backward(W, X, A, B, dY2, alpha, r)
    dY_hat = of8.dequantize(*of8.quantize(dY2))
    np.testing.assert_allclose(dX2, dY_hat @ W + olora.lora_scale(alpha, r) * (dY2 @ B) @ A, atol=1e-12)
    np.testing.assert_array_equal(dA2, p[1])
    np.testing.assert_array_equal(dB2, p[2])
