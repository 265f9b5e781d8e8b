"""The NF4 layer's backward from the 8-bit checkpoint of its input, against
the oracle in 64 bits (bounds as in test_gpu_fp8.py) and against the backward
that reads the restored input, and a training step made of these calls."""

import numpy as np
import pytest

import workloads
from gpu_helpers import dev_bf16, dev_f32, say
from oracle import fp8 as of8
from oracle import lora as olora
from oracle import nf4 as onf4
from oracle.bf16 import bits_to_float
from test_gpu_fp8 import _within

pytestmark = pytest.mark.gpu

CASES = [
    # (d_out, d_in, T, r, blocksize, double_quant, table)
    (64, 64, 1, 8, 64, True, 0),
    (256, 320, 16, 3, 64, True, 0),
    (192, 448, 40, 128, 128, True, 0),
    (320, 256, 100, 16, 64, False, 0),
    (512, 576, 600, 24, 256, True, 1),
    (576, 512, 1100, 64, 64, True, 0),
    (512, 512, 33, 0, 64, True, 0),
]


@pytest.mark.parametrize("N,K,T,r,bs,dq,table", CASES)
def test_checkpoint_backward(N, K, T, r, bs, dq, table):
    import torch
    import nf4_bit_quantized_amd as q
    say(f"checkpoint {N}x{K} T {T} r {r} blocks {bs} dq {dq} table {table}")
    alpha = 16.0
    inp = workloads.layer_inputs(N, K, T, r, seed=N + K + T)
    packed, codes, consts = q.qlora_quantize_nf4(dev_f32(inp["W"]), blocksize=bs, double_quant=dq, table=table)
    X, dY = dev_bf16(inp["X"]), dev_bf16(inp["dY"])
    A, B = (dev_bf16(inp["A"]), dev_bf16(inp["B"])) if r else (None, None)
    Xc, Xs = q.qlora_quantize_fp8(X)
    X_hat = of8.dequantize(Xc.cpu().numpy(), Xs.cpu().numpy())
    U = dev_f32(X_hat @ bits_to_float(inp["A"]).T) if r else None
    dX, dA, dB = q.qlora_linear_bwd_checkpoint(packed, codes, consts, Xc, Xs, A, B, alpha, dY, U_in=U, table=table)
    # dX does not depend on X: the plain backward's bits
    Xr = q.qlora_dequantize_fp8(Xc, Xs)
    pX, pA, pB = q.qlora_linear_bwd(packed, codes, consts, Xr, A, B, alpha, dY, U_in=U, table=table)
    assert torch.equal(dX, pX)
    if not r:
        assert dA is None and dB is None
        return
    s = olora.lora_scale(alpha, r)
    dYh, Bh, Uh = bits_to_float(inp["dY"]), bits_to_float(inp["B"]), U.double().cpu().numpy()
    c = (N + T + 16) * 2.0 ** -24
    assert _within(dA, s * (dYh @ Bh).T @ X_hat, s * (np.abs(dYh) @ np.abs(Bh)).T @ np.abs(X_hat), c, half=0.0) <= 1.0
    assert _within(dB, s * dYh.T @ Uh, s * np.abs(dYh).T @ np.abs(Uh), c, half=0.0) <= 1.0
    # without dX, and accumulated
    a0, b0 = torch.randn_like(dA), torch.randn_like(dB)
    none, dA2, dB2 = q.qlora_linear_bwd_checkpoint(packed, codes, consts, Xc, Xs, A, B, alpha, dY, U_in=U, table=table,
                                                   want_dx=False, dA=a0.clone(), dB=b0.clone(), accumulate=True)
    assert none is None and torch.equal(dA2, a0 + dA) and torch.equal(dB2, b0 + dB)
    # U recomputed from the checkpoint
    _, dA3, dB3 = q.qlora_linear_bwd_checkpoint(packed, codes, consts, Xc, Xs, A, B, alpha, dY, table=table, want_dx=False)
    Ah = bits_to_float(inp["A"])
    assert torch.equal(dA3, dA)
    assert _within(dB3, s * dYh.T @ (X_hat @ Ah.T), s * np.abs(dYh).T @ (np.abs(X_hat) @ np.abs(Ah).T),
                   c + K * 2.0 ** -24, half=0.0) <= 1.0


def test_no_tokens():
    import torch
    import nf4_bit_quantized_amd as q
    inp = workloads.layer_inputs(128, 192, 0, 8, seed=1)
    w = q.qlora_quantize_nf4(dev_f32(inp["W"]))
    Xc, Xs = q.qlora_quantize_fp8(dev_bf16(inp["X"]))
    dX, dA, dB = q.qlora_linear_bwd_checkpoint(*w, Xc, Xs, dev_bf16(inp["A"]), dev_bf16(inp["B"]), 8.0, dev_bf16(inp["dY"]))
    assert dX.shape == (0, 192) and not dA.any() and not dB.any()


def test_training_steps_of_two_layers():
    """Two steps of an NF4 layer followed by an 8-bit one: inputs kept as
    checkpoints only, gradients from them, adapters updated.  Each gradient of
    each step is the oracle's at the state the step began with."""
    import torch
    import nf4_bit_quantized_amd as q
    T, K, H, N, r, alpha = 96, 256, 384, 320, 8, 16.0
    a = workloads.layer_inputs(H, K, T, r, seed=3)
    b = workloads.layer_inputs(N, H, T, r, seed=4)
    w1 = q.qlora_quantize_nf4(dev_f32(a["W"]))
    w2 = q.qlora_quantize_fp8(dev_f32(b["W"]), block_rows=128)
    W1 = onf4.dequantize(onf4.quantize(a["W"])).astype(np.float64)
    W2 = of8.dequantize(*of8.quantize(b["W"], 128), 128)
    params = {}
    for k, inp in (("1", a), ("2", b)):
        for n in "AB":
            bf = dev_bf16(inp[n])
            p = bf.float()
            params[n + k] = (p, torch.zeros_like(p), torch.zeros_like(p), bf)
    X, dY = dev_bf16(a["X"]), dev_bf16(b["dY"])
    for step in (1, 2):
        A1, B1, A2, B2 = (params[n][3] for n in ("A1", "B1", "A2", "B2"))
        kept = [q.qlora_quantize_fp8(X)]
        Y1, U1 = q.qlora_linear_fwd(*w1, X, A1, B1, alpha)
        kept.append(q.qlora_quantize_fp8(Y1))
        Y2, U2 = q.qlora_fp8_linear_fwd(*w2, *kept[1], A2, B2, alpha)
        dY1, dA2, dB2 = q.qlora_fp8_linear_bwd(*w2, *kept[1], A2, B2, alpha, dY, U_in=U2)
        dX, dA1, dB1 = q.qlora_linear_bwd_checkpoint(*w1, *kept[0], A1, B1, alpha, dY1, U_in=U1)
        h = {n: params[n][3].double().cpu().numpy() for n in params}
        X1, X2 = (of8.dequantize(c.cpu().numpy(), s.cpu().numpy()) for c, s in kept)
        for got, inp_, X_, A_, B_, d_, U_ in ((( dA1, dB1), W1, X1, h["A1"], h["B1"], dY1, U1),
                                              (( dA2, dB2), W2, X2, h["A2"], h["B2"], dY, U2)):
            d_, U_ = d_.double().cpu().numpy(), U_.double().cpu().numpy()
            s = olora.lora_scale(alpha, r)
            c = (inp_.shape[0] + T + 16) * 2.0 ** -24
            assert _within(got[0], s * (d_ @ B_).T @ X_, s * (np.abs(d_) @ np.abs(B_)).T @ np.abs(X_), c, half=0.0) <= 1.0
            assert _within(got[1], s * d_.T @ U_, s * np.abs(d_).T @ np.abs(U_), c, half=0.0) <= 1.0
        wY, _ = of8.forward(W2, X2, h["A2"], h["B2"], alpha, r)
        mY, _ = of8.forward(np.abs(W2), np.abs(X2), np.abs(h["A2"]), np.abs(h["B2"]), alpha, r)
        assert _within(Y2, wY, mY, 2.0 ** -10) <= 1.0
        before = {n: params[n][3].clone() for n in params}
        for n, g in (("A1", dA1), ("B1", dB1), ("A2", dA2), ("B2", dB2)):
            p, m, v, bf = params[n]
            q.qlora_adamw_step(p, g, m, v, step, 1e-2, param_bf16=bf)
        torch.cuda.synchronize()
        assert all(not torch.equal(before[n], params[n][3]) for n in params)
