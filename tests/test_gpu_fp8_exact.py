"""The layer on an 8-bit weight on whole numbers (fp8_exact): every product and
every sum is exact in 32 bits, so outputs are compared bit for bit with the
definition in 64 bits, rounded once.  No tolerance covers a lost product, a
rank column, the low half of a pair or a tile in the wrong place.

Also what no such layer shows: gradients of 24-bit numbers, the codes that the
backward makes of dY, and what the matrix units drop.
"""

import numpy as np
import pytest

import fp8_exact as fe
from gpu_helpers import dev_bf16, dev_f32, say
from oracle import fp8 as of8
from oracle.bf16 import bits_to_float, float_to_bits

pytestmark = pytest.mark.gpu


def _q():
    import nf4_bit_quantized_amd as q
    return q


def _bf16(x):
    return dev_bf16(float_to_bits(np.ascontiguousarray(x, dtype=np.float32)))


def _counted(kernel, call):
    """(what call returns, launches of the kernel in it)."""
    q = _q()
    q.qlora_trace_select({kernel})
    q.qlora_trace_enable(True)
    try:
        q.qlora_trace_read(reset=True)
        out = call()
        n = q.qlora_trace_read(reset=True).get(kernel, (0, 0.0))[0]
    finally:
        q.qlora_trace_enable(False)
        q.qlora_trace_select({q.qlora_trace_kernel_name(k) for k in range(32)} - {None})
    return out, n


def _same(got, want, name):
    got = got.detach().double().cpu().numpy()
    bad = np.argwhere(got != want)
    assert len(bad) == 0, (name, len(bad), bad[0], got[tuple(bad[0])], want[tuple(bad[0])])


# (d_out, d_in, T, r, product launches of the forward, of dX): two where features are cut into 256 x 256 and 128 x 128 tiles
LAYERS = [
    (64, 64, 1, 8, 1, 1),
    (192, 320, 7, 3, 1, 1),
    (1024, 2048, 1, 64, 1, 1),
    (576, 448, 100, 128, 1, 1),
    (512, 512, 128, 12, 1, 1),         # the most tokens of the one-launch form
    (512, 512, 129, 12, 1, 1),         # one more
    (5184, 128, 128, 128, 1, 1),
    (320, 640, 700, 128, 1, 1),
    (1024, 1024, 700, 12, 1, 1),       # a rank of no whole eights on the tiles
    (448, 1088, 700, 20, 1, 1),
    (1088, 576, 1100, 64, 1, 1),
    (320, 192, 33, 0, 1, 1),           # the base alone, few tokens
    (1024, 1024, 1333, 0, 1, 1),       # and on tiles of 128 x 128
    (4096, 320, 2100, 0, 1, 1),        # of 256 x 256, half a block of contraction
    (448, 4096, 2100, 0, 1, 1),        # and backward
    (4096, 320, 2100, 8, 1, 1),
    (448, 4096, 2100, 24, 1, 1),
    (4160, 1024, 2049, 12, 1, 1),
    (9024, 1024, 2049, 20, 2, 1),      # 7168 features on 256 x 256 tiles, 1856 on 128 x 128
    (9024, 1024, 2049, 0, 2, 1),
    (1024, 4416, 4353, 16, 1, 2),      # dX: 3584 and 832
    (1024, 4416, 4353, 0, 1, 2),
]


@pytest.mark.parametrize("N,K,T,r,nf,nb", LAYERS)
def test_whole_numbers(N, K, T, r, nf, nb):
    q = _q()
    say(f"fp8 exact {N}x{K} T {T} r {r}")
    p = fe.layer(N, K, T, r, seed=N + K + T + r)
    o = fe.outputs(p)
    W = q.qlora_quantize_fp8(dev_f32(p["W"]), block_rows=128)
    X = q.qlora_quantize_fp8(_bf16(p["X"]))
    A, B = (_bf16(p["A"]), _bf16(p["B"])) if r else (None, None)
    dY = _bf16(p["dY"])
    (Y, U), n = _counted("fp8_gemm", lambda: q.qlora_fp8_linear_fwd(*W, *X, A, B, p["alpha"]))
    assert n == nf
    _same(Y, fe.rounded(o["Y"]), "Y")
    (dX, dA, dB), n = _counted("fp8_gemm", lambda: q.qlora_fp8_linear_bwd(*W, *X, A, B, p["alpha"], dY, U_in=U))
    assert n == nb
    _same(dX, fe.rounded(o["dX"]), "dX")
    if r == 0:
        assert U is None and dA is None and dB is None
        return
    _same(U, o["U"], "U")
    _same(dA, o["dA"], "dA")
    _same(dB, o["dB"], "dB")
    # U recomputed; the adapter alone, added to what is there
    a0, b0 = dev_f32(np.full((r, K), 3.0)), dev_f32(np.full((N, r), 5.0))
    none, dA, dB = q.qlora_fp8_linear_bwd(*W, *X, A, B, p["alpha"], dY, want_dx=False, dA=a0, dB=b0, accumulate=True)
    assert none is None
    _same(dA, o["dA"] + 3.0, "dA + 3")
    _same(dB, o["dB"] + 5.0, "dB + 5")


@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("N,K,T,r", [(320, 448, 5, 3), (448, 320, 100, 16), (576, 704, 300, 20), (1088, 576, 700, 64),
                                     (320, 1088, 1100, 128)])
def test_gradients_carry_all_24_bits(N, K, T, r, checkpoint):
    """Each element of dB is one element of U, and of dA one of G, which takes 24 bits: both come out whole, from the
    layer on an 8-bit weight and from an NF4 layer's checkpoint."""
    q = _q()
    say(f"24 bits {N}x{K} T {T} r {r} checkpoint {checkpoint}")
    rng = np.random.default_rng(N + T)
    X, dY = np.zeros((T, K), np.float32), np.zeros((T, N), np.float32)
    tx = rng.integers(0, T, K)                  # the token of each column of X
    X[tx, np.arange(K)] = rng.choice([-1.0, 1.0], K)
    # G[t] = 2^16 a B[0] + 2^8 b B[96] + c B[160], with a, b, c of eight bits and B of one: the products go into three
    # instructions, each adding one of them to a sum that fits 24 bits
    digits = rng.integers(128, 256, (T, 3)) * rng.choice([-1, 1], (T, 3))
    dY[:, [0, 96, 160]] = digits * 2.0 ** np.array([16, 8, 0])
    B = np.zeros((N, r), np.float32)
    B[[0, 96, 160]] = rng.choice([-1.0, 1.0], (3, r))
    G = dY.astype(np.float64) @ B
    assert np.abs(G).max() < 2 ** 24
    A = np.zeros((r, K), np.float32)
    W = dev_f32(rng.normal(size=(N, K)) * 0.02)
    Xf = q.qlora_quantize_fp8(_bf16(X))
    call = q.qlora_linear_bwd_checkpoint if checkpoint else q.qlora_fp8_linear_bwd
    w = q.qlora_quantize_nf4(W) if checkpoint else q.qlora_quantize_fp8(W, block_rows=128)
    U = rng.integers(-2 ** 24 + 1, 2 ** 24, (T, r)).astype(np.float64)
    _, dA, _ = call(*w, *Xf, _bf16(A), _bf16(B), float(r), _bf16(dY), U_in=dev_f32(U), want_dx=False)
    _same(dA, G.T @ X, "dA")
    one = np.zeros((T, N), np.float32)
    td = rng.integers(0, T, N)
    one[td, np.arange(N)] = rng.choice([-1.0, 1.0], N)
    _, _, dB = call(*w, *Xf, _bf16(A), _bf16(B), float(r), _bf16(one), U_in=dev_f32(U), want_dx=False)
    _same(dB, one.astype(np.float64).T @ U, "dB")


@pytest.mark.parametrize("T", [128, 300])
@pytest.mark.parametrize("r", [0, 8, 16, 64, 72])
@pytest.mark.parametrize("order", ["by size", "by block", "mixed"])
def test_codes_of_dy_are_the_quantizers(order, r, T):
    """Over a diagonal weight dX is the form of dY itself: for every finite bf16 value, and whichever kernel makes the
    form (r = 0 and 72: the quantizer; 8, 16, 64: the one that forms G), its values are the quantizer's.  The diagonal
    is 2^64 under small values and 2^-64 under large ones, so that dX holds each exactly."""
    import torch
    q = _q()
    say(f"codes of dY {order} r {r} T {T}")
    d = 512
    rng = np.random.default_rng(r + T)
    v = bits_to_float(np.arange(1, 0x7F80, dtype=np.uint16))
    v = v * rng.choice([-1.0, 1.0], v.size).astype(np.float32)
    for big in (False, True):
        part = v[np.abs(v) >= 1.0] if big else v[np.abs(v) < 1.0]
        if order == "mixed":                    # any sizes in a block
            part = rng.permutation(part)
        n = T * d
        part = np.resize(part, n).reshape(-1, 128)
        if order == "by block":                 # some twenty binades in a block: codes of every size, zeros among them
            scale = np.exp2(rng.integers(-10, 11, part.shape)).astype(np.float64)
            m = bits_to_float(float_to_bits(np.clip(np.abs(part * scale), 2.0 ** -133, 2.0 ** 127).astype(np.float32)))
            part = np.where((m >= 1.0) == big, m, np.abs(part)) * np.sign(part)
        part = part.astype(np.float32).reshape(T, d)
        dY = _bf16(part)
        codes, scales = q.qlora_quantize_fp8(dY)
        values = of8.dequantize(codes.cpu().numpy(), scales.cpu().numpy())
        np.testing.assert_array_equal(values, of8.dequantize(*of8.quantize(part)))
        k = 2.0 ** -64 if big else 2.0 ** 64
        W = q.qlora_quantize_fp8(torch.eye(d, device="cuda") * k, block_rows=128)
        X = q.qlora_quantize_fp8(torch.zeros((T, d), device="cuda"))
        A = torch.zeros((r, d), dtype=torch.bfloat16, device="cuda") if r else None
        B = torch.zeros((d, r), dtype=torch.bfloat16, device="cuda") if r else None
        dX, _, _ = q.qlora_fp8_linear_bwd(*W, *X, A, B, 1.0, dY)
        _same(dX, values * k, "dX")


@pytest.mark.parametrize("N,T", [(64, 700), (4096, 2100)])
@pytest.mark.parametrize("backward", [False, True])
def test_what_the_matrix_units_keep(N, T, backward):
    """In a sum of 64 products, one that is 2^-13 of the largest is kept: a row holds 2^8, 2^(8 - d) and, among the
    next 64, -2^8, over a weight of ones, so that the small product alone is left.  d = 5 .. 13, at every place."""
    import torch
    q = _q()
    say(f"kept bits {N} T {T} backward {backward}")
    t = np.arange(T)
    at, d = 1 + t % 63, 5 + t // 63 % 9
    X = np.zeros((T, 128), np.float32)
    X[:, 0], X[:, 64] = 2.0 ** 8, -2.0 ** 8
    X[t, at] = 2.0 ** (8 - d)
    ones = torch.ones((128, N) if backward else (N, 128), device="cuda")
    W = q.qlora_quantize_fp8(ones, block_rows=128)
    if backward:
        none = q.qlora_quantize_fp8(torch.zeros((T, N), device="cuda"))
        Y, _, _ = q.qlora_fp8_linear_bwd(*W, *none, None, None, 1.0, _bf16(X))
    else:
        Y, _ = q.qlora_fp8_linear_fwd(*W, *q.qlora_quantize_fp8(_bf16(X)), None, None, 1.0)
    _same(Y, np.repeat(2.0 ** (8 - d)[:, None], N, 1), "Y")


def _few_whole(rows, cols, seed):
    """A matrix of whole numbers of at most 7 on the GPU, zero but for some thousands of places and its corners."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = min(rows * cols // 8, 4000)
    M = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    i, j = (torch.randint(0, m, (n,), generator=g, device="cuda") for m in (rows, cols))
    M[i, j] = torch.randint(-7, 8, (n,), generator=g, device="cuda").to(torch.bfloat16)
    M[0, 0], M[0, -1], M[-1, 0], M[-1, -1] = 3.0, -5.0, 2.0, 7.0
    return M


def _product(a, b):
    """a b in float64, a million rows, columns and terms at a time."""
    import torch
    step = 1 << 20
    out = torch.zeros((a.shape[0], b.shape[1]), device="cuda")
    for i in range(0, a.shape[0], step):
        for j in range(0, b.shape[1], step):
            for k in range(0, a.shape[1], step):
                x = a[i:i + step, k:k + step].double().contiguous() @ b[k:k + step, j:j + step].double().contiguous()
                out[i:i + step, j:j + step] += x.float()
    return out


@pytest.mark.parametrize("N,K,T,r", [
    (64, 128, 8388000, 8),          # X and its gradient 100 KB under 2^31 bytes
    (16777152, 64, 64, 8),          # Y and B's pair
    (64, 16777152, 64, 8),          # X and A's pair
    (64, 33554368, 16, 0),          # 2^31 codes of the weight, in few rows and in many
    (33554368, 64, 16, 0),
    (46336, 46336, 3, 8),
])
def test_largest_operands(N, K, T, r):
    """Operands just under the 2^31 bytes that the kernels address, whole numbers among zeros, bit for bit."""
    import torch
    q = _q()
    say(f"largest {N}x{K} T {T} r {r}")
    W, X, dY = (_few_whole(*shape, seed) for seed, shape in enumerate(((N, K), (T, K), (T, N))))
    A, B = (_few_whole(r, K, 3), _few_whole(N, r, 4)) if r else (None, None)
    Wf, Xf = q.qlora_quantize_fp8(W, block_rows=128), q.qlora_quantize_fp8(X)
    assert torch.equal(q.qlora_dequantize_fp8(*Wf, block_rows=128), W) and torch.equal(q.qlora_dequantize_fp8(*Xf), X)
    Y, U = q.qlora_fp8_linear_fwd(*Wf, *Xf, A, B, float(max(r, 1)))
    want = _product(X, W.T)
    if r:
        u = _product(X, A.T)
        assert torch.equal(U, u)
        want += _product(u, B.T)
    assert want[-1, -1] != 0 and torch.equal(Y, want.to(torch.bfloat16))
    del want, Y
    dX, dA, dB = q.qlora_fp8_linear_bwd(*Wf, *Xf, A, B, float(max(r, 1)), dY, U_in=U)
    want = _product(dY, W)
    if r:
        G = _product(dY, B)
        want += _product(G, A)
        assert torch.equal(dA, _product(G.T, X)) and torch.equal(dB, _product(dY.T, u))
    assert want[-1, -1] != 0 and torch.equal(dX, want.to(torch.bfloat16))
