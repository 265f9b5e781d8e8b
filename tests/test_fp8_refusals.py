"""What the 8-bit entry points refuse, on the host before anything is
enqueued: through the C ABI with addresses that are never dereferenced, and
through the binding with tensors that do not fit."""

import ctypes
import os

import pytest
import torch

import nf4_bit_quantized_amd as q

pytestmark = pytest.mark.skipif(not os.path.exists(q.LIB_PATH), reason="library not built")

F = 0x10000     # an aligned address that no call below gets to use
OK, NULL, SHAPE, UNSUP, WS = (q.QLORA_OK, q.QLORA_ERR_NULL, q.QLORA_ERR_SHAPE, q.QLORA_ERR_UNSUPPORTED,
                              q.QLORA_ERR_WORKSPACE)


def test_sizes():
    assert q.qlora_fp8_sizes(4096, 8192) == (4096 * 8192, 4096 * 64)
    assert q.qlora_fp8_sizes(5, 64) == (320, 20)                 # one block, its row padded to a dword
    assert q.qlora_fp8_sizes(0, 640) == (0, 0)
    assert q.qlora_fp8_sizes(129, 576, 128) == (129 * 576, 2 * 8)


@pytest.mark.parametrize("rows,cols,br,status", [
    (-1, 64, 1, SHAPE), (1, 0, 1, SHAPE), (1, 96, 1, SHAPE), (1, 64, 2, UNSUP), (1, 64, 0, UNSUP), (1, 64, 64, UNSUP),
    (1 << 31, 64, 1, SHAPE), (1 << 30, 64, 1, SHAPE), (1, 1 << 31, 1, SHAPE), (1 << 27, 64, 1, SHAPE), ((1 << 27) - 1, 64, 1, OK)])
def test_forms_refused(rows, cols, br, status):
    L = q.lib()
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert L.qlora_fp8_sizes(rows, cols, br, ctypes.byref(a), ctypes.byref(b)) == status
    if status != OK:
        assert L.qlora_quantize_fp8(rows, cols, br, F, 0, F, F, None) == status
        assert L.qlora_dequantize_fp8(rows, cols, br, F, F, F, None) == status


@pytest.mark.parametrize("cols,br", [(512, 1), (512, 128), (1024, 1)])
def test_largest_forms(cols, br):
    """What the sizes accept, every kernel can launch: sixteen codes a thread, in a grid of fewer than 2^32 threads
    of whole workgroups of 256."""
    L = q.lib()
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    most = ((1 << 32) - 256) * 16 // cols
    for rows in range(most - 3, most + 4):
        fits = -(-(rows * cols // 16) // 256) * 256 < 1 << 32
        assert fits == (rows <= most)
        assert L.qlora_fp8_sizes(rows, cols, br, ctypes.byref(a), ctypes.byref(b)) == (OK if fits else SHAPE)
        if not fits:
            assert L.qlora_quantize_fp8(rows, cols, br, F, 0, F, F, None) == SHAPE
            assert L.qlora_dequantize_fp8(rows, cols, br, F, F, F, None) == SHAPE


def test_form_pointers():
    L = q.lib()
    a = ctypes.c_size_t()
    assert L.qlora_fp8_sizes(4, 64, 1, None, ctypes.byref(a)) == NULL
    assert L.qlora_fp8_sizes(4, 64, 1, ctypes.byref(a), None) == NULL
    for args, want in (((None, 0, F, F), NULL), ((F, 0, None, F), NULL), ((F, 0, F, None), NULL), ((F, 3, F, F), UNSUP),
                       ((F, -1, F, F), UNSUP), ((F + 8, 0, F, F), UNSUP), ((F, 0, F + 8, F), UNSUP),
                       ((F, 0, F, F + 2), UNSUP)):
        assert L.qlora_quantize_fp8(4, 64, 1, *args, None) == want, args
    for args, want in (((None, F, F), NULL), ((F, None, F), NULL), ((F, F, None), NULL), ((F + 4, F, F), UNSUP),
                       ((F, F + 1, F), UNSUP), ((F, F, F + 8), UNSUP)):
        assert L.qlora_dequantize_fp8(4, 64, 1, *args, None) == want, args
    # nothing to do needs nothing
    assert L.qlora_quantize_fp8(0, 64, 1, None, 1, None, None, None) == OK
    assert L.qlora_dequantize_fp8(0, 64, 1, None, None, None, None) == OK


LAYER = [(100, 64, 4, 8), (64, 96, 4, 8), (0, 64, 4, 8), (64, 64, -1, 8), (64, 64, 4, -1), (64, 64, 4, 129),
         (1 << 31, 64, 1, 0), (65536, 32768, 1, 0), (64, 64, 1 << 25, 0), (1 << 24, 64, 4, 64), (64, 64, 1 << 23, 128)]


@pytest.mark.parametrize("N,K,T,r", LAYER)
def test_layer_sizes_refused(N, K, T, r):
    L = q.lib()
    n = ctypes.c_size_t()
    assert L.qlora_fp8_fwd_workspace_bytes(N, K, T, r, ctypes.byref(n)) == SHAPE
    assert L.qlora_fp8_bwd_workspace_bytes(N, K, T, r, ctypes.byref(n)) == SHAPE
    assert L.qlora_fp8_linear_fwd(N, K, F, F, T, F, F, r, 1.0, F, F, F, F, F, 1 << 40, None) == SHAPE
    assert L.qlora_fp8_linear_bwd(N, K, F, F, T, F, F, r, 1.0, F, F, F, F, F, F, F, 0, F, 1 << 40, None) == SHAPE


def _each_wrong(good, wrong):
    """good with each (index, value) of wrong in turn."""
    for at, value, want in wrong:
        args = list(good)
        args[at] = value
        yield args, want


def test_forward_pointers():
    L = q.lib()
    need = q.qlora_fp8_fwd_workspace_bytes(64, 64, 4, 8)
    assert need > 0
    #        0   1   2  3  4  5  6  7  8    9  10 11 12 13 14    15
    good = [64, 64, F, F, 4, F, F, 8, 1.0, F, F, F, F, F, need, None]
    wrong = [(2, None, NULL), (3, None, NULL), (5, None, NULL), (6, None, NULL), (9, None, NULL), (10, None, NULL),
             (11, None, NULL), (2, F + 8, UNSUP), (3, F + 2, UNSUP), (5, F + 8, UNSUP), (6, F + 1, UNSUP),
             (9, F + 2, UNSUP), (10, F + 2, UNSUP), (11, F + 2, UNSUP), (12, F + 4, UNSUP), (13, F + 8, UNSUP),
             (13, None, WS), (14, need - 1, WS)]
    for args, want in _each_wrong(good, wrong):
        assert L.qlora_fp8_linear_fwd(*args) == want, args
    assert L.qlora_fp8_linear_fwd(64, 64, F, F, 0, None, None, 8, 1.0, F, F, None, None, None, 0, None) == OK
    assert L.qlora_fp8_fwd_workspace_bytes(64, 64, 4, 8, None) == NULL


def test_backward_pointers():
    L = q.lib()
    need = q.qlora_fp8_bwd_workspace_bytes(64, 64, 4, 8)
    #        0   1   2  3  4  5  6  7  8    9  10 11 12 13 14 15 16 17 18    19
    good = [64, 64, F, F, 4, F, F, 8, 1.0, F, F, F, F, F, F, F, 0, F, need, None]
    wrong = [(2, None, NULL), (3, None, NULL), (5, None, NULL), (6, None, NULL), (9, None, NULL), (10, None, NULL),
             (12, None, NULL), (14, None, NULL), (15, None, NULL), (2, F + 8, UNSUP), (3, F + 2, UNSUP),
             (5, F + 8, UNSUP), (6, F + 1, UNSUP), (9, F + 2, UNSUP), (10, F + 2, UNSUP), (11, F + 8, UNSUP),
             (12, F + 2, UNSUP), (13, F + 2, UNSUP), (14, F + 4, UNSUP), (15, F + 4, UNSUP), (17, F + 8, UNSUP),
             (17, None, WS), (18, need - 1, WS)]
    for args, want in _each_wrong(good, wrong):
        assert L.qlora_fp8_linear_bwd(*args) == want, args
    assert L.qlora_fp8_bwd_workspace_bytes(64, 64, 4, 8, None) == NULL


def test_checkpoint_backward_pointers():
    L = q.lib()
    d = q._desc(64, 64)
    D = ctypes.byref(d)
    need = q.qlora_checkpoint_workspace_bytes(64, 64, 4, 8)
    #       0  1  2  3  4  5  6  7  8    9  10 11 12 13 14 15 16 17 18    19
    good = [D, F, F, F, 4, F, F, 8, 1.0, F, F, F, F, F, F, F, 0, F, need, None]
    wrong = [(0, None, NULL), (1, None, NULL), (2, None, NULL), (3, None, NULL), (5, None, NULL), (6, None, NULL),
             (9, None, NULL), (10, None, NULL), (12, None, NULL), (14, None, NULL), (15, None, NULL),
             (4, -1, SHAPE), (7, 129, SHAPE), (1, F + 8, UNSUP), (5, F + 8, UNSUP), (6, F + 1, UNSUP), (9, F + 2, UNSUP),
             (10, F + 2, UNSUP), (11, F + 8, UNSUP), (12, F + 2, UNSUP), (13, F + 2, UNSUP), (14, F + 4, UNSUP),
             (15, F + 4, UNSUP), (17, F + 8, UNSUP), (17, None, WS), (18, need - 1, WS)]
    for args, want in _each_wrong(good, wrong):
        assert L.qlora_linear_bwd_checkpoint(*args) == want, args
    bad = q._desc(64, 64, blocksize=32)
    assert L.qlora_linear_bwd_checkpoint(ctypes.byref(bad), *good[1:]) == UNSUP
    n = ctypes.c_size_t()
    assert L.qlora_checkpoint_workspace_bytes(ctypes.byref(bad), 4, 8, ctypes.byref(n)) == UNSUP
    assert L.qlora_checkpoint_workspace_bytes(D, 4, 8, None) == NULL


# (d_out, d_in, r): A or B at 2^31 bytes, above it, and at 2^32, where a 32-bit offset is back at zero
@pytest.mark.parametrize("N,K,r", [(64, 1 << 23, 128), (64, 1 << 24, 64), (64, 1 << 24, 128), (1 << 24, 64, 64),
                                   (1 << 24, 64, 128)])
def test_checkpoint_adapter_sizes_refused(N, K, r):
    """The kernels address A and B with 32-bit byte offsets, whether U is given or not."""
    L = q.lib()
    n = ctypes.c_size_t()
    D = ctypes.byref(q._desc(N, K))
    assert L.qlora_checkpoint_workspace_bytes(D, 1, r, ctypes.byref(n)) == SHAPE
    for U in (F, None):
        assert L.qlora_linear_bwd_checkpoint(D, F, F, F, 1, F, F, r, 1.0, F, F, U, F, F, F, F, 0, F, 1 << 40, None) == SHAPE
    # as the layer on an 8-bit weight does; and the sizes below are there
    assert L.qlora_fp8_bwd_workspace_bytes(N, K, 1, r, ctypes.byref(n)) == SHAPE
    D = ctypes.byref(q._desc(min(N, (1 << 23) - 64), min(K, (1 << 23) - 64)))
    assert L.qlora_checkpoint_workspace_bytes(D, 1, r, ctypes.byref(n)) == OK


def test_workspaces_hold_what_they_are_said_to():
    """No tokens, or no adapter where only it needs scratch: none.  Else at least the 8-bit form of dY, U and G."""
    assert q.qlora_fp8_fwd_workspace_bytes(256, 256, 0, 8) == 0
    assert q.qlora_checkpoint_workspace_bytes(256, 256, 8, 0) == 0
    for T in (1, 16, 17, 100, 128, 129, 1000, 4096):
        for r in (0, 1, 8, 64, 128):
            assert q.qlora_fp8_bwd_workspace_bytes(1024, 2048, T, r) >= T * 1024 + T * 8 + T * r * 8


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------

def _t(shape, dtype=torch.uint8):
    return torch.zeros(shape, dtype=dtype)


def _layer_tensors(N=64, K=128, T=4, r=8):
    return dict(Wc=_t((N, K)), Ws=_t((1, 4)), Xc=_t((T, K)), Xs=_t((T, 4)), A=_t((r, K), torch.bfloat16),
                B=_t((N, r), torch.bfloat16), dY=_t((T, N), torch.bfloat16), U=_t((T, r), torch.float32))


BAD = [
    dict(Wc=_t((64, 128), torch.int8)), dict(Wc=_t((64, 128, 1))), dict(Ws=_t((2, 4))), dict(Ws=_t((1, 8))),
    dict(Xc=_t((4, 64)), Xs=_t((4, 4))), dict(Xs=_t((4, 1))), dict(Xs=_t((5, 4))), dict(Xs=None), dict(Wc=None),
    dict(Xc=_t((128, 4)).t()), dict(A=_t((8, 64), torch.bfloat16)), dict(B=_t((64, 7), torch.bfloat16)),
    dict(A=None), dict(A=_t((8, 128), torch.float32)),
]


@pytest.mark.parametrize("bad", range(len(BAD)))
def test_binding_refuses_layers(bad):
    t = _layer_tensors()
    t.update(BAD[bad])
    with pytest.raises((ValueError, q.QloraError)):
        q.qlora_fp8_linear_fwd(t["Wc"], t["Ws"], t["Xc"], t["Xs"], t["A"], t["B"], 16.0)
    with pytest.raises((ValueError, q.QloraError)):
        q.qlora_fp8_linear_bwd(t["Wc"], t["Ws"], t["Xc"], t["Xs"], t["A"], t["B"], 16.0, t["dY"])


@pytest.mark.parametrize("bad", [dict(dY=_t((4, 128), torch.bfloat16)), dict(dY=_t((4, 64), torch.float32)),
                                 dict(dY=None), dict(U_in=_t((4, 7), torch.float32)), dict(dX=_t((4, 64), torch.bfloat16)),
                                 dict(dA=_t((8, 128), torch.bfloat16)), dict(dB=_t((8, 64), torch.float32)),
                                 dict(accumulate=True), dict(accumulate=True, dA=_t((8, 128), torch.float32))])
def test_binding_refuses_gradients(bad):
    t = _layer_tensors()
    kw = dict(bad)
    dY = kw.pop("dY", t["dY"])
    packed, codes, consts = _t((64, 64)), _t((128,)), _t((1,), torch.float32)
    with pytest.raises(ValueError):
        q.qlora_fp8_linear_bwd(t["Wc"], t["Ws"], t["Xc"], t["Xs"], t["A"], t["B"], 16.0, dY, **kw)
    with pytest.raises(ValueError):
        q.qlora_linear_bwd_checkpoint(packed, codes, consts, t["Xc"], t["Xs"], t["A"], t["B"], 16.0, dY, **kw)


def test_binding_refuses_forms_and_host_tensors():
    for M in (_t((4, 96), torch.float32), _t((4, 64), torch.int32), _t((4, 64, 1), torch.float32), None):
        with pytest.raises((ValueError, q.QloraError)):
            q.qlora_quantize_fp8(M)
    with pytest.raises(q.QloraError):
        q.qlora_quantize_fp8(_t((4, 64), torch.float32), block_rows=16)
    with pytest.raises(ValueError, match="on the GPU"):
        q.qlora_quantize_fp8(_t((4, 64), torch.float32))
    with pytest.raises(ValueError, match="on the GPU"):
        q.qlora_dequantize_fp8(_t((4, 64)), _t((4, 4)))
    with pytest.raises(ValueError):
        q.qlora_dequantize_fp8(_t((4, 64)), _t((4, 4)), block_rows=128)
    t = _layer_tensors()
    with pytest.raises(ValueError, match="on the GPU"):
        q.qlora_fp8_linear_fwd(t["Wc"], t["Ws"], t["Xc"], t["Xs"], t["A"], t["B"], 16.0)
    with pytest.raises(ValueError, match="codes"):
        q.qlora_quantize_fp8(_t((4, 64), torch.float32), codes=_t((4, 128)))
    with pytest.raises(ValueError, match="contiguous"):
        q.qlora_quantize_fp8(_t((64, 64), torch.float32).t()[:, :64].t()[::2])


@pytest.mark.parametrize("workspace", [_t((1,)).expand(4096), _t((8192,))[::2], _t((64, 128)).t()])
def test_binding_refuses_workspaces_with_holes(workspace):
    """A workspace of enough elements that are not its bytes one after another: the kernels would write past or between
    them."""
    assert workspace.numel() >= 4096
    with pytest.raises(ValueError, match="contiguous"):
        q._workspace(4096, "cpu", workspace)
    given = _t((4096,))
    assert q._workspace(4096, "cpu", given) is given
    with pytest.raises(ValueError, match="small"):
        q._workspace(4097, "cpu", given)
