"""What the residual norm, the log probabilities and the distillation loss refuse, on the host before anything is
enqueued: through the C ABI with addresses that are never dereferenced, and through the binding."""

import ctypes
import os

import pytest
import torch

import nf4_bit_quantized_amd as q

pytestmark = pytest.mark.skipif(not os.path.exists(q.LIB_PATH), reason="library not built")

F = 0x10000     # an aligned address that no call below gets to use
OK, NULL, SHAPE, UNSUP, WS = (q.QLORA_OK, q.QLORA_ERR_NULL, q.QLORA_ERR_SHAPE, q.QLORA_ERR_UNSUPPORTED,
                              q.QLORA_ERR_WORKSPACE)
NAN, INF = float("nan"), float("inf")


def _each_wrong(good, wrong):
    for at, value, want in wrong:
        args = list(good)
        args[at] = value
        yield args, want


def test_norm_forward_arguments():
    L = q.lib()
    #       0  1   2  3  4  5  6  7  8  9    10    11 12 13 14 15 16
    good = [4, 64, F, 0, F, F, F, F, 0, 1.0, 1e-6, F, F, F, F, F, None]
    wrong = [(0, -1, SHAPE), (0, 1 << 22, SHAPE), (1, 0, SHAPE), (1, 96, SHAPE), (1, 16448, SHAPE), (3, 2, UNSUP),
             (8, 2, UNSUP), (9, NAN, UNSUP), (9, INF, UNSUP), (10, -1.0, UNSUP), (10, NAN, UNSUP), (10, INF, UNSUP),
             (2, None, NULL), (4, None, NULL), (5, None, NULL), (11, None, NULL), (13, None, NULL), (14, None, NULL),
             (15, None, NULL)]
    wrong += [(i, F + 8, UNSUP) for i in (2, 4, 5, 6, 7, 11, 12, 13)] + [(14, F + 2, UNSUP), (15, F + 2, UNSUP)]
    for args, want in _each_wrong(good, wrong):
        assert L.qlora_norm_fwd(*args) == want, args
    nothing = list(good)
    nothing[12:15] = None, None, None
    assert L.qlora_norm_fwd(*nothing) == NULL                       # neither form of x
    assert L.qlora_norm_fwd(0, 64, None, 0, None, F, None, None, 0, 1.0, 0.0, None, None, None, None, None, None) == OK


def test_norm_backward_arguments():
    L = q.lib()
    need = q.qlora_norm_bwd_workspace_bytes(4, 64)
    assert need > 0
    #       0  1   2  3  4  5  6  7  8  9  10   11 12 13 14 15 16 17 18 19 20    21
    good = [4, 64, F, F, 0, F, F, F, F, 0, 1.0, F, F, F, F, F, F, F, 0, F, need, None]
    wrong = [(0, -1, SHAPE), (0, 1 << 22, SHAPE), (1, 32, SHAPE), (4, 2, UNSUP), (9, 7, UNSUP), (10, NAN, UNSUP),
             (2, None, NULL), (3, None, NULL), (5, None, NULL), (6, None, NULL), (11, None, NULL), (13, None, NULL),
             (14, None, NULL), (15, None, NULL), (16, None, NULL), (17, None, NULL), (7, None, NULL), (8, None, NULL),
             (19, None, WS), (20, need - 1, WS), (11, F + 2, UNSUP)]
    wrong += [(i, F + 8, UNSUP) for i in (2, 3, 5, 6, 7, 8, 12, 13, 14, 15, 16, 17, 19)]
    for args, want in _each_wrong(good, wrong):
        assert L.qlora_norm_bwd(*args) == want, args
    assert L.qlora_norm_bwd_workspace_bytes(4, 64, None) == NULL
    n = ctypes.c_size_t()
    assert L.qlora_norm_bwd_workspace_bytes(4, 100, ctypes.byref(n)) == SHAPE
    empty = [0, 64, None, None, 0, None, F, None, None, 0, 1.0, None, None, None, None, None, None, None, 0, None, 0, None]
    assert L.qlora_norm_bwd(*empty) == OK


ROWS = [(0, -1, SHAPE), (0, 1 << 22, SHAPE), (1, 0, SHAPE), (1, 1 << 31, SHAPE), (4, 99, SHAPE), (4, 1 << 31, SHAPE),
        (3, 3, UNSUP), (3, -1, UNSUP), (5, 0.0, UNSUP), (5, -1.0, UNSUP), (5, NAN, UNSUP), (5, INF, UNSUP), (5, 2.0 ** 101, UNSUP),
        (2, None, NULL), (2, F + 1, UNSUP)]


def test_logprob_arguments():
    L = q.lib()
    #       0  1    2  3  4    5    6  7  8  9  10 11 12 13 14
    good = [4, 100, F, 1, 100, 1.0, 2, F, F, F, F, 5, F, F, None]
    wrong = ROWS + [(6, -1, SHAPE), (6, 129, SHAPE), (11, -1, SHAPE), (11, 101, SHAPE), (11, 129, SHAPE),
                    (7, None, NULL), (8, None, NULL), (9, None, NULL), (12, None, NULL), (13, None, NULL),
                    (7, F + 4, UNSUP), (8, F + 2, UNSUP), (9, F + 2, UNSUP), (10, F + 1, UNSUP), (12, F + 4, UNSUP),
                    (13, F + 2, UNSUP)]
    for args, want in _each_wrong(good, wrong):
        assert L.qlora_token_logprob(*args) == want, args
    assert L.qlora_token_logprob(0, 100, None, 1, 100, 1.0, 2, None, None, None, None, 5, None, None, None) == OK


def test_logprob_backward_arguments():
    L = q.lib()
    #       0  1    2  3  4    5    6  7  8  9  10 11 12      13   14   15
    good = [4, 100, F, 1, 100, 1.0, 2, F, F, F, F, F, F + 64, 100, 100, None]
    wrong = ROWS + [(6, 129, SHAPE), (13, 99, SHAPE), (14, 99, SHAPE), (13, 1 << 31, SHAPE), (14, 1 << 31, SHAPE),
                    (7, None, NULL), (8, None, NULL), (9, None, NULL), (10, None, NULL), (12, None, NULL),
                    (7, F + 4, UNSUP), (8, F + 2, UNSUP), (9, F + 2, UNSUP), (10, F + 2, UNSUP), (11, F + 2, UNSUP),
                    (12, F + 1, UNSUP)]
    for args, want in _each_wrong(good, wrong):
        assert L.qlora_token_logprob_bwd(*args) == want, args
    in_place = list(good)
    in_place[12], in_place[14] = F, 104                             # the logits' place at another stride
    assert L.qlora_token_logprob_bwd(*in_place) == UNSUP
    huge = list(good)
    huge[0], huge[4], huge[13], huge[14] = 1 << 21, 1 << 20, 1 << 20, 1 << 20
    assert L.qlora_token_logprob_bwd(*huge) == SHAPE
    assert L.qlora_token_logprob_bwd(0, 100, None, 1, 100, 1.0, 2, None, None, None, None, None, None, 100, 100, None) == OK


def test_distill_arguments():
    L = q.lib()
    #       0  1    2  3  4    5    6  7  8  9  10 11 12
    good = [4, 100, F, 1, 100, 1.0, 3, F, F, 0, F, F, None]
    wrong = ROWS + [(6, 0, SHAPE), (6, 129, SHAPE), (7, None, NULL), (8, None, NULL), (10, None, NULL), (11, None, NULL),
                    (7, F + 4, UNSUP), (8, F + 2, UNSUP), (10, F + 2, UNSUP), (11, F + 2, UNSUP)]
    for args, want in _each_wrong(good, wrong):
        assert L.qlora_distill_fwd(*args) == want, args
    #       0  1    2  3  4    5    6  7  8  9  10 11 12      13   14   15
    good = [4, 100, F, 1, 100, 1.0, 3, F, F, 0, F, F, F + 64, 100, 100, None]
    wrong = ROWS + [(6, 0, SHAPE), (6, 129, SHAPE), (13, 99, SHAPE), (14, 99, SHAPE), (7, None, NULL), (8, None, NULL),
                    (10, None, NULL), (11, None, NULL), (12, None, NULL), (7, F + 4, UNSUP), (8, F + 2, UNSUP),
                    (10, F + 2, UNSUP), (11, F + 2, UNSUP), (12, F + 1, UNSUP)]
    for args, want in _each_wrong(good, wrong):
        assert L.qlora_distill_bwd(*args) == want, args


def _refused(call, *a, **k):
    with pytest.raises(ValueError) as e:
        call(*a, **k)
    return str(e.value)


def test_binding_norm():
    h, w, b = torch.zeros(3, 128), torch.ones(128), torch.zeros(3, 128, dtype=torch.bfloat16)
    f, g = q.qlora_norm_fwd, q.qlora_norm_bwd
    assert "on the GPU" in _refused(f, h, w, block=b)
    assert "2-D" in _refused(f, h[0], w)
    assert "contiguous" in _refused(f, torch.zeros(3, 256)[:, :128], w)
    assert "float32 or bfloat16" in _refused(f, h.half(), w)
    assert "weight" in _refused(f, h, w[:64])
    assert "block" in _refused(f, h, w, block=b.float())
    assert "need a block" in _refused(f, h, w, gate=w)
    assert "post_weight" in _refused(f, h, w, block=b, post_weight=w.bfloat16())
    assert "form" in _refused(f, h, w, form="fp4")
    assert "does not write" in _refused(f, h, w, X=b, form="fp8")
    assert "h_out" in _refused(f, h, w, h_out=h)
    s = torch.zeros(3, 2)
    assert "on the GPU" in _refused(g, b, h, w, s)
    assert "dX" in _refused(g, b.float(), h, w, s)
    assert "stats" in _refused(g, b, h, w, s[:2])
    assert "dh_out" in _refused(g, b, h, w, s, dh_out=b)
    assert "dblock" in _refused(g, b, h, w, s, dblock=b)
    assert "dgate" in _refused(g, b, h, w, s, dgate=w)
    assert "dweight" in _refused(g, b, h, w, s, want_weights=False, dweight=w)
    assert "accumulate" in _refused(g, b, h, w, s, accumulate=True)


def test_binding_logits():
    z, tok = torch.zeros(3, 50), torch.zeros(3, dtype=torch.int64)
    f, g = q.qlora_token_logprob, q.qlora_token_logprob_bwd
    assert "on the GPU" in _refused(f, z, tok)
    assert "2-D" in _refused(f, z[0], tok)
    assert "float16" in _refused(f, z.double(), tok)
    assert "vocab" in _refused(f, z, tok, vocab=51)
    assert "vocab" in _refused(f, z, tok, vocab=0)
    assert "contiguous" in _refused(f, z.t(), tok)
    assert "overlap" in _refused(f, z[:1].expand(3, 50), tok)
    assert "tokens" in _refused(f, z, tok.int())
    assert "tokens" in _refused(f, z, tok[:2])
    assert "logprob needs tokens" in _refused(f, z, logprob=z[:, 0])
    assert "logprob" in _refused(f, z, tok, logprob=torch.zeros(3, 1))
    s, d = torch.zeros(3, 2), torch.zeros(3)
    assert "on the GPU" in _refused(g, z, tok, s, d)
    assert "d_logprob" in _refused(g, z, tok, s, d[:2])
    assert "stats" in _refused(g, z, tok, d, d)
    assert "entropy" in _refused(g, z, tok, s, d, d_entropy=d)
    assert "required" in _refused(g, z, None, s, None)
    ids, v = torch.zeros(3, 4, dtype=torch.int64), torch.zeros(3, 4)
    assert "on the GPU" in _refused(q.qlora_distill_fwd, z, ids, v)
    assert "2-D" in _refused(q.qlora_distill_fwd, z, tok, v)
    assert "values" in _refused(q.qlora_distill_fwd, z, ids, v[:, :3])
    assert "stats" in _refused(q.qlora_distill_bwd, z, ids, v, s, d)
    assert "d_loss" in _refused(q.qlora_distill_bwd, z, ids, v, torch.zeros(3, 4), d[:1])
