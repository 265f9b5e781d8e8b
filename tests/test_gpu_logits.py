"""Log probabilities, entropy, alternatives and the distillation loss on the GPU, with their gradients, against the
float64 oracle: every type, odd vocabularies, row strides and alignments, masked and empty rows, ties.

Tolerances.  A row's sum S is added up in at most V / 256 + 64 steps of 2^-24 each (a thread's own elements, then the
workgroup's), and a term 2^d is off by 2^-23 and by |d| 2^-24, which weighted by the terms is below 40 steps: log S is
off by at most TOL(V) = (V / 256 + 128) 2^-24 absolute.  Results have half a step of their type besides."""

import numpy as np
import pytest

from gpu_helpers import say
from oracle import logits as ol

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -24


def TOL(V):
    return (V / 256 + 128) * F32


def _logits(T, V, dtype, cols=None, offset=0, seed=0, std=2.5):
    """T rows of V logits inside rows of `cols` elements, the first `offset` elements into their allocation."""
    import torch
    cols = V if cols is None else cols
    g = torch.Generator(device="cuda").manual_seed(seed)
    store = torch.full((offset + T * cols,), float("nan"), dtype=getattr(torch, dtype), device="cuda")
    rows = store[offset:].view(T, cols)
    rows[:, :V] = (torch.randn((T, V), generator=g, device="cuda") * std).to(store.dtype)
    return rows


def _np(t):
    return t.double().cpu().numpy()


def _alike(got, want, tol, name):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), name
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), name
    err = np.abs(got[fine] - want[fine])
    assert np.all(err <= np.broadcast_to(tol, want.shape)[fine] + F32 * np.abs(want[fine])), \
        f"{name}: {err.max()} of {np.broadcast_to(tol, want.shape)[fine].max()}"


def _check_score(z, tokens, scale, top, out, vocab=None):
    logprob, stats, entropy, ids, top_lp = (None if t is None else _np(t) for t in out)
    z = _np(z)[:, :vocab]
    T, V = z.shape
    tol = TOL(V)
    tokens = tokens.cpu().numpy()
    for t in range(T):
        M, log_s = ol.statistics(z[t], scale)
        if not np.isnan(M):
            assert stats[t, 0] == M
        _alike(stats[t, 1], log_s, tol, "log S")
        lq = ol.log_q(z[t], M, log_s, scale)
        given = ol.named(tokens[t], V)
        want = np.where(given, lq[np.where(given, tokens[t], 0)], 0.0)
        _alike(logprob[t], want, tol, "logprob")
        if entropy is not None:
            H = ol.entropy(z[t], scale)
            _alike(entropy[t], H, tol * (1 + abs(H)), "entropy")
        if top:
            at = ol.largest(z[t], top)
            assert np.array_equal(ids[t], at), f"row {t}: {ids[t]} for {at}"
            _alike(top_lp[t], lq[at], tol, "top_logprob")


SCORES = [  # T, V, dtype, columns, offset, tokens per row, top, scale
    (1, 1, "float32", 1, 0, 1, 1, 1.0), (2, 7, "bfloat16", 9, 1, 3, 7, 1.0), (5, 100, "float16", 100, 3, 1, 100, 0.7),
    (3, 1000, "float32", 1003, 1, 2, 128, 2.0), (4, 4097, "bfloat16", 4097, 0, 1, 20, 1.0),
    (1, 32000, "bfloat16", 32000, 0, 1, 5, 1.25), (64, 32000, "float16", 32064, 0, 1, 0, 1.0),
    (3, 50257, "float32", 50257, 2, 128, 64, 0.5), (1, 128256, "bfloat16", 128256, 0, 1, 20, 1.0),
    (2, 151937, "bfloat16", 151940, 5, 1, 128, 1.0), (600, 2049, "bfloat16", 2049, 0, 1, 3, 1.0),
    (1100, 517, "float32", 520, 0, 1, 10, 1.0), (1, 300001, "float32", 300001, 0, 1, 50, 1.0)]


@pytest.mark.parametrize("T,V,dtype,cols,offset,n,top,scale", SCORES)
def test_score(T, V, dtype, cols, offset, n, top, scale):
    import nf4_bit_quantized_amd as q
    import torch
    say(f"score T {T} V {V} {dtype} columns {cols} offset {offset} n {n} top {top} scale {scale}")
    z = _logits(T, V, dtype, cols, offset, seed=V)
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens = torch.randint(0, V, (T, n), generator=g, device="cuda")
    if T > 1:
        tokens[1::3, 0] = -100
        tokens[0, -1] = V
    out = q.qlora_token_logprob(z, tokens, scale=scale, top=top, want_entropy=True, vocab=V)
    _check_score(z, tokens, scale, top, out, V)
    # the parts that are not asked for change nothing
    plain = q.qlora_token_logprob(z, tokens, scale=scale, vocab=V)
    assert torch.equal(plain[0], out[0]) and torch.equal(plain[1], out[1])
    assert plain[2] is plain[3] is plain[4] is None
    alone = q.qlora_token_logprob(z, scale=scale, top=top, vocab=V)
    assert alone[0] is None and (top == 0 or torch.equal(alone[3], out[3]) and torch.equal(alone[4], out[4]))


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("V,T", [(333, 9), (40000, 9), (40000, 1100)])
def test_masked_rows(V, T, dtype):
    """Masks of -inf and of the type's lowest value, rows that they leave empty, NaN and infinities, equal logits."""
    import nf4_bit_quantized_amd as q
    import torch
    say(f"masked rows V {V} T {T} {dtype}")
    dt = getattr(torch, dtype)
    low, inf = torch.finfo(dt).min, float("inf")
    z = _logits(T, V, dtype, seed=2)
    z[0, :] = -inf
    z[1, :] = low
    z[2, 5:] = -inf
    z[3, :V // 2] = low
    z[4, 17] = float("nan")
    z[5, 3] = inf
    z[6, :] = 1.5
    z[7, :] = -inf
    z[7, 300] = low
    z[8, ::2] = 0.0
    z[8, 1::2] = -0.0
    tokens = torch.full((T, 2), 300, dtype=torch.int64, device="cuda")
    tokens[:, 1] = 2
    out = q.qlora_token_logprob(z, tokens, top=20, want_entropy=True)
    rows = slice(0, 9)
    _check_score(z[rows], tokens[rows], 1.0, 20, [t[rows] for t in out])
    d, d_H = torch.randn((T, 2), device="cuda"), torch.randn(T, device="cuda")
    got = q.qlora_token_logprob_bwd(z, tokens, out[1], d, entropy=out[2], d_entropy=d_H)
    assert not got[[0]].any() and got[4].isnan().any() and got[5].isnan().any()
    zn, s = _np(z[:9]), _np(out[1])
    for t in (1, 2, 3, 6, 7, 8):                          # a given token that the mask takes still has d (1 - 0)
        want, mag = ol.score_gradient(zn[t], 1.0, [300, 2], _np(d[t]), s[t, 0], s[t, 1], float(out[2][t]), float(d_H[t]))
        _near(got[t:t + 1], want[None], mag[None], "dlogits")
    none = torch.zeros_like(d)
    assert not q.qlora_token_logprob_bwd(z, tokens, out[1], none).any()      # whatever the row holds


def _half(t):
    import torch
    return torch.finfo(t).eps / 2


def _near(got, want, mag, name):
    """Half a step of the type (of its least value, below its normal range), and 2^-21 of the magnitude: a
    probability is off by |log q| 2^-23 + 2^-22 relative, which the magnitude counts as (4 + |log q|) 2^-22."""
    import torch
    low = torch.finfo(got.dtype)
    tiny = low.smallest_normal * low.eps / 2 if got.dtype == torch.float16 else 1e-37
    half, got = _half(got.dtype), _np(got)
    over = np.abs(got - want) - (half * np.abs(want) + 2.0 ** -21 * mag + tiny)
    at = np.unravel_index(np.argmax(over), over.shape)
    assert over[at] <= 0, f"{name}{list(at)}: {got[at]} for {want[at]}, magnitude {mag[at]}"


GRADS = [(1, 1, "float32", 1, 0, 1), (3, 9, "bfloat16", 16, 0, 2), (4, 1001, "float16", 1001, 1, 1),
         (2, 32000, "bfloat16", 32064, 0, 128), (33, 8191, "bfloat16", 8191, 3, 1), (5, 50257, "float32", 50260, 1, 3),
         (700, 640, "bfloat16", 640, 0, 1)]


@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("T,V,dtype,cols,offset,n", GRADS)
def test_score_gradient(T, V, dtype, cols, offset, n, entropy):
    import nf4_bit_quantized_amd as q
    import torch
    say(f"score gradient T {T} V {V} {dtype} columns {cols} offset {offset} n {n} entropy {entropy}")
    scale = 1.25
    z = _logits(T, V, dtype, cols, offset, seed=V)
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens = torch.randint(-1, V + 1, (T, n), generator=g, device="cuda")
    if n > 1:
        tokens[:, 1] = tokens[:, 0]                       # the same token twice
    _, stats, H, _, _ = q.qlora_token_logprob(z, tokens, scale=scale, want_entropy=True, vocab=V)
    d, d_H = torch.randn((T, n), generator=g, device="cuda"), torch.randn(T, generator=g, device="cuda")
    d[T // 2] = 0.0
    more = dict(entropy=H, d_entropy=d_H) if entropy else {}
    got = q.qlora_token_logprob_bwd(z, tokens, stats, d, scale=scale, vocab=V, **more)
    assert got.shape == z.shape and got.dtype == z.dtype
    want, mag = np.zeros((T, V)), np.zeros((T, V))
    zn, s, dn = _np(z)[:, :V], _np(stats), _np(d)
    for t in range(T):
        want[t], mag[t] = ol.score_gradient(zn[t], scale, tokens[t].cpu().numpy(), dn[t], s[t, 0], s[t, 1],
                                            float(H[t]) if entropy else 0.0, float(d_H[t]) if entropy else 0.0)
    _near(got[:, :V], want, mag, "dlogits")
    assert not got[:, V:].any()
    # in the logits' place, and into rows of another stride and alignment
    place = torch.empty_strided(z.shape, z.stride(), dtype=z.dtype, device="cuda").copy_(z)
    assert q.qlora_token_logprob_bwd(place, tokens, stats, d, scale=scale, vocab=V, dlogits=place, **more) is place
    assert torch.equal(place, got)
    wide = torch.full((T, cols + 5), 9.0, dtype=z.dtype, device="cuda")
    q.qlora_token_logprob_bwd(z, tokens, stats, d, scale=scale, vocab=V, dlogits=wide[:, 3:cols + 3], **more)
    assert torch.equal(wide[:, 3:cols + 3], got) and (wide[:, :3] == 9).all() and (wide[:, cols + 3:] == 9).all()


def test_entropy_gradient_alone():
    import nf4_bit_quantized_amd as q
    import torch
    z = _logits(3, 8192, "float32", seed=5)
    _, stats, H, _, _ = q.qlora_token_logprob(z, want_entropy=True)
    d_H = torch.tensor([1.0, 0.0, -2.0], device="cuda")
    got = q.qlora_token_logprob_bwd(z, None, stats, None, entropy=H, d_entropy=d_H)
    rows = [ol.score_gradient(_np(z)[t], 1.0, [], [], *_np(stats)[t], float(H[t]), float(d_H[t])) for t in range(3)]
    _near(got, np.stack([w for w, _ in rows]), np.stack([m for _, m in rows]), "dlogits")
    assert not got[1].any()


DISTILL = [  # T, V, dtype, columns, offset, k, scale
    (1, 1, "float32", 1, 0, 1, 1.0), (3, 11, "bfloat16", 12, 1, 11, 1.0), (4, 1000, "float16", 1000, 0, 128, 0.5),
    (2, 32000, "bfloat16", 32064, 0, 64, 1.0), (70, 4096, "float32", 4099, 3, 16, 2.0),
    (3, 50257, "float32", 50257, 0, 7, 1.0), (2, 151937, "bfloat16", 151937, 0, 100, 1.0),
    (1, 280001, "float32", 280001, 1, 33, 1.0), (1100, 700, "bfloat16", 704, 0, 5, 1.0)]


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("T,V,dtype,cols,offset,k,scale", DISTILL)
def test_distill(T, V, dtype, cols, offset, k, scale, rest):
    import nf4_bit_quantized_amd as q
    import torch
    say(f"distill T {T} V {V} {dtype} columns {cols} offset {offset} k {k} scale {scale} rest {rest}")
    z = _logits(T, V, dtype, cols, offset, seed=V)
    teacher = _logits(T, V, "float32", seed=V + 1)
    teacher += z[:, :V].float()
    _, _, _, ids, values = q.qlora_token_logprob(teacher, scale=scale, top=k)
    if k > 3:                                             # shorter lists, a token twice, one with nothing, one without mass
        ids[::2, 2] = -1
        ids[::3, 3] = ids[::3, 0]
        ids[T // 2] = V
        values[0, 1] = float("-inf")
    loss, stats = q.qlora_distill_fwd(z, ids, values, scale=scale, rest=rest, vocab=V)
    d = torch.randn(T, device="cuda")
    d[T // 3] = 0.0
    got = q.qlora_distill_bwd(z, ids, values, stats, d, scale=scale, rest=rest, vocab=V)
    zn, sn, dn, idn, vn = _np(z)[:, :V], _np(stats), _np(d), ids.cpu().numpy(), _np(values)
    want, mag, tol = np.zeros((T, V)), np.zeros((T, V)), TOL(V)
    for t in range(T):
        l, M, log_s, whole, ratio = ol.distill(zn[t], scale, idn[t], vn[t], rest)
        _alike(loss[t].item(), l, 2 * tol, "loss")
        assert sn[t, 0] == M
        _alike(sn[t, 1], log_s, tol, "log S")
        # sum p is formed in 64 bits; q_r has the error of two sums
        _alike(sn[t, 2:], [whole, ratio], np.array([F32, 3 * tol * ratio]), "whole, ratio")
        want[t], mag[t] = ol.distill_gradient(zn[t], scale, idn[t], vn[t], rest, dn[t], *sn[t])
    _near(got[:, :V], want, mag, "dlogits")
    assert not got[:, V:].any()
    place = torch.empty_strided(z.shape, z.stride(), dtype=z.dtype, device="cuda").copy_(z)
    q.qlora_distill_bwd(place, ids, values, stats, d, scale=scale, rest=rest, vocab=V, dlogits=place)
    assert torch.equal(place, got)


@pytest.mark.parametrize("V", [200, 20000])
def test_distill_masked(V):
    import nf4_bit_quantized_amd as q
    import torch
    say(f"distill masked V {V}")
    inf = float("inf")
    z = _logits(6, V, "float32", seed=9)
    ids = torch.arange(6 * 8, device="cuda").view(6, 8) * 4
    values = torch.log_softmax(torch.randn((6, 8), device="cuda"), 1) - 0.5
    z[0, :] = -inf                                        # nothing left
    z[1].scatter_(0, ids[1, :1], -inf)                    # a token that the student cannot say
    z[2, 1::2] = -inf                                     # a mask that leaves the list whole
    keep = torch.zeros(V, dtype=torch.bool, device="cuda")
    keep[ids[3]] = True
    z[3, ~keep] = -inf                                    # nothing outside the list: the bucket is left out
    z[4, 3] = float("nan")
    ids[5] = -1                                           # no teacher
    z[5, 7] = float("nan")
    zn, idn, vn = _np(z), ids.cpu().numpy(), _np(values)
    for rest in (False, True):
        loss, stats = q.qlora_distill_fwd(z, ids, values, rest=rest)
        grad = q.qlora_distill_bwd(z, ids, values, stats, torch.ones(6, device="cuda"), rest=rest)
        for t in range(6):
            l, M, log_s, whole, ratio = ol.distill(zn[t], 1.0, idn[t], vn[t], rest)
            _alike(loss[t].item(), l, 2 * TOL(V), "loss")
            if t != 4 and t != 5:
                _alike(_np(stats)[t], [M, log_s, whole, ratio], TOL(V) * 3 * (1 + ratio), "stats")
                want, mag = ol.distill_gradient(zn[t], 1.0, idn[t], vn[t], rest, 1.0, *_np(stats)[t])
                _near(grad[t:t + 1], want[None], mag[None], "dlogits")
        assert not grad[0].any() and not grad[5].any() and grad[4].isnan().any()


def test_no_rows():
    import nf4_bit_quantized_amd as q
    import torch
    z, tokens = torch.empty((0, 50), device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    out = q.qlora_token_logprob(z, tokens, top=5, want_entropy=True)
    assert [tuple(t.shape) for t in out] == [(0,), (0, 2), (0,), (0, 5), (0, 5)]
    assert q.qlora_token_logprob_bwd(z, tokens, out[1], out[0]).shape == (0, 50)
    loss, stats = q.qlora_distill_fwd(z, out[3], out[4])
    assert loss.shape == (0,) and q.qlora_distill_bwd(z, out[3], out[4], stats, loss).shape == (0, 50)
