"""Rows of logits that are masked with large finite values between those of the data and the type's lowest: whole
threads see nothing but the mask, and a mask's value times the scale is far from a whole number that 32 bits hold.
Against the float64 oracle, with the tolerances of test_gpu_logits.py: a masked token has probability 0 in both, and
log q = scale (z - M) - log S in 64 bits, rounded once."""

import numpy as np
import pytest

from gpu_helpers import say
from oracle import logits as ol
from test_gpu_logits import TOL, F32, _alike, _check_score, _logits, _near, _np

pytestmark = pytest.mark.gpu

MASKS = {"bfloat16": (-1e9, -1e10, -1e20, -1e30), "float32": (-1e9, -1e10, -1e20, -1e30),
         "float16": (-1e3, -1e4, -6e4, -65504.0)}
KEPT = 5


def _masked(T, V, dtype, seed):
    """T rows: each mask over the front, over the back, over all but KEPT tokens; then one of these with NaN among the
    masked, then rows as they are.  Returns the logits and the number of rows to look at."""
    import torch
    z = _logits(T, V, dtype, seed=seed)
    kept = torch.randperm(V, generator=torch.Generator().manual_seed(seed))[:KEPT].cuda()
    row = 0
    for value in MASKS[dtype]:
        z[row, :V - V // 4] = value
        z[row + 1, V // 4:] = value
        some = z[row + 2, kept].clone()
        z[row + 2] = value
        z[row + 2, kept] = some
        row += 3
    z[row, V // 8:] = MASKS[dtype][1]
    z[row, V - V // 8] = float("nan")
    return z, kept, row + 2


@pytest.mark.parametrize("scale", [0.5, 1.0, 1.25, 2.0])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32", "float16"])
@pytest.mark.parametrize("T,V", [(16, 700), (16, 40000), (300, 60001)])
def test_score(T, V, dtype, scale):
    import nf4_bit_quantized_amd as q
    import torch
    say(f"finite masks T {T} V {V} {dtype} scale {scale}")
    z, kept, rows = _masked(T, V, dtype, seed=V)
    tokens = torch.full((T, 3), V - 1, dtype=torch.int64, device="cuda")
    tokens[:, 1] = kept[0]
    tokens[:, 2] = 0
    d, d_H = torch.randn((T, 3), device="cuda"), torch.randn(T, device="cuda")
    out = q.qlora_token_logprob(z, tokens, scale=scale, top=20, want_entropy=True)
    plain = q.qlora_token_logprob(z, tokens, scale=scale)
    few = slice(0, rows)
    _check_score(z[few], tokens[few], scale, 20, [t[few] for t in out])
    _check_score(z[few], tokens[few], scale, 0, [None if t is None else t[few] for t in plain])
    got = q.qlora_token_logprob_bwd(z, tokens, out[1], d, scale=scale, entropy=out[2], d_entropy=d_H)
    assert got[rows - 2].isnan().all()
    zn, s = _np(z[few]), _np(out[1])
    for t in range(rows):
        if t != rows - 2:
            want, mag = ol.score_gradient(zn[t], scale, tokens[t].cpu().numpy(), _np(d[t]), *s[t], float(out[2][t]),
                                          float(d_H[t]))
            _near(got[t:t + 1], want[None], mag[None], "dlogits")


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32", "float16"])
@pytest.mark.parametrize("T,V", [(16, 700), (16, 40000), (300, 60001)])
def test_distill(T, V, dtype, rest):
    import nf4_bit_quantized_amd as q
    import torch
    say(f"finite masks, distill T {T} V {V} {dtype} rest {rest}")
    scale = 1.25
    z, kept, rows = _masked(T, V, dtype, seed=V + 1)
    ids = torch.cat([kept, torch.tensor([0, V - 1], device="cuda")]).unique().expand(T, -1).contiguous()
    values = torch.log_softmax(torch.randn(ids.shape, device="cuda"), 1) - 0.25
    loss, stats = q.qlora_distill_fwd(z, ids, values, scale=scale, rest=rest)
    d = torch.randn(T, device="cuda")
    got = q.qlora_distill_bwd(z, ids, values, stats, d, scale=scale, rest=rest)
    zn, sn, idn, vn = _np(z[:rows]), _np(stats), ids.cpu().numpy(), _np(values)
    for t in range(rows):
        l, M, log_s, whole, ratio = ol.distill(zn[t], scale, idn[t], vn[t], rest)
        # two of log q, weighted by p, which add up to at most 1; the far tokens' terms are rounded with the loss
        _alike(loss[t].item(), l, 2 * TOL(V), "loss")
        if t == rows - 2:
            assert np.isnan(l) and got[t].isnan().all()
            continue
        assert sn[t, 0] == M
        _alike(sn[t, 1], log_s, TOL(V), "log S")
        _alike(sn[t, 2:], [whole, ratio], np.array([F32, 3 * TOL(V) * ratio]), "whole, ratio")
        want, mag = ol.distill_gradient(zn[t], scale, idn[t], vn[t], rest, float(d[t]), *sn[t])
        _near(got[t:t + 1], want[None], mag[None], "dlogits")


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("weight", [1e9, -1e20, 1e36])
def test_large_weights_of_the_entropy(weight, dtype):
    """A masked token's q is 0, and so is its gradient, at any weight."""
    import nf4_bit_quantized_amd as q
    import torch
    say(f"weight {weight} of the entropy, {dtype}")
    V = 3000
    z = _logits(4, V, dtype, seed=12)
    z[0, ::3] = float("-inf")
    z[1, V // 2:] = -1e30
    z[2, 1:] = -200.0
    _, stats, H, _, _ = q.qlora_token_logprob(z, want_entropy=True)
    d_H = torch.full((4,), weight, device="cuda")
    got = q.qlora_token_logprob_bwd(z, None, stats, None, entropy=H, d_entropy=d_H)
    assert not got[0, ::3].any() and not got[1, V // 2:].any()
    rows = [ol.score_gradient(_np(z)[t], 1.0, [], [], *_np(stats)[t], float(H[t]), float(d_H[t])) for t in range(4)]
    _near(got, np.stack([w for w, _ in rows]), np.stack([m for _, m in rows]), "dlogits")


@pytest.mark.parametrize("V", [6, 300, 20000])
@pytest.mark.parametrize("value", ["nan", "inf"])
def test_not_finite_in_the_list_alone(value, V):
    """Nothing else is left of the row, listed or not: the loss and the gradient are NaN all the same."""
    import nf4_bit_quantized_amd as q
    import torch
    say(f"{value} in the list alone, V {V}")
    z = torch.full((3, V), float("-inf"), device="cuda")
    z[0, 2] = float(value)
    z[1, 1:6] = float(value)
    z[2, 4] = 1.0
    ids = torch.arange(1, 6, device="cuda").repeat(3, 1)
    values = torch.full((3, 5), -2.0, device="cuda")
    for rest in (False, True):
        loss, stats = q.qlora_distill_fwd(z, ids, values, rest=rest)
        got = q.qlora_distill_bwd(z, ids, values, stats, torch.ones(3, device="cuda"), rest=rest)
        for t in range(3):
            l, *_ = ol.distill(_np(z)[t], 1.0, ids[t].cpu().numpy(), _np(values)[t], rest)
            _alike(loss[t].item(), l, 2 * TOL(V), "loss")
        assert got[:2].isnan().all() and got[2].isfinite().all()


def test_rows_without_entries_take_any_weight():
    import nf4_bit_quantized_amd as q
    import torch
    say("rows without entries")
    z = _logits(3, 500, "float32", seed=13)
    ids = torch.tensor([[1, 2], [-1, 500], [-100, -1]], device="cuda")
    values = torch.tensor([[-1.0, -2.0]] * 3, device="cuda")
    d = torch.tensor([1.0, float("nan"), float("inf")], device="cuda")
    for rest in (False, True):
        loss, stats = q.qlora_distill_fwd(z, ids, values, rest=rest)
        got = q.qlora_distill_bwd(z, ids, values, stats, d, rest=rest)
        assert not loss[1:].any() and got[0].any() and not got[1:].any()
    _, stats, _, _, _ = q.qlora_token_logprob(z, ids)
    got = q.qlora_token_logprob_bwd(z, ids, stats, d[:, None].expand(3, 2).contiguous())
    assert got[0].any() and not got[1:].any()
