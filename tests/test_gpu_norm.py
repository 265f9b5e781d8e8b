"""The residual norm and its backward on the GPU against the float64 oracle: every form, stream and weight type, with
and without a block, its norm and its gate, at the widths where the work is cut differently.

Tolerances.  An output is off by half a step of its type, finfo.eps / 2 relative, and by what 32-bit arithmetic leaves:
at most FINE of its magnitude (the sum of the absolute values it is added up from).  A sum of squares is added up in at
most 16 + 6 + 16 steps of 2^-24 each and its root halves that; with the rounding of h', of the branch (four products)
and of x (three) this stays below 2^-18.  The sums over tokens take T / 256 + 16 + 16 steps more, fewer than 64 here."""

import numpy as np
import pytest

from gpu_helpers import say
from oracle import fp8 as of8
from oracle import norm as on

pytestmark = pytest.mark.gpu

FINE = 2.0 ** -18


def _half(t):
    import torch
    return torch.finfo(t).eps / 2


def _inputs(T, D, stream, weights, post, gate, block=True, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    h = rand(T, D)
    h[:, D // 3] *= 50
    v = dict(h=h.to(stream), weight=(1 + rand(D) / 4).to(weights))
    if block:
        v["block"] = (rand(T, D) * torch.exp(rand(T, 1))).bfloat16()
    if post:
        v["post_weight"] = rand(D).to(weights)
    if gate:
        v["gate"] = rand(D).to(weights)
    return v


def _np(t):
    return t.double().cpu().numpy()


def _near(got, want, mag, name):
    got, half = _np(got), _half(got.dtype)
    over = np.abs(got - want) - (half * np.abs(want) + FINE * mag + 1e-37)
    at = np.unravel_index(np.argmax(over), over.shape)
    assert over[at] <= 0, f"{name}{list(at)}: {got[at]} for {want[at]}, magnitude {mag[at]}"


def _check_form(codes, scales, x, mag):
    """The 8-bit form of x, x being known to within FINE of mag: the scale is the rule's for some x that near, and the
    values are within half a step."""
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy().astype(np.int64)
    T, D = x.shape
    for b in range(-(-D // 128)):
        at = np.s_[:, 128 * b:128 * (b + 1)]
        big, slack = np.abs(x[at]).max(1), FINE * mag[at].max(1)
        e = scales[:, b]
        limit = 448.0 * 2.0 ** (e - 127.0)
        assert np.all(big - slack <= limit) and np.all((big + slack > limit / 2) | (e == 1))
    assert np.all(scales[:, -(-D // 128):] == 127)
    k = 2.0 ** (scales - 127.0)[:, np.arange(D) // 128]
    err = np.abs(of8.e4m3_values()[codes] * k - x)
    assert np.all(err <= 2.0 ** -4 * np.abs(x) + 2.0 ** -10 * k + FINE * mag)


CASES = [  # T, D, stream, weights, post, gate
    (1, 64, "bfloat16", "bfloat16", False, False), (3, 192, "float32", "float32", True, True),
    (5, 576, "bfloat16", "float32", True, False), (2, 1024, "float32", "bfloat16", False, True),
    (1, 4096, "float32", "float32", True, True), (37, 5120, "bfloat16", "bfloat16", True, True),
    (9, 8192, "bfloat16", "bfloat16", False, False), (300, 8192, "float32", "bfloat16", True, False),
    (4, 8256, "bfloat16", "float32", True, True), (3, 16384, "float32", "float32", True, True),
    (600, 704, "float32", "bfloat16", True, True)]


@pytest.mark.parametrize("T,D,stream,weights,post,gate", CASES)
def test_forward_and_backward(T, D, stream, weights, post, gate):
    import nf4_bit_quantized_amd as q
    import torch
    say(f"norm T {T} D {D} stream {stream} weights {weights} post {post} gate {gate}")
    scale, eps = 0.375, 1e-5
    v = _inputs(T, D, getattr(torch, stream), getattr(torch, weights), post, gate, seed=T + D)
    want, mag = on.forward(**{k: _np(t) for k, t in v.items()}, scale=scale, eps=eps)
    (X, codes, scales), h, stats = q.qlora_norm_fwd(scale=scale, eps=eps, form="both", **v)
    _near(X, want["x"], mag["x"], "x")
    _near(h, want["h"], mag["h"], "h")
    np.testing.assert_allclose(_np(stats), np.stack([want["r"], want["r_b"]], 1), rtol=2.0 ** -18)
    _check_form(codes, scales, want["x"], mag["x"])
    # each form alone is the same
    x1, h1, s1 = q.qlora_norm_fwd(scale=scale, eps=eps, **v)
    (c2, sc2), h2, s2 = q.qlora_norm_fwd(scale=scale, eps=eps, form="fp8", **v)
    assert torch.equal(x1, X) and torch.equal(h1, h) and torch.equal(h2, h) and torch.equal(s1, stats)
    assert torch.equal(c2, codes) and torch.equal(sc2, scales) and torch.equal(s2, stats)

    rest = {k: t for k, t in v.items() if k != "h"}
    g = torch.Generator(device="cuda").manual_seed(1)
    dX = torch.randn((T, D), generator=g, device="cuda").bfloat16()
    later = torch.randn((T, D), generator=g, device="cuda").to(h.dtype)
    want, mag = on.backward(_np(dX), _np(h), r=_np(stats)[:, 0], r_b=_np(stats)[:, 1], scale=scale, dh_out=_np(later),
                            **{k: _np(t) for k, t in rest.items()})
    got = dict(zip(("dh", "dblock", "dweight", "dpost_weight", "dgate"),
                   q.qlora_norm_bwd(dX, h, stats=stats, scale=scale, dh_out=later, **rest)))
    assert {k for k, t in got.items() if t is not None} == set(want)
    for k in want:
        _near(got[k], want[k], mag[k], k)
    # the same again is the same; in place; frozen weights; added to what is there
    again = q.qlora_norm_bwd(dX, h, stats=stats, scale=scale, dh_out=later, **rest)
    assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(again, got.values()))
    place = later.clone()
    frozen = q.qlora_norm_bwd(dX, h, stats=stats, scale=scale, dh_out=place, dh=place, want_weights=False, **rest)
    assert frozen[0] is place and torch.equal(place, got["dh"]) and torch.equal(frozen[1], got["dblock"])
    assert frozen[2] is frozen[3] is frozen[4] is None
    sums = {k: torch.full((D,), 3.0, device="cuda") for k in want if k not in ("dh", "dblock")}
    q.qlora_norm_bwd(dX, h, stats=stats, scale=scale, dh_out=later, accumulate=True, **sums, **rest)
    for k, t in sums.items():
        assert torch.equal(t, got[k] + 3.0)


@pytest.mark.parametrize("T,D,stream", [(1, 64, "float32"), (7, 320, "bfloat16"), (260, 2048, "float32")])
def test_without_a_block(T, D, stream):
    import nf4_bit_quantized_amd as q
    import torch
    say(f"norm without a block T {T} D {D} {stream}")
    v = _inputs(T, D, getattr(torch, stream), torch.float32, False, False, block=False, seed=3)
    want, mag = on.forward(**{k: _np(t) for k, t in v.items()})
    X, h, stats = q.qlora_norm_fwd(v["h"], v["weight"])
    assert h is v["h"]
    _near(X, want["x"], mag["x"], "x")
    dX = torch.randn((T, D), device="cuda").bfloat16()
    want, mag = on.backward(_np(dX), _np(h), _np(v["weight"]), _np(stats)[:, 0], _np(stats)[:, 1])
    dh, dblock, dweight, dpost, dgate = q.qlora_norm_bwd(dX, h, v["weight"], stats)
    assert dblock is dpost is dgate is None
    _near(dh, want["dh"], mag["dh"], "dh")
    _near(dweight, want["dweight"], mag["dweight"], "dweight")


def test_in_place_stream_and_given_outputs():
    import nf4_bit_quantized_amd as q
    import torch
    v = _inputs(11, 640, torch.bfloat16, torch.bfloat16, True, True, seed=4)
    X, h, stats = q.qlora_norm_fwd(**v)
    place, X2, s2 = v["h"].clone(), torch.full_like(X, 7.0), torch.empty_like(stats)
    out = q.qlora_norm_fwd(**{**v, "h": place}, h_out=place, X=X2, stats=s2)
    assert out[0] is X2 and out[1] is place and out[2] is s2
    assert torch.equal(place, h) and torch.equal(X2, X) and torch.equal(s2, stats)


def test_no_tokens():
    import nf4_bit_quantized_amd as q
    import torch
    v = _inputs(0, 128, torch.float32, torch.float32, True, True)
    X, h, stats = q.qlora_norm_fwd(**v)
    assert X.shape == h.shape == (0, 128) and stats.shape == (0, 2)
    rest = {k: t for k, t in v.items() if k != "h"}
    out = q.qlora_norm_bwd(X, h, stats=stats, **rest)
    assert out[0].shape == (0, 128) and all(not t.any() for t in out[2:])
    kept = [torch.ones(128, device="cuda") for _ in range(3)]
    q.qlora_norm_bwd(X, h, stats=stats, accumulate=True, dweight=kept[0], dpost_weight=kept[1], dgate=kept[2], **rest)
    assert all((t == 1).all() for t in kept)


def test_not_finite_stays_in_its_token():
    import nf4_bit_quantized_amd as q
    import torch
    v = _inputs(6, 1024, torch.float32, torch.float32, True, False, seed=5)
    clean, _, _ = q.qlora_norm_fwd(**v)
    v["block"][2, 100] = float("nan")
    v["h"][4, 1] = float("inf")
    X, _, _ = q.qlora_norm_fwd(**v)
    fine = [0, 1, 3, 5]
    assert torch.equal(X[fine], clean[fine]) and X[2].isnan().all() and X[4, 1].isnan()


@pytest.mark.parametrize("T,D,stream,post", [(70000, 512, "bfloat16", False), (20000, 1024, "float32", True),
                                             (9000, 8192, "bfloat16", True), (3000, 16384, "float32", True)])
def test_calls_that_pass_the_caches(T, D, stream, post):
    """A large call's tokens are the small call's, bit for bit."""
    import nf4_bit_quantized_amd as q
    import torch
    say(f"norm past the caches T {T} D {D} {stream} post {post}")
    v = _inputs(T, D, getattr(torch, stream), torch.float32, post, post, seed=6)
    x, h, stats = q.qlora_norm_fwd(form="both", **v)
    dX, later = x[0].clone(), h.clone()
    rest = {k: t for k, t in v.items() if k != "h"}
    g = q.qlora_norm_bwd(dX, h, stats=stats, dh_out=later, **rest)
    for rows in (slice(0, 600), slice(T - 600, T)):
        few = {k: t[rows].clone() if t.dim() == 2 else t for k, t in v.items()}
        x2, h2, s2 = q.qlora_norm_fwd(form="both", **few)
        assert all(torch.equal(a[rows], b) for a, b in zip(x, x2)) and torch.equal(h[rows], h2)
        assert torch.equal(stats[rows], s2)
        few.pop("h")
        g2 = q.qlora_norm_bwd(dX[rows].clone(), h2, stats=s2, dh_out=later[rows].clone(), **few)
        assert torch.equal(g[0][rows], g2[0]) and torch.equal(g[1][rows], g2[1])
    # the sums over all tokens: of the stored h, in 64 bits, a block of tokens at a time
    want, mag = torch.zeros(D, dtype=torch.float64, device="cuda"), torch.zeros(D, dtype=torch.float64, device="cuda")
    for t in range(0, T, 5000):
        term = dX[t:t + 5000].double() * h[t:t + 5000].double() * stats[t:t + 5000, :1].double()
        want += term.sum(0)
        mag += term.abs().sum(0)
    # T / 256 + 32 steps of a sum, and three roundings of a term
    assert ((g[2].double() - want).abs() <= (T / 256 + 40) * 2.0 ** -24 * mag + 2.0 ** -24 * want.abs()).all()
