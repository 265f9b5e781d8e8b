"""The float64 oracles of the residual norm, the log probabilities and the distillation loss: their gradients against
central differences, their definitions against each other, and the rows that a mask leaves empty."""

import numpy as np
import pytest

from oracle import logits as ol
from oracle import norm as on


def _difference(f, x, at, step=1e-5):
    up, down = x.copy(), x.copy()
    up[at] += step
    down[at] -= step
    return (f(up) - f(down)) / (2 * step)


# a central difference of step s is off by s^2 times a third derivative (of order 10 here) and by 2^-52 / s
DIFF = dict(rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("post,gate,with_block", [(True, True, True), (False, True, True), (True, False, True),
                                                  (False, False, True), (False, False, False)])
def test_norm_gradients_against_differences(post, gate, with_block):
    rng = np.random.default_rng(5)
    T, D, scale = 3, 64, 0.7
    v = {"h": rng.normal(size=(T, D)), "weight": 1 + rng.normal(size=D) / 4}
    if with_block:
        v["block"] = rng.normal(size=(T, D))
    if post:
        v["post_weight"] = rng.normal(size=D)
    if gate:
        v["gate"] = rng.normal(size=D)
    dx, later = rng.normal(size=(T, D)), rng.normal(size=(T, D))

    def total(v):
        out, _ = on.forward(scale=scale, eps=1e-3, **v)
        return (out["x"] * dx).sum() + (out["h"] * later).sum()

    out, _ = on.forward(scale=scale, eps=1e-3, **v)
    g, mag = on.backward(dx, out["h"], v["weight"], out["r"], out["r_b"], block=v.get("block"),
                         post_weight=v.get("post_weight"), gate=v.get("gate"), scale=scale, dh_out=later)
    assert set(g) == {"dh" if k == "h" else "d" + k for k in v}
    for k in v:
        grad = g["dh" if k == "h" else "d" + k]
        assert np.all(np.abs(grad) <= mag["dh" if k == "h" else "d" + k] * (1 + 1e-12))
        for at in [tuple(rng.integers(0, s) for s in v[k].shape) for _ in range(6)]:
            np.testing.assert_allclose(_difference(lambda x: total({**v, k: x}), v[k], at), grad[at], **DIFF)


def test_score_gradient_against_differences():
    rng = np.random.default_rng(6)
    V, scale = 37, 1.3
    z = rng.normal(size=V) * 2
    z[[3, 30]] = -np.inf
    tokens, d, d_H = [4, -100, 4, 9, 37], [0.3, 5.0, -1.1, 0.4, 2.0], 0.6

    def total(z):
        M, log_s = ol.statistics(z, scale)
        lq = ol.log_q(z, M, log_s, scale)
        return sum(w * lq[t] for t, w in zip(tokens, d) if 0 <= t < V) + d_H * ol.entropy(z, scale)

    M, log_s = ol.statistics(z, scale)
    grad, mag = ol.score_gradient(z, scale, tokens, d, M, log_s, ol.entropy(z, scale), d_H)
    assert grad[3] == grad[30] == 0 and np.all(np.abs(grad) <= mag)
    for j in (0, 4, 9, 20):
        np.testing.assert_allclose(_difference(total, z, j), grad[j], **DIFF)


@pytest.mark.parametrize("rest", [False, True])
def test_distill_gradient_against_differences(rest):
    rng = np.random.default_rng(7)
    V, scale = 41, 0.8
    z = rng.normal(size=V) * 2
    ids = np.array([5, 40, -1, 5, 0, 41])                   # a token twice, two that are none
    values = np.log(np.array([0.2, 0.1, 0.3, 0.15, 0.25, 0.5]))
    loss, M, log_s, whole, ratio = ol.distill(z, scale, ids, values, rest)
    grad, mag = ol.distill_gradient(z, scale, ids, values, rest, 1.7, M, log_s, whole, ratio)
    assert np.all(np.abs(grad) <= mag * (1 + 1e-12)) and abs(grad.sum()) < 1e-12
    for j in (0, 5, 40, 17):
        np.testing.assert_allclose(_difference(lambda z: 1.7 * ol.distill(z, scale, ids, values, rest)[0], z, j),
                                   grad[j], **DIFF)


def test_distillation_is_a_divergence():
    """Against a teacher with the student's own probabilities the loss is 0, and so is its gradient."""
    rng = np.random.default_rng(8)
    z = rng.normal(size=50)
    M, log_s = ol.statistics(z, 1.0)
    lq = ol.log_q(z, M, log_s, 1.0)
    for ids, rest in ((np.arange(50), False), (ol.largest(z, 7), True)):
        loss, M, log_s, whole, ratio = ol.distill(z, 1.0, ids, lq[ids], rest)
        assert abs(loss) < 1e-14
        grad, _ = ol.distill_gradient(z, 1.0, ids, lq[ids], rest, 1.0, M, log_s, whole, ratio)
        assert np.abs(grad).max() < 1e-14


def test_largest_breaks_ties_by_index():
    z = np.array([1.0, 3.0, -0.0, 3.0, 0.0, np.nan, -np.inf, 3.0])
    assert list(ol.largest(z, 8)) == [1, 3, 7, 0, 2, 4, 6, 5]


def test_empty_rows():
    z = np.full(5, -np.inf)
    M, log_s = ol.statistics(z, 1.0)
    assert M == log_s == -np.inf and ol.entropy(z, 1.0) == 0.0
    assert not ol.score_gradient(z, 1.0, [2], [1.0], M, log_s)[0].any()
    assert ol.distill(z, 1.0, [1], [0.0], False)[0] == np.inf
    assert ol.distill(z, 1.0, [-1], [0.0], True) == (0.0, -np.inf, -np.inf, 0.0, 0.0)
    low = np.full(5, float(np.finfo(np.float32).min))         # a mask of the lowest value leaves all tokens alike
    assert abs(ol.entropy(low, 1.0) - np.log(5)) < 1e-12
