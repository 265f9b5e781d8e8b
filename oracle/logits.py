"""Log probabilities, entropy, the most likely tokens and the distillation loss of rows of logits, and their
gradients, in float64, from the definitions, a row at a time.

q = softmax(scale * z).  A logit of -inf has probability 0; a row of nothing else has M = log S = -inf, log
probabilities -inf, entropy 0 and no gradient; NaN or +inf makes the row's results NaN.
"""

import numpy as np

NONE = -np.inf


def statistics(z, scale):
    """(M, log S) of one row."""
    z = np.asarray(z, np.float64)
    if np.isnan(z).any():
        return np.nan, np.nan
    M = z.max()
    if M == NONE:
        return NONE, NONE
    if M == np.inf:
        return np.inf, np.nan
    return M, np.log(np.exp(scale * (z - M)).sum())


def log_q(z, M, log_s, scale):
    z = np.asarray(z, np.float64)
    if M == NONE:
        return np.full(z.shape, NONE)
    with np.errstate(invalid="ignore"):
        return scale * (z - M) - log_s


def entropy(z, scale):
    M, log_s = statistics(z, scale)
    if M == NONE:
        return 0.0
    lq = log_q(z, M, log_s, scale)
    q = np.exp(lq)
    with np.errstate(invalid="ignore"):
        return -np.where(q == 0, 0.0, q * lq).sum()


def largest(z, k):
    """The k largest, ties to the lower index, NaN last."""
    z = np.asarray(z, np.float64)
    order = np.where(np.isnan(z), np.inf, -z)
    return np.lexsort((np.arange(z.size), order, np.isnan(z)))[:k]


def named(tokens, V):
    return (np.asarray(tokens) >= 0) & (np.asarray(tokens) < V)


def score_gradient(z, scale, tokens, d, M, log_s, H=0.0, d_H=0.0):
    """(gradient, magnitude) of one row: d of each given token, d_H of the entropy."""
    V = len(z)
    tokens, d = np.asarray(tokens, np.int64), np.asarray(d, np.float64)
    in_ = named(tokens, V)
    w = np.zeros(V)
    np.add.at(w, tokens[in_], d[in_])
    A = d[in_].sum()
    size = np.abs(d[in_]).sum()
    if M == NONE or (not d[in_].any() and d_H == 0):
        return np.zeros(V), np.zeros(V)
    lq = log_q(z, M, log_s, scale)
    q = np.exp(lq)
    lq = np.where(q == 0, 0.0, lq)
    grad = scale * (w - q * (A + d_H * (lq + H)))
    return grad, scale * (np.abs(w) + q * (size + abs(d_H) * (np.abs(lq) + abs(H))) * (4 + np.abs(lq)))


def _teacher(ids, values, V, rest):
    in_ = named(ids, V)
    t = np.where(in_, np.asarray(values, np.float64), NONE)
    if not in_.any():
        return in_, t, np.zeros(len(t)), 0.0
    if rest:
        p = np.exp(t)
        return in_, t, p, max(0.0, 1.0 - p.sum())
    if t.max() == NONE:
        return in_, t, np.zeros(len(t)), 0.0
    t = t - t.max()
    t = t - np.log(np.exp(t).sum())
    return in_, t, np.exp(t), 0.0


def distill(z, scale, ids, values, rest):
    """(loss, M, log S, whole, ratio) of one row."""
    z = np.asarray(z, np.float64)
    V = len(z)
    M, log_s = statistics(z, scale)
    in_, lp, p, left = _teacher(ids, values, V, rest)
    if not in_.any():
        return 0.0, M, log_s, 0.0, 0.0
    others = np.ones(V, bool)
    others[np.asarray(ids)[in_]] = False
    lq = log_q(z, M, log_s, scale)
    q_r = np.exp(lq[others]).sum()
    whole = p.sum() if rest else float(p.sum() > 0)
    ratio = 0.0
    on = p > 0
    if M == NONE:
        return (np.inf if on.any() else 0.0), M, log_s, whole, 0.0
    loss = (p[on] * (lp[on] - lq[np.asarray(ids)[on]])).sum()
    if left > 0 and q_r > 0:
        loss += left * (np.log(left) - np.log(q_r))
        ratio, whole = min(left / q_r, 1e30), 1.0
    if np.isnan(log_s):
        loss = np.nan
    return loss, M, log_s, whole, ratio


def distill_gradient(z, scale, ids, values, rest, d_loss, M, log_s, whole, ratio):
    """(gradient, magnitude) of one row, from its statistics.  p counts twice: in 32 bits it is an exponential (two
    half steps and one), a sum of at most 128 of them in a tree (eight), its reciprocal and two products: fourteen half
    steps, where a magnitude's measure, 2^-21, has eight."""
    z = np.asarray(z, np.float64)
    V = len(z)
    in_, _, p, _ = _teacher(ids, values, V, rest)
    if M == NONE or d_loss == 0 or (whole == 0 and ratio == 0 and not p.any()):
        return np.zeros(V), np.zeros(V)
    w = np.zeros(V)
    np.add.at(w, np.asarray(ids)[in_], p[in_])
    listed = np.zeros(V, bool)
    listed[np.asarray(ids)[in_]] = True
    lq = log_q(z, M, log_s, scale)
    q = np.exp(lq)
    lq = np.where(q == 0, 0.0, lq)
    share = np.where(listed, whole, whole - ratio)
    size = np.where(listed, whole, whole + ratio)
    return scale * d_loss * (share * q - w), scale * abs(d_loss) * (2 * w + q * size * (4 + np.abs(lq)))
