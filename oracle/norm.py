"""The residual norm and its backward in float64, from the definition.

    m  = block * r_b,  r_b = 1 / sqrt(mean(block^2) + eps)    (m = block without a norm behind the block)
    h' = h + scale * gate * post_weight * m
    x  = weight * h' * r,  r = 1 / sqrt(mean(h'^2) + eps)

Next to each result stands its magnitude: the sum of the absolute values that it is added up from, the measure of what
rounding in 32 bits can do to it.
"""

import numpy as np


def _vector(v, D):
    return np.ones(D) if v is None else np.asarray(v, np.float64)


def forward(h, weight, block=None, post_weight=None, gate=None, scale=1.0, eps=1e-6):
    """{"x", "h", "r", "r_b"} and the magnitudes {"x", "h"}."""
    h = np.asarray(h, np.float64)
    T, D = h.shape
    r_b = np.ones(T)
    branch = np.zeros_like(h)
    if block is not None:
        block = np.asarray(block, np.float64)
        if post_weight is not None:
            r_b = 1.0 / np.sqrt((block ** 2).mean(1) + eps)
        branch = scale * _vector(gate, D) * _vector(post_weight, D) * block * r_b[:, None]
    new = h + branch
    r = 1.0 / np.sqrt((new ** 2).mean(1) + eps)
    w = _vector(weight, D)
    mag = np.abs(h) + np.abs(branch)
    return ({"x": new * r[:, None] * w, "h": new, "r": r, "r_b": r_b},
            {"x": mag * r[:, None] * np.abs(w), "h": mag})


def backward(dx, h_out, weight, r, r_b, block=None, post_weight=None, gate=None, scale=1.0, dh_out=None):
    """{"dh", "dblock", "dweight", "dpost_weight", "dgate"} (those that there are) and their magnitudes; r and r_b as
    the forward gave them."""
    dx, h = np.asarray(dx, np.float64), np.asarray(h_out, np.float64)
    T, D = h.shape
    r, r_b = np.asarray(r, np.float64)[:, None], np.asarray(r_b, np.float64)[:, None]
    later = np.zeros_like(h) if dh_out is None else np.asarray(dh_out, np.float64)
    n = h * r
    dn = dx * _vector(weight, D)
    dh = later + r * (dn - n * (dn * n).mean(1, keepdims=True))
    size = np.abs(later) + r * (np.abs(dn) + np.abs(n) * np.abs(dn * n).mean(1, keepdims=True))
    out = {"dh": dh, "dweight": (dx * n).sum(0)}
    mag = {"dh": size, "dweight": np.abs(dx * n).sum(0)}
    if block is None:
        return out, mag
    w, g = _vector(post_weight, D), _vector(gate, D)
    m = np.asarray(block, np.float64) * (r_b if post_weight is not None else 1.0)
    if gate is not None:
        out["dgate"], mag["dgate"] = scale * w * (dh * m).sum(0), np.abs(scale * w) * (size * np.abs(m)).sum(0)
    dm, dm_size = scale * g * w * dh, np.abs(scale * g * w) * size
    if post_weight is not None:
        out["dpost_weight"], mag["dpost_weight"] = scale * g * (dh * m).sum(0), np.abs(scale * g) * (size * np.abs(m)).sum(0)
        out["dblock"] = r_b * (dm - m * (dm * m).mean(1, keepdims=True))
        mag["dblock"] = r_b * (dm_size + np.abs(m) * (dm_size * np.abs(m)).mean(1, keepdims=True))
    else:
        out["dblock"], mag["dblock"] = dm, dm_size
    return out, mag
