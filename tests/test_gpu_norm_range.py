"""The residual norm and its backward where a block's values are far from 1: the forward normalises them, so the
gradients of block, gate and post_weight have their means at every magnitude whose squares fp32 holds.  Tolerances as in
test_gpu_norm.py."""

import numpy as np
import pytest

from gpu_helpers import say
from oracle import norm as on
from test_gpu_norm import _inputs, _near, _np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stream", ["float32", "bfloat16"])
@pytest.mark.parametrize("D", [64, 4096, 8256])
@pytest.mark.parametrize("eps,sizes", [
    (0.0, (1e-16, 1e-14, 1e-13, 1e-10, 1e-5, 1.0, 1e5, 1e10, 1e13, 1e14, 1e15, 1e16)),
    (1e-30, (0.0, 1e-16, 1e-15, 1e-13, 1e-10, 1.0, 1e16))])
def test_block_of_any_size(D, stream, eps, sizes):
    import nf4_bit_quantized_amd as q
    import torch
    say(f"blocks of any size D {D} {stream} eps {eps}")
    T, scale = len(sizes), 0.375
    v = _inputs(T, D, getattr(torch, stream), torch.float32, True, True, seed=D)
    unit = torch.randn((T, D), device="cuda")
    v["block"] = (unit * torch.tensor(sizes, device="cuda")[:, None]).bfloat16()
    want, mag = on.forward(**{k: _np(t) for k, t in v.items()}, scale=scale, eps=eps)
    X, h, stats = q.qlora_norm_fwd(scale=scale, eps=eps, **v)
    _near(X, want["x"], mag["x"], "x")
    _near(h, want["h"], mag["h"], "h")
    np.testing.assert_allclose(_np(stats), np.stack([want["r"], want["r_b"]], 1), rtol=2.0 ** -18)
    rest = {k: t for k, t in v.items() if k != "h"}
    dX = torch.randn((T, D), device="cuda").bfloat16()
    # a gradient that follows the block, so that its mean with the block counts
    later = (unit / (rest["post_weight"] * rest["gate"]).abs().clamp(min=0.1) + torch.randn_like(unit) / 4).to(h.dtype)
    want, mag = on.backward(_np(dX), _np(h), r=_np(stats)[:, 0], r_b=_np(stats)[:, 1], scale=scale, dh_out=_np(later),
                            **{k: _np(t) for k, t in rest.items()})
    got = dict(zip(("dh", "dblock", "dweight", "dpost_weight", "dgate"),
                   q.qlora_norm_bwd(dX, h, stats=stats, scale=scale, dh_out=later, **rest)))
    for k in want:
        _near(got[k], want[k], mag[k], k)
