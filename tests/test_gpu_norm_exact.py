"""x of the residual norm bit for bit from what else the call writes: with an fp32 stream h' and r come whole, and
x = (h' r) weight has its two roundings in this order, then one to bf16, or the 8-bit form's own."""

import pytest

from gpu_helpers import say
from test_gpu_norm import _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block", [False, True])
@pytest.mark.parametrize("weights", ["float32", "bfloat16"])
@pytest.mark.parametrize("T,D", [(1, 64), (7, 4096), (600, 5120), (5, 8256), (1100, 16384)])
def test_x_from_the_stream_and_its_factor(T, D, weights, block):
    import nf4_bit_quantized_amd as q
    import torch
    say(f"x from h' and r, T {T} D {D} weights {weights} block {block}")
    v = _inputs(T, D, torch.float32, getattr(torch, weights), block, block, block=block, seed=D)
    (X, codes, scales), h, stats = q.qlora_norm_fwd(form="both", **v)
    x = h * stats[:, :1] * v["weight"].float()
    assert torch.equal(X, x.bfloat16())
    want_codes, want_scales = q.qlora_quantize_fp8(x)
    assert torch.equal(codes, want_codes) and torch.equal(scales, want_scales)
