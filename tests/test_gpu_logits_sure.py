"""Rows that are sure of one token, whose log S, log probability and entropy are small: they are as exact as 32 bits can
say, not only next to log S of a flat row.

Tolerances.  The largest element's term is 1 in 64 bits; at most nine additions in 32 bits (seven of a chain, two that
join the chains) round a sum between 1 and 2, each by 2^-24 at most.  The other terms are off by 2^-23 and by |d| 2^-24
with d above -60 where a term counts, and by the additions among them: 80 steps of 2^-24 of their sum.  In the entropy
each term is multiplied by its d, so the same holds of the sum of |d| terms.  Results are rounded once more."""

import numpy as np
import pytest

from gpu_helpers import say
from oracle import logits as ol
from test_gpu_logits import F32, _np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [0.5, 1.0, 1.25])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("T,V", [(200, 900), (200, 32000), (300, 60001), (20, 128256)])
def test_sure_rows(T, V, dtype, scale):
    import nf4_bit_quantized_amd as q
    import torch
    say(f"sure rows T {T} V {V} {dtype} scale {scale}")
    g = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn((T, V), generator=g, device="cuda") * 2
    at = torch.randint(0, V, (T,), generator=g, device="cuda")
    z[torch.arange(T, device="cuda"), at] = 14 + torch.rand(T, generator=g, device="cuda") * 8
    z = (z / scale).to(getattr(torch, dtype))
    logprob, stats, entropy, _, _ = q.qlora_token_logprob(z, at, scale=scale, want_entropy=True)
    plain = q.qlora_token_logprob(z, at, scale=scale)
    assert q.qlora_token_logprob(z, at, scale=scale, top=1)[3].squeeze(1).equal(at)
    ids = torch.stack([at, (at + 1) % V], 1).contiguous()
    values = torch.tensor([[-0.01, -6.0]], device="cuda").expand(T, 2).contiguous()
    losses = [q.qlora_distill_fwd(z, ids, values, scale=scale, rest=rest) for rest in (False, True)]
    zn, lp, lp2, log_s, H = _np(z), _np(logprob), _np(plain[0]), _np(stats)[:, 1], _np(entropy)
    for t in range(T):
        d = scale * (zn[t] - zn[t].max())
        e = np.exp(d)
        S, spread = e.sum(), (e * -d).sum()
        tol = (9 + 80 * (S - 1)) * F32
        want = np.log1p(S - 1)
        for got, sign in ((log_s[t], 1), (lp[t], -1), (lp2[t], -1)):
            assert abs(sign * got - want) <= tol + F32 * want, f"row {t}: {got} for {want}"
        want = want + spread / S
        assert abs(H[t] - want) <= tol + 80 * F32 * spread + F32 * want, f"row {t}: entropy {H[t]} for {want}"
        for rest, (loss, _) in zip((False, True), losses):
            want = ol.distill(zn[t], scale, ids[t].cpu().numpy(), _np(values[t]), rest)[0]
            # with a bucket log q_r is off, too, by what its own sum is
            more = (80 * F32 if rest else 0.0) + F32 * abs(want)
            assert abs(loss[t].item() - want) <= tol + more, f"row {t}: loss {loss[t].item()} for {want}"
