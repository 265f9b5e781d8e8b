"""The residual norm, the losses and the layers between them as a training step uses them: one step against the float64
oracles, on a side stream, captured and replayed; and operands beyond 2^31 elements and beyond the caches."""

import numpy as np
import pytest

from gpu_helpers import TOL, normwise_err, say
from oracle import logits as ol
from oracle import lora as olora
from oracle import norm as on
from test_gpu_logits import _alike, _check_score, _logits, _near, _np
from test_gpu_logits import TOL as row_tol

pytestmark = pytest.mark.gpu


def _step_inputs(T=48, D=256, N=576, V=531, k=12, r=8, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    s = dict(T=T, D=D, V=V, r=r, W=rand(N, D) * 0.08, h=rand(T, D), block=rand(T, D).bfloat16(), weight=1 + rand(D) / 5,
             post_weight=rand(D) / 2, gate=rand(D) / 3, A=(rand(r, D) / r).bfloat16(), B=(rand(N, r) * 0.05).bfloat16())
    teacher = rand(T, V) * 2
    s["values"], s["ids"] = torch.log_softmax(teacher, 1).topk(k, dim=1)
    s["ids"] = s["ids"].contiguous()
    s["d_loss"] = torch.full((T,), 1.0 / T, device="cuda")
    return s


def _norm_args(s):
    return dict(block=s["block"], post_weight=s["post_weight"], gate=s["gate"], scale=0.5)


def _step(q, s, stored, kind="nf4"):
    """Norm, head, distillation and the way back: every output of the step."""
    alpha, V = 16.0, s["V"]
    x, h, stats = q.qlora_norm_fwd(s["h"], s["weight"], form="fp8" if kind == "fp8" else "bf16", **_norm_args(s))
    if kind == "fp8":
        logits, U = q.qlora_fp8_linear_fwd(*stored, *x, s["A"], s["B"], alpha)
    else:
        logits, U = q.qlora_linear_fwd(*stored, x, s["A"], s["B"], alpha)
    loss, row = q.qlora_distill_fwd(logits, s["ids"], s["values"], rest=True, vocab=V)
    dY = q.qlora_distill_bwd(logits, s["ids"], s["values"], row, s["d_loss"], rest=True, vocab=V)
    if kind == "fp8":
        dX, dA, dB = q.qlora_fp8_linear_bwd(*stored, *x, s["A"], s["B"], alpha, dY, U_in=U)
    else:
        dX, dA, dB = q.qlora_linear_bwd(*stored, x, s["A"], s["B"], alpha, dY, U_in=U)
    dh, dblock, dw, dp, dg = q.qlora_norm_bwd(dX, h, s["weight"], stats, dh_out=None, **_norm_args(s))
    return dict(h=h, stats=stats, logits=logits, loss=loss, row=row, dY=dY, dX=dX, dA=dA, dB=dB, dh=dh, dblock=dblock,
                dweight=dw, dpost_weight=dp, dgate=dg, x=x[0] if kind == "fp8" else x)


def _store(q, s, kind="nf4"):
    return q.qlora_quantize_fp8(s["W"], block_rows=128) if kind == "fp8" else q.qlora_quantize_nf4(s["W"])


@pytest.mark.parametrize("kind", ["nf4", "fp8"])
def test_training_step(kind):
    """Against the whole step in float64 on the stored weight.  The bf16 logits (at most 4, off by 2^-8 of that) put a
    relative 2^-6 into q, a bf16 X half of that into the logits, and with 8-bit X and dY 2^-4 of single elements enter
    sums over 256 and 576 of them; the layers' bar, TOL normwise, holds for the 16-bit step and four times it for the
    8-bit one."""
    import nf4_bit_quantized_amd as q
    say(f"training step {kind}")
    s = _step_inputs()
    stored = _store(q, s, kind)
    out = _step(q, s, stored, kind)
    W = _np(q.qlora_dequantize_fp8(*stored, block_rows=128) if kind == "fp8" else q.qlora_dequantize_nf4(*stored))
    n = {k: _np(v) for k, v in s.items() if hasattr(v, "cpu")}
    kw = {k: n[k] for k in ("block", "post_weight", "gate")}
    f, _ = on.forward(n["h"], n["weight"], scale=0.5, **kw)
    Y, _ = olora.forward(W, f["x"], n["A"], n["B"], 16.0, s["r"])
    V, T = s["V"], s["T"]
    loss, dY = np.zeros(T), np.zeros_like(Y)
    for t in range(T):
        loss[t], *row = ol.distill(Y[t, :V], 1.0, s["ids"][t].cpu().numpy(), n["values"][t], True)
        dY[t, :V], _ = ol.distill_gradient(Y[t, :V], 1.0, s["ids"][t].cpu().numpy(), n["values"][t], True, 1.0 / T, *row)
    dX, dA, dB = olora.backward(W, f["x"], n["A"], n["B"], dY, 16.0, s["r"])
    g, _ = on.backward(dX, f["h"], n["weight"], f["r"], f["r_b"], scale=0.5, **kw)
    want = dict(h=f["h"], logits=Y, loss=loss, dY=dY, dX=dX, dA=dA, dB=dB, **g)
    for k, w in want.items():
        e = normwise_err(_np(out[k]), w)
        assert e <= TOL * (4 if kind == "fp8" else 1), f"{k}: {e}"
    assert not out["dY"][:, V:].any()
    # the optimizer takes the norm's gradients as it takes an adapter's
    import torch
    m, v, w16 = torch.zeros_like(s["weight"]), torch.zeros_like(s["weight"]), s["weight"].bfloat16()
    before = s["weight"].clone()
    q.qlora_adamw_step(s["weight"], out["dweight"], m, v, 1, 1e-3, param_bf16=w16)
    assert torch.equal(w16, s["weight"].bfloat16())
    moved = (s["weight"] - before).abs()                  # the first step is lr in size, off by eps / |grad|
    big = out["dweight"].abs() > 1e-5
    assert ((moved[big] - 1e-3).abs() <= 1e-5).all()


@pytest.mark.parametrize("kind", ["nf4", "fp8"])
def test_side_stream_and_replays(kind):
    import nf4_bit_quantized_amd as q
    import torch
    say(f"side stream and replays {kind}")
    a, b = _step_inputs(seed=1), _step_inputs(seed=2)
    stored = _store(q, a, kind)
    b["W"] = a["W"]
    want = {0: _step(q, a, stored, kind), 1: _step(q, b, stored, kind)}
    torch.cuda.synchronize()

    def same(got, ref):
        for k in ref:
            assert torch.equal(got[k], ref[k]), k

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        late = {k: v.clone() if torch.is_tensor(v) else v for k, v in a.items()}
        got = _step(q, late, stored, kind)
    side.synchronize()
    same(got, want[0])

    place = {k: v.clone() if torch.is_tensor(v) else v for k, v in a.items()}
    with torch.cuda.stream(side):
        _step(q, place, stored, kind)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = _step(q, place, stored, kind)
    for turn in (1, 0, 1, 1, 0):
        for k, v in (a, b)[turn].items():
            if torch.is_tensor(v):
                place[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        same(got, want[turn])
        same(_step(q, (a, b)[1 - turn], stored, kind), want[1 - turn])      # eager work between the replays


def test_given_stream_and_workspace():
    """stream= enqueues there and allocates there; one workspace serves calls in turn, captured ones too."""
    import nf4_bit_quantized_amd as q
    import torch
    say("given stream and workspace")
    s = _step_inputs(seed=4)
    side = torch.cuda.Stream()
    x, h, stats = q.qlora_norm_fwd(s["h"], s["weight"], **_norm_args(s))
    want = q.qlora_norm_bwd(x, h, s["weight"], stats, **_norm_args(s))
    z = _logits(6, 3001, "float16", seed=8)
    tokens = torch.arange(6, device="cuda")
    ref = q.qlora_token_logprob(z, tokens, top=4)
    ws = torch.empty(q.qlora_norm_bwd_workspace_bytes(*s["h"].shape), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    x2, h2, s2 = q.qlora_norm_fwd(s["h"], s["weight"], stream=side, **_norm_args(s))
    got = q.qlora_norm_bwd(x2, h2, s["weight"], s2, workspace=ws, stream=side, **_norm_args(s))
    out = q.qlora_token_logprob(z, tokens, top=4, stream=side)
    loss = q.qlora_distill_fwd(z, out[3], out[4], stream=side)
    d = q.qlora_distill_bwd(z, out[3], out[4], loss[1], torch.ones_like(loss[0]), stream=side)
    side.synchronize()
    assert torch.equal(x, x2) and all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(out, ref) if a is not None) and d.isfinite().all()
    graphs = []
    for rows in (slice(0, 48), slice(0, 17)):
        few = {k: v[rows].clone() if k in ("h", "block") else v for k, v in s.items()}
        a = q.qlora_norm_fwd(few["h"], few["weight"], **_norm_args(few))
        expect = q.qlora_norm_bwd(a[0], a[1], few["weight"], a[2], **_norm_args(few))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            r = q.qlora_norm_bwd(a[0], a[1], few["weight"], a[2], workspace=ws, **_norm_args(few))
        graphs.append((graph, r, expect, a, few))
    for turn in (0, 1, 1, 0):
        graph, r, expect = graphs[turn][:3]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(r, expect))


def test_scores_on_a_side_stream_and_replayed():
    import nf4_bit_quantized_amd as q
    import torch
    say("scores captured")
    z = [_logits(5, 40001, "bfloat16", seed=i) for i in range(2)]
    tokens = torch.arange(5, device="cuda") * 7
    d, d_H = torch.randn(5, device="cuda"), torch.randn(5, device="cuda")

    def run(z):
        out = q.qlora_token_logprob(z, tokens, top=20, want_entropy=True)
        return (*out, q.qlora_token_logprob_bwd(z, tokens, out[1], d, entropy=out[2], d_entropy=d_H))

    want = [run(x) for x in z]
    place = z[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = run(place)
    for turn in (1, 0, 0, 1):
        place.copy_(z[turn])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want[turn]))
        assert all(torch.equal(x, y) for x, y in zip(run(z[1 - turn]), want[1 - turn]))


@pytest.mark.parametrize("T,V,dtype", [
    (1100, 128256, "bfloat16"), (20000, 8000, "bfloat16"), (4000, 40000, "float16"), (256, 300001, "float32"),
    (300, 60001, "bfloat16")])
def test_beyond_the_caches(T, V, dtype):
    """Sizes that pass the caches by (256 MB of logits and more), and every number of threads."""
    import nf4_bit_quantized_amd as q
    import torch
    say(f"beyond the caches T {T} V {V} {dtype}")
    z = _logits(T, V, dtype, seed=3)
    rows = [0, 1, T // 2, T - 1]
    tokens = torch.randint(0, V, (T, 1), device="cuda")
    at = torch.tensor(rows, device="cuda")
    for top, ent in ((0, False), (0, True), (9, False)):
        out = q.qlora_token_logprob(z, tokens, top=top, want_entropy=ent)
        _check_score(z[at], tokens[at], 1.0, top, [t if t is None else t[at] for t in out])
    _, stats, _, ids, values = q.qlora_token_logprob(z, top=40)
    d = torch.randn((T, 1), device="cuda")
    values = torch.where(torch.rand((T, 40), device="cuda") < 0.5, values - 1, values)
    grad = q.qlora_token_logprob_bwd(z, tokens, stats, d)
    want = [ol.score_gradient(_np(z[t]), 1.0, tokens[t].cpu().numpy(), _np(d[t]), *_np(stats[t])) for t in rows]
    _near(grad[at], np.stack([w for w, _ in want]), np.stack([m for _, m in want]), "dlogits")
    for rest in (False, True):
        loss, stats = q.qlora_distill_fwd(z, ids, values, rest=rest)
        grad = q.qlora_distill_bwd(z, ids, values, stats, d[:, 0].contiguous(), rest=rest)
        want = []
        for t in rows:
            l, *row = ol.distill(_np(z[t]), 1.0, ids[t].cpu().numpy(), _np(values[t]), rest)
            _alike(loss[t].item(), l, 2 * row_tol(V), "loss")
            want.append(ol.distill_gradient(_np(z[t]), 1.0, ids[t].cpu().numpy(), _np(values[t]), rest, float(d[t, 0]),
                                            *_np(stats[t])))
        _near(grad[at], np.stack([w for w, _ in want]), np.stack([m for _, m in want]), "dlogits")


@pytest.mark.parametrize("T,V,k", [(300, 70001, 128), (40, 70001, 128), (600, 9000, 7)])
def test_alternatives_of_like_logits(T, V, k):
    """Rows with more ties than the candidates' place holds: few levels, ascending, one value."""
    import nf4_bit_quantized_amd as q
    import torch
    say(f"alternatives of like logits T {T} V {V} k {k}")
    z = torch.randint(-2, 3, (T, V), device="cuda").bfloat16()
    z[1] = torch.arange(V, device="cuda").float().bfloat16()
    z[2] = -z[1]
    z[3] = 4.0
    z[4] = -1.0
    z[4, V - 1] = 0.0
    z[5, :] = float("-inf")
    z[5, V // 2:] = -3.0
    ids = q.qlora_token_logprob(z, top=k)[3].cpu().numpy()
    for t in (0, 1, 2, 3, 4, 5, T - 1):
        assert np.array_equal(ids[t], ol.largest(_np(z[t]), k)), t


def test_offsets_past_32_bits():
    import nf4_bit_quantized_amd as q
    import torch
    say("logits of more than 2^31 elements")
    T, V = 17000, 128256                                  # 2.18e9 elements
    z = torch.empty((T, V), dtype=torch.bfloat16, device="cuda")
    for t in range(0, T, 1000):
        z[t:t + 1000].normal_()
    tokens = torch.full((T,), V - 1, dtype=torch.int64, device="cuda")
    out = q.qlora_token_logprob(z, tokens, top=3)
    d = torch.ones(T, device="cuda")
    last = z[-2:].clone()
    alone = q.qlora_token_logprob(last, tokens[-2:], top=3)
    assert torch.equal(out[3][-2:], alone[3])
    # a row alone is summed by another number of threads
    assert (out[0][-2:] - alone[0]).abs().max() <= 2 * row_tol(V) + 2.0 ** -20
    want = q.qlora_token_logprob_bwd(last, tokens[-2:], out[1][-2:].contiguous(), d[-2:])
    q.qlora_token_logprob_bwd(z, tokens, out[1], d, dlogits=z)
    assert torch.equal(z[-2:], want)
    del z
    say("norm over more than 2^31 elements")
    T, D = 270000, 8192                                   # 2.21e9 elements
    h = torch.zeros((T, D), dtype=torch.bfloat16, device="cuda")
    h[-3:] = torch.randn((3, D), device="cuda").bfloat16()
    block = torch.zeros_like(h)
    block[-3:] = torch.randn((3, D), device="cuda").bfloat16()
    w = torch.rand(D, device="cuda")
    x, h2, stats = q.qlora_norm_fwd(h, w, block=block, h_out=h, form="both")
    xs, hs, ss = q.qlora_norm_fwd(h2[-3:].clone(), w, form="both")
    assert (x[0][:5] == 0).all()
    # the norm of the rounded h' is the norm of h' to half a step of h'
    assert ((x[0][-3:].float() - xs[0].float()).abs() <= 2.0 ** -6 * xs[0].float().abs() + 2.0 ** -8).all()
    dx = x[0]
    g = q.qlora_norm_bwd(dx, h2, w, stats, block=block, dh_out=h2)
    one = q.qlora_norm_bwd(dx[-3:].clone(), h2[-3:].clone(), w, stats[-3:].clone(), block=block[-3:].clone(),
                           dh_out=h2[-3:].clone())
    assert torch.equal(g[0][-3:], one[0]) and torch.equal(g[1][-3:], one[1])
