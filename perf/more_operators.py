"""Cases of what stands at the two ends of the library's layers: the residual norm that forms a layer's input (bf16
or its 8-bit form) and takes its gradient back, the log probabilities of given tokens from the logits of the last
layer, and the distillation loss from a teacher's top logits, each with its gradient.

``own`` False: ``run`` computes the operators in plain torch operations in 32 bits, rounded once at the end.
``own`` True: ``run`` calls ``nf4_bit_quantized_amd``.

Residual norm, per token, over D channels: a block's output b joins the residual stream h, and the stream is
normalised for the next layer:
    m = b * r_b,  r_b = 1 / sqrt(mean(b^2) + eps)      (with a norm behind the block; m = b without one)
    h' = h + scale * gate * post_weight * m
    x = weight * h' * r,  r = 1 / sqrt(mean(h'^2) + eps)
Log probabilities: q = softmax(scale * z) over the first `vocab` columns of the logits z; log q of the given tokens,
the entropy of q, and the `top` largest with their tokens, ties to the lower token.  A token that is none (-100) has
log probability 0 and no gradient.
Distillation: p from the teacher's k values t: softmax(t) over the k tokens, or with `rest` exp(t) and what is left
to 1 as one more bucket, against which stands what q has outside the k tokens.  Loss: the sum of p (log p - log q).
"""

import math

import torch

own = False

BLOCK = 128
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# --------------------------------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------------------------------

def listed():
    return [
        # serving, one token, 65B-class width: the norm between two layers, where latency counts
        dict(name="norm_token", op="norm", T=1, D=8192, stream="bf16", weights="bf16", post=False, gate=False,
             scale=1.0, form="bf16"),
        # a ragged batch, 7B-class width, fp32 stream, norms before and after the block, a gate per channel
        dict(name="norm_sandwich", op="norm", T=1333, D=4096, stream="f32", weights="f32", post=True, gate=True,
             scale=0.5, form="bf16"),
        # 65B-class training forward whose next layer takes the 8-bit form
        dict(name="norm_fp8_65b", op="norm", T=4096, D=8192, stream="bf16", weights="bf16", post=False, gate=False,
             scale=1.0, form="fp8"),
        # the backward passes of the last two
        dict(name="norm_bwd_sandwich", op="norm_bwd", T=1333, D=4096, stream="f32", weights="f32", post=True, gate=True,
             scale=0.5),
        dict(name="norm_bwd_65b", op="norm_bwd", T=4096, D=8192, stream="bf16", weights="bf16", post=False, gate=False,
             scale=1.0),
        # serving: the log probability of the token that was sampled, with twenty alternatives, at a temperature
        dict(name="score_token", op="score", T=1, V=128256, dtype="bf16", top=20, entropy=False, scale=1.25),
        # scoring a short text, odd vocabulary, fp32 logits, with entropy and five alternatives
        dict(name="score_odd", op="score", T=77, V=50257, dtype="f32", top=5, entropy=True, scale=1.0),
        # a teacher's pass over a batch: its 64 largest for later distillation
        dict(name="score_teacher", op="score", T=2048, V=128256, dtype="bf16", top=64, entropy=False, scale=1.0),
        # fine-tuning on given tokens, 4096 of them, prompt masked: the gradient of the logits
        dict(name="score_grad_sft", op="score_grad", T=4096, V=32000, dtype="bf16", entropy=False, scale=1.0),
        # policy gradient with an entropy bonus over a short answer, odd vocabulary
        dict(name="score_grad_policy", op="score_grad", T=217, V=50257, dtype="f32", entropy=True, scale=1.0),
        # distillation of a short sequence, with the rest of the teacher's mass as a bucket
        dict(name="distill_rest", op="distill", T=129, V=32000, dtype="f32", k=16, rest=True, scale=0.5),
        # distillation of a batch over a large vocabulary
        dict(name="distill_large", op="distill", T=4096, V=128256, dtype="bf16", k=64, rest=False, scale=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "norm_bwd", "score", "score", "score", "score_grad", "distill", "distill"])
    if op in ("norm", "norm_bwd"):
        T, D = _log_int(rng, 1, 8192), 64 * max(1, round(_log_int(rng, 512, 16384) / 64))
        while T * D > 4096 * 8192:
            T = _log_int(rng, 1, 8192)
        post = rng.random() < 0.5
        case = dict(op=op, T=T, D=D, stream=rng.choice(["bf16", "f32"]), weights=rng.choice(["bf16", "f32"]), post=post,
                    gate=rng.random() < 0.5, scale=rng.choice([1.0, 0.5, 0.22]))
        if op == "norm":
            case["form"] = rng.choice(["bf16", "fp8"])
        elif T * D > 2048 * 8192 and (post or case["gate"]):
            case["T"] = T // 2
        return case
    T, V = _log_int(rng, 1, 4096), _log_int(rng, 8000, 160000)
    most = 2048 * 128256 if op == "score" else 4096 * 32000 if op == "score_grad" else 4096 * 128256
    while T * V > most:
        T = _log_int(rng, 1, 4096)
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if dtype == "f32" and T * V > most // 4:
        T = max(1, T // 4)
    case = dict(op=op, T=T, V=V, dtype=dtype, scale=rng.choice([1.0, 1.0, 0.5, 1.25]))
    if op == "score":
        case.update(top=rng.choice([0, 1, 5, 20, rng.randint(2, 64)]), entropy=rng.random() < 0.4)
    elif op == "score_grad":
        case.update(entropy=rng.random() < 0.4)
    else:
        case.update(k=rng.choice([8, 32, 64, rng.randint(1, 100)]), rest=rng.random() < 0.5)
    return case


def work(case):
    op, T = case["op"], case["T"]
    if op in ("norm", "norm_bwd"):
        n, wide = T * case["D"], 4 if case["stream"] == "f32" else 2
        arrays = 1 + case["post"] + case["gate"]
        weights = case["D"] * arrays * (4 if case["weights"] == "f32" else 2)
        if op == "norm":     # h, b read; h', x written
            out = 2 if case["form"] == "bf16" else 1 + 1 / BLOCK
            return {"bytes": n * (2 * wide + 2 + out) + weights + 8 * T, "flops": 8.0 * n}
        # dx, h', dh' read, b where its norm or gate needs it; dh, db written
        extra = 2 if case["post"] or case["gate"] else 0
        return {"bytes": n * (3 * wide + 2 + 2 + extra) + weights + 4 * case["D"] * arrays + 8 * T, "flops": 14.0 * n}
    n, wide = T * case["V"], 4 if case["dtype"] == "f32" else 2
    if op == "score":
        return {"bytes": n * wide + T * (20 + 12 * case["top"]), "flops": (7.0 if case["entropy"] else 5.0) * n}
    if op == "score_grad":
        return {"bytes": 2 * n * wide + 20 * T, "flops": 5.0 * n}
    # the row's sum has to be known before its first gradient, so the logits are read twice
    return {"bytes": 3 * n * wide + T * (20 + 12 * case["k"]), "flops": 9.0 * n}


# --------------------------------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------------------------------

def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device=g.device) * std).to(dtype)


def _prepare_norm(case, g):
    T, D = case["T"], case["D"]
    stream, weights = TYPES[case["stream"]], TYPES[case["weights"]]
    h = torch.randn((T, D), generator=g, device=g.device)
    h[:, torch.randint(0, D, (max(1, D // 512),), generator=g, device=g.device)] *= 30.0
    b = torch.randn((T, D), generator=g, device=g.device) * torch.exp(0.5 * torch.randn((T, 1), generator=g, device=g.device))
    s = dict(case=case, eps=1e-6, h=h.to(stream), block=b.to(torch.bfloat16), post_weight=None, gate=None)
    s["weight"] = (1.0 + 0.2 * torch.randn(D, generator=g, device=g.device)).to(weights)
    if case["post"]:
        s["post_weight"] = (0.5 + 0.1 * torch.randn(D, generator=g, device=g.device)).to(weights)
    if case["gate"]:
        s["gate"] = _normal(g, (D,), 0.3, weights)
    if case["op"] == "norm_bwd":
        _, total, s["stats"] = _norm(s)
        s["h_out"] = total.to(stream)
        del s["h"]
        s["dX"] = _normal(g, (T, D), 1.0, torch.bfloat16)
        s["dh"] = _normal(g, (T, D), 1.0, stream)
    return s


def _logits(g, T, V, dtype):
    """Logits of a language model: a broad bell, and in each row a few tokens far above it."""
    z = torch.randn((T, V), generator=g, device=g.device) * 2.0
    likely = torch.randint(0, V, (T, 6), generator=g, device=g.device)
    z.scatter_add_(1, likely, 6.0 + 3.0 * torch.randn((T, 6), generator=g, device=g.device))
    return z.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=_device())
    g.manual_seed(int(seed))
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        return _prepare_norm(case, g)
    T, V = case["T"], case["V"]
    s = dict(case=case, logits=_logits(g, T, V, TYPES[case["dtype"]]))
    if op == "distill":
        teacher = s["logits"].float() + torch.randn((T, V), generator=g, device=g.device)
        teacher *= case["scale"]
        values, s["ids"] = teacher.topk(case["k"], dim=1)
        s["values"] = values - teacher.logsumexp(1, keepdim=True)
        s["d_loss"] = torch.full((T,), 1.0 / T, device=g.device) * (torch.rand(T, generator=g, device=g.device) > 0.1)
        return s
    s["tokens"] = torch.randint(0, V, (T,), generator=g, device=g.device)
    often = torch.rand(T, generator=g, device=g.device) < 0.6
    s["tokens"] = torch.where(often, s["logits"].float().argmax(1), s["tokens"])
    if T > 1:   # the prompt's tokens are not trained on, nor scored
        s["tokens"][torch.rand(T, generator=g, device=g.device) < 0.2] = -100
    if op == "score_grad":
        top = s["logits"].float().amax(1)
        spread = (s["logits"].float() - top[:, None]) * case["scale"]
        total = spread.exp().sum(1)
        s["stats"] = torch.stack([top, total.log()], 1).contiguous()
        s["d_logprob"] = torch.randn(T, generator=g, device=g.device) / T
        if case["entropy"]:
            s["entropy"] = total.log() - (spread.exp() * spread).sum(1) / total
            s["d_entropy"] = torch.randn(T, generator=g, device=g.device) / T
    return s


# --------------------------------------------------------------------------------------------------
# The plain forms
# --------------------------------------------------------------------------------------------------

def _norm(s):
    """(x, h', the two factors 1 / rms) in 32 bits."""
    case = s["case"]
    m = s["block"].float()
    r_b = torch.rsqrt(m.square().mean(1) + s["eps"]) if case["post"] else torch.ones(m.shape[0], device=m.device)
    if case["post"]:
        m = m * r_b[:, None] * s["post_weight"].float()
    if case["gate"]:
        m = m * s["gate"].float()
    total = s["h"].float() + case["scale"] * m
    r = torch.rsqrt(total.square().mean(1) + s["eps"])
    return total * r[:, None] * s["weight"].float(), total, torch.stack([r, r_b], 1)


def _form(x):
    """The 8-bit form by rows: codes and scales 2^(e - 127), e the smallest byte in 1 .. 254 with
    (largest |x| of 128) <= 448 * 2^(e - 127)."""
    R, C = x.shape
    blocks = torch.nn.functional.pad(x, (0, -C % BLOCK)).reshape(R, -1, BLOCK)
    size = blocks.abs().amax(2)
    byte = (((size.view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp(1, 254)
    power = ((254 - byte) << 23).to(torch.int32).view(torch.float32)
    codes = (blocks * power[:, :, None]).reshape(R, -1)[:, :C].to(torch.float8_e4m3fn)
    scales = torch.nn.functional.pad(byte, (0, -byte.shape[1] % 4), value=127).to(torch.uint8)
    return codes.contiguous(), scales.contiguous().view(torch.float8_e8m0fnu)


def _plain_norm(s):
    x, total, stats = _norm(s)
    out = {"h": total.to(s["h"].dtype), "stats": stats}
    if s["case"]["form"] == "fp8":
        out["codes"], out["scales"] = _form(x)
    else:
        out["x"] = x.to(torch.bfloat16)
    return out


def _plain_norm_bwd(s):
    case = s["case"]
    dx, h = s["dX"].float(), s["h_out"].float()
    r, r_b = s["stats"][:, :1], s["stats"][:, 1:]
    n = h * r
    dn = dx * s["weight"].float()
    dh = s["dh"].float() + r * (dn - n * (dn * n).mean(1, keepdim=True))
    out = {"dh": dh.to(s["dh"].dtype), "dweight": (dx * n).sum(0)}
    dp = case["scale"] * dh
    m = s["block"].float()
    if case["post"]:
        m = m * r_b
    if case["gate"]:
        p = m * s["post_weight"].float() if case["post"] else m
        out["dgate"] = (dp * p).sum(0)
        dp = dp * s["gate"].float()
    if case["post"]:
        out["dpost_weight"] = (dp * m).sum(0)
        dm = dp * s["post_weight"].float()
        dp = r_b * (dm - m * (dm * m).mean(1, keepdim=True))
    out["dblock"] = dp.to(torch.bfloat16)
    return out


def _plain_score(s):
    case = s["case"]
    z = s["logits"].float()
    T, V = z.shape
    top = z.amax(1)
    d = (z - top[:, None]) * case["scale"]
    e = d.exp()
    total = e.sum(1)
    log_sum = total.log()
    given = s["tokens"] >= 0
    lp = d.gather(1, s["tokens"].clamp(min=0)[:, None])[:, 0] - log_sum
    out = {"logprob": torch.where(given, lp, 0.0), "stats": torch.stack([top, log_sum], 1)}
    if case["entropy"]:
        out["entropy"] = log_sum - (e * d).sum(1) / total
    if case["top"]:
        bits = (z + 0.0).view(torch.int32)
        order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long()
        key = (order << 32) | (0x7FFFFFFF - torch.arange(V, device=z.device))
        out["top_ids"] = 0x7FFFFFFF - (key.topk(case["top"], dim=1).values & 0x7FFFFFFF)
        out["top_logprob"] = d.gather(1, out["top_ids"]) - log_sum[:, None]
    return out


def _plain_score_grad(s):
    case = s["case"]
    z = s["logits"].float()
    lq = (z - s["stats"][:, :1]) * case["scale"] - s["stats"][:, 1:]
    q = lq.exp()
    given = (s["tokens"] >= 0).float()
    d = s["d_logprob"] * given
    grad = -q * d[:, None]
    if case["entropy"]:
        grad -= s["d_entropy"][:, None] * q * (lq + s["entropy"][:, None])
    grad.scatter_add_(1, s["tokens"].clamp(min=0)[:, None], d[:, None])
    return {"dlogits": (grad * case["scale"]).to(s["logits"].dtype)}


def _plain_distill(s):
    """The loss is a small difference of large terms: its sums and logarithms are taken in 64 bits."""
    case = s["case"]
    z = s["logits"].float()
    top = z.amax(1, keepdim=True)
    d = (z - top) * case["scale"]
    e = d.exp()
    picked = e.gather(1, s["ids"])
    others = e.scatter(1, s["ids"], 0.0).sum(1, dtype=torch.float64) if case["rest"] else None
    total = others + picked.double().sum(1) if case["rest"] else e.sum(1, dtype=torch.float64)
    log_sum = total.log()
    lq = d.gather(1, s["ids"]).double() - log_sum[:, None]
    lp = s["values"].double()
    if not case["rest"]:
        lp = lp - lp.logsumexp(1, keepdim=True)
    p = lp.exp()
    loss = (p * (lp - lq)).sum(1)
    whole, ratio = torch.ones_like(loss), torch.zeros_like(loss)
    q = e / total.float()[:, None]
    grad = q
    if case["rest"]:
        left = (1.0 - p.sum(1)).clamp(min=0.0)
        others = others / total
        loss = loss + torch.where(left > 0, left * (left.log() - others.log()), 0.0)
        ratio = left / others
        whole = p.sum(1).clamp(min=1.0)
        grad = q * (whole - ratio).float()[:, None]
        grad.scatter_(1, s["ids"], whole.float()[:, None] * q.gather(1, s["ids"]))
    grad = grad.scatter_add(1, s["ids"], -p.float())
    grad = grad * (case["scale"] * s["d_loss"])[:, None]
    stats = torch.stack([top[:, 0], log_sum.float(), whole.float(), ratio.float()], 1)
    return {"loss": loss.float(), "stats": stats, "dlogits": grad.to(s["logits"].dtype)}


PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "score": _plain_score, "score_grad": _plain_score_grad,
         "distill": _plain_distill}


# --------------------------------------------------------------------------------------------------
# The library's calls
# --------------------------------------------------------------------------------------------------

def _kernels(s):
    import nf4_bit_quantized_amd as q

    case = s["case"]
    op = case["op"]
    if op == "norm":
        x, h, stats = q.qlora_norm_fwd(s["h"], s["weight"], block=s["block"], post_weight=s["post_weight"],
                                       gate=s["gate"], scale=case["scale"], eps=s["eps"], form=case["form"])
        if case["form"] == "fp8":
            return {"h": h, "stats": stats, "codes": x[0].view(torch.float8_e4m3fn),
                    "scales": x[1].view(torch.float8_e8m0fnu)}
        return {"h": h, "stats": stats, "x": x}
    if op == "norm_bwd":
        g = q.qlora_norm_bwd(s["dX"], s["h_out"], s["weight"], s["stats"], block=s["block"],
                             post_weight=s["post_weight"], gate=s["gate"], scale=case["scale"], dh_out=s["dh"])
        dh, dblock, dweight, dpost_weight, dgate = g
        out = {"dh": dh, "dblock": dblock, "dweight": dweight}
        if case["post"]:
            out["dpost_weight"] = dpost_weight
        if case["gate"]:
            out["dgate"] = dgate
        return out
    if op == "score":
        logprob, stats, entropy, ids, top = q.qlora_token_logprob(s["logits"], s["tokens"], scale=case["scale"],
                                                                  top=case["top"], want_entropy=case["entropy"])
        out = {"logprob": logprob, "stats": stats}
        if case["entropy"]:
            out["entropy"] = entropy
        if case["top"]:
            out["top_ids"], out["top_logprob"] = ids, top
        return out
    if op == "score_grad":
        return {"dlogits": q.qlora_token_logprob_bwd(s["logits"], s["tokens"], s["stats"], s["d_logprob"],
                                                     scale=case["scale"], entropy=s.get("entropy"),
                                                     d_entropy=s.get("d_entropy"))}
    loss, stats = q.qlora_distill_fwd(s["logits"], s["ids"], s["values"], scale=case["scale"], rest=case["rest"])
    dlogits = q.qlora_distill_bwd(s["logits"], s["ids"], s["values"], stats, s["d_loss"], scale=case["scale"],
                                  rest=case["rest"])
    return {"loss": loss, "stats": stats, "dlogits": dlogits}


def run(state):
    return _kernels(state) if own else PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------------------------------

def _two_to(e):
    """2^e in float64 for whole e in -1022 .. 1023, exactly: e becomes the exponent field."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_form(x):
    """(values of the codes, values of the scales), float64."""
    R, C = x.shape
    nc = -(-C // BLOCK)
    full = torch.zeros((R, nc * BLOCK), dtype=torch.float64, device=x.device)
    full[:, :C] = x
    m = full.abs().reshape(R, nc, BLOCK).amax(2)
    half, e = torch.frexp(m)                       # m = half * 2^e, half in [0.5, 1)
    e = torch.where(half > 0.875, e - 8, e - 9)    # 448 = 0.875 * 2^9
    power = _two_to(torch.where(m > 0, e, -126).clamp(-126, 127))
    v = full / power.repeat_interleave(BLOCK, 1)
    step = _two_to(torch.frexp(v)[1].clamp(min=-5) - 4)   # four significant bits, 2^-9 the least
    scales = torch.ones((R, -(-nc // 4) * 4), dtype=torch.float64, device=x.device)
    scales[:, :nc] = power
    return (torch.round(v / step) * step)[:, :C], scales


def _exact_norm(s):
    case = s["case"]
    h, b = s["h"].double(), s["block"].double()
    T, D = h.shape
    one = torch.ones(D, dtype=torch.float64, device=h.device)
    w_b = s["post_weight"].double() if case["post"] else one
    gate = s["gate"].double() if case["gate"] else one
    r_b = torch.ones(T, dtype=torch.float64, device=h.device)
    if case["post"]:
        r_b = 1.0 / torch.sqrt(torch.sum(b * b, 1) / D + s["eps"])
    new = h + torch.einsum("td,t,d->td", b, r_b, case["scale"] * gate * w_b)
    r = 1.0 / torch.sqrt(torch.sum(new * new, 1) / D + s["eps"])
    x = torch.einsum("td,t,d->td", new, r, s["weight"].double())
    out = {"h": new, "stats": torch.stack([r, r_b], 1)}
    if case["form"] == "fp8":
        out["codes"], out["scales"] = _exact_form(x)
    else:
        out["x"] = x
    return out


def _exact_norm_bwd(s):
    """Through the Jacobian of v / rms(v) applied from the left: J^T a = r a - r^3 v (v . a) / D."""
    case = s["case"]
    D = s["h_out"].shape[1]
    dx, h, b = s["dX"].double(), s["h_out"].double(), s["block"].double()
    r, r_b = s["stats"].double().unbind(1)
    a = dx * s["weight"].double()
    dh = s["dh"].double() + a * r[:, None] - h * (r ** 3 * (h * a).sum(1) / D)[:, None]
    out = {"dh": dh, "dweight": torch.matmul(r, dx * h)}
    one = torch.ones(D, dtype=torch.float64, device=h.device)
    w_b = s["post_weight"].double() if case["post"] else one
    gate = s["gate"].double() if case["gate"] else one
    f = r_b if case["post"] else torch.ones_like(r_b)
    common = torch.matmul(f, b * dh) * case["scale"]
    if case["gate"]:
        out["dgate"] = common * w_b
    a = dh * (case["scale"] * gate * w_b)
    if case["post"]:
        out["dpost_weight"] = common * gate
        a = a * r_b[:, None] - b * (r_b ** 3 * (b * a).sum(1) / D)[:, None]
    out["dblock"] = a
    return out


def _exact_score(s):
    case = s["case"]
    z = s["logits"].double() * case["scale"]
    lse = torch.logsumexp(z, 1)
    where = torch.where(s["tokens"] < 0, 0, s["tokens"])
    lp = z[torch.arange(z.shape[0], device=z.device), where] - lse
    most = torch.max(z, 1).values
    out = {"logprob": lp * (s["tokens"] >= 0), "stats": torch.stack([most / case["scale"], lse - most], 1)}
    if case["entropy"]:
        out["entropy"] = lse - torch.sum(torch.exp(z - lse[:, None]) * z, 1)
    if case["top"]:
        if z.shape[0] * z.shape[1] > 1 << 26:
            out["top_ids"] = None
            out["top_logprob"] = torch.topk(z, case["top"], dim=1).values - lse[:, None]
        else:
            value, at = torch.sort(z, dim=1, descending=True, stable=True)
            out["top_ids"] = at[:, :case["top"]].contiguous()
            out["top_logprob"] = value[:, :case["top"]] - lse[:, None]
    return out


def _exact_score_grad(s):
    case = s["case"]
    z = s["logits"].double()
    log_q = case["scale"] * z - (case["scale"] * s["stats"][:, 0].double() + s["stats"][:, 1].double())[:, None]
    q = torch.exp(log_q)
    T = z.shape[0]
    rows = torch.arange(T, device=z.device)[s["tokens"] >= 0]
    d = torch.where(s["tokens"] >= 0, s["d_logprob"].double(), 0.0)
    weight = d[:, None].expand_as(q)
    if case["entropy"]:
        weight = weight + s["d_entropy"].double()[:, None] * (log_q + s["entropy"].double()[:, None])
    grad = -q * weight
    grad[rows, s["tokens"][rows]] += d[rows]
    return {"dlogits": grad * case["scale"]}


def _exact_distill(s):
    case = s["case"]
    z = s["logits"].double()
    T = z.shape[0]
    most = z.amax(1)
    lse = torch.logsumexp(case["scale"] * z, 1)
    q = torch.exp(case["scale"] * z - lse[:, None])
    t = s["values"].double()
    p = torch.exp(t) if case["rest"] else torch.softmax(t, 1)
    rows = torch.arange(T, device=z.device)[:, None]
    picked = q[rows, s["ids"]]
    loss = torch.sum(torch.xlogy(p, p / picked), 1)
    grad = q.clone()
    whole, ratio = torch.ones_like(loss), torch.zeros_like(loss)
    if case["rest"]:
        left = torch.clamp(1.0 - p.sum(1), min=0.0)
        out_of = q.clone()
        out_of[rows, s["ids"]] = 0.0
        mass = out_of.sum(1)
        loss = loss + torch.xlogy(left, left / mass)
        ratio = left / mass
        whole = p.sum(1) + left
        grad = grad * whole[:, None] - out_of * ratio[:, None]
    grad[rows, s["ids"]] -= p
    grad *= (s["d_loss"].double() * case["scale"])[:, None]
    return {"loss": loss, "stats": torch.stack([most, lse - case["scale"] * most, whole, ratio], 1), "dlogits": grad}


EXACT = {"norm": _exact_norm, "norm_bwd": _exact_norm_bwd, "score": _exact_score, "score_grad": _exact_score_grad,
         "distill": _exact_distill}


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))
