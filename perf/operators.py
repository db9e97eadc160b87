"""Timed cases of the operators around a language model's linear layers:
token embedding (lookup and gradient), root-mean-square norm (residual
addition, 8-bit checkpoint, gradient) and the output layer's softmax cross
entropy (loss, and the gradients of the hidden states and of the table).

``listed()`` names fixed cases, ``draw(rng)`` makes one more of the same
ranges.  ``prepare(case, seed)`` makes the inputs on the GPU and
``run(state)`` is one call of the operator: in plain torch operations in 32
bits where ``own`` is false, through this package where it is true.
``exact(case, seed)`` is the same result from the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5
IGNORE = -100
# the output layer of GPT-2 on 8 sequences of 1024 tokens
LARGEST = 8192 * 768 * 50257


def listed():
    return [
        # a decoding step of eight sequences: latency
        dict(name="embed_step", op="embed", grad=False, tokens=8, width=768, vocab=50257, dtype="bf16"),
        # the token embedding of a GPT-2 training step and its gradient
        dict(name="embed_gpt2_grad", op="embed", grad=True, tokens=8192, width=768, vocab=50257, dtype="bf16"),
        # an odd width in 32 bits, a smaller vocabulary, many repeated tokens
        dict(name="embed_odd_grad", op="embed", grad=True, tokens=5001, width=515, vocab=8191, dtype="f32"),
        # the norm in a decoding step of one token: latency
        dict(name="norm_step", op="norm", grad=False, tokens=1, width=768, dtype="bf16", residual=True, bits8=False),
        # the norm of a GPT-2 training step, with the residual's addition and the 8-bit checkpoint
        dict(name="norm_gpt2_8bit", op="norm", grad=False, tokens=8192, width=768, dtype="bf16", residual=True, bits8=True),
        # its gradient from the stored residual stream
        dict(name="norm_gpt2_grad", op="norm", grad=True, tokens=8192, width=768, dtype="bf16", residual=True, bits8=False),
        # its gradient from the 8-bit checkpoint, fp16, a wider layer, a ragged token count
        dict(name="norm_wide_grad_8bit", op="norm", grad=True, tokens=3001, width=2048, dtype="f16", residual=True, bits8=True),
        # the toy MLP's width in 32 bits, no residual
        dict(name="norm_toy_grad", op="norm", grad=True, tokens=512, width=512, dtype="f32", residual=False, bits8=False),
        # scoring one token against a vocabulary: the table is read once
        dict(name="loss_one", op="loss", grad=False, tokens=1, width=768, vocab=50257, dtype="bf16", kept=1.0),
        # evaluation loss of a GPT-2 batch
        dict(name="loss_gpt2", op="loss", grad=False, tokens=8192, width=768, vocab=50257, dtype="bf16", kept=1.0),
        # a short ragged batch with padded positions, fp16 with a scaled loss
        dict(name="loss_ragged_grad", op="loss", grad=True, tokens=509, width=512, vocab=32003, dtype="f16", kept=0.8),
        # the output layer of a GPT-2 training step
        dict(name="loss_gpt2_grad", op="loss", grad=True, tokens=8192, width=768, vocab=50257, dtype="bf16", kept=1.0),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "norm", "loss"])
    grad = rng.random() < 0.6
    if op == "embed":
        return dict(op=op, grad=grad, tokens=_spread(rng, 1, 16384), width=_spread(rng, 64, 1600),
                    vocab=_spread(rng, 1000, 131072), dtype=rng.choice(["bf16", "f16", "f32"]))
    if op == "norm":
        # a linear layer's widths: mostly whole vectors, sometimes odd
        width = _spread(rng, 64, 4096)
        if rng.random() < 0.75:
            width = (width + 7) // 8 * 8
        return dict(op=op, grad=grad, tokens=_spread(rng, 1, 16384), width=width,
                    dtype=rng.choice(["bf16", "f16", "f32"]), residual=rng.random() < 0.7, bits8=rng.random() < 0.4)
    while True:
        c = dict(op=op, grad=grad, tokens=_spread(rng, 1, 8192), width=8 * _spread(rng, 8, 256),
                 vocab=_spread(rng, 1000, 131072), dtype=rng.choice(["bf16", "f16"]), kept=rng.choice([1.0, 0.8, 0.3]))
        if c["tokens"] * c["width"] * c["vocab"] <= LARGEST:
            return c


def _ids(case, g):
    """Token ids whose frequencies fall off like those of text: a few very common, many seen once."""
    u = torch.rand(case["tokens"], generator=g, device="cuda", dtype=torch.float64)
    rank = torch.exp(u * math.log(case["vocab"])) - 1.0
    # a fixed permutation spreads the common ids over the table
    return (rank.long().clamp_(0, case["vocab"] - 1) * 7919 + 13) % case["vocab"]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)

    M, D = case["tokens"], case["width"]
    s = {"case": case}
    if case["op"] == "embed":
        s["ids"] = _ids(case, g)
        s["scale"] = math.sqrt(D)
        if case["grad"]:
            s["dy"] = normal(M, D, std=1e-2)
        else:
            s["table"] = normal(case["vocab"], D, std=0.02)
    elif case["op"] == "norm":
        s["gamma"] = (1.0 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(dt)
        if case["grad"]:
            h = torch.randn(M, D, generator=g, device="cuda") * 2.0
            rstd = torch.rsqrt(h.square().mean(1) + EPS)
            s["rstd"] = rstd
            s["dy"] = normal(M, D, std=1e-2)
            s["dh"] = normal(M, D, std=1e-2) if case["residual"] else None
            if case["bits8"]:
                xn = h * rstd[:, None]
                s["scales"] = xn.abs().amax(1) / 127.0
                s["codes"] = torch.round(xn / s["scales"][:, None]).clamp_(-127, 127).to(torch.int8)
            else:
                s["h"] = h.to(dt)
        else:
            s["x"] = normal(M, D)
            s["residual"] = normal(M, D, std=2.0) if case["residual"] else None
    else:
        V = case["vocab"]
        s["x"] = normal(M, D)
        s["table"] = normal(V, D, std=2.0 / math.sqrt(D))
        t = _ids(case, g)
        if case["kept"] < 1.0:
            t[torch.rand(M, generator=g, device="cuda") >= case["kept"]] = IGNORE
        s["targets"] = t
        # fp16 training scales its loss so that small gradients stay in range
        s["grad"] = torch.full((), 4096.0 if case["dtype"] == "f16" else 1.0, device="cuda")
    return s


def _embed(s, wide):
    c = s["case"]
    if not c["grad"]:
        return (s["table"][s["ids"]].to(wide) * s["scale"])
    out = torch.zeros(c["vocab"], c["width"], dtype=wide, device="cuda")
    out.index_add_(0, s["ids"], s["dy"].to(wide))
    return out * s["scale"]


def _norm(s, wide):
    c = s["case"]
    gamma = s["gamma"].to(wide)
    if not c["grad"]:
        h = s["x"].to(wide)
        if s["residual"] is not None:
            h = h + s["residual"].to(wide)
        rstd = torch.rsqrt(h.square().mean(1) + EPS)
        xn = h * rstd[:, None]
        out = {"y": xn * gamma, "h": h if c["residual"] else None, "rstd": rstd, "read_back": None}
        if c["bits8"]:
            scales = xn.abs().amax(1, keepdim=True) / 127.0
            out["read_back"] = torch.round(xn / scales) * scales
        return out
    if c["bits8"]:
        xn = s["codes"].to(wide) * s["scales"].to(wide)[:, None]
    else:
        xn = s["h"].to(wide) * s["rstd"].to(wide)[:, None]
    dy = s["dy"].to(wide)
    gdy = gamma * dy
    dx = s["rstd"].to(wide)[:, None] * (gdy - xn * (gdy * xn).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].to(wide)
    return {"dx": dx, "dgamma": (dy * xn).sum(0), "y": xn * gamma if c["bits8"] else None}


def _loss(s, wide):
    c = s["case"]
    x, w, t = s["x"].to(wide), s["table"].to(wide), s["targets"]
    keep = t != IGNORE
    row = torch.arange(t.numel(), device="cuda")
    at = torch.where(keep, t, torch.zeros_like(t))
    z = x @ w.t()
    top = z.amax(1)
    lse = top + torch.log(torch.exp(z - top[:, None]).sum(1))
    lse = torch.where(keep, lse, torch.zeros_like(lse))        # nothing is asked of a padded position
    loss = torch.where(keep, lse - z[row, at], torch.zeros_like(lse))
    if not c["grad"]:
        return {"loss": loss, "lse": lse}
    count = keep.sum().clamp(min=1)
    # the gradient of the mean over kept positions, written over the logits
    p = z.sub_(lse[:, None]).exp_()
    p[row, at] -= 1.0
    p.mul_((keep.to(wide) * (s["grad"].to(wide) / count))[:, None])
    return {"loss": loss.sum() / count, "dx": p @ w, "dtable": p.t() @ x}


_plain = {"embed": _embed, "norm": _norm, "loss": _loss}
_stats = ("rstd", "loss", "lse")          # 32-bit whatever the inputs' type


def _round(out, dt):
    """The one rounding at the end; the 8-bit values are read back as 16-bit ones."""
    if torch.is_tensor(out):
        return out.to(dt)
    low = dt if dt != torch.float32 else torch.bfloat16
    return {k: v if v is None else v.to(torch.float32 if k in _stats else low if k == "read_back" else dt)
            for k, v in out.items()}


def _own(s):
    import deterministic_invariant_gemm_fwd_gb300 as cg
    c = s["case"]
    if c["op"] == "embed":
        if c["grad"]:
            return cg.embedding_bwd(s["dy"], s["ids"], c["vocab"], scale=s["scale"])
        return cg.embedding_fwd(s["table"], s["ids"], scale=s["scale"])
    if c["op"] == "norm":
        if c["grad"]:
            if c["bits8"]:
                dx, dgamma, y = cg.rms_norm_bwd(s["dy"], s["gamma"], s["rstd"], codes=s["codes"],
                                                scales=s["scales"], dh=s["dh"], recompute=True)
                return {"dx": dx, "dgamma": dgamma, "y": y}
            dx, dgamma = cg.rms_norm_bwd(s["dy"], s["gamma"], s["rstd"], h=s["h"], dh=s["dh"])
            return {"dx": dx, "dgamma": dgamma, "y": None}
        r = cg.rms_norm_fwd(s["x"], s["gamma"], residual=s["residual"], eps=EPS, quantize=c["bits8"])
        out = {"y": r.y, "h": r.h if c["residual"] else None, "rstd": r.rstd, "read_back": None}
        if c["bits8"]:
            low = s["x"].dtype if s["x"].dtype != torch.float32 else torch.bfloat16
            out["read_back"] = cg.rms_norm_expand(r.codes, r.scales, dtype=low)
        return out
    if not c["grad"]:
        loss, lse = cg.linear_cross_entropy_fwd(s["x"], s["table"], s["targets"], ignore_index=IGNORE,
                                                   reduction="none")
        return {"loss": loss, "lse": lse}
    loss, lse = cg.linear_cross_entropy_fwd(s["x"], s["table"], s["targets"], ignore_index=IGNORE,
                                                   reduction="mean")
    dx, dtable = cg.linear_cross_entropy_bwd(s["grad"], s["x"], s["table"], s["targets"], lse,
                                             ignore_index=IGNORE, reduction="mean")
    return {"loss": loss, "dx": dx, "dtable": dtable}


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    return _round(_plain[c["op"]](state, torch.float32), DTYPES[c["dtype"]])


def work(case):
    """Bytes: each input read once, each output written once.  Flops: the products."""
    M, D, e = case["tokens"], case["width"], SIZE[case["dtype"]]
    if case["op"] == "embed":
        if case["grad"]:
            return {"bytes": M * D * e + M * 8 + case["vocab"] * D * e, "flops": M * D}
        return {"bytes": 2 * M * D * e + M * 8, "flops": M * D}
    if case["op"] == "norm":
        if case["grad"]:
            kept = M * D * (1 if case["bits8"] else e) + 4 * M * (2 if case["bits8"] else 1)
            moved = M * D * e * (2 + (1 if case["residual"] else 0) + (1 if case["bits8"] else 0))
            return {"bytes": kept + moved + 2 * D * e, "flops": 10 * M * D}
        moved = M * D * e * (4 if case["residual"] else 2)
        if case["bits8"]:       # the codes, and their values as they are read back
            moved += M * D * (1 + 2) + 4 * M
        return {"bytes": moved + D * e + 4 * M, "flops": 5 * M * D}
    # a padded position needs no product: only its zeros are written
    V, kept = case["vocab"], case["kept"] * M
    read = (kept + V) * D * e + 8 * M
    if case["grad"]:
        # logits, logits again (they are not kept), and the two gradients
        return {"bytes": read + (M + V) * D * e + 4, "flops": 8 * kept * D * V}
    return {"bytes": read + 8 * M, "flops": 2 * kept * D * V}


# ---- the same results from the definitions, in 64 bits, written apart from the plain form

def _exact_embed(s):
    c = s["case"]
    if not c["grad"]:
        return torch.gather(s["table"].double(), 0, s["ids"][:, None].expand(-1, c["width"])) * s["scale"]
    order = torch.argsort(s["ids"], stable=True)
    sums = torch.cumsum(s["dy"].double()[order], 0)
    ids, n = torch.unique_consecutive(s["ids"][order], return_counts=True)
    last = torch.cumsum(n, 0) - 1
    run_sums = sums[last]
    run_sums[1:] -= sums[last[:-1]]
    out = torch.zeros(c["vocab"], c["width"], dtype=torch.float64, device="cuda")
    out[ids] = run_sums * s["scale"]
    return out


def _exact_norm(s):
    c = s["case"]
    gamma = s["gamma"].double()
    if not c["grad"]:
        h = s["x"].double() + (s["residual"].double() if c["residual"] else 0.0)
        rms = torch.sqrt((h * h).sum(1) / c["width"] + EPS)
        n = h / rms[:, None]
        back = None
        if c["bits8"]:
            unit = n.abs().max(1).values[:, None] / 127
            back = torch.floor(n / unit + 0.5) * unit
        return {"y": n * gamma, "h": h if c["residual"] else None, "rstd": 1 / rms, "read_back": back}
    r = s["rstd"].double()[:, None]
    n = s["codes"].double() * s["scales"].double()[:, None] if c["bits8"] else s["h"].double() * r
    dy = s["dy"].double()
    dn = dy * gamma
    dot = torch.einsum("md,md->m", dn, n) / c["width"]
    dx = r * dn - r * n * dot[:, None]
    if c["residual"]:
        dx = dx + s["dh"].double()
    return {"dx": dx, "dgamma": torch.einsum("md,md->d", dy, n), "y": n * gamma if c["bits8"] else None}


def _exact_loss(s):
    c = s["case"]
    x, w, t = s["x"].double(), s["table"].double(), s["targets"]
    M, V = c["tokens"], c["vocab"]
    kept = torch.nonzero(t >= 0).squeeze(1)
    logits = torch.mm(x, w.T)
    lse = torch.logsumexp(logits, 1)
    loss = torch.zeros(M, dtype=torch.float64, device="cuda")
    loss[kept] = lse[kept] - (x[kept] * w[t[kept]]).sum(1)
    if not c["grad"]:
        return {"loss": loss, "lse": torch.zeros_like(lse).index_copy_(0, kept, lse[kept])}
    weight = torch.zeros(M, dtype=torch.float64, device="cuda")
    weight[kept] = float(s["grad"]) / max(1, kept.numel())
    soft = torch.softmax(logits, 1)
    del logits
    soft *= weight[:, None]
    # the softmax's part, then the targets' rows
    dx = torch.mm(soft, w)
    dtable = torch.mm(soft.T, x)
    dx[kept] -= weight[kept, None] * w[t[kept]]
    dtable.index_add_(0, t[kept], -weight[kept, None] * x[kept])
    return {"loss": loss.sum() / max(1, kept.numel()), "dx": dx, "dtable": dtable}


def exact(case, seed):
    return {"embed": _exact_embed, "norm": _exact_norm, "loss": _exact_loss}[case["op"]](prepare(case, seed))
