"""Timed cases of the operators of fine-tuning and scoring a language model:
low-rank adapters beside a shared linear layer (many requests or sequences,
each with its own adapter), log probabilities of given tokens with the
entropy and the top alternatives, and the norm of all gradients with their
clipping.

``listed()`` names fixed cases, ``draw(rng)`` makes one more of the same
ranges.  ``prepare(case, seed)`` makes the inputs on the GPU and
``run(state)`` is one call of the operator (with its gradient where the case
has one): in plain torch operations in 32 bits where ``own`` is false, through
this package where it is true.  ``exact(case, seed)`` is the same result from
the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
IGNORE = -100
CLIP_EPS = 1e-6
# beyond these, a drawn case would cost more than the largest listed one
LARGEST_LORA = 8192 * 1600 * 6400
LARGEST_LOGP = 8192 * 768 * 50257
LARGEST_CLIP = 99_000_000


def listed():
    return [
        # one request's next token through a projection with its adapter: latency
        dict(name="lora_one", op="lora", grad=False, tokens=1, inner=768, outer=768, adapters=4, rank=16,
             mean=1, bias=True, dtype="bf16"),
        # a decoding step of 64 requests with 24 adapters among them
        dict(name="lora_step", op="lora", grad=False, tokens=64, inner=768, outer=2304, adapters=24, rank=16,
             mean=1, bias=True, dtype="bf16"),
        # fine-tuning a GPT-2 layer's adapters: sequences of some hundred tokens, four tasks
        dict(name="lora_gpt2_grad", op="lora", grad=True, tokens=8192, inner=768, outer=2304, adapters=4, rank=16,
             mean=512, bias=True, dtype="bf16"),
        # an odd token count, fp16, a high rank, short sequences of many tasks
        dict(name="lora_ragged_grad", op="lora", grad=True, tokens=3001, inner=520, outer=776, adapters=9, rank=64,
             mean=37, bias=False, dtype="f16"),
        # prompts of several requests through a wide layer
        dict(name="lora_wide", op="lora", grad=False, tokens=8192, inner=1600, outer=6400, adapters=8, rank=32,
             mean=1000, bias=False, dtype="bf16"),
        # a decoding step of eight sequences: the sampled tokens' log probabilities and five alternatives
        dict(name="logp_step", op="logp", grad=False, tokens=8, width=768, vocab=50257, top=5, kept=1.0,
             entropy=True, temperature=0.7, dtype="bf16"),
        # scoring a batch of sequences with eight alternatives per token
        dict(name="logp_score", op="logp", grad=False, tokens=8192, width=768, vocab=50257, top=8, kept=1.0,
             entropy=True, temperature=1.0, dtype="bf16"),
        # a policy's update on a ragged batch: prompts do not count, fp16
        dict(name="logp_ragged_grad", op="logp", grad=True, tokens=1003, width=512, vocab=32003, top=0, kept=0.6,
             entropy=True, temperature=0.9, dtype="f16"),
        # a policy's update on a full batch, with a bonus for entropy
        dict(name="logp_update", op="logp", grad=True, tokens=8192, width=768, vocab=50257, top=0, kept=1.0,
             entropy=True, temperature=1.0, dtype="bf16"),
        # the toy MLP's gradients: latency
        dict(name="clip_toy", op="clip", blocks=0, width=256, vocab=0, odd=0, max_norm=1.0, dtype="f32"),
        # gradients of adapters: many small tensors of odd sizes and both types
        dict(name="clip_adapters", op="clip", blocks=40, width=0, vocab=0, odd=5003, max_norm=0.5, dtype="mixed"),
        # gradients of a small language model, embedding included
        dict(name="clip_model", op="clip", blocks=16, width=640, vocab=32003, odd=0, max_norm=1.0, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lora", "logp", "clip"])
    if op == "lora":
        while True:
            c = dict(op=op, grad=rng.random() < 0.6, tokens=_spread(rng, 1, 8192), inner=8 * _spread(rng, 8, 512),
                     outer=8 * _spread(rng, 8, 512), adapters=_spread(rng, 1, 32), rank=8 * rng.randint(1, 16),
                     mean=_spread(rng, 1, 1000), bias=rng.random() < 0.5, dtype=rng.choice(["bf16", "f16"]))
            if c["tokens"] * c["inner"] * c["outer"] * (3 if c["grad"] else 1) <= LARGEST_LORA:
                return c
    if op == "logp":
        while True:
            grad = rng.random() < 0.5
            c = dict(op=op, grad=grad, tokens=_spread(rng, 1, 8192), width=8 * _spread(rng, 8, 256),
                     vocab=_spread(rng, 1000, 131072), top=0 if grad else rng.choice([0, 1, 5, 8, 20]),
                     kept=rng.choice([1.0, 0.7, 0.3]), entropy=rng.random() < 0.8,
                     temperature=rng.choice([1.0, 0.7, 1.3]), dtype=rng.choice(["bf16", "f16"]))
            if c["tokens"] * c["width"] * c["vocab"] <= LARGEST_LOGP:
                return c
    while True:
        c = dict(op=op, blocks=rng.randint(0, 24), width=8 * _spread(rng, 4, 96), vocab=_spread(rng, 100, 40000),
                 odd=rng.choice([0, _spread(rng, 1, 100000)]), max_norm=rng.choice([0.1, 1.0, 1e6]),
                 dtype=rng.choice(["f32", "bf16", "f16", "mixed"]))
        if sum(_sizes(c)) <= LARGEST_CLIP:
            return c


def _sizes(case):
    """Elements of each gradient tensor of a clipping case."""
    D, n = case["width"], []
    if case["vocab"]:
        n.append(case["vocab"] * D)
    for _ in range(case["blocks"]):
        if D:           # a block: two norms, attention's and the MLP's matrices and biases
            n += [D, 3 * D * D, 3 * D, D * D, D, D, 4 * D * D, 4 * D, 4 * D * D, D]
        if case["odd"]:     # an adapter's two matrices, and a vector that moves the next one off its alignment
            n += [case["odd"] * 2, case["odd"] * 6, 1 + case["odd"] % 97]
    if not case["blocks"] or not n:
        n += [D * 2 * D, 2 * D, 4 * D * D, 2 * D, 2 * D * D, D] if D else [case["odd"] or 1]
    return n


def _adapters(case, g):
    """An adapter for each token: sequences of a random length share one, and
    about one sequence in ten has none."""
    M, n = case["tokens"], case["adapters"]
    starts = torch.rand(M, generator=g, device="cuda") < 1.0 / case["mean"]
    which = torch.randint(0, n, (M + 1,), generator=g, device="cuda")
    which[torch.rand(M + 1, generator=g, device="cuda") < 0.1] = -1
    which[0] = 0
    return which[torch.cumsum(starts.long(), 0)]


def _ids(case, g):
    """Token ids whose frequencies fall off like those of text."""
    u = torch.rand(case["tokens"], generator=g, device="cuda", dtype=torch.float64)
    rank = torch.exp(u * math.log(case["vocab"])) - 1.0
    return (rank.long().clamp_(0, case["vocab"] - 1) * 7919 + 13) % case["vocab"]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}

    if case["op"] == "clip":
        kinds = [torch.bfloat16, torch.float32] if case["dtype"] == "mixed" else [DTYPES[case["dtype"]]]
        by_kind = {k: [i for i, _ in enumerate(_sizes(case)) if kinds[i % len(kinds)] is k] for k in kinds}
        sizes = _sizes(case)
        std = 2.0 / math.sqrt(sum(sizes))               # a norm of about 2
        s["grads"], s["out"] = [None] * len(sizes), [None] * len(sizes)
        s["flat"], s["flat_out"] = [], []               # one buffer per type, its tensors one behind another
        for k, which in by_kind.items():
            n = [sizes[i] for i in which]
            s["flat"].append((torch.randn(sum(n), generator=g, device="cuda") * std).to(k))
            s["flat_out"].append(torch.empty_like(s["flat"][-1]))
            for i, t, o in zip(which, s["flat"][-1].split(n), s["flat_out"][-1].split(n)):
                s["grads"][i], s["out"][i] = t, o
        return s

    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)

    M = case["tokens"]
    if case["op"] == "lora":
        K, N, n, r = case["inner"], case["outer"], case["adapters"], case["rank"]
        s["x"] = normal(M, K)
        s["weight"] = normal(K, N, std=1.0 / math.sqrt(K))
        s["bias"] = normal(N, std=0.1) if case["bias"] else None
        s["a"] = normal(n, K, r, std=1.0 / math.sqrt(K))
        s["b"] = normal(n, r, N, std=0.5 / math.sqrt(r))
        s["scales"] = 0.5 + torch.rand(n, generator=g, device="cuda")
        s["adapters"] = _adapters(case, g)
        if case["grad"]:
            s["dy"] = normal(M, N, std=1e-2)
        return s

    V, D = case["vocab"], case["width"]
    s["x"] = normal(M, D)
    s["table"] = normal(V, D, std=2.0 / math.sqrt(D))
    t = _ids(case, g)
    if case["kept"] < 1.0:
        left_out = torch.rand(M, generator=g, device="cuda") >= case["kept"]
        left_out[0] = False
        t[left_out] = IGNORE
    s["tokens"] = t
    if case["grad"]:
        # advantages over the number of tokens (fp16 training scales them up), and the entropy's weight
        up = (4096.0 if case["dtype"] == "f16" else 1.0) / M
        s["dlogp"] = torch.randn(M, generator=g, device="cuda") * up
        s["dentropy"] = torch.full((M,), 0.01 * up, device="cuda") if case["entropy"] else None
    return s


# ---- the plain forms ------------------------------------------------------------

def _lora(s):
    c, ids, n = s["case"], s["adapters"], s["case"]["adapters"]
    x, w, a, b = (s[k].float() for k in ("x", "weight", "a", "b"))
    y = x @ w
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if c["tokens"] <= 64 and not c["grad"]:         # few tokens: each one's own matrices
        at = ids.clamp(min=0)
        scale = torch.where(ids >= 0, s["scales"][at], torch.zeros((), device="cuda"))
        u = (x[:, :, None] * a[at]).sum(1)
        return {"y": y + scale[:, None] * (u[:, :, None] * b[at]).sum(1)}
    here = [(ids == i)[:, None] for i in range(n)]
    us = []
    for i in range(n):
        us.append(x @ a[i] * s["scales"][i])
        y = y + torch.where(here[i], us[i] @ b[i], 0.0)
    if not c["grad"]:
        return {"y": y}
    dy = s["dy"].float()
    dx, da, db = dy @ w.t(), torch.empty_like(a), torch.empty_like(b)
    for i in range(n):
        mine = torch.where(here[i], dy, 0.0)
        du = mine @ b[i].t() * s["scales"][i]
        dx = dx + du @ a[i].t()
        da[i] = x.t() @ du
        db[i] = us[i].t() @ mine
    return {"y": y, "dx": dx, "da": da, "db": db}


def _top(z, x, table, keep, top):
    """Ids and logits of the largest logits, by their values in 64 bits (what
    32 bits cannot tell apart is decided there), equal ones by the lower id."""
    some = min(top + 4, z.shape[1])
    ids = torch.sort(torch.topk(z, some, dim=1).indices, dim=1).values
    value = (table[ids].double() * x.double()[:, None, :]).sum(2)
    order = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :top]
    ids, value = torch.gather(ids, 1, order), torch.gather(value, 1, order)
    return torch.where(keep[:, None], ids, -1), value


def _logp(s):
    c = s["case"]
    x, w, t = s["x"].float(), s["table"].float(), s["tokens"]
    keep = t != IGNORE
    row = torch.arange(t.numel(), device="cuda")
    at = torch.where(keep, t, torch.zeros_like(t))
    zero = torch.zeros((), device="cuda")
    z = x @ w.t()
    out = {"top_ids": None, "top_log_probs": None}
    if c["top"]:
        out["top_ids"], best = _top(z, x, w, keep, c["top"])
    z = z / c["temperature"]
    high = z.amax(1)
    e = torch.exp(z - high[:, None])
    total = e.sum(1)
    lse = high + torch.log(total)
    # the entropy from differences to the largest logit, so that nothing cancels
    ent = torch.log(total) - (e.mul_(z - high[:, None])).sum(1) / total
    del e
    if c["top"]:
        logp = (best / c["temperature"] - lse.double()[:, None]).float()
        out["top_log_probs"] = torch.where(keep[:, None], logp, zero)
    out["log_probs"] = torch.where(keep, z[row, at] - lse, zero)
    out["entropy"] = torch.where(keep, ent, zero)
    if not c["grad"]:
        return out
    gl = torch.where(keep, s["dlogp"], zero)
    logp = z.sub_(lse[:, None])
    p = torch.exp(logp)
    if s["dentropy"] is not None:
        ge = torch.where(keep, s["dentropy"], zero)
        g = logp.add_(ent[:, None]).mul_(ge[:, None]).add_(gl[:, None]).mul_(p).neg_()
    else:
        g = p.mul_(-gl[:, None])
    g[row, at] += gl
    g /= c["temperature"]
    out["dx"], out["dtable"] = g @ w, g.t() @ x
    return out


def _clip(s):
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for t in s["grads"]:
        total = total + t.float().square().sum(dtype=torch.float64)
    norm = torch.sqrt(total).float()
    factor = torch.clamp(s["case"]["max_norm"] / (norm + CLIP_EPS), max=1.0)
    for t, o in zip(s["grads"], s["out"]):
        o.copy_(t.float() * factor)                     # rounds
    return {"norm": norm, "grads": s["flat_out"]}


_plain = {"lora": _lora, "logp": _logp, "clip": _clip}
_stats = ("log_probs", "entropy", "top_log_probs", "norm")          # 32-bit whatever the inputs' type


def _round(out, s):
    """The one rounding at the end."""
    if "grads" in out:
        return out
    dt = s["x"].dtype
    return {k: v if v is None or k == "top_ids" or k in _stats else v.to(dt) for k, v in out.items()}


# ---- this package's calls ---------------------------------------------------------

def _own(s):
    import deterministic_invariant_gemm_fwd_gb300 as cg
    c = s["case"]
    if c["op"] == "clip":
        norm = cg.clip_grads(s["grads"], c["max_norm"], eps=CLIP_EPS, out=s["out"])
        return {"norm": norm, "grads": s["flat_out"]}
    if c["op"] == "lora":
        r = cg.lora_linear_fwd(s["x"], s["weight"], s["a"], s["b"], s["adapters"], s["scales"], bias=s["bias"],
                               keep=c["grad"])
        if not c["grad"]:
            return {"y": r}
        y, u = r
        dx, da, db = cg.lora_linear_bwd(s["dy"], s["x"], s["weight"], s["a"], s["b"], s["adapters"], s["scales"], u)
        return {"y": y, "dx": dx, "da": da, "db": db}
    r = cg.linear_log_probs_fwd(s["x"], s["table"], s["tokens"], temperature=c["temperature"], top=c["top"],
                                ignore_index=IGNORE)
    out = {"top_ids": r.top_ids, "top_log_probs": r.top_log_probs, "log_probs": r.log_probs, "entropy": r.entropy}
    if c["grad"]:
        out["dx"], out["dtable"] = cg.linear_log_probs_bwd(s["dlogp"], s["dentropy"], s["x"], s["table"], s["tokens"],
                                                           r.lse, r.entropy, temperature=c["temperature"],
                                                           ignore_index=IGNORE)
    return out


def run(state):
    return _own(state) if own else _round(_plain[state["case"]["op"]](state), state)


def work(case):
    """Bytes: each input read once, each output written once.  Flops: the products."""
    if case["op"] == "clip":
        sizes = _sizes(case)
        if case["dtype"] == "mixed":
            moved = sum(n * (2 if i % 2 == 0 else 4) for i, n in enumerate(sizes))
        else:
            moved = sum(sizes) * SIZE[case["dtype"]]
        return {"bytes": 2 * moved + 4, "flops": 3 * sum(sizes)}
    M, e = case["tokens"], SIZE[case["dtype"]]
    if case["op"] == "lora":
        K, N, r = case["inner"], case["outer"], case["rank"]
        n = min(case["adapters"], M)                     # adapters that a token can name
        read = M * K * e + K * N * e + n * (K + N) * r * e + 8 * M + 4 * n + (N * e if case["bias"] else 0)
        base, low = 2 * M * K * N, 2 * M * (K + N) * r
        if case["grad"]:
            # dy, dx, the adapters' gradients; the layer's own dx; dU, its product, and the two gradients
            return {"bytes": read + 2 * M * N * e + M * K * e + case["adapters"] * (K + N) * r * e,
                    "flops": 2 * base + 3 * low}
        return {"bytes": read + M * N * e, "flops": base + low}
    # a position that does not count needs no product
    V, D, kept = case["vocab"], case["width"], case["kept"] * M
    read = (kept + V) * D * e + 8 * M
    out = 8 * M + 12 * M * case["top"]
    if case["grad"]:
        # logits, logits again (they are not kept), and the two gradients
        return {"bytes": read + out + (M + V) * D * e + 8 * M, "flops": 8 * kept * D * V}
    return {"bytes": read + out, "flops": 2 * kept * D * V}


# ---- the same results from the definitions, in 64 bits, written apart from the plain form

def _exact_lora(s):
    c, ids = s["case"], s["adapters"]
    x, w = s["x"].double(), s["weight"].double()
    y = torch.mm(x, w)
    if s["bias"] is not None:
        y += s["bias"].double()
    out = {"y": y}
    if c["grad"]:
        dy = s["dy"].double()
        out["dx"] = torch.mm(dy, w.T)
        out["da"] = torch.zeros(s["a"].shape, dtype=torch.float64, device="cuda")
        out["db"] = torch.zeros(s["b"].shape, dtype=torch.float64, device="cuda")
    for i in range(c["adapters"]):
        rows = torch.nonzero(ids == i).squeeze(1)
        if rows.numel() == 0:
            continue
        a, b, scale = s["a"][i].double(), s["b"][i].double(), float(s["scales"][i])
        u = torch.mm(x[rows], a)
        y[rows] += scale * torch.mm(u, b)
        if c["grad"]:
            du = scale * torch.mm(dy[rows], b.T)
            out["dx"][rows] += torch.mm(du, a.T)
            out["da"][i] = torch.mm(x[rows].T, du)
            out["db"][i] = scale * torch.mm(u.T, dy[rows])
    return out


def _exact_logp(s):
    c = s["case"]
    x, w, t, M = s["x"].double(), s["table"].double(), s["tokens"], s["case"]["tokens"]
    kept = torch.nonzero(t >= 0).squeeze(1)
    out = {"top_ids": None, "top_log_probs": None, "log_probs": torch.zeros(M, dtype=torch.float64, device="cuda"),
           "entropy": torch.zeros(M, dtype=torch.float64, device="cuda")}
    logits = torch.mm(x[kept], w.T)
    if c["top"]:
        best = torch.topk(logits, c["top"], dim=1)
        out["top_ids"] = torch.full((M, c["top"]), -1, dtype=torch.long, device="cuda")
        out["top_ids"][kept] = best.indices
    logits /= c["temperature"]
    logp = torch.log_softmax(logits, 1)
    del logits
    out["log_probs"][kept] = logp[torch.arange(kept.numel(), device="cuda"), t[kept]]
    if c["top"]:
        out["top_log_probs"] = torch.zeros((M, c["top"]), dtype=torch.float64, device="cuda")
        out["top_log_probs"][kept] = torch.gather(logp, 1, best.indices)
    p = torch.exp(logp)
    ent = -torch.einsum("mv,mv->m", p, logp)
    out["entropy"][kept] = ent
    if not c["grad"]:
        return out
    gl = s["dlogp"].double()[kept]
    # d log p[t] = onehot - p;  d entropy = -p (log p + entropy)
    if s["dentropy"] is not None:
        ge = s["dentropy"].double()[kept]
        logp += ent[:, None]
        logp *= ge[:, None]
        logp += gl[:, None]
        p *= logp
    else:
        p *= gl[:, None]
    del logp
    p /= c["temperature"]
    step = gl / c["temperature"]
    out["dx"] = torch.zeros(M, c["width"], dtype=torch.float64, device="cuda")
    out["dx"][kept] = step[:, None] * w[t[kept]] - torch.mm(p, w)
    out["dtable"] = -torch.mm(p.T, x[kept])
    out["dtable"].index_add_(0, t[kept], step[:, None] * x[kept])
    return out


def _exact_clip(s):
    parts = [torch.linalg.vector_norm(t.double()) for t in s["grads"]]
    norm = torch.linalg.vector_norm(torch.stack(parts))
    factor = min(1.0, s["case"]["max_norm"] / (float(norm) + CLIP_EPS))
    return {"norm": norm, "grads": [t.double() * factor for t in s["flat"]]}


def exact(case, seed):
    return {"lora": _exact_lora, "logp": _exact_logp, "clip": _exact_clip}[case["op"]](prepare(case, seed))
