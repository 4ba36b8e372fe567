"""Cases that time the operators between a model's outputs and the step that updates it, and those
operators in their plain form.

    score        log probabilities of given tokens, with their distribution's entropy and its top
                 alternatives: what a worker reports beside its answers, and a trainer's forward pass
    grad         the logits' gradient from those of the log probabilities and the entropy
    route        a mixture's router: the experts of each token and their weights, how many tokens
                 each expert got, and the balance loss
    route_train  the same with the gradient of the router's logits

Where `own` is false, `run` computes them with elementary torch operations in 32 bits; where it
is true, it calls the library.
"""
from __future__ import annotations

import math
import random

import torch

own = False

BALANCE = 0.01                   # the balance loss's share of a training loss


def listed():
    return [
        # ---- log probabilities
        # one new token of one request, with its alternatives: the latency of a call
        dict(name="score_1row_top20", op="score", rows=1, vocab=151936, pad=0, dtype="bf16", top=20,
             entropy=False, temperature=0.7, each=False, left=0.0, masked=0.0),
        # a batch of single tokens: temperatures of their own, a third of the rows confined to a
        # grammar's few tokens
        dict(name="score_64rows_top20", op="score", rows=64, vocab=151936, pad=0, dtype="bf16",
             top=20, entropy=True, temperature=1.0, each=True, left=0.0, masked=0.33),
        # prompts scored in 32 bits, odd vocabulary in padded rows, padding between the prompts
        dict(name="score_1500rows_odd_fp32", op="score", rows=1500, vocab=32001, pad=63,
             dtype="fp32", top=5, entropy=False, temperature=1.0, each=False, left=0.25, masked=0.0),
        # answers behind long prompts: most rows are left out
        dict(name="score_4096rows_left", op="score", rows=4096, vocab=32000, pad=0, dtype="bf16",
             top=0, entropy=True, temperature=1.0, each=False, left=0.6, masked=0.0),
        # a trainer's forward pass, the largest
        dict(name="score_8192rows", op="score", rows=8192, vocab=151936, pad=0, dtype="bf16", top=0,
             entropy=True, temperature=1.0, each=False, left=0.0, masked=0.0),
        # ---- their gradient
        # an ordinary micro-batch of a policy gradient, prompts left out
        dict(name="grad_2048rows", op="grad", rows=2048, vocab=32000, pad=0, dtype="bf16",
             entropy=False, temperature=1.0, each=False, left=0.25, masked=0.0),
        # odd vocabulary, 32 bits, another temperature
        dict(name="grad_333rows_odd_fp32", op="grad", rows=333, vocab=32001, pad=0, dtype="fp32",
             entropy=True, temperature=0.8, each=False, left=0.1, masked=0.0),
        # a large vocabulary with an entropy bonus
        dict(name="grad_4096rows", op="grad", rows=4096, vocab=151936, pad=0, dtype="bf16",
             entropy=True, temperature=1.0, each=False, left=0.0, masked=0.0),
        # ---- routers
        # a decode batch: the latency of a call
        dict(name="route_64tokens", op="route", tokens=64, experts=128, k=8, dtype="bf16",
             normalize=True, padding=0.0),
        # long prompts of many requests
        dict(name="route_262144tokens", op="route", tokens=262144, experts=128, k=8, dtype="bf16",
             normalize=True, padding=0.0),
        # odd sizes, weights that are the probabilities themselves, padded sequences
        dict(name="route_train_5001tokens_odd", op="route_train", tokens=5001, experts=60, k=4,
             dtype="fp32", normalize=False, padding=0.2),
        # a training step's micro-batch with router logits in 32 bits
        dict(name="route_train_32768tokens", op="route_train", tokens=32768, experts=128, k=8,
             dtype="fp32", normalize=True, padding=0.1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(["score", "score", "grad", "grad", "route", "route_train"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("route", "route_train"):
        experts = _log_int(rng, 4, 512)
        experts = max(4, experts // 8 * 8) if rng.random() < 0.7 else experts
        return dict(op=op, tokens=_log_int(rng, 1, 65536), experts=experts,
                    k=_log_int(rng, 1, min(16, experts)), dtype=dtype,
                    normalize=rng.random() < 0.6, padding=rng.choice([0.0, 0.0, 0.1, 0.5]))
    vocab = _log_int(rng, 1000, 160000)
    vocab = vocab // 64 * 64 if rng.random() < 0.6 else vocab
    rows = _log_int(rng, 1, min(4096, 300_000_000 // vocab))
    case = dict(op=op, rows=rows, vocab=vocab, pad=rng.choice([0, 0, 0, -vocab % 64, 8]),
                dtype=dtype, entropy=rng.random() < 0.5, temperature=rng.choice([1.0, 1.0, 0.6, 1.3]),
                each=rng.random() < 0.3, left=rng.choice([0.0, 0.0, 0.25, 0.6]),
                masked=rng.choice([0.0, 0.0, 0.0, 0.3]))
    if op == "score":
        case["top"] = rng.choice([0, 0, 1, 5, 20, rng.randint(1, 32)])
    return case


# ------------------------------------------------------------------------------------- inputs

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_CHUNK = 1 << 28                 # elements of a chunk of rows


def _left_out(case):
    return int(case["rows"] * case["left"])


def _prepare_tokens(case, gen):
    rows, vocab = case["rows"], case["vocab"]

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=gen, device="cuda") * (hi - lo) + lo

    memory = torch.empty(rows, vocab + case["pad"], dtype=_TYPES[case["dtype"]], device="cuda")
    memory[:, vocab:] = 0
    s = dict(case=case, logits=memory[:, :vocab])
    tokens = torch.empty(rows, dtype=torch.int64, device="cuda")
    confined = uniform(rows) < case["masked"]
    step = max(1, _CHUNK // vocab)
    for a in range(0, rows, step):
        b = min(rows, a + step)
        # some rows near one-hot, some flat; a few likely tokens; a level of its own each
        z = torch.randn(b - a, vocab, generator=gen, device="cuda") * uniform(b - a, 1, lo=0.5, hi=2.5)
        likely = torch.randint(vocab, (b - a, 8), generator=gen, device="cuda")
        z.scatter_(1, likely, uniform(b - a, 8, lo=4.0, hi=16.0))
        z += uniform(b - a, 1, lo=-5.0, hi=5.0)
        if case["masked"]:
            allowed = torch.zeros(b - a, vocab, dtype=torch.bool, device="cuda")
            few = torch.randint(vocab, (b - a, 300), generator=gen, device="cuda")
            allowed.scatter_(1, few, True)
            z.masked_fill_(confined[a:b, None] & ~allowed, -math.inf)
        s["logits"][a:b] = z
        # tokens as they are sampled from these rows
        z = torch.exp(z - z.amax(1, keepdim=True))
        tokens[a:b] = (z / torch.empty_like(z).exponential_(generator=gen)).argmax(1)
    tokens[torch.randperm(rows, generator=gen, device="cuda")[:_left_out(case)]] = -1
    s["tokens"] = tokens
    s["temperature"] = uniform(rows, lo=0.5, hi=1.5) if case["each"] else case["temperature"]
    if case["op"] == "grad":
        s["d_logprobs"] = torch.randn(rows, generator=gen, device="cuda") * 0.1
        s["d_entropy"] = torch.full((rows,), -0.01, device="cuda") if case["entropy"] else None
        s["saved"] = torch.empty(2, rows, device="cuda")       # what the forward pass keeps
        for a in range(0, rows, step):
            s["saved"][:, a:a + step] = torch.stack(_statistics(s, a, a + step)[1:])
        s["out"] = torch.empty_like(memory)[:, :vocab]
    if own:
        import lossless_bf16_weight_old_gb300 as bd
        s["scores"] = bd.TokenLogprobs(rows, vocab, top=case.get("top", 0), entropy=case["entropy"])
        if case["op"] == "grad":
            s["scores"].run(s["logits"], tokens, s["temperature"])
    return s


def _prepare_router(case, gen):
    t, e = case["tokens"], case["experts"]

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * scale

    s = dict(case=case)
    # some experts are likelier than others
    s["logits"] = (normal(t, e, scale=1.5) + normal(1, e, scale=0.7)).to(_TYPES[case["dtype"]])
    s["mask"] = None
    if case["padding"]:
        s["mask"] = torch.ones(t, dtype=torch.bool, device="cuda")
        s["mask"][torch.randperm(t, generator=gen, device="cuda")[:int(t * case["padding"])]] = False
    if case["op"] == "route_train":
        s["d_weights"] = normal(t, case["k"], scale=0.05)
        s["out"] = torch.empty_like(s["logits"])
    if own:
        import lossless_bf16_weight_old_gb300 as bd
        s["routing"] = bd.ExpertRouting(t, e, case["k"], normalize=case["normalize"])
    return s


# --------------------------------------------------------------------------------- plain forms

def _order(x):
    """Whole numbers that order values, and equal values by their place, the lowest first."""
    i = (x.float() + 0.0).view(torch.int32).to(torch.int64)
    i = torch.where(i < 0, i ^ 0x7FFFFFFF, i)
    places = torch.arange(x.shape[1], device=x.device)
    return i * (1 << 20) + ((1 << 20) - 1 - places)


def _greatest(x, k):
    """Places of the k greatest of each row, in order."""
    best = _order(x).topk(k, dim=1).values
    return (1 << 20) - 1 - (best & ((1 << 20) - 1))


def _heat(s, a=0, b=None):
    t = s["temperature"]
    return t[a:b, None] if s["case"]["each"] else t


def _statistics(s, a=0, b=None):
    """Scaled logits, their log-sum-exp and the entropy, by rows."""
    z = s["logits"][a:b].float() / _heat(s, a, b)
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1)
    mean = torch.where(e > 0, e * (z - top), 0.0).sum(1) / total
    return z, top.squeeze(1) + total.log(), total.log() - mean


def _run_score(s):
    case, tokens = s["case"], s["tokens"]
    if own:
        r = s["scores"]
        r.run(s["logits"], tokens, s["temperature"])
        out = dict(logprobs=r.logprobs)
        if case["entropy"]:
            out["entropy"] = r.entropy
        if case["top"]:
            out.update(top_logprobs=r.top_logprobs, top_tokens=r.top_tokens)
        return out
    z, lse, entropy = _statistics(s)
    has = tokens >= 0
    given = z.gather(1, tokens.clamp(min=0)[:, None]).squeeze(1)
    out = dict(logprobs=torch.where(has, given - lse, 0.0))
    if case["entropy"]:
        out["entropy"] = torch.where(has, entropy, 0.0)
    if case["top"]:
        places = _greatest(s["logits"], case["top"])
        best = z.gather(1, places) - lse[:, None]
        out["top_logprobs"] = torch.where(has[:, None], best, 0.0)
        out["top_tokens"] = torch.where(has[:, None], places, -1).int()
    return out


def _run_grad(s):
    if own:
        return s["scores"].backward(s["logits"], s["d_logprobs"], s["d_entropy"], out=s["out"])
    tokens = s["tokens"]
    has = (tokens >= 0)[:, None]
    lse, entropy = s["saved"]
    logp = s["logits"].float() / _heat(s) - lse[:, None]
    p = torch.exp(logp)
    g = s["d_logprobs"][:, None]
    d = -g * p
    if s["d_entropy"] is not None:
        d -= s["d_entropy"][:, None] * torch.where(p > 0, p * (logp + entropy[:, None]), 0.0)
    d.scatter_add_(1, tokens.clamp(min=0)[:, None], g)
    s["out"].copy_(torch.where(has, d / _heat(s), 0.0))
    return s["out"]


def _run_router(s):
    case = s["case"]
    train = case["op"] == "route_train"
    if own:
        r = s["routing"]
        r.run(s["logits"], s["mask"])
        out = dict(weights=r.weights, experts=r.experts, counts=r.counts, probs=r.probs, loss=r.loss)
        if train:
            out["d_logits"] = r.backward(s["logits"], s["d_weights"], BALANCE, out=s["out"])
        return out
    t, e, k = case["tokens"], case["experts"], case["k"]
    z = s["logits"].float()
    p = torch.exp(z - z.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    places = _greatest(s["logits"], k)
    w = p.gather(1, places)
    total = w.sum(1, keepdim=True) if case["normalize"] else 1.0
    w = w / total
    real = torch.ones(t, 1, device="cuda") if s["mask"] is None else s["mask"][:, None].float()
    n = real.sum()
    chosen = torch.zeros(t, e, device="cuda").scatter_(1, places, real.expand(t, k))
    counts = chosen.sum(0)
    probs = (p * real).sum(0) / n
    share = counts / (n * k)
    out = dict(weights=w * real, experts=torch.where(real > 0, places, -1).int(), counts=counts.int(),
               probs=probs, loss=e * (share * probs).sum().reshape(1))
    if train:
        dw = s["d_weights"]
        if case["normalize"]:
            d = torch.zeros(t, e, device="cuda").scatter_(1, places, w * (dw - (w * dw).sum(1, keepdim=True)))
            dp = (BALANCE * e / n * share)[None, :].expand(t, e)
        else:
            d = 0.0
            dp = (BALANCE * e / n * share)[None, :].repeat(t, 1).scatter_add_(1, places, dw)
        d = (d + p * (dp - (p * dp).sum(1, keepdim=True))) * real
        s["out"].copy_(d)
        out["d_logits"] = s["out"]
    return out


# --------------------------------------------------------------------------- exact, in 64 bits

def _exact_tokens(s):
    case, parts = s["case"], []
    rows, vocab = case["rows"], case["vocab"]
    step = max(1, (1 << 26) // vocab)
    heat = s["temperature"].double() if case["each"] else torch.full((rows,), case["temperature"]).double().cuda()
    for a in range(0, rows, step):
        x, t = s["logits"][a:a + step].double(), s["tokens"][a:a + step]
        logp = torch.log_softmax(x / heat[a:a + step, None], 1)
        p = logp.exp()
        entropy = -(p * logp.masked_fill(p == 0, 0.0)).sum(1)
        out = t < 0
        row = torch.arange(x.shape[0], device="cuda")
        if case["op"] == "score":
            r = {"logprobs": logp[row, t.clamp(min=0)].masked_fill(out, 0.0)}
            if case["entropy"]:
                r["entropy"] = entropy.masked_fill(out, 0.0)
            if case["top"]:
                _, places = x.sort(dim=1, descending=True, stable=True)
                places = places[:, :case["top"]]
                r["top_logprobs"] = logp.gather(1, places).masked_fill(out[:, None], 0.0)
                r["top_tokens"] = places.masked_fill(out[:, None], -1).int()
        else:
            g = s["d_logprobs"][a:a + step].double()
            one = torch.zeros_like(p)
            one[row, t.clamp(min=0)] = 1.0
            d = g[:, None] * (one - p)
            if case["entropy"]:
                h = s["d_entropy"][a:a + step].double()
                d -= h[:, None] * p * (logp.masked_fill(p == 0, 0.0) + entropy[:, None])
            r = {"out": (d / heat[a:a + step, None]).masked_fill(out[:, None], 0.0)}
            if rows * vocab > 1 << 28:     # (half the memory, and still 2^-24)
                r["out"] = r["out"].float()
        parts.append(r)
    both = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    return both if case["op"] == "score" else both["out"]


def _exact_router(s):
    case = s["case"]
    t, e, k = case["tokens"], case["experts"], case["k"]
    x = s["logits"].double()
    mask = torch.ones(t, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    n = int(mask.sum())
    p = torch.softmax(x, 1)
    places = x.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, places)
    if case["normalize"]:
        w = w / w.sum(1, keepdim=True)
    counts = torch.bincount(places[mask].reshape(-1), minlength=e)
    probs = p[mask].mean(0)
    f = counts.double() / (n * k)
    out = dict(weights=w.masked_fill(~mask[:, None], 0.0), experts=places.masked_fill(~mask[:, None], -1).int(),
               counts=counts.int(), probs=probs, loss=e * torch.dot(f, probs).reshape(1))
    if case["op"] == "route_train":
        dw = s["d_weights"].double()
        if case["normalize"]:              # w = p_i / q, q = the sum of the chosen ones
            q = p.gather(1, places).sum(1, keepdim=True)
            dw = (dw - (dw * w).sum(1, keepdim=True)) / q
        dp = (BALANCE * e / n * f).expand(t, e).clone()
        dp.scatter_add_(1, places, dw)
        out["d_logits"] = (p * (dp - (p * dp).sum(1, keepdim=True))).masked_fill(~mask[:, None], 0.0)
    return out


# ------------------------------------------------------------------------------------ interface

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return _prepare_router(case, gen) if case["op"].startswith("route") else _prepare_tokens(case, gen)


def run(state):
    op = state["case"]["op"]
    return _run_score(state) if op == "score" else _run_grad(state) if op == "grad" else _run_router(state)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_router(s) if case["op"].startswith("route") else _exact_tokens(s)


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("route"):
        t, e, k = case["tokens"], case["experts"], case["k"]
        real = t - int(t * case["padding"])
        work = {"bytes": real * e * size + t * k * 8 + (t if case["padding"] else 0) + 8 * e, "flops": 6 * real * e}
        if case["op"] == "route_train":    # the weights' gradients in, the logits' out
            work["bytes"] += real * k * 4 + t * e * size
            work["flops"] += 8 * real * e
        return work
    rows, vocab = case["rows"], case["vocab"]
    real = rows - _left_out(case)
    if case["op"] == "score":
        return {"bytes": real * vocab * size + rows * (12 + (4 if case["entropy"] else 0) + 8 * case["top"]),
                "flops": real * vocab * (6 if case["entropy"] else 4)}
    return {"bytes": (real + rows) * vocab * size + rows * 20, "flops": real * vocab * (9 if case["entropy"] else 5)}
