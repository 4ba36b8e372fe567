"""Cases that time the operators around the weight sync, and those operators in their plain form.

    adamw   one AdamW step over many tensors at once (states in 32 or in 8 bits, with or without
            clipping by the global gradient norm): what a trainer runs before the compress
    serve   low-rank adapters of many requests added to a shared projection's output
    train   the same with the backward pass: a training step of adapters

Where `own` is false, `run` computes them with elementary torch operations in 32 bits; where it
is true, it calls the library.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

BLOCK = 256                      # elements that share a scale in the 8-bit states
GAMMA = 0x9E3779B97F4A7C15
LR, BETA1, BETA2, EPS, DECAY, MAX_NORM = 1e-4, 0.9, 0.95, 1e-8, 0.1, 1.0
FIRST_STEP, NOISE_SEED = 100, 1234


def listed():
    return [
        # ---- AdamW, 32-bit states
        # the adapters of one decoder layer, rank 8: 14 small tensors, the latency of a step
        dict(name="adamw32_adapters_1layer", op="adamw", bits=32, kind="adapters", layers=1,
             hidden=4096, inter=11008, rank=8, experts=0, weights="master", grads="bf16",
             clip=False, stochastic=False),
        # two layers of the 7B decoder with their norms, clipped: an ordinary trainer shard
        dict(name="adamw32_dense_2layers_clip", op="adamw", bits=32, kind="dense", layers=2,
             hidden=4096, inter=11008, rank=0, experts=0, weights="master", grads="bf16",
             clip=True, stochastic=False),
        # one layer of the 30B mixture of experts: 389 tensors, the largest step
        dict(name="adamw32_experts_1layer", op="adamw", bits=32, kind="experts", layers=1,
             hidden=2048, inter=768, rank=0, experts=128, weights="master", grads="bf16",
             clip=False, stochastic=False),
        # odd sizes throughout, 32-bit weights and gradients
        dict(name="adamw32_odd_fp32", op="adamw", bits=32, kind="dense", layers=3, hidden=1001,
             inter=2731, rank=0, experts=0, weights="fp32", grads="fp32", clip=True,
             stochastic=False),
        # ---- AdamW, 8-bit states (a pass is a step and the read-out of both moments, as a
        # checkpoint takes them)
        dict(name="adamw8_dense_1layer_clip", op="adamw", bits=8, kind="dense", layers=1,
             hidden=4096, inter=11008, rank=0, experts=0, weights="master", grads="bf16",
             clip=True, stochastic=False),
        # adapters of a whole 32-layer model, BF16 weights alone with stochastic rounding
        dict(name="adamw8_adapters_32layers", op="adamw", bits=8, kind="adapters", layers=32,
             hidden=4096, inter=11008, rank=16, experts=0, weights="bf16", grads="bf16",
             clip=False, stochastic=True),
        # ---- adapters, serving
        # one new token of one request
        dict(name="serve_1row", op="serve", rows=1, requests=1, adapters=1, rank=16, mixed=False,
             hidden=4096, out=4096, none=0.0),
        # a batch of single tokens, nearly each request with an adapter of its own, a few without
        dict(name="serve_decode_64rows", op="serve", rows=64, requests=64, adapters=48, rank=16,
             mixed=False, hidden=4096, out=11008, none=0.1),
        # ragged chunks of prompts of several requests, adapters of different rank
        dict(name="serve_ragged_1500rows", op="serve", rows=1500, requests=9, adapters=5,
             rank=32, mixed=True, hidden=2048, out=4096, none=0.1),
        # long prompts
        dict(name="serve_16384rows", op="serve", rows=16384, requests=24, adapters=8, rank=64,
             mixed=False, hidden=4096, out=14336, none=0.0),
        # ---- adapters, training
        dict(name="train_2048rows", op="train", rows=2048, requests=1, adapters=1, rank=16,
             mixed=False, hidden=4096, out=4096, none=0.0),
        # several policies' adapters in one batch of sequences, odd row count
        dict(name="train_8191rows_4adapters", op="train", rows=8191, requests=16, adapters=4,
             rank=64, mixed=False, hidden=4096, out=11008, none=0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A layer's width: mostly a multiple of 64, sometimes of 8, sometimes anything."""
    n, p = _log_int(rng, lo, hi), rng.random()
    m = 64 if p < 0.7 else 8 if p < 0.85 else 1
    return max(lo, n // m * m)


def draw(rng: random.Random):
    op = rng.choice(["adamw", "adamw", "serve", "serve", "train"])
    if op == "adamw":
        kind = rng.choice(["adapters", "dense", "experts"])
        weights = rng.choice(["master", "master", "bf16", "fp32"])
        c = dict(op=op, bits=rng.choice([32, 8]), kind=kind, layers=1, hidden=_width(rng, 256, 4096),
                 inter=_width(rng, 512, 8192), rank=0, experts=0, weights=weights,
                 grads=rng.choice(["bf16", "fp32"]), clip=rng.random() < 0.5,
                 stochastic=weights == "bf16" and rng.random() < 0.7)
        if kind == "adapters":
            c["layers"], c["rank"] = _log_int(rng, 1, 32), _log_int(rng, 1, 64)
        elif kind == "experts":
            c["hidden"], c["inter"] = _width(rng, 256, 2048), _width(rng, 128, 1024)
            c["experts"] = _log_int(rng, 2, 64)
        return c
    rows = _log_int(rng, 1 if op == "serve" else 64, 8192)
    requests = _log_int(rng, 1, max(1, min(rows, 256)))
    return dict(op=op, rows=rows, requests=requests,
                adapters=_log_int(rng, 1, 64 if op == "serve" else 8), rank=_log_int(rng, 1, 64),
                mixed=rng.random() < 0.5, hidden=_width(rng, 256, 8192), out=_width(rng, 256, 8192),
                none=rng.choice([0.0, 0.0, 0.1, 0.5]))


# ------------------------------------------------------------------------------ AdamW: inputs

def _shapes(case):
    """(shape, weight decay) of every tensor of a step."""
    h, f, r = case["hidden"], case["inter"], case["rank"]
    if case["kind"] == "adapters":
        wide = [(h, h)] * 4 + [(h, f)] * 2 + [(f, h)]          # in, out of each projection
        one = [s for i, o in wide for s in (((r, i), 0.0), ((o, r), 0.0))]
    elif case["kind"] == "dense":
        one = [((h, h), DECAY)] * 4 + [((f, h), DECAY)] * 2 + [((h, f), DECAY), ((h,), 0.0), ((h,), 0.0)]
    else:
        one = [((f, h), DECAY), ((f, h), DECAY), ((h, f), DECAY)] * case["experts"]
        one = one + [((2 * h, h), DECAY), ((h // 4, h), DECAY), ((h // 4, h), DECAY),
                     ((h, 2 * h), DECAY), ((case["experts"], h), DECAY)]
    return one * case["layers"]


def _views(arena, shapes):
    """The tensors of a step, each starting at a block of the flat arena that holds them all."""
    numels = [math.prod(s) for s, _ in shapes]
    starts = np.cumsum([0] + [-(-n // BLOCK) * BLOCK for n in numels])
    return [arena[b:b + n].view(s) for b, n, (s, _) in zip(starts.tolist(), numels, shapes)]


def _prepare_adamw(case, gen):
    shapes = _shapes(case)
    numels = torch.tensor([math.prod(s) for s, _ in shapes])
    blocks = -(-numels // BLOCK)
    total = int(blocks.sum())

    def normal(scale):
        return torch.randn(total * BLOCK, generator=gen, device="cuda") * scale

    # which elements are padding behind a tensor's end: zero in every arena, and stay zero
    within = torch.arange(total) - torch.repeat_interleave(torch.cumsum(blocks, 0) - blocks, blocks)
    used = (torch.repeat_interleave(numels, blocks) - within * BLOCK).clamp(max=BLOCK).cuda()
    real = (torch.arange(BLOCK, device="cuda")[None, :] < used[:, None]).reshape(-1)
    # gradients whose size differs from block to block, as those of different rows do; one tenth
    # of the blocks have none at all (rows of a table, or experts, that no token reached)
    size = torch.exp(torch.randn(total, 1, generator=gen, device="cuda")) * 1e-4
    size = size * (torch.rand(total, 1, generator=gen, device="cuda") > 0.1)

    def sized(x):
        return (x.view(-1, BLOCK) * size).view(-1)

    s = dict(case=case, step=FIRST_STEP)
    grads = sized(normal(1.0)) * real
    s["grads"] = grads.bfloat16() if case["grads"] == "bf16" else grads
    del grads
    weights = normal(0.02) * real
    s["weights"] = weights if case["weights"] == "fp32" else weights.bfloat16()
    if case["weights"] == "master":
        s["master"] = weights
    del weights
    m, v = sized(normal(0.3)) * real, sized(normal(1.0)).square_() * real
    if case["bits"] == 32:
        s["m"], s["v"] = m, v
    else:
        m, v = m.view(-1, BLOCK), v.view(-1, BLOCK)
        s["m_scale"], s["v_scale"] = m.abs().amax(1), v.amax(1)
        s["m"], s["v"] = torch.empty(total * BLOCK, dtype=torch.int8, device="cuda"), torch.empty(total * BLOCK, dtype=torch.uint8, device="cuda")
        s["m"].copy_((_ratio(m.abs(), s["m_scale"]).sqrt() * 127).round().mul_(m.sign()).view(-1))
        s["v"].copy_((_ratio(v, s["v_scale"]).sqrt().sqrt() * 255).ceil().clamp_(max=255).view(-1))
    del m, v
    decays = [d for _, d in shapes]
    s["decay"] = torch.repeat_interleave(torch.tensor(decays), blocks).cuda().unsqueeze(1)
    if own:
        import lossless_bf16_weight_old_gb300 as bd
        state = {k: s[k] for k in ("master", "m", "v", "m_scale", "v_scale") if k in s}
        s["adam"] = bd.AdamWBatch(
            _views(s["weights"], shapes), _views(s["grads"], shapes), state=state,
            state_bits=case["bits"], master=case["weights"] == "master", lr=LR,
            betas=(BETA1, BETA2), eps=EPS, weight_decay=decays,
            max_norm=MAX_NORM if case["clip"] else None, stochastic=case["stochastic"],
            seed=NOISE_SEED, step=FIRST_STEP)
    return s


# --------------------------------------------------------------------------- AdamW: plain form

def _ratio(x, scale):
    """x / scale by rows, zero where the scale is zero."""
    return torch.where(scale[:, None] > 0, x / scale[:, None], torch.zeros((), device=x.device))


def _signed(x):
    x &= (1 << 64) - 1
    return x - (1 << 64) if x >> 63 else x


def _shift(x, k):
    return (x >> k) & ((1 << (64 - k)) - 1)


def _mix(z):
    """SplitMix64's output function on int64 tensors (whose products wrap)."""
    z = (z ^ _shift(z, 30)) * _signed(0xBF58476D1CE4E5B9)
    z = (z ^ _shift(z, 27)) * _signed(0x94D049BB133111EB)
    return z ^ _shift(z, 31)


def _noise(count, step):
    """32 random bits for each of `count` elements, as int64: two to a draw of the stream."""
    key = _mix(torch.tensor(_signed(NOISE_SEED ^ (step * GAMMA)), device="cuda"))
    j = torch.arange(1, count // 2 + 1, device="cuda")
    r = _mix(key + j * _signed(GAMMA))
    return torch.stack([r & 0xFFFFFFFF, _shift(r, 32)], 1).view(-1)


def _round_stochastic(x, bits16):
    """BF16 values next to x, away from zero with the probability of the part cut off."""
    whole = x.contiguous().view(torch.int32).to(torch.int64) & 0xFFFFFFFF
    cut = (whole + bits16) >> 16
    return (cut - ((cut >> 15) << 16)).to(torch.int16).view(torch.bfloat16)


def _run_adamw(s):
    case = s["case"]
    if own:
        s["adam"].run()
        out = {k: s[k] for k in ("weights", "master") if k in s}
        if case["bits"] == 32:
            return {**out, "m": s["m"], "v": s["v"]}
        m, v = s["adam"].moments(dtype=torch.bfloat16)
        return {**out, "m": m, "v": v}
    s["step"] += 1
    t = s["step"]
    g = s["grads"].float().view(-1, BLOCK)
    if case["clip"]:
        norm = g.square().sum().sqrt()
        g = g * (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)
    m, v = s["m"].float().view(-1, BLOCK), s["v"].float().view(-1, BLOCK)
    if case["bits"] == 8:
        m = m * m.abs() * (1 / 127 ** 2) * s["m_scale"][:, None]
        v = (v * (1 / 255)).square().square() * s["v_scale"][:, None]
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g.square() * (1 - BETA2)
    p = (s["master"] if "master" in s else s["weights"].float()).view(-1, BLOCK)
    update = (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
    p = p * (1 - LR * s["decay"]) - LR * update
    noise = _noise(p.numel(), t) if case["bits"] == 8 or case["stochastic"] else None
    if "master" in s:
        s["master"].copy_(p.view(-1))
    if case["stochastic"]:
        s["weights"].copy_(_round_stochastic(p.view(-1), noise & 0xFFFF))
    else:
        s["weights"].copy_(p.view(-1))
    out = {k: s[k] for k in ("weights", "master") if k in s}
    if case["bits"] == 32:
        s["m"].copy_(m.view(-1))
        s["v"].copy_(v.view(-1))
        return {**out, "m": s["m"], "v": s["v"]}
    sm, sv = m.abs().amax(1), v.amax(1)
    cm = (_ratio(m.abs(), sm).sqrt() * 127).round() * m.sign()
    x = _ratio(v, sv)
    low = (x.sqrt().sqrt() * 255).floor().clamp(max=254)
    a, b = (low * (1 / 255)).square().square(), ((low + 1) * (1 / 255)).square().square()
    up = (noise >> 16).float().view(-1, BLOCK) * (1 / 65536) * (b - a) < x - a
    cv = torch.where(v > 0, (low + up).clamp(min=1), torch.zeros((), device="cuda"))
    s["m"].copy_(cm.view(-1))
    s["v"].copy_(cv.view(-1))
    s["m_scale"].copy_(sm)
    s["v_scale"].copy_(sv)
    out["m"] = (cm * cm.abs() * (1 / 127 ** 2) * sm[:, None]).bfloat16().view(-1)
    out["v"] = ((cv * (1 / 255)).square().square() * sv[:, None]).bfloat16().view(-1)
    return out


def _exact_noise(count, step):
    """The random bits once more, on the host in unsigned 64 bits."""
    with np.errstate(over="ignore"):
        def mix(z):
            z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
            z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
            return z ^ (z >> np.uint64(31))
        key = mix(np.array([NOISE_SEED ^ ((step * GAMMA) & ((1 << 64) - 1))], dtype=np.uint64))
        parts = []
        for j0 in range(0, count // 2, 1 << 22):
            j = np.arange(j0 + 1, min(count // 2, j0 + (1 << 22)) + 1, dtype=np.uint64)
            parts.append(mix(key + j * np.uint64(GAMMA)).view(np.int64))
    r = torch.from_numpy(np.concatenate(parts)).cuda()
    halves = r.view(torch.int32).to(torch.int64) & 0xFFFFFFFF   # little-endian: low half first
    return halves & 0xFFFF, halves >> 16


def _exact_adamw(s):
    case, t = s["case"], FIRST_STEP + 1
    d = torch.float64
    g = s["grads"].to(d)
    if case["clip"]:
        norm = math.sqrt(float((g * g).sum()))
        g *= min(1.0, MAX_NORM / (norm + 1e-6))
    m, v = s["m"].to(d), s["v"].to(d)
    if case["bits"] == 8:
        m = torch.sign(m) * (m / 127) ** 2 * s["m_scale"].to(d).repeat_interleave(BLOCK)
        v = (v / 255) ** 4 * s["v_scale"].to(d).repeat_interleave(BLOCK)
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    del g
    p = (s["master"] if "master" in s else s["weights"]).to(d)
    decay = s["decay"].to(d).repeat_interleave(BLOCK, 0).view(-1)
    p = p - LR * (decay * p + (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS))
    del decay
    low16, high16 = _exact_noise(p.numel(), t) if case["bits"] == 8 or case["stochastic"] else (None, None)
    out = {"weights": p}
    if case["stochastic"]:
        step = torch.exp2(torch.floor(torch.log2(p.abs().clamp(min=2.0 ** -126))) - 7)
        down = torch.floor(p.abs() / step)
        frac = torch.floor((p.abs() / step - down) * 65536)
        out["weights"] = torch.sign(p) * (down + (frac + low16 >= 65536)) * step
    if "master" in s:
        out["master"] = p
    if case["bits"] == 32:
        return {**out, "m": m, "v": v}
    sm = m.abs().view(-1, BLOCK).amax(1).float().to(d).repeat_interleave(BLOCK)
    sv = v.view(-1, BLOCK).amax(1).float().to(d).repeat_interleave(BLOCK)
    qm = torch.where(sm > 0, m.abs() / sm, 0.0)
    out["m"] = torch.sign(m) * (torch.round(127 * qm.sqrt()) / 127) ** 2 * sm
    del qm, m, sm
    qv = torch.where(sv > 0, v / sv, 0.0)
    low = torch.floor(255 * qv ** 0.25).clamp(max=254)
    chance = (qv - (low / 255) ** 4) / (((low + 1) / 255) ** 4 - (low / 255) ** 4)
    code = torch.where(v > 0, (low + (high16 / 65536 < chance)).clamp(min=1), 0.0)
    out["v"] = (code / 255) ** 4 * sv
    return out


# ------------------------------------------------------------------------------ adapters: inputs

def _prepare_adapters(case, gen, seed):
    t, n, r, h, o = (case[k] for k in ("rows", "adapters", "rank", "hidden", "out"))
    host = random.Random(seed)
    cuts = sorted(host.sample(range(1, t), case["requests"] - 1))
    lengths = [b - a for a, b in zip([0] + cuts, cuts + [t])]
    owner = [-1 if host.random() < case["none"] else host.randrange(n) for _ in lengths]
    index = np.repeat(np.array(owner, dtype=np.int64), lengths)     # adapter of each row
    ranks = [host.randint(1, r) if case["mixed"] and i else r for i in range(n)]

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).bfloat16()

    real = (torch.arange(r)[None, :] < torch.tensor(ranks)[:, None]).cuda()
    s = dict(case=case, ranks=ranks)
    s["x"], s["y"] = normal(t, h), normal(t, o)                     # y: the projection's output
    s["a"] = normal(n, r, h, scale=h ** -0.5) * real[:, :, None]
    s["b"] = normal(n, o, r, scale=0.25 * r ** -0.5) * real[:, None, :]
    scales = [2.0 ** host.choice([-1, 0, 1]) for _ in range(n)]
    s["scale"] = torch.tensor(scales, device="cuda")
    s["index"] = torch.from_numpy(index.astype(np.int32)).cuda()
    # the plain form's plan: rows grouped by adapter and padded to the largest group
    groups = [np.flatnonzero(index == i) for i in range(n)]
    most = max(1, max(len(q) for q in groups))
    group, place = np.zeros((n, most), np.int64), np.zeros(t, np.int64)
    for i, q in enumerate(groups):
        group[i, :len(q)] = q
        place[q] = i * most + np.arange(len(q))
    s["group"], s["place"] = torch.from_numpy(group).cuda(), torch.from_numpy(place).cuda()
    s["valid"] = (torch.arange(most)[None, :] < torch.tensor([len(q) for q in groups])[:, None]).cuda().unsqueeze(2)
    s["has"] = (s["index"] >= 0).unsqueeze(1)
    if case["op"] == "train":
        s["dy"], s["dx"] = normal(t, o, scale=0.01), normal(t, h, scale=0.01)
        s["da"], s["db"] = torch.zeros_like(s["a"]), torch.zeros_like(s["b"])
    if own:
        import lossless_bf16_weight_old_gb300 as bd
        grads = {}
        if case["op"] == "train":
            grads = dict(d_downs=[s["da"][i, :k] for i, k in enumerate(ranks)],
                         d_ups=[s["db"][i, :, :k] for i, k in enumerate(ranks)])
        s["set"] = bd.AdapterSet([s["a"][i, :k] for i, k in enumerate(ranks)],
                                 [s["b"][i, :, :k] for i, k in enumerate(ranks)], scales, **grads)
        s["plan"] = bd.AdapterRows(s["index"], n)
        if case["op"] == "train":
            s["low"] = torch.empty(t, s["set"].rank, dtype=torch.bfloat16, device="cuda")
    return s


# --------------------------------------------------------------------------- adapters: plain form

def _run_adapters(s):
    train = s["case"]["op"] == "train"
    if own:
        import lossless_bf16_weight_old_gb300 as bd
        if not train:
            return bd.adapter_forward(s["x"], s["y"], s["set"], s["plan"])
        bd.adapter_forward(s["x"], s["y"], s["set"], s["plan"], low=s["low"])
        bd.adapter_backward(s["x"], s["dy"], s["low"], s["dx"], s["set"], s["plan"])
        return {k: s[k] for k in ("y", "dx", "da", "db")}
    a, b, scale = s["a"].float(), s["b"].float(), s["scale"][:, None, None]

    def spread(grouped):
        return torch.where(s["has"], grouped.reshape(-1, grouped.shape[2])[s["place"]], 0.0)

    x = s["x"][s["group"]].float() * s["valid"]                     # [n, most, hidden]
    u = torch.bmm(x, a.transpose(1, 2)) * scale
    s["y"].copy_(s["y"].float() + spread(torch.bmm(u, b.transpose(1, 2))))
    if not train:
        return s["y"]
    dy = s["dy"][s["group"]].float() * s["valid"]
    du = torch.bmm(dy, b) * scale
    s["dx"].copy_(s["dx"].float() + spread(torch.bmm(du, a)))
    s["da"].copy_(torch.bmm(du.transpose(1, 2), x))
    s["db"].copy_(torch.bmm(dy.transpose(1, 2), u))
    return {k: s[k] for k in ("y", "dx", "da", "db")}


def _exact_adapters(s):
    d = torch.float64
    x, y = s["x"].to(d), s["y"].to(d)
    train = s["case"]["op"] == "train"
    if train:
        dy, dx = s["dy"].to(d), s["dx"].to(d)
        da, db = torch.zeros_like(s["a"], dtype=d), torch.zeros_like(s["b"], dtype=d)
    index = s["index"].cpu()
    for i in range(s["case"]["adapters"]):
        rows = (index == i).nonzero().squeeze(1).cuda()
        a, b, scale = s["a"][i].to(d), s["b"][i].to(d), float(s["scale"][i])
        low = scale * (x[rows] @ a.T)
        y[rows] += low @ b.T
        if train:
            dlow = scale * (dy[rows] @ b)
            dx[rows] += dlow @ a
            da[i], db[i] = dlow.T @ x[rows], dy[rows].T @ low
    return dict(y=y, dx=dx, da=da, db=db) if train else y


# ------------------------------------------------------------------------------------ interface

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return _prepare_adamw(case, gen) if case["op"] == "adamw" else _prepare_adapters(case, gen, seed)


def run(state):
    return _run_adamw(state) if state["case"]["op"] == "adamw" else _run_adapters(state)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_adamw(s) if case["op"] == "adamw" else _exact_adapters(s)


def work(case):
    if case["op"] == "adamw":
        n = sum(math.prod(s) for s, _ in _shapes(case))
        weight = {"master": 4 + 4 + 2, "bf16": 4, "fp32": 8}[case["weights"]]
        # 8 bits: both codes and both blocks' scales in and out, then the moments' BF16 values
        state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK + 4
        return {"bytes": n * ((2 if case["grads"] == "bf16" else 4) + weight + state), "flops": n * 18}
    t, r, h, o = (case[k] for k in ("rows", "rank", "hidden", "out"))
    used = max(1, min(case["adapters"], case["requests"]))
    rows = t * (1 - case["none"])
    factors = used * r * (h + o) * 2
    if case["op"] == "serve":
        return {"bytes": rows * (h + 2 * o) * 2 + factors + 4 * t, "flops": 2 * rows * r * (h + o)}
    # x, dy once; y, dx in and out; the factors and their gradients
    return {"bytes": rows * (3 * h + 3 * o) * 2 + 2 * factors + 4 * t, "flops": 6 * rows * r * (h + o)}
