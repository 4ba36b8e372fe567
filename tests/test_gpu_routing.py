"""Routing to experts, counts, the balance loss and the gradient against their formulas in 64 bits
(GPU).

Tolerances, with u = 2^-24 (half an FP32 step): d = x - max carries one rounding and its product with
log2 e two, 2^x by the hardware 4 u, so e^d is off by (4 + 4 |d|) u of itself; a token's sum adds a
rounding for each of at most 32 + 5 additions, its reciprocal and the product two more."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("lossless_bf16_weight_old_gb300")

U = 2.0 ** -24
BF16, FP32 = torch.bfloat16, torch.float32
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    bd._ops_lib.load()


def _logits(tokens, experts, dtype, *, seed=0, ld=None, offset=0, scale=2.0):
    gen = torch.Generator(device="cuda").manual_seed(seed + 1000 * tokens + experts)
    ld = ld or experts
    memory = torch.empty(offset + tokens * ld + 64, dtype=dtype, device="cuda").fill_(77.0)
    x = memory[offset:offset + tokens * ld].view(tokens, ld)[:, :experts]
    x.copy_(torch.randn(tokens, experts, generator=gen, device="cuda") * scale)
    return x


def _reference(x, k, normalize, mask, gw=None, gl=0.0, counts=None):
    t, e = x.shape
    x = x.double()
    mask = torch.ones(t, dtype=torch.bool, device="cuda") if mask is None else mask.bool()
    mask = mask & (x > -INF).any(1)
    p = torch.softmax(x, 1).masked_fill(~mask[:, None], 0.0)
    places = (x + 0.0).sort(dim=1, descending=True, stable=True).indices[:, :k]
    chosen = p.gather(1, places)
    q = chosen.sum(1, keepdim=True).masked_fill(~mask[:, None], 1.0)
    w = chosen / q if normalize else chosen
    n = int(mask.sum())
    c = torch.bincount(places[mask].reshape(-1), minlength=e)
    probs = p.sum(0) / max(n, 1)
    r = dict(weights=w, experts=torch.where(mask[:, None], places, -1), counts=c, probs=probs, real=n,
             loss=e * float((c.double() / max(1, n * k) * probs).sum()), p=p, mask=mask,
             d=(x - x.amax(1, keepdim=True)).clamp(min=-200).nan_to_num(0.0).abs())
    use = c if counts is None else counts
    dp = (gl * e / max(n, 1) * use.double() / max(1, int(use.sum()))).expand(t, e)
    gw = torch.zeros(t, k, device="cuda") if gw is None else gw
    gw = gw.double()
    full = dp if normalize else dp.clone().scatter_add_(1, places, gw)
    dx = p * (full - (p * full).sum(1, keepdim=True))
    if normalize:   # (a softmax over the chosen alone: exactly nothing for the others)
        dx = dx.scatter_add(1, places, w * (gw - (gw * w).sum(1, keepdim=True)))
    r["dx"] = dx.masked_fill(~mask[:, None], 0.0)
    # what is added up in a gradient, without its signs
    size = p * (dp.abs() + (p * dp.abs()).sum(1, keepdim=True))
    part = w * (gw.abs() + (w * gw.abs()).sum(1, keepdim=True))
    if not normalize:
        size = size + p * (w * gw.abs()).sum(1, keepdim=True)
    r["size"] = size.scatter_add(1, places, part)
    return r


def _near(got, want, tol, what):
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: off by {off[bad][0].item():.3g}, allowed " \
                          f"{torch.as_tensor(tol).expand_as(off)[bad][0].item():.3g}"


def _check_forward(a, r, tokens):
    assert torch.equal(a.experts[:tokens].long(), r["experts"])
    assert torch.equal(a.counts.long(), r["counts"]) and int(a.real) == r["real"]
    most = r["d"].amax(1, keepdim=True).clamp(max=60)
    _near(a.weights[:tokens], r["weights"], r["weights"] * U * (64 + 8 * most) + 1e-37, "weights")
    # a token's p is off by 64 + 4 |d|; an expert's sum goes through at most tokens / 256 + 64 additions
    slack = (r["p"] * r["d"]).sum(0) / max(1, r["real"]) * 4 * U
    _near(a.probs, r["probs"], r["probs"] * U * (128 + tokens / 256) + slack + 1e-37, "probs")
    _near(a.loss, torch.tensor([r["loss"]], device="cuda").double(),
          U * (r["loss"] * (160 + tokens / 256) + 4 * float((r["p"] * r["d"]).sum(1).max()) * r["loss"]) + 1e-37, "loss")


def _check_grad(dx, r, dtype):
    most = r["d"].amax(1, keepdim=True).clamp(max=60)
    tol = r["size"] * U * (96 + 8 * r["d"] + 8 * most) + r["dx"].abs() * (2.0 ** -8 if dtype == BF16 else 4 * U) + 1e-36
    _near(dx, r["dx"], tol, "gradient")


CASES = [  # tokens, experts, k, dtype, ld, offset, normalize
    (1, 1, 1, BF16, None, 0, True), (1, 1, 1, FP32, None, 0, False), (3, 2, 2, BF16, 5, 1, True),
    (1, 128, 8, BF16, None, 0, True), (7, 4, 2, BF16, None, 0, True), (64, 8, 2, FP32, None, 0, True), (64, 31, 5, BF16, 33, 3, False),
    (64, 128, 8, BF16, None, 0, True), (64, 128, 8, FP32, None, 0, True), (100, 33, 32, FP32, None, 1, True),
    (333, 60, 4, FP32, None, 0, False), (333, 64, 6, BF16, 64, 0, True), (333, 64, 6, BF16, 72, 1, True),
    (1000, 128, 8, BF16, None, 0, False), (1001, 128, 8, BF16, 136, 0, True), (1001, 128, 9, BF16, 131, 2, True),
    (500, 129, 16, BF16, None, 0, True), (500, 256, 8, FP32, None, 0, False), (500, 256, 8, BF16, None, 0, True),
    (300, 512, 10, BF16, None, 0, True), (200, 1000, 32, FP32, 1003, 5, True), (200, 1024, 32, BF16, None, 0, False),
    (20000, 128, 8, BF16, None, 0, True), (20001, 128, 8, FP32, None, 0, True), (40000, 16, 2, BF16, None, 0, True),
    (5001, 60, 4, BF16, 61, 1, True),
]


@pytest.mark.parametrize("tokens,experts,k,dtype,ld,offset,normalize", CASES)
@pytest.mark.parametrize("masked", [False, True])
def test_forward_and_gradient(tokens, experts, k, dtype, ld, offset, normalize, masked):
    x = _logits(tokens, experts, dtype, ld=ld, offset=offset)
    before = x.clone()
    mask = None
    if masked:
        mask = torch.rand(tokens, device="cuda") < 0.7
        mask[0] = True
    a = bd.ExpertRouting(tokens + 3, experts, k, normalize=normalize)
    a.run(x, mask)
    gw = torch.randn(tokens, k, device="cuda")
    r = _reference(x, k, normalize, mask, gw, 3.0)
    _check_forward(a, r, tokens)
    assert not a.weights[tokens:].any() and not a.experts[tokens:].any()
    dx = a.backward(x, gw, 3.0)
    assert torch.equal(x, before) and dx.shape == x.shape
    _check_grad(dx, r, dtype)
    rate = torch.tensor([3.0], device="cuda")
    assert torch.equal(a.backward(x, gw, rate), dx)
    for w, l in ((None, 5.0), (gw, 0.0)):
        _check_grad(a.backward(x, w, l), _reference(x, k, normalize, mask, w, l), dtype)
    a.backward(x, gw, rate, out=x)
    assert torch.equal(x, dx)
    if ld and ld > experts:
        assert (x.as_strided((tokens - 1, ld - experts), (ld, 1), x.storage_offset() + experts) == 77.0).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("experts,k", [(4, 2), (60, 8), (128, 8), (128, 32), (200, 20), (1024, 32)])
def test_equal_logits(dtype, experts, k):
    t = torch.arange(300, device="cuda")[:, None]
    e = torch.arange(experts, device="cuda")[None, :]
    for x in (torch.zeros(300, experts, device="cuda"), ((t + e * 7) % 3).float(),
              torch.where((e + t) % 2 == 0, 0.0, -0.0), (e - t) * 0.01, (e % 5 == t % 5) * 2.0):
        x = x.to(dtype).expand(300, experts).contiguous()
        a = bd.ExpertRouting(300, experts, k)
        a.run(x)
        _check_forward(a, _reference(x, k, True, None), 300)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("experts,k", [(9, 4), (128, 8), (300, 8)])
def test_experts_and_tokens_without_a_probability(dtype, normalize, experts, k):
    x = _logits(200, experts, dtype)
    x[:, 5] = -INF                      # an expert that is switched off
    x[10:20, 2:] = -INF                 # fewer left than are chosen
    x[30:33] = -INF                     # nothing left
    x[40:44] = torch.finfo(dtype).min   # all alike
    x[50, :3] = torch.finfo(dtype).max
    mask = torch.ones(200, dtype=torch.uint8, device="cuda")
    mask[31], mask[60:70] = 0, 0
    x[65] = NAN                         # in a place that the mask leaves out
    a = bd.ExpertRouting(200, experts, k, normalize=normalize)
    a.run(x, mask)
    gw = torch.randn(200, k, device="cuda")
    ref = x.clone()
    ref[65] = 0
    r = _reference(ref, k, normalize, mask, gw, 2.0)
    _check_forward(a, r, 200)
    _check_grad(a.backward(x, gw, 2.0), r, dtype)
    assert a.counts[5] < 200


def test_nothing_counts():
    a = bd.ExpertRouting(20, 16, 2)
    x = _logits(20, 16, BF16)
    a.run(x, torch.zeros(20, dtype=torch.bool, device="cuda"))
    assert not a.counts.any() and not a.probs.any() and float(a.loss) == 0 and int(a.real) == 0
    assert (a.experts == -1).all() and not a.weights.any()
    assert not a.backward(x, torch.ones(20, 2, device="cuda"), 1.0).any()
    a.run(x)
    assert int(a.real) == 20
    a.run(x[:0])
    assert float(a.loss) == 0 and int(a.real) == 0 and not a.counts.any()
    assert a.backward(x[:0], None, 1.0).shape == (0, 16)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("value", [NAN, INF])
def test_values_that_are_not_finite(dtype, value):
    x = _logits(50, 128, dtype)
    clean = x.clone()
    x[7, 100] = value
    a, b = bd.ExpertRouting(50, 128, 8), bd.ExpertRouting(50, 128, 8)
    a.run(x)
    b.run(clean)
    assert a.experts[7, 0] == 100 and a.weights[7].isnan().all() and a.loss.isnan().all()
    rest = torch.arange(50, device="cuda") != 7
    assert torch.equal(a.experts[rest], b.experts[rest]) and torch.equal(a.weights[rest], b.weights[rest])
    gw = torch.randn(50, 8, device="cuda")
    dx, dc = a.backward(x, gw), b.backward(clean, gw)
    assert dx[7].isnan().all() and torch.equal(dx[rest], dc[rest])


def test_strides_masks_and_counts_of_several_batches():
    x = _logits(300, 64, BF16)
    mask = (torch.rand(300, 3, device="cuda") < 0.8)[:, 1]
    a = bd.ExpertRouting(300, 64, 4)
    a.run(x, mask)
    gw = torch.randn(4, 300, device="cuda").T
    _check_grad(a.backward(x, gw, 1.0), _reference(x, 4, True, mask, gw, 1.0), BF16)
    one = torch.tensor(0.5, device="cuda").expand(300, 4)
    _check_grad(a.backward(x, one, 1.0), _reference(x, 4, True, mask, one, 1.0), BF16)
    counts = a.counts + torch.arange(64, device="cuda", dtype=torch.int32) * 100
    _check_grad(a.backward(x, gw, 10.0, counts=counts), _reference(x, 4, True, mask, gw, 10.0, counts), BF16)
    counts = torch.full_like(counts, 2 ** 31 - 1)      # (a sum past 32 bits)
    _check_grad(a.backward(x, gw, 10.0, counts=counts), _reference(x, 4, True, mask, gw, 10.0, counts), BF16)


@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_against_differences(normalize):
    x = _logits(6, 10, FP32, scale=1.0)
    a = bd.ExpertRouting(6, 10, 3, normalize=normalize)
    a.run(x)
    gw = torch.randn(6, 3, device="cuda")
    dx = a.backward(x, gw, 0.8)
    counts, places = a.counts.double(), a.experts.long()

    def loss(x):
        p = torch.softmax(x, 1)
        w = p.gather(1, places)
        w = w / w.sum(1, keepdim=True) if normalize else w
        balance = 10 * (counts / 18 * p.mean(0)).sum()
        return float((w * gw).sum() + 0.8 * balance)

    e = 1e-4
    for i in range(6):
        for j in (0, 4, 9, int(places[i, 0])):
            up, down = x.double(), x.double()
            up[i, j] += e
            down[i, j] -= e
            # a softmax's third derivatives are below 2 in size
            bound = e * e * 2 * (float(gw[i].abs().sum()) + 8) + 1e-5
            assert abs((loss(up) - loss(down)) / (2 * e) - float(dx[i, j])) < bound


def test_calls_repeat_and_a_token_is_as_by_itself():
    x = _logits(9000, 128, BF16)
    a = bd.ExpertRouting(9000, 128, 8)
    a.run(x)
    first = [t.clone() for t in (a.weights, a.experts, a.counts, a.probs, a.loss)]
    gw = torch.randn(9000, 8, device="cuda")
    dx = a.backward(x, gw, 1.0)
    for _ in range(3):
        a.run(x)
        for p, q in zip(first, (a.weights, a.experts, a.counts, a.probs, a.loss)):
            assert torch.equal(p, q)
        assert torch.equal(dx, a.backward(x, gw, 1.0))
    a.run(x[77:78])
    assert torch.equal(a.weights[0], first[0][77]) and torch.equal(a.experts[0], first[1][77])
    assert torch.equal(a.weights[1:], first[0][1:])


def test_the_gradient_of_the_first_tokens():
    """Their share of the balance loss is that among all of the run's."""
    x = _logits(300, 64, FP32)
    a = bd.ExpertRouting(400, 64, 4)
    a.run(x)
    gw = torch.randn(300, 4, device="cuda")
    assert torch.equal(a.backward(x[:77], gw[:77], 3.0), a.backward(x, gw, 3.0)[:77])


def test_columns_of_one_buffer():
    both = torch.randn(500, 256, device="cuda").bfloat16()
    x, out = both[:, :128], both[:, 128:]
    a = bd.ExpertRouting(500, 128, 8)
    a.run(x)
    gw = torch.randn(500, 8, device="cuda")
    _check_grad(a.backward(x, gw, 1.0, out=out), _reference(x, 8, True, None, gw, 1.0), BF16)
