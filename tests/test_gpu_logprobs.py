"""Token log probabilities, entropies, top tokens and the logits' gradient against their formulas in
64 bits (GPU).

Tolerances, with u = 2^-24 (half an FP32 step): an FP32 operation adds a relative u, 2^x by the
hardware 4 u (its documented error is 2 steps).  d = (x - max) / T carries three roundings, so
e^d is off by (4 + 4 |d|) u of itself.  A sum of positive numbers is off by u for each addition that
a term goes through, at most `adds` below.  A logarithm turns relative errors into absolute ones.
Weighted by p, |d| sums to D and d^2 to Q."""
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


def _logits(rows, vocab, dtype, *, seed=0, ld=None, offset=0, scale=3.0):
    """Rows of normal logits, `offset` elements into their memory, `ld` elements apart."""
    gen = torch.Generator(device="cuda").manual_seed(seed + 1000 * rows + vocab)
    ld = ld or vocab
    memory = torch.empty(offset + rows * ld + 64, dtype=dtype, device="cuda").fill_(77.0)
    x = memory[offset:offset + rows * ld].view(rows, ld)[:, :vocab]
    x.copy_(torch.randn(rows, vocab, generator=gen, device="cuda") * scale)
    tokens = torch.randint(vocab, (rows,), generator=gen, device="cuda")
    return x, tokens


def _reference(x, tokens, temperature):
    """The formulas in 64 bits, for rows with a distribution and a token."""
    z = x.double() / (temperature.double()[:, None] if isinstance(temperature, torch.Tensor) else temperature)
    d = z - z.amax(1, keepdim=True)
    lp = d - d.exp().sum(1, keepdim=True).log()
    p = lp.exp()
    d0 = torch.where(p > 0, d, 0.0)
    r = dict(z=z, d=d0, lp=lp, p=p, D=(p * d0.abs()).sum(1), Q=(p * d0 * d0).sum(1))
    r["entropy"] = -(p * torch.where(p > 0, lp, 0.0)).sum(1)
    r["logprob"] = lp.gather(1, tokens.long().clamp(min=0)[:, None]).squeeze(1)
    return r


def _adds(vocab):
    """Additions that a term of a row's sum goes through: 256 threads take windows of at least 16
    elements in turn, with at least two sums each (then 64 for all that joins them)."""
    return vocab / 512 + 16 + 64


def _sum_error(r, vocab):
    return U * (8 + 4 * r["D"] + _adds(vocab))


def _near(got, want, tol, what):
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: off by {off[bad][0].item():.3g}, allowed " \
                          f"{torch.as_tensor(tol).expand_as(off)[bad][0].item():.3g}"


def _check_forward(lp, x, tokens, temperature, rows):
    r = _reference(x, tokens, temperature)
    v = x.shape[1]
    has = tokens >= 0
    tol = _sum_error(r, v)
    _near(lp.logprobs[:rows], torch.where(has, r["logprob"], 0.0), tol + U * 6 * (r["logprob"].abs() + 40), "logprobs")
    if lp.entropy is not None:
        # sum e d over sum e: each factor's error, and that of d beside d
        _near(lp.entropy[:rows], torch.where(has, r["entropy"], 0.0),
              tol + U * (r["D"] * (16 + 2 * _adds(v)) + 8 * r["Q"] + 4 * (r["entropy"] + 1)), "entropy")
    if lp.top:
        places = x.float().sort(dim=1, descending=True, stable=True).indices[:, :lp.top]
        want = torch.where(has[:, None], places, -1)
        assert torch.equal(lp.top_tokens[:rows].long(), want)
        best = torch.where(has[:, None], r["lp"].gather(1, places), 0.0)
        fine = torch.isfinite(best)
        assert torch.equal(lp.top_logprobs[:rows][~fine].double(), best[~fine])
        _near(lp.top_logprobs[:rows][fine], best[fine],
              (tol[:, None] + U * 6 * (best.abs() + 40))[fine], "top_logprobs")
    return r


def _check_grad(dx, r, tokens, temperature, g, h, dtype):
    heat = temperature.double()[:, None] if isinstance(temperature, torch.Tensor) else temperature
    g, h = g.double()[:, None], (h.double()[:, None] if h is not None else torch.zeros(1, 1, device="cuda").double())
    one = torch.zeros_like(r["p"]).scatter_(1, tokens.long().clamp(min=0)[:, None], 1.0)
    lp = torch.where(r["p"] > 0, r["lp"], 0.0)
    want = (g * (one - r["p"]) - h * r["p"] * (lp + r["entropy"][:, None])) / heat
    want = torch.where((tokens >= 0)[:, None], want, 0.0)
    size = r["p"] * (g.abs() + h.abs() * (lp.abs() + r["entropy"][:, None] + 1)) / heat
    tol = size * U * (24 + 8 * r["d"].abs()) + size * 2 * _sum_error(r, dx.shape[1])[:, None]
    tol = tol + one * g.abs() / heat * 8 * U + want.abs() * (2.0 ** -8 if dtype == BF16 else 4 * U) + 1e-30
    _near(dx, want, tol, "gradient")


CASES = [  # rows, vocab, dtype, ld, offset, top, entropy
    (1, 1, BF16, None, 0, 1, True), (2, 1, FP32, 3, 1, 1, True), (3, 2, BF16, None, 1, 2, True),
    (5, 31, BF16, 33, 1, 31, False), (4, 32, BF16, None, 0, 32, True), (4, 33, FP32, 35, 3, 32, True),
    (7, 100, BF16, 101, 5, 20, True), (600, 1000, BF16, None, 0, 5, True), (600, 1000, FP32, 1001, 7, 5, True),
    (1, 4113, FP32, None, 0, 32, True), (1300, 4113, BF16, None, 0, 20, False),
    (130, 8191, BF16, 8200, 3, 32, True), (1, 32001, BF16, None, 0, 0, True), (9, 32001, FP32, None, 0, 20, True),
    (40, 32000, BF16, None, 0, 20, True), (1000, 32000, BF16, None, 0, 0, True),
    (1, 151936, BF16, None, 0, 20, True), (1, 151936, FP32, None, 0, 20, True),
    (70, 151936, BF16, None, 0, 1, False), (5, 151937, FP32, 151940, 1, 32, True),
    (240, 140001, BF16, 140004, 3, 0, True), (240, 140001, BF16, None, 0, 20, True), (250, 70001, FP32, None, 1, 0, False),
    (250, 70001, FP32, None, 0, 20, True), (130, 32000, FP32, None, 0, 5, True), (180, 151936, BF16, None, 0, 0, True),
    (3000, 1000, BF16, None, 0, 5, True), (3000, 777, FP32, 779, 1, 32, True), (5000, 4099, FP32, None, 0, 0, True),
    (1300, 32001, BF16, None, 0, 20, True), (1300, 16001, FP32, None, 0, 32, True), (2500, 60001, BF16, None, 1, 0, True),
    (2, 600001, BF16, None, 0, 32, True), (700, 300001, BF16, None, 0, 3, True), (650, 140001, FP32, None, 0, 3, True),
]


@pytest.mark.parametrize("rows,vocab,dtype,ld,offset,top,entropy", CASES)
def test_forward_and_gradient(rows, vocab, dtype, ld, offset, top, entropy):
    x, tokens = _logits(rows, vocab, dtype, ld=ld, offset=offset)
    tokens[1::5] = -1
    before = x.clone()
    lp = bd.TokenLogprobs(rows + 2, vocab, top=top, entropy=entropy)
    lp.run(x, tokens)
    step = max(1, (1 << 25) // vocab)
    g = torch.randn(rows, device="cuda")
    h = torch.randn(rows, device="cuda") if entropy else None
    dx = lp.backward(x, g, h)
    assert torch.equal(x, before) and dx.shape == x.shape and dx.dtype == dtype
    for a in range(0, rows, step):     # (the reference in 64 bits, some rows at a time)
        part = _View(lp, a, min(rows, a + step))
        r = _check_forward(part, x[a:a + step], tokens[a:a + step], 1.0, part.rows)
        _check_grad(dx[a:a + step], r, tokens[a:a + step], 1.0, g[a:a + step], None if h is None else h[a:a + step], dtype)
    assert not lp.logprobs[rows:].any()        # rows behind the last one stay as they were


class _View:
    def __init__(self, lp, a, b):
        self.rows, self.top = b - a, lp.top
        self.logprobs, self.top_logprobs, self.top_tokens = lp.logprobs[a:b], lp.top_logprobs[a:b], lp.top_tokens[a:b]
        self.entropy = None if lp.entropy is None else lp.entropy[a:b]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("each", [False, True])
@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
def test_temperatures_and_token_types(dtype, each, kind):
    x, tokens = _logits(37, 5003, dtype)
    tokens = tokens.to(kind)
    heat = torch.rand(37, device="cuda") * 2 + 0.1 if each else 0.37
    lp = bd.TokenLogprobs(37, 5003, top=7, entropy=True)
    lp.run(x, tokens, heat)
    r = _check_forward(lp, x, tokens, heat, 37)
    g, h = torch.randn(37, device="cuda"), torch.randn(37, device="cuda")
    _check_grad(lp.backward(x, g, h), r, tokens, heat, g, h, dtype)
    _check_grad(lp.backward(x, None, h), r, tokens, heat, torch.zeros_like(g), h, dtype)
    _check_grad(lp.backward(x, g), r, tokens, heat, g, None, dtype)


def test_strided_vectors_and_one_number_for_all_rows():
    x, tokens = _logits(50, 777, BF16)
    wide = torch.stack([tokens, tokens - 1, tokens + 5], 1)
    heat = torch.rand(50, 2, device="cuda") + 0.5
    lp = bd.TokenLogprobs(50, 777, entropy=True)
    lp.run(x, wide[:, 0], heat[:, 1])
    r = _check_forward(lp, x, tokens, heat[:, 1], 50)
    g, h = torch.randn(50, 4, device="cuda")[:, 2], torch.tensor([-0.3], device="cuda").expand(50)
    _check_grad(lp.backward(x, g, h), r, tokens, heat[:, 1], g, h, BF16)
    lp.run(x, torch.tensor([5], device="cuda").expand(50), torch.tensor([2.0], device="cuda").expand(50))
    _check_forward(lp, x, torch.full((50,), 5, device="cuda"), 2.0, 50)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("ld,ld_out,shift", [(1001, 1001, 0), (1001, 1001, 1), (1008, 1001, 0), (1001, 1024, 3),
                                             (1001, 1002, 16), (1024, 1024, 16)])
def test_where_the_gradient_goes(dtype, ld, ld_out, shift):
    """Rows that begin differently in the two, and memory around them that stays as it was."""
    rows, vocab = 45, 1001
    x, tokens = _logits(rows, vocab, dtype, ld=ld)
    tokens[3] = -1
    g = torch.randn(rows, device="cuda")
    lp = bd.TokenLogprobs(rows, vocab)
    lp.run(x, tokens)
    memory = torch.full((shift + rows * ld_out + 50,), 7.0, dtype=dtype, device="cuda")
    out = memory[shift:shift + rows * ld_out].view(rows, ld_out)[:, :vocab]
    assert lp.backward(x, g, out=out) is out
    _check_grad(out, _reference(x, tokens, 1.0), tokens, 1.0, g, None, dtype)
    want = out.clone()
    out.fill_(7.0)
    assert (memory == 7.0).all()
    own = lp.backward(x, g)
    assert torch.equal(own, want)
    lp.backward(x, g, out=x)                   # in place
    assert torch.equal(x, want)
    if ld > vocab:
        assert (x.as_strided((rows - 1, ld - vocab), (ld, 1), x.storage_offset() + vocab) == 77.0).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("vocab", [50, 4099, 151936])
def test_masked_vocabularies(dtype, vocab):
    """Logits of -inf, and of the type's lowest value, in all but a few places."""
    rows, low = 24, torch.finfo(dtype).min
    x, tokens = _logits(rows, vocab, dtype)
    keep = torch.rand(rows, vocab, device="cuda") < 8 / vocab
    keep.scatter_(1, tokens[:, None], True)
    x[:12] = torch.where(keep[:12], x[:12], -INF)
    x[12:18] = torch.where(keep[12:18], x[12:18], low)
    x[18:20] = low                              # even rows of the lowest value: all alike
    x[20] = -INF
    x[20, vocab - 1], tokens[20] = low, vocab - 1     # one token, of the lowest value
    tokens[5] = int((~keep[5]).nonzero()[0])    # a token that the mask forbids
    lp = bd.TokenLogprobs(rows, vocab, top=min(32, vocab), entropy=True)
    lp.run(x, tokens)
    some = torch.arange(rows, device="cuda") != 5
    r = _reference(x, tokens, 1.0)
    assert lp.logprobs[5] == -INF and r["logprob"][5] == -INF
    part = _View(lp, 6, rows)
    _check_forward(part, x[6:], tokens[6:], 1.0, part.rows)
    part = _View(lp, 0, 5)
    _check_forward(part, x[:5], tokens[:5], 1.0, 5)
    g, h = torch.randn(rows, device="cuda"), torch.randn(rows, device="cuda")
    _check_grad(lp.backward(x, g, h), r, tokens, 1.0, g, h, dtype)
    assert some.sum() == rows - 1


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("vocab", [3, 70, 5000, 151936])
def test_rows_without_a_distribution(dtype, vocab):
    x, tokens = _logits(6, vocab, dtype)
    x[1], x[4] = -INF, -INF
    top = min(5, vocab)
    lp = bd.TokenLogprobs(6, vocab, top=top, entropy=True)
    lp.run(x, tokens)
    dx = lp.backward(x, torch.ones(6, device="cuda"), torch.ones(6, device="cuda"))
    for i in (1, 4):
        assert lp.logprobs[i] == -INF and lp.entropy[i] == 0 and not dx[i].any()
        assert (lp.top_logprobs[i] == -INF).all() and lp.top_tokens[i].tolist() == list(range(top))
    assert torch.isfinite(lp.logprobs[[0, 2, 3, 5]]).all() and torch.isfinite(dx).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("vocab", [70, 151937])
def test_values_that_are_not_finite_and_tokens_that_do_not_exist(dtype, vocab):
    x, tokens = _logits(9, vocab, dtype)
    x[0, vocab // 2], x[1, vocab - 1], x[2, 3] = NAN, INF, -NAN
    tokens[3], tokens[4], tokens[5] = vocab, 1 << 40, -(1 << 40)
    heat = torch.ones(9, device="cuda")
    heat[6], heat[7] = 0.0, NAN
    lp = bd.TokenLogprobs(9, vocab, top=4, entropy=True)
    lp.run(x, tokens, heat)
    dx = lp.backward(x, torch.ones(9, device="cuda"), torch.zeros(9, device="cuda"))
    bad = [0, 1, 2, 3, 4, 6, 7]
    assert lp.logprobs[bad].isnan().all() and dx[bad].isnan().all()
    assert lp.entropy[[0, 1, 2, 6, 7]].isnan().all()
    assert torch.isfinite(lp.entropy[[3, 4]]).all() and torch.isfinite(lp.top_logprobs[[3, 4, 8]]).all()
    assert lp.logprobs[5] == 0 and not dx[5].any() and (lp.top_tokens[5] == -1).all()
    assert lp.top_tokens[0, 0] == vocab // 2 and lp.top_tokens[1, 0] == vocab - 1 and lp.top_tokens[2, 0] == 3
    part = _View(lp, 8, 9)
    r = _check_forward(part, x[8:], tokens[8:], 1.0, 1)
    _check_grad(dx[8:], r, tokens[8:], 1.0, torch.ones(1, device="cuda"), None, dtype)
    # no gradient wanted: none, whatever the row holds
    assert not lp.backward(x, torch.zeros(9, device="cuda"), torch.zeros(9, device="cuda")).any()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("rows,vocab", [(3, 64), (2, 5001), (1, 151936), (700, 33333), (2, 524288), (1300, 3000), (1300, 20000)])
def test_top_tokens_of_equal_values(dtype, rows, vocab):
    """Constant rows, few distinct values, zeros of both signs, ascending and descending rows."""
    for kind in range(5):
        n = torch.arange(vocab, device="cuda")
        row = [torch.zeros(vocab, device="cuda"), (n * 7919 % 5).float(), torch.where(n % 3 == 1, -0.0, 0.0),
               n * (8.0 / vocab), -(n * (8.0 / vocab))][kind]
        x = row.to(dtype).expand(rows, vocab).contiguous()
        lp = bd.TokenLogprobs(rows, vocab, top=32)
        tokens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        lp.run(x, tokens)
        want = x[0].float().add(0.0).sort(descending=True, stable=True).indices[:32]
        assert torch.equal(lp.top_tokens.long(), want.expand(rows, 32)), kind


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_large_values(dtype):
    """Logits whose differences, and scaled ones, pass the FP32 range."""
    big = torch.finfo(dtype).max
    x = torch.tensor([[big, -big, 0.0, big], [-big, -big, -big, -INF], [1e30, 1e30, -1e30, 0.0]],
                     dtype=dtype, device="cuda")
    tokens = torch.tensor([0, 1, 0], device="cuda")
    lp = bd.TokenLogprobs(3, 4, top=2, entropy=True)
    for heat in (1.0, 1e-6, 100.0):
        lp.run(x, tokens, heat)
        want = torch.tensor([2.0, 3.0, 2.0], dtype=torch.float64, device="cuda").log()
        _near(lp.logprobs, -want, 64 * U, "logprobs")
        _near(lp.entropy, want, 64 * U, "entropy")
        dx = lp.backward(x, torch.ones(3, device="cuda"), torch.ones(3, device="cuda"))
        want = torch.tensor([[0.5, 0, 0, -0.5], [-1 / 3, 2 / 3, -1 / 3, 0], [0.5, -0.5, 0, 0]], device="cuda").double() / heat
        _near(dx, want, want.abs() * (2.0 ** -8 if dtype == BF16 else 128 * U), "gradient")


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("rows,vocab", [(3, 50000), (240, 140000), (1000, 3001), (3000, 3001), (1300, 20001)])
@pytest.mark.parametrize("heat", [1e-7, 1e6])
def test_far_from_ordinary_temperatures(dtype, rows, vocab, heat):
    """So cold that a row's shift passes its bound, and so hot that all tokens are alike."""
    x, tokens = _logits(rows, vocab, dtype)
    tokens[::9] = -1
    lp = bd.TokenLogprobs(rows, vocab, top=6, entropy=True)
    lp.run(x, tokens, heat)
    g, h = torch.randn(rows, device="cuda"), torch.randn(rows, device="cuda")
    dx = lp.backward(x, g, h)
    step = max(1, (1 << 25) // vocab)
    for a in range(0, rows, step):
        part = _View(lp, a, min(rows, a + step))
        r = _check_forward(part, x[a:a + step], tokens[a:a + step], heat, part.rows)
        _check_grad(dx[a:a + step], r, tokens[a:a + step], heat, g[a:a + step], h[a:a + step], dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_one_likely_token(dtype):
    """-lp and the entropy are small, and as right as the sum and l are."""
    rows, vocab = 64, 32000
    x, tokens = _logits(rows, vocab, dtype, scale=0.5)
    at = torch.arange(rows, device="cuda")
    x[at, tokens] = (12.0 + at / 4).to(dtype)
    lp = bd.TokenLogprobs(rows, vocab, entropy=True)
    lp.run(x, tokens)
    r = _reference(x, tokens, 1.0)
    # Each of the others' terms is off by (8 + 4 |d|) u.  The greatest term is the sum's size, and each
    # addition that it goes through rounds by u of it, however small the others are: _adds(vocab) u in
    # the sum over the greatest term, and as much in its logarithm.
    rest = 1 - r["p"].amax(1)
    size = rest * U * (8 + 8 * 30) * 30 + U * _adds(vocab)
    _near(lp.entropy, r["entropy"], size + 4 * U * r["entropy"], "entropy")
    # and z, l and ln S each by u of their size
    z = x.double()[at, tokens].abs()
    _near(lp.logprobs, r["logprob"], size + 2 * U * (z + 1), "logprobs")
    assert (lp.logprobs <= 0).all() and (lp.entropy >= 0).all()


def test_gradient_against_differences():
    x, tokens = _logits(4, 60, FP32, scale=1.0)
    lp = bd.TokenLogprobs(4, 60, entropy=True)
    lp.run(x, tokens, 0.7)
    g, h = torch.randn(4, device="cuda"), torch.randn(4, device="cuda")
    dx = lp.backward(x, g, h)

    def loss(x):
        r = _reference(x, tokens, 0.7)
        return (g.double() * r["logprob"] + h.double() * r["entropy"]).sum().item()

    e = 1e-4
    for i, j in [(0, 0), (1, 59), (2, int(tokens[2])), (3, 31), (3, int(tokens[3]))]:
        a, b = x.double(), x.double()
        a[i, j] += e
        b[i, j] -= e
        # the third derivative of either part is at most 8 / T^3 times the gradients' size
        bound = e * e * 8 / 0.7 ** 3 * (g[i].abs() + 5 * h[i].abs()).item() + 1e-5 * (g[i].abs() + h[i].abs()).item()
        assert abs((loss(a) - loss(b)) / (2 * e) - dx[i, j].item()) < bound + 1e-9


def test_a_row_of_a_batch_is_as_by_itself_and_calls_repeat():
    x, tokens = _logits(900, 32000, BF16)
    lp = bd.TokenLogprobs(900, 32000, top=20, entropy=True)
    lp.run(x, tokens)
    first = [t.clone() for t in (lp.logprobs, lp.entropy, lp.top_logprobs, lp.top_tokens)]
    g = torch.randn(900, device="cuda")
    dx = lp.backward(x, g, g)
    for _ in range(3):
        lp.run(x, tokens)
        for a, b in zip(first, (lp.logprobs, lp.entropy, lp.top_logprobs, lp.top_tokens)):
            assert torch.equal(a, b)
        assert torch.equal(dx, lp.backward(x, g, g))
    lp.run(x[5:6], tokens[5:6])
    assert torch.equal(lp.top_tokens[0], first[3][5]) and abs(float(lp.logprobs[0] - first[0][5])) < 1e-5
    assert torch.equal(lp.logprobs[1:], first[0][1:])     # rows behind the last one


def test_offsets_past_32_bits():
    """A matrix of more than 2^32 bytes, whose last rows count."""
    rows, vocab = 17000, 151936
    x = torch.zeros(rows, vocab, dtype=BF16, device="cuda")
    tokens = torch.full((rows,), -1, device="cuda")
    for i in (0, 14200, rows - 1):
        x[i] = torch.randn(vocab, device="cuda") * 3
        tokens[i] = vocab - 1
    lp = bd.TokenLogprobs(rows, vocab, top=3, entropy=True)
    lp.run(x, tokens)
    at = torch.tensor([0, 14200, rows - 1], device="cuda")
    part = _View(lp, 0, 3)
    part.logprobs, part.entropy, part.top_logprobs, part.top_tokens = (
        t[at] for t in (lp.logprobs, lp.entropy, lp.top_logprobs, lp.top_tokens))
    r = _check_forward(part, x[at], tokens[at], 1.0, 3)
    g = torch.ones(rows, device="cuda")
    x0 = x[at].clone()
    dx = lp.backward(x, g, out=x)
    _check_grad(dx[at], r, tokens[at], 1.0, g[at], None, BF16)
    assert x0.shape == dx[at].shape and not dx[1:14200].any() and not dx[14201:-1].any()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_the_largest_vocabulary(dtype):
    rows, vocab = 2, 1 << 24
    x, tokens = _logits(rows, vocab, dtype)
    x[1, -1], tokens[1] = 30.0, vocab - 1
    lp = bd.TokenLogprobs(rows, vocab, top=32, entropy=True)
    lp.run(x, tokens)
    g, h = torch.randn(rows, device="cuda"), torch.randn(rows, device="cuda")
    dx = lp.backward(x, g, h)
    for i in range(rows):
        part = _View(lp, i, i + 1)
        r = _check_forward(part, x[i:i + 1], tokens[i:i + 1], 1.0, 1)
        _check_grad(dx[i:i + 1], r, tokens[i:i + 1], 1.0, g[i:i + 1], h[i:i + 1], dtype)


def test_the_gradient_of_the_first_rows():
    x, tokens = _logits(50, 3000, BF16)
    lp = bd.TokenLogprobs(50, 3000, entropy=True)
    lp.run(x, tokens)
    g = torch.randn(50, device="cuda")
    assert torch.equal(lp.backward(x[:20], g[:20], g[:20]), lp.backward(x, g, g)[:20])


def test_no_rows():
    lp = bd.TokenLogprobs(4, 10, top=2)
    x = torch.empty(0, 10, dtype=BF16, device="cuda")
    lp.run(x, torch.empty(0, dtype=torch.int64, device="cuda"))
    assert lp.backward(x, torch.empty(0, device="cuda")).shape == (0, 10)
    lp = bd.TokenLogprobs(0, 10)
    lp.run(x, torch.empty(0, dtype=torch.int32, device="cuda"))
    assert lp.logprobs.shape == (0,)
