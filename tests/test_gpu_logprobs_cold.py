"""Token log probabilities at very low temperatures (GPU).

With u = 2^-24: d = (x - max) / T carries a rounding in the difference and one in the quotient, its
product with log2 e two more, and 2^x by the hardware 4 u: e^d is off by (4 + 4 |d|) u of itself.  A sum
goes through at most vocab / 32 + 16 additions a thread and 20 that join the threads', each off by u of a
sum of numbers of one sign.  The rest as for other rows, but for e^d below 2^-126, the least normal
number, which FP32's 2^x takes as 0: a probability is off by 2^-126 there at most, and a gradient by that
times (|g| + |h| (|lp| + H + 1)) / T, which 1 / T makes large beside the 1e-30 of other tests."""
import math

import pytest
import torch

from test_gpu_logprobs import BF16, FP32, U, _near, _reference

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("lossless_bf16_weight_old_gb300")

INF = math.inf
COLD = [1e-8, 4e-9, 1e-9, 1e-12, 1e-20, 1e-30]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    bd._ops_lib.load()


def _number(heat):
    """The temperature as FP32 has it."""
    return torch.tensor(heat, dtype=torch.float32).double().item()


def _rows(vocab, dtype, heat):
    """Rows whose maximum is 0 or nearly so, with and without values that are masked out."""
    gen = torch.Generator(device="cuda").manual_seed(vocab)
    low = torch.finfo(dtype).min
    x = torch.zeros(14, vocab, device="cuda")
    x[0, 1:] = -INF                                # one token
    x[1, 1:] = low
    x[2, :-1] = -INF
    x[3, 1:] = -torch.rand(vocab - 1, generator=gen, device="cuda") - 1.0
    x[4, vocab // 2:] = -INF                       # many alike (and row 5: all)
    x[6] = -1e-6
    x[6, 1:] = -1.0
    for i, scale in ((7, 1), (8, 4), (9, 20)):     # differences that are as small as the temperature
        x[i] = -(torch.randint(0, 8, (vocab,), generator=gen, device="cuda") * scale).double().mul(heat)
        x[i, 0] = 0.0
    x[10], x[11] = x[8], x[9]
    x[10, 1::2] = -INF
    x[11, 1::3] = low
    x[12] = x[8] - 4 * heat                        # (the maximum is not 0)
    x[13] = x[3] + 1.0                             # (nor here, and far from it in temperatures)
    tokens = torch.randint(vocab, (14,), generator=gen, device="cuda")
    tokens[:2] = 0
    tokens[2] = vocab - 1
    return x.to(dtype), tokens


def _check(lp, x, tokens, heat, has_entropy):
    """Of one temperature, or one a row."""
    r = _reference(x, tokens, heat)
    v = x.shape[1]
    adds = v / 32 + 36
    tol = U * (8 + 4 * r["D"] + adds)
    far = torch.isinf(r["logprob"])
    big = r["logprob"].abs() > torch.finfo(FP32).max
    got = lp.logprobs
    assert (got[far | big] == -INF).all()
    some = ~(far | big)
    _near(got[some], r["logprob"][some], (tol + U * 6 * r["logprob"].abs())[some], "logprobs")
    if has_entropy:
        _near(lp.entropy, r["entropy"], tol + U * (r["D"] * (16 + 2 * adds) + 8 * r["Q"] + 4 * r["entropy"]), "entropy")
    if lp.top:
        places = x.float().sort(dim=1, descending=True, stable=True).indices[:, :lp.top]
        assert torch.equal(lp.top_tokens.long(), places)
    return r


def _check_gradient(dx, r, tokens, heat, g, h, dtype, least=0.0):
    """Where the type has the gradient, and 0 where nothing is to be learned."""
    heats = heat.double()[:, None] if isinstance(heat, torch.Tensor) else heat
    g, h = g.double()[:, None], (torch.zeros_like(g) if h is None else h).double()[:, None]
    one = torch.zeros_like(r["p"]).scatter_(1, tokens[:, None], 1.0)
    lp, entropy = torch.where(r["p"] > 0, r["lp"], 0.0), r["entropy"][:, None]
    want = (g * (one - r["p"]) - h * r["p"] * (lp + entropy)) / heats
    most = torch.finfo(dtype).max
    over = want.abs() > most
    assert not dx.isnan().any()
    assert (dx[over].double().sign() == want[over].sign()).all() and (dx[over].double().abs() >= most / 2).all()
    assert not dx[(r["p"] == 0) & (one == 0)].any()
    each = (g.abs() + h.abs() * (lp.abs() + entropy + 1)) / heats
    sums = U * (8 + 4 * r["D"] + dx.shape[1] / 32 + 36)[:, None]
    tol = r["p"] * each * (U * (24 + 8 * r["d"].abs()) + 2 * sums) + 2.0 ** -126 * each + least / heats
    tol = tol + one * g.abs() / heats * 8 * U + want.abs() * (2.0 ** -8 if dtype == BF16 else 4 * U)
    fine = (each < most / 4).expand_as(dx)
    _near(dx[fine], want[fine], tol[fine], "gradient")


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("vocab", [3, 70, 1024, 5001, 32000])
@pytest.mark.parametrize("heat", COLD)
def test_very_low_temperatures(dtype, vocab, heat):
    heat = _number(heat)
    x, tokens = _rows(vocab, dtype, heat)
    gen = torch.Generator(device="cuda").manual_seed(1)
    g, h = torch.randn(14, generator=gen, device="cuda"), torch.randn(14, generator=gen, device="cuda")
    for entropy in (True, False):
        lp = bd.TokenLogprobs(14, vocab, top=min(3, vocab), entropy=entropy)
        lp.run(x, tokens, heat)
        r = _check(lp, x, tokens, heat, entropy)
        _check_gradient(lp.backward(x, g), r, tokens, heat, g, None, dtype)
        if entropy:
            _check_gradient(lp.backward(x, g, h), r, tokens, heat, g, h, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_many_short_rows_and_few_long_ones(dtype):
    """The other blocks that a row may get."""
    for rows, vocab in ((4000, 70), (2000, 5001), (300, 70001), (3, 151937)):
        x = torch.full((rows, vocab), -INF, dtype=dtype, device="cuda")
        at = torch.arange(rows, device="cuda") * 31 % vocab
        x[torch.arange(rows, device="cuda"), at] = 0.0
        g = torch.ones(rows, device="cuda")
        for entropy in (True, False):
            lp = bd.TokenLogprobs(rows, vocab, entropy=entropy)
            lp.run(x, at, 1e-9)
            assert not lp.logprobs.any() and not lp.backward(x, g).any()
            if entropy:
                assert not lp.entropy.any() and not lp.backward(x, g, g).any() and not lp.backward(x, None, g).any()
