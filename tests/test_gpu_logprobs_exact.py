"""Log probabilities are as exact as the row's sum, wherever its logits lie (GPU).

With u = 2^-24.  lp = (x - max) / T - ln S, S = sum e^((x - max) / T): both parts have one sign, so each is
at most |lp| in size.  The first carries two roundings, the second that of its logarithm (2 u), and their
difference one: 6 u |lp| covers them.  An error of S is one of ln S.  S lies between 1 and the vocabulary;
its terms are off by (8 + 4 |d|) u of themselves, and a rounding of S is off by u of it, or by what is
added where that is less (a term that is lost).

The greatest term's way: a thread adds what its windows hold (in four sums), three additions join them, ten
the lanes' and the warps', five the cluster's; the quotient by the greatest term and its 2^x add 5 u.  So
beside the thread's own terms 24 u cover it."""
import pytest
import torch

from test_gpu_logprobs import BF16, FP32, U, _near, _reference

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("lossless_bf16_weight_old_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    bd._ops_lib.load()


def _tolerance(r, lp, own):
    """own: the share of a row's other terms that one thread may add, all of which could be lost."""
    rest = 1 - r["p"].amax(1)
    return rest * U * 8 + U * 4 * r["D"] + own * rest + U * 24 + U * 6 * lp.abs()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("top", [0, 3])
@pytest.mark.parametrize("at", [100.0, 128.0, 120.0, -90.0, 30.0, 2.0])
def test_one_likely_token_anywhere(dtype, top, at):
    """The others 23 below it: -lp is 3e-6."""
    rows, vocab = 64, 32000
    x = torch.full((rows, vocab), at - 23.0, dtype=dtype, device="cuda")
    tokens = torch.arange(rows, device="cuda") * 499
    x[torch.arange(rows, device="cuda"), tokens] = at
    lp = bd.TokenLogprobs(rows, vocab, top=top)
    lp.run(x, tokens)
    r = _reference(x, tokens, 1.0)
    assert (r["logprob"] < -2e-6).all()
    # (a thread has at most 4 of 2000 FP32 windows, two blocks a row: a 500th of the row)
    _near(lp.logprobs, r["logprob"], _tolerance(r, r["logprob"], 1 / 500), "logprobs")
    if top:
        best = r["lp"].sort(dim=1, descending=True, stable=True).values[:, :top]
        _near(lp.top_logprobs, best, _tolerance(r, r["logprob"], 1 / 500)[:, None] + U * 6 * best.abs(), "top_logprobs")


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("at", [0.0, 60.0, 110.0, -110.0, 126.0])
def test_few_tokens_far_from_zero(dtype, at):
    """One window a thread at most: 8 additions, and the joins."""
    rows, vocab = 640, 90
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = (torch.randn(rows, vocab, generator=gen, device="cuda") * 2 + at).to(dtype)
    x[::2, 7] = at + 9.0
    tokens = torch.randint(vocab, (rows,), generator=gen, device="cuda")
    tokens[::4] = 7
    lp = bd.TokenLogprobs(rows, vocab)
    lp.run(x, tokens)
    r = _reference(x, tokens, 1.0)
    tol = U * (8 + 4 * r["D"] + 8 + 24 + 6 * r["logprob"].abs())
    _near(lp.logprobs, r["logprob"], tol, "logprobs")


@pytest.mark.parametrize("at", [0.0, 100.0, -100.0, 500.0])
def test_tokens_far_below(at):
    """z of -1000 and less beside a likely token: relative to lp."""
    x = torch.tensor([[at, at - 3.0, at - 700.5, at - 5000.25]], device="cuda").expand(4, 4).contiguous()
    lp = bd.TokenLogprobs(4, 4)
    lp.run(x, torch.arange(4, device="cuda"), 0.75)
    r = _reference(x, torch.arange(4, device="cuda"), 0.75)
    _near(lp.logprobs, r["logprob"], U * (8 + 4 * r["D"] + 32 + 6 * r["logprob"].abs()), "logprobs")
