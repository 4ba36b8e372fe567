"""Token log probabilities at the least and the greatest temperatures of FP32, whose reciprocals it does not
have or has with few bits, and of logits whose differences it does not have (GPU).

Tolerances as for very low temperatures.  Gradients g of 1e35 T and less keep g / T in FP32's range; products
with them below 2^-126 are denormal and round by 2^-150 each, four of them to an element, before they are
divided by T; gradients below 2^-126 are denormal and round by half their spacing, 2^-150 or, of BF16, 2^-134."""
import pytest
import torch

from test_gpu_logprobs import BF16, FP32, U, _near, _reference
from test_gpu_logprobs_cold import _check, _check_gradient, _number, _rows

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("lossless_bf16_weight_old_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    bd._ops_lib.load()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("vocab", [3, 70, 5001, 32000])
@pytest.mark.parametrize("heat", [1e-36, 1e-37, 2.0 ** -126, 3e-39, 2e-39, 1e-40, 2.0 ** -149])
@pytest.mark.parametrize("each", [False, True])
def test_the_least_temperatures(dtype, vocab, heat, each):
    heat = _number(heat)
    x, tokens = _rows(vocab, dtype, heat)
    heats = torch.full((14,), heat, device="cuda") if each else heat
    gen = torch.Generator(device="cuda").manual_seed(1)
    g, h = torch.randn(14, generator=gen, device="cuda"), torch.randn(14, generator=gen, device="cuda")
    small = min(1.0, heat * 1e35)
    for entropy in (True, False):
        lp = bd.TokenLogprobs(14, vocab, top=min(3, vocab), entropy=entropy)
        lp.run(x, tokens, heats)
        r = _check(lp, x, tokens, heats, entropy)
        for of in (1.0, small):
            _check_gradient(lp.backward(x, g * of), r, tokens, heats, g * of, None, dtype, 2.0 ** -148)
            if entropy:
                _check_gradient(lp.backward(x, g * of, h * of), r, tokens, heats, g * of, h * of, dtype, 2.0 ** -148)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("vocab", [4, 1003, 40000])
@pytest.mark.parametrize("heat", [1e36, 1e37, 1e38, 3.4e38])
def test_differences_past_the_range(dtype, vocab, heat):
    heat = _number(heat)
    big = torch.finfo(dtype).max
    x = torch.zeros(6, vocab, device="cuda")
    x[0, 0], x[0, 1:] = big, -big
    x[1, ::2], x[1, 1::2] = big, -big
    x[2, 0], x[2, 1] = 2e38, -2e38
    x[3, 1:] = -big
    x[4, 0], x[4, 1], x[4, 2:] = -big, -big, -float("inf")
    x[5, 0], x[5, 1:] = big, -float("inf")
    x = x.to(dtype)
    tokens = torch.tensor([1, 1, 1, 1, 1, 0], device="cuda")
    g, h = torch.randn(6, device="cuda"), torch.randn(6, device="cuda")
    least = heat * (2.0 ** -134 if dtype == BF16 else 2.0 ** -148)
    for entropy in (True, False):
        lp = bd.TokenLogprobs(6, vocab, top=3, entropy=entropy)
        lp.run(x, tokens, heat)
        r = _check(lp, x, tokens, heat, entropy)
        places = x.double().sort(dim=1, descending=True, stable=True).indices[:, :3]
        best = r["lp"].gather(1, places)
        far = torch.isinf(best)
        assert torch.equal(lp.top_logprobs.double()[far], best[far])
        tol = (U * (8 + 4 * r["D"] + vocab / 32 + 36))[:, None] + U * 6 * best.abs()
        _near(lp.top_logprobs[~far], best[~far], tol[~far], "top_logprobs")
        _check_gradient(lp.backward(x, g), r, tokens, heat, g, None, dtype, least)
        if entropy:
            _check_gradient(lp.backward(x, g, h), r, tokens, heat, g, h, dtype, least)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("vocab", [4, 1003, 40000])
@pytest.mark.parametrize("heat", [1e-5, 1e-18, 1e-25, 1e-37, 4e-39, 2e-39, 1e-40, 2.0 ** -149])
def test_large_logits_at_low_temperatures(dtype, vocab, heat):
    """Maxima so large that their next neighbours are infinitely far below them."""
    heat = _number(heat)
    rows = 8
    x = torch.zeros(rows, vocab, device="cuda")
    for i, most in enumerate((1e20, -1e20, 2.0 ** 60, 2.0 ** 59, 1e38, -3e38, torch.finfo(dtype).max, -1e10)):
        x[i] = most - abs(most) / 64 if i != 6 else -most
        x[i, 1] = x[i, vocab - 1] = most
    x[1, 0] = x[5, 0] = -float("inf")
    x = x.to(dtype)
    tokens = torch.tensor([1, 1, 0, 1, 2, 1, 1, 1], device="cuda")
    g, h = torch.randn(rows, device="cuda"), torch.randn(rows, device="cuda")
    small = min(1.0, heat * 1e35)
    for entropy in (True, False):
        lp = bd.TokenLogprobs(rows, vocab, top=3, entropy=entropy)
        lp.run(x, tokens, heat)
        r = _check(lp, x, tokens, heat, entropy)
        for of in (1.0, small):
            _check_gradient(lp.backward(x, g * of), r, tokens, heat, g * of, None, dtype, 2.0 ** -148)
            if entropy:
                _check_gradient(lp.backward(x, g * of, h * of), r, tokens, heat, g * of, h * of, dtype, 2.0 ** -148)
