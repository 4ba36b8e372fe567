"""Routing of many tokens, which a warp takes 32 at a time: logits whose order hangs on their last bits,
equal ones, infinities and NaN, against the formulas (GPU)."""
import math

import pytest
import torch

from test_gpu_routing import BF16, FP32, _check_forward, _check_grad, _logits, _reference

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("lossless_bf16_weight_old_gb300")

INF, NAN = math.inf, math.nan
TOKENS = 21507     # more than the bound of any number of experts


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    bd._ops_lib.load()


SHAPES = [(2, 1), (5, 4), (8, 2), (16, 8), (16, 16), (17, 5), (48, 6), (64, 9), (100, 4), (128, 1), (128, 8),
          (128, 16), (160, 8), (250, 10), (256, 8), (256, 16)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("experts,k", SHAPES)
def test_shapes(dtype, experts, k):
    x = _logits(TOKENS, experts, dtype, ld=experts + 3, offset=1)
    mask = torch.rand(TOKENS, device="cuda") < 0.9
    for normalize in (True, False):
        a = bd.ExpertRouting(TOKENS, experts, k, normalize=normalize)
        a.run(x, mask)
        gw = torch.randn(TOKENS, k, device="cuda")
        r = _reference(x, k, normalize, mask, gw, 2.0)
        _check_forward(a, r, TOKENS)
        _check_grad(a.backward(x, gw, 2.0), r, dtype)


@pytest.mark.parametrize("experts,k", [(8, 2), (64, 6), (128, 8), (256, 16)])
@pytest.mark.parametrize("kind", ["last bits", "few values", "from BF16", "zeros", "constant", "powers"])
def test_order_in_32_bits(experts, k, kind):
    """FP32 logits that differ in their last bits alone, or not at all."""
    gen = torch.Generator(device="cuda").manual_seed(experts)
    shape = TOKENS, experts
    if kind == "last bits":      # neighbours of a few numbers, of both signs
        base = torch.randint(-3, 4, shape, generator=gen, device="cuda").float() * 0.7
        x = (base.view(torch.int32) + torch.randint(0, 700, shape, generator=gen, device="cuda", dtype=torch.int32)).view(FP32)
    elif kind == "few values":
        x = torch.randint(-2, 3, shape, generator=gen, device="cuda").float()
    elif kind == "from BF16":
        x = (torch.randn(shape, generator=gen, device="cuda") * 2).bfloat16().float()
    elif kind == "zeros":
        x = torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.5, 0.0, -0.0)
    elif kind == "constant":
        x = torch.full(shape, 1.5, device="cuda")
    else:                        # denormal and large numbers
        x = torch.exp2(torch.randint(-149, 6, shape, generator=gen, device="cuda").float())
        x = x * torch.randint(-1, 2, shape, generator=gen, device="cuda")
    a = bd.ExpertRouting(TOKENS, experts, k)
    a.run(x)
    _check_forward(a, _reference(x, k, True, None), TOKENS)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("experts,k", [(9, 4), (128, 8), (256, 16)])
def test_infinities(dtype, experts, k):
    x = _logits(TOKENS, experts, dtype)
    x[:, 5] = -INF
    x[100:300, 2:] = -INF               # fewer left than are chosen
    x[300:333] = -INF                   # nothing left
    x[400:444] = torch.finfo(dtype).min
    x[500, :3] = torch.finfo(dtype).max
    x[600:640, 1:] = torch.where(torch.rand(40, experts - 1, device="cuda") < 0.5, -INF, torch.finfo(dtype).min).to(dtype)
    mask = torch.ones(TOKENS, dtype=torch.uint8, device="cuda")
    mask[310], mask[1000:1100] = 0, 0
    ref = x.clone()
    x[1050] = NAN                       # in a place that the mask leaves out
    a = bd.ExpertRouting(TOKENS, experts, k)
    a.run(x, mask)
    gw = torch.randn(TOKENS, k, device="cuda")
    r = _reference(ref, k, True, mask, gw, 2.0)
    _check_forward(a, r, TOKENS)
    _check_grad(a.backward(x, gw, 2.0), r, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_not_a_number(dtype):
    """NaN of either sign and any payload counts as the greatest; the other tokens are as without it."""
    x = _logits(TOKENS, 128, dtype)
    clean = x.clone()
    bits = torch.int16 if dtype == BF16 else torch.int32
    inf = 0x7F80 if dtype == BF16 else 0x7F800000
    raw = x.view(bits)
    raw[3, 100], raw[40, 7], raw[50, 0] = inf + 1, -1, inf + 5
    raw[50, 127] = -2                   # two of them: the lower expert first
    x[60, 9] = INF
    a, b = bd.ExpertRouting(TOKENS, 128, 8), bd.ExpertRouting(TOKENS, 128, 8)
    a.run(x)
    b.run(clean)
    assert a.experts[[3, 40, 50, 60], 0].tolist() == [100, 7, 0, 9] and int(a.experts[50, 1]) == 127
    bad = torch.zeros(TOKENS, dtype=torch.bool, device="cuda")
    bad[[3, 40, 50, 60]] = True
    assert a.weights[bad].isnan().all() and a.loss.isnan().all()
    assert torch.equal(a.experts[~bad], b.experts[~bad]) and torch.equal(a.weights[~bad], b.weights[~bad])


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_calls_repeat_and_tokens_are_as_by_themselves(dtype):
    x = _logits(TOKENS, 128, dtype)
    a = bd.ExpertRouting(TOKENS, 128, 8)
    a.run(x)
    first = [t.clone() for t in (a.weights, a.experts, a.counts, a.probs, a.loss)]
    for _ in range(3):
        a.run(x)
        for p, q in zip(first, (a.weights, a.experts, a.counts, a.probs, a.loss)):
            assert torch.equal(p, q)
    a.run(x[777:1000])
    assert torch.equal(a.weights[:223], first[0][777:1000]) and torch.equal(a.experts[:223], first[1][777:1000])


def test_offsets_past_32_bits():
    """Rows 2^18 elements apart: the last ones begin behind 2^32 bytes."""
    rows, ld = 21000, 1 << 18
    memory = torch.empty(rows * ld, dtype=BF16, device="cuda")
    x = memory.view(rows, ld)[:, 1:65]
    x.copy_(torch.randn(rows, 64, device="cuda"))
    a = bd.ExpertRouting(rows, 64, 4)
    a.run(x)
    gw = torch.randn(rows, 4, device="cuda")
    r = _reference(x, 4, True, None, gw, 1.0)
    _check_forward(a, r, rows)
    _check_grad(a.backward(x, gw, 1.0, out=memory.view(rows, ld)[:, 100:164]), r, BF16)
