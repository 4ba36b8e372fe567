"""A token routed by itself and among others, with weights that are divided by their sum and that are not (GPU).

Experts are the same in any case.  Weights that are divided by their sum are the same bits; others are
divided by the sum over all experts, whose order few and many tokens have each their own of: both are within
(64 + 8 |d|) u of the formula's, d the chosen logit's distance from the greatest."""
import pytest
import torch

from test_gpu_routing import BF16, FP32, U, _logits

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("lossless_bf16_weight_old_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    bd._ops_lib.load()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("experts,k", [(8, 2), (60, 4), (128, 8), (256, 16)])
def test_a_token_by_itself_and_among_others(dtype, normalize, experts, k):
    x = _logits(21507, experts, dtype)
    a = bd.ExpertRouting(21507, experts, k, normalize=normalize)

    def of(begin, end):
        a.run(x[begin:end])
        return a.experts[:end - begin].clone(), a.weights[:end - begin].clone()
    most, many, some, one = of(0, 21507), of(0, 9000), of(0, 700), of(77, 78)
    for few in (many, some):
        n = few[0].shape[0]
        assert torch.equal(few[0], most[0][:n])
    assert torch.equal(one[0], most[0][77:78])
    # calls that take the same form
    assert torch.equal(many[1], most[1][:9000]) and torch.equal(one[1], some[1][77:78])
    if normalize:
        assert torch.equal(some[1], most[1][:700])
    else:
        d = (x[:700].double().amax(1, keepdim=True) - x[:700].double().gather(1, some[0].long())).clamp(min=0)
        off = (some[1].double() - most[1][:700].double()).abs()
        assert (off <= 2 * U * (64 + 8 * d) * most[1][:700].double()).all()
