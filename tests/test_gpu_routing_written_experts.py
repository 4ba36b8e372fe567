"""The gradient of routing reads the run's experts from its results, where a caller may have written (GPU)."""
import pytest
import torch

from test_gpu_routing import BF16, FP32, _logits

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("lossless_bf16_weight_old_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    bd._ops_lib.load()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("tokens,experts,k", [(5, 16, 2), (700, 60, 4), (9000, 128, 8), (200, 1000, 32)])
def test_numbers_that_are_no_experts(dtype, tokens, experts, k):
    """As of tokens that are left out; memory behind the logits' gradient stays as it was."""
    x = _logits(tokens, experts, dtype)
    gw = torch.randn(tokens, k, device="cuda")
    a = bd.ExpertRouting(tokens, experts, k)
    a.run(x)
    want = a.backward(x, gw, 2.0)
    memory = torch.full(((tokens + 64) * experts,), 7.0, dtype=dtype, device="cuda")
    out = memory[32 * experts:(tokens + 32) * experts].view(tokens, experts)
    far = torch.zeros(tokens, dtype=torch.bool, device="cuda")
    far[::3] = True
    kept = a.experts.clone()
    for number in (experts, experts + 31, -2, 1 << 30, -(1 << 31)):
        a.experts[far] = number
        a.backward(x, gw, 2.0, out=out)
        assert not out[far].any() and torch.equal(out[~far], want[~far])
        assert (memory[:32 * experts] == 7.0).all() and (memory[(tokens + 32) * experts:] == 7.0).all()
        a.experts.copy_(kept)
    assert torch.equal(a.backward(x, gw, 2.0), want)
