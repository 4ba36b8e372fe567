"""Tensors that autograd records, beside the logits: calls that would lose their gradient are refused (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("lossless_bf16_weight_old_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    bd._ops_lib.load()


def _calls():
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(20, 500, generator=gen, device="cuda")
    t = torch.randint(500, (20,), generator=gen, device="cuda")
    r = torch.randn(20, 16, generator=gen, device="cuda")
    lp, a = bd.TokenLogprobs(20, 500, entropy=True), bd.ExpertRouting(20, 16, 2)
    lp.run(x, t)
    a.run(r)
    heat, g, gw, one = (torch.rand(n, device="cuda") + 0.5 for n in ((20,), (20,), (20, 2), (1,)))
    return {
        "temperature": (heat, lambda v: lp.run(x, t, v)),
        "d_logprobs": (g, lambda v: lp.backward(x, v)),
        "d_entropy": (g, lambda v: lp.backward(x, None, v)),
        "out of log probabilities": (torch.zeros_like(x), lambda v: lp.backward(x, g, out=v)),
        "d_weights": (gw, lambda v: a.backward(r, v)),
        "d_loss": (one, lambda v: a.backward(r, None, v)),
        "out of routing": (torch.zeros_like(r), lambda v: a.backward(r, gw, out=v)),
    }


NAMES = ["temperature", "d_logprobs", "d_entropy", "out of log probabilities", "d_weights", "d_loss", "out of routing"]


@pytest.mark.parametrize("name", NAMES)
def test_recorded(name):
    value, call = _calls()[name]
    leaf = value.clone().requires_grad_()
    for recorded in (leaf, leaf * 2):
        with pytest.raises(ValueError, match="autograd records"):
            call(recorded)


@pytest.mark.parametrize("name", NAMES)
def test_not_recorded(name):
    value, call = _calls()[name]
    call(value)
    leaf = value.clone().requires_grad_()
    call((leaf * 2).detach())
    with torch.no_grad():
        call(leaf)
