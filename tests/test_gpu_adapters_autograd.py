"""Tensors that autograd records are refused, not passed by (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("lossless_bf16_weight_old_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    bd._ops_lib.load()


class _Adapter(torch.autograd.Function):
    """The two calls as autograd takes them."""

    @staticmethod
    def forward(ctx, x, y, s, plan, low):
        ctx.save_for_backward(x, low)
        ctx.s, ctx.plan = s, plan
        return bd.adapter_forward(x, y.clone(), s, plan, low=low)

    @staticmethod
    def backward(ctx, dy):
        x, low = ctx.saved_tensors
        dx = torch.zeros_like(x)
        bd.adapter_backward(x, dy.contiguous(), low, dx, ctx.s, ctx.plan)
        return dx, dy, None, None, None


def test_recorded_tensors():
    gen = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").bfloat16()

    x, y, dy, dx = normal(20, 64), normal(20, 32), normal(20, 32), normal(20, 64)
    down, up = torch.nn.Parameter(normal(8, 64)), torch.nn.Parameter(normal(32, 8))
    s = bd.AdapterSet([down], [up], d_downs=[torch.zeros(8, 64, device="cuda")],
                      d_ups=[torch.zeros(32, 8, device="cuda")])
    plan = bd.AdapterRows(torch.zeros(20, dtype=torch.int32, device="cuda"), 1)
    low = torch.zeros(20, s.rank, dtype=torch.bfloat16, device="cuda")
    want = bd.adapter_forward(x, y.clone(), s, plan, low=low)
    for which in (x, y):
        which.requires_grad_()
        y0 = y.detach().clone()
        with pytest.raises(ValueError, match="autograd"):
            bd.adapter_forward(x, y, s, plan)
        assert torch.equal(y.detach(), y0)
        with torch.no_grad():
            assert torch.equal(bd.adapter_forward(x, y.clone(), s, plan), want)
        which.requires_grad_(False)
    for which in (dy, dx):
        which.requires_grad_()
        with pytest.raises(ValueError, match="autograd"):
            bd.adapter_backward(x, dy, low, dx, s, plan)
        which.requires_grad_(False)
    # through an autograd function, where nothing is recorded inside
    g = normal(20, 32)
    x.requires_grad_()
    out = _Adapter.apply(x, y, s, plan, low)
    assert torch.equal(out.detach(), want)
    out.backward(g)
    bd.adapter_backward(x.detach(), g, low, ref := torch.zeros_like(dx), s, plan)
    assert torch.equal(x.grad, ref) and bool(ref.any())
