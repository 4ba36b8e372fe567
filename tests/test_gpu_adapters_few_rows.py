"""The product with low in two BF16 numbers, which batches of few rows take (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("lossless_bf16_weight_old_gb300")

U, F = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    bd._ops_lib.load()


def _rows(n):
    return bd.AdapterRows(torch.zeros(n, dtype=torch.int32, device="cuda"), 1)


@pytest.mark.parametrize("rows", [1, 20])
@pytest.mark.parametrize("rank,out", [(5, 96), (16, 512), (24, 512), (64, 512)])
def test_low_is_not_rounded_to_one_number(rows, rank, out):
    """y starts where the sum ends at next to nothing, so that y's own rounding hides no error of
    low.  Of the two numbers the second is rounded: u^2 |low| and the FP32 sum's error in low (K f
    of the sizes of its terms), r + 1 FP32 sums in y, and one rounding of what is left."""
    hidden = 64
    gen = torch.Generator(device="cuda").manual_seed(rank)
    x = torch.randn(rows, hidden, generator=gen, device="cuda").bfloat16()
    down = (torch.randn(rank, hidden, generator=gen, device="cuda") * 0.125).bfloat16()
    up = torch.randn(out, rank, generator=gen, device="cuda").bfloat16()
    low = x.double() @ down.double().T
    part = low @ up.double().T
    y = (-part).bfloat16()
    want = y.double() + part
    e_low = U * U * low.abs() + hidden * F * (x.double().abs() @ down.double().abs().T)
    size = low.abs() @ up.double().abs().T
    tol = e_low @ up.double().abs().T + (rank + 1) * F * (y.double().abs() + size)
    tol = tol * (1 + U) + U * want.abs()
    got = bd.adapter_forward(x, y.clone(), bd.AdapterSet([down], [up]), _rows(rows)).double()
    assert bool(((got - want).abs() <= tol).all())
    # (one rounding of low would be seen)
    once = (y.double() + low.bfloat16().double() @ up.double().T).bfloat16().double()
    assert not bool(((once - want).abs() <= tol).all())


@pytest.mark.parametrize("rows", [4, 600, 3000])
@pytest.mark.parametrize("rank", [8, 24])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_a_low_that_rounds_to_infinity(rows, rank, sign):
    """Beyond BF16's largest number and within FP32's: infinity in low, and in y with a factor's
    sign, however many rows there are."""
    x = torch.zeros(rows, 64, dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1] = sign * 3.3895e38, sign * 1.2e36       # their sum: 3.4015e38
    down = torch.zeros(rank, 64, dtype=torch.bfloat16, device="cuda")
    down[:, :2] = 1.0
    up = torch.full((64, rank), 0.25, dtype=torch.bfloat16, device="cuda")
    up[3] = -0.5
    y = torch.ones(rows, 64, dtype=torch.bfloat16, device="cuda")
    s = bd.AdapterSet([down], [up])
    low = torch.empty(rows, s.rank, dtype=torch.bfloat16, device="cuda")
    bd.adapter_forward(x, y, s, _rows(rows), low=low)
    want = torch.full((64,), sign * float("inf"), dtype=torch.bfloat16, device="cuda")
    assert bool((low[:, :rank] == want[0]).all()) and not bool(low[:, rank:].any())
    want[3] = -want[3]
    assert bool((y == want).all())
