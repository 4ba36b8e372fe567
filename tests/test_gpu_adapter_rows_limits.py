"""The operators at the ends of what they take (GPU): counts past 32 bits, and more adapters than a
block of the grouping has threads."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("lossless_bf16_weight_old_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    bd._ops_lib.load()


def test_counts_past_32_bits_are_refused():
    index = torch.zeros(4, dtype=torch.int32, device="cuda")
    for k in (0, -1, 65536, (1 << 32) + 1, (1 << 33) + 5):
        with pytest.raises(ValueError, match="65535"):
            bd.AdapterRows(index, k)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    for rows in ((1 << 30) + 1, (1 << 32) + 4):
        with pytest.raises(ValueError, match="at most"):
            bd.AdapterRows(one.expand(rows), 1)
    wide = torch.empty(1, (1 << 32) + 64, dtype=torch.bfloat16, device="cuda")
    tall = torch.empty((1 << 32) + 64, 1, dtype=torch.bfloat16, device="cuda")
    small = torch.zeros(1, 8, dtype=torch.bfloat16, device="cuda")
    for down, up in ((wide, small.T), (small, tall), (wide[:, :(1 << 24) + 1], small.T),
                     (small[:, :0], small.T), (small, small.T[:0])):
        with pytest.raises(ValueError, match="widths"):
            bd.AdapterSet([down], [up])
    for step in (-1, (1 << 64) + 5):
        with pytest.raises(ValueError, match="step"):
            bd.AdamWBatch([small], [small.clone()], step=step)
    del wide, tall
    torch.cuda.empty_cache()


@pytest.mark.parametrize("k,rows", [(257, 300), (700, 5000), (700, 3), (65535, 4000)])
def test_more_adapters_than_threads(k, rows):
    """Adapters of rank 1 whose factors are small whole numbers: every product is exact in FP32, and
    whole numbers below 256 in BF16, so that the results are equal to the formula's."""
    rng = np.random.default_rng(k + rows)
    gen = torch.Generator(device="cuda").manual_seed(rows)

    def whole(*shape):
        return torch.randint(-2, 3, shape, generator=gen, device="cuda").bfloat16()

    x, y, downs, ups = whole(rows, 16), whole(rows, 8), whole(k, 1, 16), whole(k, 8, 1)
    x[:, 8:] = 0     # low is at most 32
    d_downs, d_ups = torch.full((k, 1, 16), 9.0, device="cuda"), torch.full((k, 8, 1), 9.0, device="cuda")
    s = bd.AdapterSet(list(downs), list(ups), d_downs=list(d_downs), d_ups=list(d_ups))
    index = torch.from_numpy(rng.integers(-1, k, rows).astype(np.int32)).cuda()
    index[-1], index[0] = k - 1, 256 if k > 256 else 0
    plan = bd.AdapterRows(index, k)
    low = torch.zeros(rows, s.rank, dtype=torch.bfloat16, device="cuda")
    dy, dx = whole(rows, 8), torch.zeros(rows, 16, dtype=torch.bfloat16, device="cuda")
    want = y.double()
    at = index.clamp(min=0).long()
    has = (index >= 0).double()[:, None]
    p = (x.double()[:, None, :] * downs[at, 0].double()[:, None, :]).sum(2) * has
    q = (dy.double() * ups[at, :, 0].double()).sum(1, keepdim=True) * has
    want += p * ups[at, :, 0].double()
    bd.adapter_forward(x, y, s, plan, low=low)
    bd.adapter_backward(x, dy, low, dx, s, plan)
    assert int(plan.status.item()) == bd.OK
    assert torch.equal(y.double(), want)
    assert torch.equal(dx.double(), q * downs[at, 0].double())
    ga, gb = torch.zeros(k, 16, dtype=torch.double, device="cuda"), torch.zeros(k, 8, dtype=torch.double, device="cuda")
    ga.index_add_(0, at, q * x.double())
    gb.index_add_(0, at, p * dy.double())
    assert torch.equal(d_downs[:, 0].double(), ga) and torch.equal(d_ups[:, :, 0].double(), gb)
