"""The bounded waits of the adapters' kernels on the tensor cores' own memory (GPU).

A flag of the set keeps the first stage of every block from being reported, which is all that the
others wait for.  The waits (two seconds each) run out, the call ends by itself and says so in the
rows' status, and the context, the memory and the same objects serve the next call."""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("lossless_bf16_weight_old_gb300")

STALL = 0x80000000


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    bd._ops_lib.load()


def _objects(rows, hidden, out, rank):
    gen = torch.Generator(device="cuda").manual_seed(rank)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").bfloat16()

    down, up = normal(rank, hidden), normal(out, rank)
    d = [torch.zeros_like(down)], [torch.zeros_like(up)]
    s = bd.AdapterSet([down], [up], d_downs=d[0], d_ups=d[1])
    index = torch.zeros(rows, dtype=torch.int32, device="cuda")
    return normal(rows, hidden), normal(rows, out), s, bd.AdapterRows(index, 1), index, d


def _stalled(s, plan, call):
    torch.cuda.synchronize()
    s.handle.wide |= STALL
    t0 = time.monotonic()
    call()
    torch.cuda.synchronize()
    took = time.monotonic() - t0
    s.handle.wide &= ~STALL & 0xFFFFFFFF
    assert int(plan.status.item()) == bd.ERR_CUDA
    assert 1.0 < took < 30, took


@pytest.mark.parametrize("rank,hidden", [(16, 4096), (64, 128)])   # (clusters, many stages; one stage)
def test_low(rank, hidden):
    rows = int(2e8 / (2 * (hidden + 2 * 16384))) + 1
    x, y, s, plan, index, _ = _objects(rows, hidden, 16384, rank)
    assert s._low_rows <= rows
    low = torch.empty(rows, s.rank, dtype=torch.bfloat16, device="cuda")
    want = bd.adapter_forward(x, y.clone(), s, plan, low=low)
    want_low = low.clone()
    _stalled(s, plan, lambda: bd.adapter_forward(x, y.clone(), s, plan, low=low))
    plan.update(index)
    assert torch.equal(bd.adapter_forward(x, y.clone(), s, plan, low=low), want)
    assert torch.equal(low, want_low) and int(plan.status.item()) == bd.OK


@pytest.mark.parametrize("rank", [16, 128])
def test_weight_gradients(rank):
    x, dy, s, plan, index, d = _objects(900, 1024, 2048, rank)
    low = torch.randn(900, s.rank, device="cuda").bfloat16()
    ws = torch.empty(int(bd._ops_lib.load().bo_adapter_backward_workspace_size(s._ref, 900)),
                     dtype=torch.uint8, device="cuda")

    def go():
        bd.adapter_backward(x, dy, low, None, s, plan, workspace=ws)

    go()
    want = [d[0][0].clone(), d[1][0].clone()]
    _stalled(s, plan, go)
    plan.update(index)
    go()
    assert torch.equal(d[0][0], want[0]) and torch.equal(d[1][0], want[1])
    assert int(plan.status.item()) == bd.OK and bool(want[0].any()) and bool(want[1].any())
