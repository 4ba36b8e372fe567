"""What bo_adapter_set_init refuses of the gradients that it is given: nothing is launched, so
addresses that lead nowhere do."""
import ctypes

import pytest
import torch

import lossless_bf16_weight_old_gb300 as bd
from lossless_bf16_weight_old_gb300 import _ops_lib as ol

P = ctypes.c_void_p
BAD = 1
HIDDEN, OUT, RANK = 64, 32, 16


def _init(items, grad=0, ws=1 << 40):
    k = len(items)
    arr = (ol.Adapter * k)(*[ol.Adapter(*i) for i in items])
    h = ol.AdapterSet()
    return ol.load().bo_adapter_set_init(arr, k, HIDDEN, OUT, grad, P(ws), 1 << 20, ctypes.byref(h), None)


def _item(i, gd=None, gu=None, ldgd=HIDDEN, ldgu=RANK):
    return (1 << 20) + 4096 * i, (1 << 21) + 4096 * i, HIDDEN, RANK, gd, gu, ldgd, ldgu, RANK, 1.0


def test_gradients_of_some_adapters_only():
    a, b = _item(0), _item(1, 1 << 22, 1 << 23)
    assert _init([a, b]) == BAD and _init([b, a]) == BAD
    assert _init([b, _item(0, 1 << 24, None)]) == BAD and _init([b, _item(0, None, 1 << 24)]) == BAD
    assert _init([_item(0, 1 << 24, None)]) == BAD and _init([_item(0, None, 1 << 24)]) == BAD


def test_gradients_over_others_and_over_factors():
    d, u = 1 << 22, 1 << 23                    # 16 x 64 and 32 x 16 values: 2048 and 1024 bytes
    for gd, gu in ((d, u + 4096), (d + 2046, u + 4096), (d + 4096, u), (d + 4096, u - 1022),
                   (u, u + 4096), (d + 4096, d), (d + 4096, d + 4096), ((1 << 20) + 4096, u + 4096),
                   (1 << 20, u + 4096), (d + 4096, 1 << 21), (d + 4096, (1 << 21) + 1022)):
        items = [_item(0, d, u), _item(1, gd, gu)]
        assert _init(items) == BAD and _init(items[::-1]) == BAD, (gd - d, gu - u)
    # twice the size in FP32
    assert _init([_item(0, d, u), _item(1, d + 2048, u + 4096)], grad=1) == BAD
    # columns of one buffer with an element in common
    assert _init([_item(0, d, u, ldgu=31), _item(1, d + 4096, u + 30, ldgu=31)]) == BAD
    # among many
    items = [_item(i, d + 4096 * i, u + (1 << 22) + 4096 * i) for i in range(300)]
    items[271] = _item(271, d + 4096 * 271, items[13][5])
    assert _init(items) == BAD


@pytest.mark.gpu
def test_gradients_that_lie_apart():
    """Columns of one buffer, neighbours in memory, and shared factors are taken, and written where
    they belong: as of sets of one adapter each."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    gen = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").bfloat16()

    k, rows, hidden, out, ranks = 3, 200, 72, 40, [8, 5, 16]
    index = torch.arange(rows, device="cuda", dtype=torch.int32) % k
    x, dy, dx = normal(rows, hidden), normal(rows, out), normal(rows, hidden)
    down, up = normal(16, hidden), normal(out, 16)
    downs, ups = [down[:r] for r in ranks], [up[:, :r] for r in ranks]
    all_downs = torch.zeros(sum(ranks), hidden, device="cuda")
    all_ups = torch.zeros(out, sum(ranks), device="cuda")
    s = bd.AdapterSet(downs, ups, 0.5, d_downs=all_downs.split(ranks), d_ups=all_ups.split(ranks, 1))
    plan = bd.AdapterRows(index, k)
    low = torch.empty(rows, s.rank, dtype=torch.bfloat16, device="cuda")
    bd.adapter_forward(x, normal(rows, out), s, plan, low=low)
    bd.adapter_backward(x, dy, low, dx, s, plan)
    for i, r in enumerate(ranks):
        d = torch.zeros(r, hidden, device="cuda"), torch.zeros(out, r, device="cuda")
        one = bd.AdapterSet([downs[i]], [ups[i]], 0.5, d_downs=[d[0]], d_ups=[d[1]])
        mine = torch.nonzero(index == i).squeeze(1)
        p1 = bd.AdapterRows(torch.zeros(len(mine), dtype=torch.int32, device="cuda"), 1)
        low1 = low[mine][:, :one.rank].contiguous()
        bd.adapter_backward(x[mine], dy[mine], low1, None, one, p1)
        a = sum(ranks[:i])
        # dlow is one rounding to BF16 of a sum whose order the batch may decide: a unit, 2^-7, of
        # each term between the two, and as much again for all FP32 sums
        for got, want, p, q in ((all_downs[a:a + r], d[0], 0.5 * dy[mine].float() @ ups[i].float(), x[mine]),
                                (all_ups[:, a:a + r].T, d[1].T, low1[:, :r].float(), dy[mine])):
            size = p.abs().T @ q.float().abs()
            assert bool(((got - want).abs() <= 2.0 ** -6 * size).all())
            assert bool((got != 0).any())
