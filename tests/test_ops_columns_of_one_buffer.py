"""Matrices whose rows lie between one another's, as columns of one buffer do, share no memory and
are taken; those that share an element are refused."""
import ctypes
import random

import pytest
import torch

import lossless_bf16_weight_old_gb300 as bd
from lossless_bf16_weight_old_gb300 import _ops_lib as ol

P = ctypes.c_void_p
BAD, NO_GPU = 1, 5


def _elements(at, ld, width, rows):
    return {at + 2 * (r * ld + c) for r in range(rows) for c in range(width)}


def test_which_are_refused():
    """Where a call's arguments are in order it goes on to the GPU, which is not there."""
    if torch.cuda.is_available():
        pytest.skip("the calls that are not refused would run")
    lib, rng = ol.load(), random.Random(5)
    base, seen = 1 << 20, {BAD: 0, NO_GPU: 0}
    for _ in range(4000):
        hidden, out, n = rng.randint(1, 9), rng.randint(1, 9), rng.randint(1, 5)
        ldx = max(hidden, rng.randint(1, 20))
        ldy = ldx if rng.random() < 0.8 and ldx >= out else max(out, rng.randint(1, 20))
        at = base + 2 * rng.randint(-60, 60)
        s = ol.AdapterSet(1 << 30, 2, hidden, out, 16, 0, 0, 0)
        r = ol.AdapterRows()
        r.d_perm, r.d_offsets, r.d_blocks, r.d_ntiles, r.rows, r.k = 4096, 8192, 1 << 14, 1 << 15, n, 2
        for i in range(3):
            r.d_tiles[i] = 1 << 16
        x, y = _elements(base, ldx, hidden, n), _elements(at, ldy, out, n)
        rc = lib.bo_adapter_forward(ctypes.byref(s), ctypes.byref(r), P(base), ldx, P(at), ldy, None, None)
        assert rc in (BAD, NO_GPU)
        if x & y:
            assert rc == BAD, (hidden, out, n, ldx, ldy, at - base)
        elif ldx == ldy or n == 1 or max(x) < min(y) or max(y) < min(x):
            assert rc == NO_GPU, (hidden, out, n, ldx, ldy, at - base)
        seen[rc] += 1
    assert min(seen.values()) > 500


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [3, 700, 2500])
@pytest.mark.parametrize("hidden,out", [(64, 128), (61, 67)])
def test_columns_of_one_buffer(rows, hidden, out):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    gen = torch.Generator(device="cuda").manual_seed(rows)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").bfloat16()

    down, up = normal(8, hidden), normal(out, 8)
    d = dict(d_downs=[torch.zeros_like(down)], d_ups=[torch.zeros_like(up)])
    s = bd.AdapterSet([down], [up], 0.5, **d)
    plan = bd.AdapterRows(torch.zeros(rows, dtype=torch.int32, device="cuda"), 1)
    low = torch.empty(rows, s.rank, dtype=torch.bfloat16, device="cuda")
    apart = [normal(rows, n) for n in (hidden, out, out, hidden)]
    buf = torch.cat(apart, 1)
    joined = buf.split([hidden, out, out, hidden], 1)
    got = []
    for x, y, dy, dx in (apart, joined):
        bd.adapter_forward(x, y, s, plan, low=low)
        bd.adapter_backward(x, dy, low, dx, s, plan)
        got.append([t.clone() for t in (x, y, dy, dx, d["d_downs"][0], d["d_ups"][0])])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    with pytest.raises(bd.OpsError):
        bd.adapter_forward(buf[:, :hidden], buf[:, hidden - 1:hidden - 1 + out], s, plan)
