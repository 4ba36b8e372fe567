"""bo_adamw_plan refuses memory that a step would write twice, or read while another block of it
writes: nothing is launched, so addresses that lead nowhere do."""
import ctypes

import pytest
import torch

import lossless_bf16_weight_old_gb300 as bd
from lossless_bf16_weight_old_gb300 import _ops_lib as ol

P = ctypes.c_void_p
BAD = 1
W, O, G = 1 << 20, 1 << 21, 1 << 22       # weights, outputs, gradients


def _plan(items, kind=1, bits=32, state=None, ws=1 << 30):
    lib = ol.load()
    k = len(items)
    arr = (ol.AdamWItem * k)(*[ol.AdamWItem(w, o, g, n, b, 0.0, 0) for w, o, g, n, b in items])
    st = ol.AdamWState(1 << 24, 1 << 25, 1 << 26, 1 << 27, 1 << 28, 64)
    for name, v in (state or {}).items():
        setattr(st, name, v)
    h = ol.AdamW()
    return lib.bo_adamw_plan(arr, k, ctypes.byref(st), kind, 0, bits, 0, 0, P(ws), 1 << 20,
                             ctypes.byref(h), None)


def _two(**second):
    """Two items of 1000 elements side by side, the second with what is given instead."""
    a = dict(w=W, o=O, g=G, n=1000, b=0)
    b = dict(w=W + 4096, o=O + 4096, g=G + 4096, n=1000, b=4)
    b.update(second)
    return [tuple(a.values()), tuple(b[x] for x in "wognb")]


@pytest.mark.parametrize("second", [
    dict(o=O), dict(o=O + 1984), dict(o=O - 1984),             # the same output, or a part of it
    dict(o=W), dict(o=W + 1984),                               # the other's weights
    dict(o=G), dict(o=G + 1984), dict(g=O), dict(w=O),         # ... gradients, output
    dict(b=0), dict(b=3),                                      # its blocks
    dict(w=W, o=W),                                            # tied weights, in place
])
@pytest.mark.parametrize("in_place", [False, True])
def test_two_items(second, in_place):
    items = _two(**second)
    if in_place:
        items = [(o if i == 0 else w, o, g, n, b) for i, (w, o, g, n, b) in enumerate(items)]
        if second in (dict(o=W), dict(o=W + 1984), dict(w=W, o=W)):
            return                                             # (the first's weights are elsewhere then)
    assert _plan(items) == BAD


@pytest.mark.parametrize("bits,state", [
    (32, dict(d_v=1 << 24)), (32, dict(d_v=(1 << 24) + 256)), (32, dict(d_m=O)),
    (32, dict(d_v=(1 << 30) + 256)), (8, dict(d_m_scale=1 << 24)), (8, dict(d_v_scale=O + 256)),
    (8, dict(d_v_scale=1 << 26)), (8, dict(d_m=1 << 30)),
])
def test_arenas(bits, state):
    assert _plan(_two(), bits=bits, state=state) == BAD


def test_a_master_over_gradients():
    assert _plan(_two(), kind=0, state=dict(d_master=G)) == BAD
    assert _plan(_two(), kind=0, state=dict(d_master=1 << 25)) == BAD
    assert _plan(_two(o=O), kind=0) == BAD


@pytest.mark.gpu
def test_tensors():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    w = torch.zeros(1024, dtype=torch.bfloat16, device="cuda")
    g, h = torch.ones_like(w), torch.ones_like(w)
    for kw in (dict(master=True), dict(master=False)):
        with pytest.raises(bd.OpsError):
            bd.AdamWBatch([w, w], [g, h], **kw)                # tied
        with pytest.raises(bd.OpsError):
            bd.AdamWBatch([w[:512], w[256:768]], [g[:512], h[:512]], **kw)
    new = torch.zeros_like(w)
    with pytest.raises(bd.OpsError):
        bd.AdamWBatch([w[:512], w[512:]], [g[:512], g[512:]], news=[new[:512], new[:512]])
    with pytest.raises(bd.OpsError):                           # out of place over another's weights
        bd.AdamWBatch([w[:512], w[512:]], [g[:512], g[512:]], news=[new[:512], w[:512]], master=False)
    # what does not meet is taken: neighbours, one gradient for two tensors, empty tensors anywhere
    ad = bd.AdamWBatch([w[:512], w[512:], w[:0]], [g[:512], g[:512], g[:0]], lr=0.125, eps=0.0)
    ad.run()
    assert bool((w == -0.125).all())
    ad = bd.AdamWBatch([w[:512], w[512:]], [g[:512], g[512:]], news=[new[:512], new[512:]], lr=0.125,
                       master=False)
    ad.run()
    assert bool((w == -0.125).all()) and bool((new == -0.25).all())
