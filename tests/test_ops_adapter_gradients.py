"""What bo_adapter_set_init refuses of the gradients that it is given: nothing is launched, so
addresses that lead nowhere do."""
import ctypes

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
