"""Calls with another current device than the tensors', the handles' or the stream's are refused
before anything is launched.  One device is enough: the other is a number that no handle is made
with, or a stand-in.  (Handles that do not go together need no GPU.)"""
import ctypes
import types

import pytest
import torch

import lossless_bf16_weight_old_gb300 as bd
from lossless_bf16_weight_old_gb300 import _ops_lib as ol

P = ctypes.c_void_p


def test_a_set_and_rows_of_different_devices():
    lib = ol.load()
    s = ol.AdapterSet(1 << 20, 2, 64, 32, 16, 0, 0, 1)
    r = ol.AdapterRows()
    r.d_perm, r.d_offsets, r.d_blocks, r.d_ntiles, r.rows, r.k = 4096, 8192, 1 << 14, 1 << 15, 10, 2
    for i in range(3):
        r.d_tiles[i] = 1 << 16
    r.device = 1
    assert lib.bo_adapter_forward(ctypes.byref(s), ctypes.byref(r), P(1 << 24), 64, P(1 << 25), 32,
                                  None, None) == 1
    n = lib.bo_adapter_backward_workspace_size(ctypes.byref(s), 10)
    assert lib.bo_adapter_backward(ctypes.byref(s), ctypes.byref(r), P(1 << 24), 64, P(1 << 25), 32,
                                   P(1 << 26), P(1 << 27), 64, 0, P(1 << 30), n, None) == 1


def _objects():
    def z(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device="cuda")
    t = dict(x=z(4, 64), y=z(4, 32), dx=z(4, 64), w=z(100), g=z(100) + 1, down=z(8, 64), up=z(32, 8),
             index=z(4, dtype=torch.int32))
    s = bd.AdapterSet([t["down"]], [t["up"]], d_downs=[z(8, 64)], d_ups=[z(32, 8)])
    t["low"] = z(4, s.rank)
    return t, s, bd.AdapterRows(t["index"], 1), bd.AdamWBatch([t["w"]], [t["g"]], state_bits=8, max_norm=1.0)


def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


@pytest.mark.gpu
def test_handles_of_another_device():
    _gpu()
    t, s, rows, adam = _objects()
    s.handle.device = rows.handle.device = adam.handle.device = 1
    calls = [lambda: bd.adapter_forward(t["x"], t["y"], s, rows),
             lambda: bd.adapter_backward(t["x"], t["y"], t["low"], t["dx"], s, rows),
             adam.run, adam.grad_norm, adam.moments]
    for call in calls:
        with pytest.raises(bd.OpsError):
            call()
    torch.cuda.synchronize()
    assert int(adam.steps.item()) == 0 and not t["w"].any() and float(adam.norm.item()) == 0
    s.handle.device = rows.handle.device = adam.handle.device = 0
    for call in calls:
        call()
    assert int(adam.steps.item()) == 1


@pytest.mark.gpu
def test_tensors_of_another_device(monkeypatch):
    _gpu()
    t, s, rows, adam = _objects()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (lambda: bd.AdamWBatch([t["w"]], [t["g"]]),
                 lambda: bd.AdapterSet([t["down"]], [t["up"]]),
                 lambda: bd.AdapterRows(t["index"], 1),
                 lambda: rows.update(t["index"])):
        with pytest.raises(ValueError, match="current device"):
            call()


@pytest.mark.gpu
def test_streams_and_rates_of_another_device():
    _gpu()
    t, s, rows, adam = _objects()
    far = types.SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=0)
    for call in (lambda: bd.AdamWBatch([t["w"]], [t["g"]], stream=far),
                 lambda: bd.AdapterSet([t["down"]], [t["up"]], stream=far),
                 lambda: bd.AdapterRows(t["index"], 1, stream=far),
                 lambda: rows.update(t["index"], far),
                 lambda: adam.run(stream=far), lambda: adam.grad_norm(far),
                 lambda: adam.moments(stream=far),
                 lambda: bd.adapter_forward(t["x"], t["y"], s, rows, stream=far),
                 lambda: bd.adapter_backward(t["x"], t["y"], t["low"], t["dx"], s, rows, stream=far)):
        with pytest.raises(ValueError, match="the stream is on"):
            call()
    with pytest.raises(ValueError, match="lr"):
        adam.run(lr=torch.zeros(1))
    torch.cuda.synchronize()
    assert int(adam.steps.item()) == 0
