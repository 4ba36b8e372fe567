"""What adapter_backward takes as its workspace: memory that nothing else of the call lies in, and a
tensor whose elements lie in one piece on the right device."""
import ctypes

import pytest
import torch

import lossless_bf16_weight_old_gb300 as bd
from lossless_bf16_weight_old_gb300 import _ops_lib as ol

P = ctypes.c_void_p
BAD = 1


def test_a_workspace_over_an_input():
    lib = ol.load()
    s = ol.AdapterSet(1 << 20, 2, 64, 32, 16, 0, 0, 1)
    r = ol.AdapterRows()
    r.d_perm, r.d_offsets, r.d_blocks, r.d_ntiles, r.rows, r.k = 4096, 8192, 1 << 14, 1 << 15, 10, 2
    for i in range(3):
        r.d_tiles[i] = 1 << 16
    need = lib.bo_adapter_backward_workspace_size(ctypes.byref(s), 10)
    ws = 1 << 30

    def backward(x=1 << 24, dy=1 << 25, low=1 << 26, dx=1 << 27):
        return lib.bo_adapter_backward(ctypes.byref(s), ctypes.byref(r), P(x), 64, P(dy), 32, P(low),
                                       P(dx), 64, 0, P(ws), need, None)

    last = ws + need - 16
    for kw in (dict(x=ws), dict(x=last), dict(x=ws - 10 * 64 * 2 + 16), dict(dy=ws + 256), dict(dy=last),
               dict(low=ws), dict(low=last), dict(low=ws - 16), dict(dx=last)):
        assert backward(**kw) == BAD, kw


@pytest.mark.gpu
def test_workspace_tensors():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")

    def z(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")

    s = bd.AdapterSet([z(8, 64)], [z(32, 8)], d_downs=[z(8, 64)], d_ups=[z(32, 8)])
    rows = bd.AdapterRows(torch.zeros(10, dtype=torch.int32, device="cuda"), 1)
    args = z(10, 64), z(10, 32), z(10, s.rank), z(10, 64), s, rows
    need = int(ol.load().bo_adapter_backward_workspace_size(s._ref, 10))
    wide = torch.empty(need // 256 + 1, 512, dtype=torch.uint8, device="cuda")
    for ws in (wide[:, :256], wide[::2], torch.empty(need, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="workspace"):
            bd.adapter_backward(*args, workspace=ws)
    with pytest.raises(bd.OpsError):
        bd.adapter_backward(*args, workspace=wide.view(-1)[:need - 256])
    bd.adapter_backward(*args, workspace=wide.view(-1)[:need])
    torch.cuda.synchronize()
