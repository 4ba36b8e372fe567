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
