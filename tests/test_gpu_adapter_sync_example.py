"""The example that trains adapters, sends them as deltas and serves them (GPU)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_learns_and_keeps_the_worker_in_step():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    spec = importlib.util.spec_from_file_location(
        "adapter_sync", os.path.join(ROOT, "examples", "adapter_sync.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.main(12)   # (raises when a worker's answer differs in any bit)
    assert losses[-1] < 0.8 * losses[0]
