"""Calls whose blocks take about 48 KB of shared memory, or more: each by itself in a process that has
launched nothing larger, and different ones from two threads at once (GPU)."""
import json
import subprocess
import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("lossless_bf16_weight_old_gb300")

# tokens, experts, k, type: the dynamic part is at most 48 KB, with the kernel's own it is more
SIZES = [(9000, 208, 8, "bfloat16"), (9000, 84, 8, "float32"), (262144, 58, 8, "bfloat16"), (64, 491, 8, "bfloat16"),
         (128, 491, 8, "float32"), (24, 722, 8, "bfloat16"), (12, 944, 8, "bfloat16"), (16, 945, 32, "float32")]
CHILD = """
import json, sys, torch
sys.path[:0] = sys.argv[1:3]
import lossless_bf16_weight_old_gb300 as bd
from test_gpu_routing import _check_forward, _logits, _reference
said = {}
for size in json.loads(sys.argv[3]):
    tokens, experts, k, kind = size
    x = _logits(tokens, experts, getattr(torch, kind))
    a = bd.ExpertRouting(tokens, experts, k)
    try:
        a.run(x)
        _check_forward(a, _reference(x, k, True, None), tokens)
        said[json.dumps(size)] = ""
    except (bd.OpsError, AssertionError) as e:
        said[json.dumps(size)] = repr(e)
print(json.dumps(said))
"""


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    bd._ops_lib.load()


@pytest.fixture(scope="module")
def said(request):
    """What a new process says of each size.  (None of them raises the limit for those after it.)"""
    here = request.path.parent
    r = subprocess.run([sys.executable, "-c", CHILD, str(here.parent), str(here), json.dumps(SIZES)],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout.splitlines()[-1])


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_about_48_kb(said, size):
    assert said[json.dumps(list(size))] == ""


def test_two_threads_of_different_sizes():
    """Both launch the same kernel, with 100 KB and with 78."""
    failed = []

    def work(experts):
        try:
            stream = torch.cuda.Stream()
            x = torch.zeros(64, experts, dtype=torch.bfloat16, device="cuda")
            a = bd.ExpertRouting(64, experts, 8, stream=stream)
            torch.cuda.synchronize()
            for _ in range(20000):
                a.run(x, stream=stream)
            stream.synchronize()
            if a.experts.tolist() != [list(range(8))] * 64:
                failed.append("experts")
        except Exception as e:      # (raised in a thread of its own)
            failed.append(repr(e))

    threads = [threading.Thread(target=work, args=(n,)) for n in (1024, 800)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
