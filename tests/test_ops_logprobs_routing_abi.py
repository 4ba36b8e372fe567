"""CPU tests of the C boundary of token log probabilities and routing: sizes, structures, and
arguments that are refused before any CUDA call.  No call here launches GPU work."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

from lossless_bf16_weight_old_gb300 import _ops_lib as ol

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
BAD, NO_GPU = 1, 5


@pytest.fixture(scope="module")
def lib():
    return ol.load()


def test_structures_have_the_headers_layout(tmp_path):
    names = {"bo_logprobs": ol.Logprobs, "bo_routing": ol.Routing}
    lines = []
    for c, s in names.items():
        lines.append(f'printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'printf("{c}.{f[0]} %zu\\n", offsetof({c}, {f[0]}));' for f in s._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include "ops/bf16ops.h"\n#include <stddef.h>\n#include <stdio.h>\n'
                   "int main(void) {" + "\n".join(lines) + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", f"-I{ROOT}/include", str(src), "-o", str(exe)], check=True)
    got = dict(line.split() for line in
               subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for c, s in names.items():
        assert int(got[c]) == ctypes.sizeof(s), c
        for f in s._fields_:
            assert int(got[f"{c}.{f[0]}"]) == getattr(s, f[0]).offset, f"{c}.{f[0]}"


def test_sizes(lib):
    size = lib.bo_logprobs_size
    assert size(0, 1, 0, 0) > 0 and size(100, 1000, 32, 1) >= 100 * (4 + 4 + 8 * 32 + 32)
    for bad in ((1, 0, 0, 0), (1, (1 << 24) + 1, 0, 0), ((1 << 28) + 1, 10, 0, 0), (1, 10, 11, 0), (1, 100, 33, 0),
                (1, 10, 0, 2)):
        assert size(*bad) == 0, bad
    size = lib.bo_routing_size
    assert size(0, 1, 1) > 0 and size(100, 128, 8) >= 100 * 64 + 1024
    for bad in ((1, 0, 1), (1, 1025, 1), ((1 << 28) + 1, 8, 1), (1, 8, 9), (1, 64, 33), (1, 8, 0)):
        assert size(*bad) == 0, bad


def test_init_refusals(lib):
    h, r = ol.Logprobs(), ol.Routing()

    def logprobs(rows=10, vocab=100, top=5, entropy=1, mem=1 << 30, n=1 << 20, out=h):
        return lib.bo_logprobs_init(rows, vocab, top, entropy, P(mem), n, ctypes.byref(out) if out else None, None)

    def routing(tokens=10, experts=16, k=2, normalize=1, mem=1 << 30, n=1 << 20, out=r):
        return lib.bo_routing_init(tokens, experts, k, normalize, P(mem), n, ctypes.byref(out) if out else None, None)

    for kw in (dict(vocab=0), dict(top=33), dict(vocab=4), dict(entropy=2), dict(mem=0), dict(mem=(1 << 30) + 128),
               dict(n=64), dict(out=None)):
        assert logprobs(**kw) == BAD, kw
    for kw in (dict(experts=0), dict(k=0), dict(k=17), dict(normalize=2), dict(mem=0), dict(mem=(1 << 30) + 16),
               dict(n=64), dict(out=None)):
        assert routing(**kw) == BAD, kw


def _logprobs(rows=10, vocab=100, top=5, entropy=True):
    base = 1 << 32
    return ol.Logprobs(base, base + 256 if entropy else None, base + 512, base + 1024, base + 1536, rows, vocab, top, 0)


def test_logprobs_forward_refusals(lib):
    if torch.cuda.is_available():
        pytest.skip("the calls that are not refused would run")

    def forward(h=None, x=1 << 34, dtype=0, ld=100, rows=10, tokens=1 << 36, tb=8, ts=1, t=1.0, temps=None, tst=1):
        return lib.bo_logprobs_forward(ctypes.byref(h or _logprobs()), P(x), dtype, ld, rows, P(tokens), tb, ts, t,
                                       P(temps), tst, None)

    for kw in (dict(), dict(ld=1000), dict(dtype=1), dict(tb=4, ts=0), dict(temps=1 << 37, tst=0), dict(rows=0, x=0),
               dict(t=1e-30), dict(temps=1 << 37, t=0.0), dict(rows=1, ld=0)):
        assert forward(**kw) == NO_GPU, kw
    for kw in (dict(x=0), dict(x=(1 << 34) + 1), dict(dtype=1, x=(1 << 34) + 2), dict(dtype=2), dict(ld=99),
               dict(ld=1 << 41), dict(rows=11), dict(tokens=0), dict(tokens=(1 << 36) + 4), dict(tb=2),
               dict(ts=1 << 41), dict(t=0.0), dict(t=-1.0), dict(t=math.nan), dict(t=math.inf),
               dict(temps=(1 << 37) + 2), dict(x=(1 << 32) - 200), dict(tokens=1 << 32), dict(temps=(1 << 32) + 512),
               dict(h=ol.Logprobs())):
        assert forward(**kw) == BAD, kw


def test_logprobs_backward_refusals(lib):
    if torch.cuda.is_available():
        pytest.skip("the calls that are not refused would run")
    x0, d0 = 1 << 34, 1 << 35

    def backward(h=None, x=x0, dtype=0, ld=100, rows=10, g=1 << 36, gs=1, e=1 << 37, es=1, dx=d0, ldx=100):
        return lib.bo_logprobs_backward(ctypes.byref(h or _logprobs()), P(x), dtype, ld, rows, P(g), gs, P(e), es,
                                        P(dx), ldx, None)

    for kw in (dict(), dict(dx=x0), dict(g=None), dict(e=None), dict(gs=0, es=0), dict(ldx=333), dict(dx=x0 + 2000),
               dict(ld=300, ldx=300, dx=x0 + 200), dict(rows=1, dx=x0, ldx=500), dict(rows=0)):
        assert backward(**kw) == NO_GPU, kw
    for kw in (dict(g=None, e=None), dict(x=0), dict(dx=0), dict(dx=x0, ldx=101), dict(dx=x0 + 2), dict(dx=x0 + 1998),
               dict(ld=300, ldx=300, dx=x0 + 198), dict(ldx=99), dict(dtype=2), dict(dtype=1, dx=d0 + 2),
               dict(dx=1 << 36), dict(dx=(1 << 36) + 4 * 9), dict(dx=1 << 37), dict(dx=(1 << 32) + 1500),
               dict(g=(1 << 36) + 2), dict(rows=11), dict(h=_logprobs(entropy=False)), dict(h=ol.Logprobs())):
        assert backward(**kw) == BAD, kw
    assert backward(h=_logprobs(entropy=False), e=None) == NO_GPU


def _routing(tokens=10, experts=16, k=2):
    base = 1 << 32
    return ol.Routing(base, base + 256, base + 512, base + 768, base + 1024, base + 1280, base + 1536, tokens,
                      experts, k, 1, 0)


def test_routing_refusals(lib):
    if torch.cuda.is_available():
        pytest.skip("the calls that are not refused would run")
    x0, d0 = 1 << 34, 1 << 35

    def forward(h=None, x=x0, dtype=0, ld=16, tokens=10, mask=None, ms=1):
        return lib.bo_routing_forward(ctypes.byref(h or _routing()), P(x), dtype, ld, tokens, P(mask), ms, None)

    def backward(h=None, x=x0, dtype=0, ld=16, tokens=10, gw=1 << 36, s0=2, s1=1, gl=1.0, dgl=None, counts=None,
                 dx=d0, ldx=16):
        return lib.bo_routing_backward(ctypes.byref(h or _routing()), P(x), dtype, ld, tokens, P(gw), s0, s1, gl,
                                       P(dgl), P(counts), P(dx), ldx, None)

    for kw in (dict(), dict(ld=40), dict(dtype=1), dict(mask=(1 << 36) + 1, ms=0), dict(tokens=0, x=0), dict(tokens=1, ld=0)):
        assert forward(**kw) == NO_GPU, kw
    for kw in (dict(x=0), dict(x=x0 + 1), dict(dtype=2), dict(ld=15), dict(tokens=11), dict(ms=1 << 41),
               dict(mask=(1 << 32) + 100), dict(x=(1 << 32) + 2), dict(h=ol.Routing()), dict(h=_routing(k=17)),
               dict(h=_routing(experts=2000))):
        assert forward(**kw) == BAD, kw
    for kw in (dict(), dict(dx=x0), dict(gw=None), dict(s0=0, s1=0), dict(dgl=1 << 37, counts=1 << 38), dict(tokens=0),
               dict(ld=40, ldx=40, dx=x0 + 32)):
        assert backward(**kw) == NO_GPU, kw
    for kw in (dict(x=0), dict(dx=0), dict(dx=x0 + 2), dict(dx=x0, ldx=17), dict(ldx=15), dict(gw=(1 << 36) + 2),
               dict(dgl=2), dict(counts=6), dict(dx=1 << 36), dict(gw=d0 - 4 * 19), dict(dgl=d0 + 4), dict(counts=d0 - 60),
               dict(dx=(1 << 32) + 1600), dict(tokens=11), dict(s0=1 << 41), dict(s1=1 << 35),
               dict(ld=40, ldx=40, dx=x0 + 30), dict(h=ol.Routing())):
        assert backward(**kw) == BAD, kw


@pytest.mark.gpu
def test_handles_of_another_device(lib):
    """Of a device that is not current; nothing is launched."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    h, r = _logprobs(), _routing()
    h.device = r.device = 1
    assert lib.bo_logprobs_forward(ctypes.byref(h), P(1 << 34), 0, 100, 10, P(1 << 36), 8, 1, 1.0, None, 0, None) == BAD
    assert lib.bo_logprobs_backward(ctypes.byref(h), P(1 << 34), 0, 100, 10, P(1 << 36), 1, None, 0, P(1 << 35), 100,
                                    None) == BAD
    assert lib.bo_routing_forward(ctypes.byref(r), P(1 << 34), 0, 16, 10, None, 0, None) == BAD
    assert lib.bo_routing_backward(ctypes.byref(r), P(1 << 34), 0, 16, 10, None, 0, 0, 1.0, None, None, P(1 << 35), 16,
                                   None) == BAD
