"""CPU tests of libbf16ops' C-ABI boundary: it builds for sm_103a, loads without a GPU, exports
exactly what include/ops/bf16ops.h declares, its ctypes structures have the header's layout, and
bad arguments are refused before any CUDA call.  No call here launches GPU work."""
import ctypes
import math
import os
import re
import subprocess

import pytest

from lossless_bf16_weight_old_gb300 import _ops_lib as ol

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ops", "bf16ops.h")
P = ctypes.c_void_p
BAD = 1


@pytest.fixture(scope="module")
def lib():
    return ol.load()


def _declared() -> set[str]:
    return set(re.findall(r"^BD_API\s+[\w\s\*]*?\b(bo_\w+)\s*\(", open(HEADER).read(), flags=re.M))


def test_library_exports_every_declared_symbol_and_no_other(lib):
    out = subprocess.run(["nm", "-D", "--defined-only", ol.path()], capture_output=True, text=True,
                         check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines()
                if line.split()[-1].startswith(("bo_", "bd_"))}
    assert exported == _declared() == set(ol.SIGNATURES)


def test_structures_have_the_headers_layout(tmp_path):
    names = {"bo_adamw_item": ol.AdamWItem, "bo_adamw_state": ol.AdamWState, "bo_adamw": ol.AdamW,
             "bo_adamw_step_args": ol.AdamWStepArgs, "bo_adapter": ol.Adapter,
             "bo_adapter_set": ol.AdapterSet, "bo_adapter_rows": ol.AdapterRows}
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


def _adamw(n=1000, blocks=4, **over):
    item = (ol.AdamWItem * 1)(ol.AdamWItem(1 << 20, 1 << 20, 1 << 22, n, 0, 0.0, 0))
    state = ol.AdamWState(1 << 24, 1 << 25, 1 << 26, 1 << 27, 1 << 28, blocks)
    for k, v in over.items():
        setattr(item[0] if hasattr(item[0], k) else state, k, v)
    return item, state


def test_adamw_plan_refusals(lib):
    h = ol.AdamW()

    def plan(item, state, kind=0, grad=0, bits=32, flags=0, step=0, ws=1 << 30, ws_bytes=1 << 20):
        return lib.bo_adamw_plan(item, 1, ctypes.byref(state), kind, grad, bits, flags, step, P(ws),
                                 ws_bytes, ctypes.byref(h), None)

    ok = _adamw()
    assert lib.bo_adamw_plan_size(ok[0], 1) > 0
    assert lib.bo_adamw_plan_size(None, 1) == 0
    assert lib.bo_adamw_plan_size(_adamw(n=(1 << 40) + 1)[0], 1) == 0
    for kw in (dict(kind=3), dict(grad=2), dict(bits=16), dict(flags=2), dict(flags=1), dict(step=-1),
               dict(ws=(1 << 30) + 16), dict(ws=0), dict(ws_bytes=64)):
        assert plan(*ok, **kw) == BAD, kw
    for over in (dict(n=1025), dict(first_block=1), dict(first_block=1 << 60), dict(reserved=1),
                 dict(d_out=0), dict(d_out=(1 << 20) + 8), dict(d_grad=0), dict(d_grad=(1 << 22) + 2),
                 dict(d_out=1 << 22), dict(d_out=1 << 24), dict(d_out=1 << 28), dict(d_out=1 << 30),
                 dict(d_m=0), dict(d_v=(1 << 25) + 16), dict(d_master=0), dict(blocks=1 << 50)):
        assert plan(*_adamw(**over)) == BAD, over
    # without a master the weights are read
    for over in (dict(d_weight=0), dict(d_weight=(1 << 20) + 4), dict(d_out=(1 << 20) + 64)):
        assert plan(*_adamw(**over), kind=1) == BAD, over
    # 8 bits need scales
    for over in (dict(d_m_scale=0), dict(d_v_scale=(1 << 27) + 4)):
        assert plan(*_adamw(**over), bits=8) == BAD, over
    assert lib.bo_adamw_plan(None, 1, ctypes.byref(ok[1]), 0, 0, 32, 0, 0, P(1 << 30), 1 << 20,
                             ctypes.byref(h), None) == BAD


def test_adamw_step_refusals(lib):
    h = ol.AdamW()
    args = ol.AdamWStepArgs(1e-3, None, 0.9, 0.999, 1e-8, 0.0, 0)
    assert lib.bo_adamw_step(ctypes.byref(h), ctypes.byref(args), None) == BAD     # an empty handle
    h.d_control, h.d_chunks, h.d_partials, h.state_bits = 4096, 8192, 1 << 14, 32
    for over in (dict(beta1=1.0), dict(beta2=-0.1), dict(beta1=math.nan), dict(eps=-1.0),
                 dict(max_norm=-1.0), dict(max_norm=math.nan), dict(lr=math.nan), dict(lr=math.inf),
                 dict(d_lr=4098)):
        bad = ol.AdamWStepArgs(1e-3, None, 0.9, 0.999, 1e-8, 0.0, 0)
        for k, v in over.items():
            setattr(bad, k, v)
        assert lib.bo_adamw_step(ctypes.byref(h), ctypes.byref(bad), None) == BAD, over
    assert lib.bo_adamw_step(ctypes.byref(h), None, None) == BAD
    assert lib.bo_adamw_norm(ctypes.byref(h), -1.0, None) == BAD
    assert lib.bo_adamw_moments(ctypes.byref(h), 1, P(1 << 20), P(1 << 21), None) == BAD   # 32 bits
    h.state_bits = 8
    assert lib.bo_adamw_moments(ctypes.byref(h), 2, P(1 << 20), P(1 << 21), None) == BAD
    assert lib.bo_adamw_moments(ctypes.byref(h), 1, P((1 << 20) + 4), P(1 << 21), None) == BAD


def _adapter(**over):
    a = (ol.Adapter * 1)(ol.Adapter(1 << 20, 1 << 21, 64, 16, None, None, 0, 0, 16, 1.0))
    for k, v in over.items():
        setattr(a[0], k, v)
    return a


def test_adapter_set_refusals(lib):
    h = ol.AdapterSet()

    def init(a, k=1, hidden=64, out=32, grad=0, ws=1 << 30, ws_bytes=1 << 20):
        return lib.bo_adapter_set_init(a, k, hidden, out, grad, P(ws), ws_bytes, ctypes.byref(h), None)

    assert lib.bo_adapter_set_size(0) == 0 and lib.bo_adapter_set_size(65536) == 0
    assert lib.bo_adapter_set_size(65535) > 0
    for kw in (dict(k=0), dict(k=65536), dict(hidden=0), dict(out=0), dict(hidden=(1 << 24) + 1),
               dict(grad=2), dict(ws=0), dict(ws=(1 << 30) + 16), dict(ws_bytes=16)):
        assert init(_adapter(), **kw) == BAD, kw
    for over in (dict(rank=0), dict(rank=129), dict(d_down=None), dict(d_up=(1 << 21) + 1),
                 dict(ld_down=63), dict(ld_up=15), dict(d_grad_down=1 << 22),
                 dict(d_grad_down=1 << 22, d_grad_up=1 << 23, ld_grad_down=63, ld_grad_up=16),
                 dict(d_grad_down=1 << 22, d_grad_up=1 << 23, ld_grad_down=64, ld_grad_up=15)):
        assert init(_adapter(**over)) == BAD, over
    assert lib.bo_adapter_set_init(None, 1, 64, 32, 0, P(1 << 30), 1 << 20, ctypes.byref(h), None) == BAD


def _handles():
    s = ol.AdapterSet(1 << 20, 2, 64, 32, 16, 0, 0, 1)
    r = ol.AdapterRows()
    r.d_perm, r.d_offsets, r.d_blocks, r.d_ntiles, r.rows, r.k = 4096, 8192, 1 << 14, 1 << 15, 10, 2
    for i in range(3):
        r.d_tiles[i] = 1 << 16
    return s, r


def test_adapter_call_refusals(lib):
    s, r = _handles()
    x, y, ws = 1 << 24, 1 << 25, 1 << 30

    def forward(s, r, x=x, ldx=64, y=y, ldy=32, low=None):
        return lib.bo_adapter_forward(ctypes.byref(s), ctypes.byref(r), P(x), ldx, P(y), ldy, low, None)

    for kw in (dict(x=0), dict(y=0), dict(x=x + 1), dict(ldx=63), dict(ldy=31), dict(y=x + 64),
               dict(low=P(1 << 26 | 4)), dict(low=P(y)), dict(low=P(x + 128))):
        assert forward(s, r, **kw) == BAD, kw
    other = _handles()[1]
    other.k = 3
    assert forward(s, other) == BAD
    assert forward(ol.AdapterSet(), r) == BAD and forward(s, ol.AdapterRows()) == BAD
    r.rows = lib.bo_adapter_low_rows(ctypes.byref(s))       # many rows need low
    assert r.rows > 10 and forward(s, r, y=1 << 40) == BAD
    r.rows = 10
    need = lib.bo_adapter_backward_workspace_size(ctypes.byref(s), 10)
    assert need > 0 and lib.bo_adapter_backward_workspace_size(ctypes.byref(ol.AdapterSet()), 10) == 0

    def backward(x=x, ldx=64, dy=y, lddy=32, low=1 << 26, dx=1 << 27, lddx=64, ws=ws, n=need):
        return lib.bo_adapter_backward(ctypes.byref(s), ctypes.byref(r), P(x), ldx, P(dy), lddy, P(low),
                                       P(dx), lddx, 0, P(ws), n, None)

    for kw in (dict(x=0), dict(dy=0), dict(low=0), dict(low=(1 << 26) + 8), dict(ldx=63), dict(lddy=31),
               dict(lddx=63), dict(dx=x), dict(dx=y + 16), dict(dx=1 << 26), dict(dx=ws), dict(ws=0),
               dict(ws=ws + 16), dict(n=need - 1)):
        assert backward(**kw) == BAD, kw


def test_adapter_rows_refusals(lib):
    h = ol.AdapterRows()

    def init(index=1 << 20, rows=10, k=2, ws=1 << 30, ws_bytes=1 << 20, status=1 << 21):
        return lib.bo_adapter_rows_init(P(index), rows, k, P(ws), ws_bytes, ctypes.byref(h), P(status), None)

    assert lib.bo_adapter_rows_size(10, 0) == 0 and lib.bo_adapter_rows_size((1 << 30) + 1, 2) == 0
    assert lib.bo_adapter_rows_size(0, 1) > 0
    for kw in (dict(k=0), dict(k=65536), dict(rows=(1 << 30) + 1), dict(index=0), dict(index=(1 << 20) + 2),
               dict(ws=0), dict(ws=(1 << 30) + 128), dict(ws_bytes=64), dict(status=(1 << 21) + 2),
               dict(index=(1 << 30) + 256)):
        assert init(**kw) == BAD, kw


def test_status_strings(lib):
    for code, word in [(0, b"ok"), (1, b"argument"), (5, b"CUDA"), (16, b"norm"), (99, b"unknown")]:
        assert word in lib.bo_status_string(code)
