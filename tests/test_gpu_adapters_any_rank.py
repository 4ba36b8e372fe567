"""Adapters whose ranks are no multiples of 8: their second factors' rows start anywhere, beside
rows of x and y that are read 16 bytes at a time (GPU).

Against the formulas in 64 bits with the bounds of tests/test_gpu_adapters_many_rows.py, whose
check this calls where there are many rows; the same bounds below for fewer.
"""
import pytest
import torch

import test_gpu_adapters_many_rows as many

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("lossless_bf16_weight_old_gb300")

U, F = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    bd._ops_lib.load()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows,hidden,out,ranks,kind,pad,gtype", [
    (4500, 4104, 16392, [13, 1], "runs", 0, torch.bfloat16),
    (4500, 4096, 16384, [27, 30], "mixed", 0, torch.float32),
    (4099, 8192, 11008, [50, 33, 3], "runs", 0, torch.bfloat16),
    (4500, 4104, 16392, [127, 66], "runs", 8, torch.bfloat16),
])
def test_many_rows(rows, hidden, out, ranks, kind, pad, gtype):
    many.test_forward_and_backward(rows, hidden, out, ranks, kind, pad, gtype)


@pytest.mark.parametrize("rows", [1, 37, 700])
@pytest.mark.parametrize("ranks", [[13, 2], [31, 17, 5], [50, 64, 7], [101, 128]])
@pytest.mark.parametrize("gtype,accumulate", [(torch.bfloat16, False), (torch.float32, True)])
def test_forward_and_gradients(rows, ranks, gtype, accumulate):
    hidden, out, k = 520, 1032, len(ranks)
    gen = torch.Generator(device="cuda").manual_seed(rows + ranks[0])
    x, y = many._wide((rows, hidden), 1.0, gen, 0), many._wide((rows, out), 1.0, gen, 0)
    dy, dx = many._wide((rows, out), 0.1, gen, 0), many._wide((rows, hidden), 0.1, gen, 0)
    downs = [many._wide((r, hidden), hidden ** -0.5, gen, 0) for r in ranks]
    ups = [many._wide((out, r), 0.3, gen, i) for i, r in enumerate(ranks)]
    d_downs = [torch.full((r, hidden), 0.5, dtype=gtype, device="cuda") for r in ranks]
    d_ups = [torch.full((out, r), 0.5, dtype=gtype, device="cuda") for r in ranks]
    s = bd.AdapterSet(downs, ups, 1.0, d_downs=d_downs, d_ups=d_ups)
    index = many._index(rows, k, "mixed", rows).cuda()
    plan = bd.AdapterRows(index, k)
    low = torch.full((rows, s.rank), float("nan"), dtype=torch.bfloat16, device="cuda")
    y0, dx0 = y.clone(), dx.clone()
    bd.adapter_forward(x, y, s, plan, low=low)
    bd.adapter_backward(x, dy, low, dx, s, plan, accumulate=accumulate)
    torch.cuda.synchronize()
    assert int(plan.status.item()) == bd.OK
    gu, base_g = (U if gtype == torch.bfloat16 else F), (0.5 if accumulate else 0.0)
    for i, r in enumerate(ranks):
        m = (index == i).nonzero().squeeze(1)
        a, b = downs[i].double(), ups[i].double()
        xs, dys = x[m].double(), dy[m].double()
        wl, wd = xs @ a.T, dys @ b
        e_l = U * wl.abs() + (hidden * F + U * U) * xs.abs() @ a.abs().T
        e_d = U * wd.abs() + (out * F + U * U) * dys.abs() @ b.abs()
        got = low[m].double()
        assert bool(((got[:, :r] - wl).abs() <= e_l).all()) and not bool(got[:, r:].any())
        for res, base, p, e, f in ((y, y0, wl, e_l, b.T), (dx, dx0, wd, e_d, a)):
            want = base[m].double() + p @ f
            tol = (e @ f.abs() + r * F * p.abs() @ f.abs()) * (1 + U) + U * want.abs()
            assert bool(((res[m].double() - want).abs() <= tol).all())
        t = m.numel()
        for res, p, e, q in ((d_downs[i], wd, e_d, xs), (d_ups[i].T, wl, e_l, dys)):
            want = p.T @ q
            tol = e.T @ q.abs() + t * F * (p.abs() + e).T @ q.abs()
            want = want + base_g
            tol = tol * (1 + gu) + gu * want.abs()
            assert bool(((res.double() - want).abs() <= tol).all())
