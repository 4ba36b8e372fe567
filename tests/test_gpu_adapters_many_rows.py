"""adapter_forward and adapter_backward at sizes that take the forms for many rows (GPU).

Against the formulas in 64 bits on the GPU, with the bounds that tests/test_gpu_adapters.py
derives: u = 2^-8 for each rounding to BF16, K 2^-24 of a sum of K terms' sizes.
"""
import pytest
import torch

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


def _index(rows, k, kind, seed):
    gen = torch.Generator().manual_seed(seed)
    if kind == "runs":          # requests, of any length, some without an adapter
        cuts = torch.sort(torch.randint(1, rows, (3 * k,), generator=gen)).values.tolist()
        index = torch.empty(rows, dtype=torch.int32)
        for a, b in zip([0] + cuts, cuts + [rows]):
            index[a:b] = int(torch.randint(-1, k, (1,), generator=gen))
        return index
    if kind == "mixed":         # neighbouring rows of different adapters
        return torch.randint(-1, k, (rows,), generator=gen, dtype=torch.int32)
    return torch.full((rows,), k - 1, dtype=torch.int32)     # all of one; the others have none


def _wide(shape, scale, gen, pad):
    buf = torch.full((shape[0], shape[1] + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
    t = buf[:, :shape[1]]
    t.copy_(torch.randn(shape, generator=gen, device="cuda") * scale)
    return t


@pytest.mark.parametrize("rows,hidden,out,ranks,kind,pad,gtype", [
    (4500, 4104, 16392, [16, 8], "runs", 0, torch.bfloat16),
    (4501, 4104, 16392, [16, 5, 1], "mixed", 0, torch.float32),
    (4500, 4096, 16384, [32, 24], "runs", 8, torch.bfloat16),
    (4099, 8192, 11008, [64, 64, 40], "runs", 0, torch.bfloat16),
    (4500, 4104, 16392, [64], "one", 8, torch.float32),
    (4500, 4104, 16392, [128, 72], "runs", 0, torch.bfloat16),
    (9001, 4096, 4160, [8, 16, 16], "one", 0, torch.bfloat16),
])
def test_forward_and_backward(rows, hidden, out, ranks, kind, pad, gtype):
    k = len(ranks)
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x, y = _wide((rows, hidden), 1.0, gen, pad), _wide((rows, out), 1.0, gen, pad)
    dy, dx = _wide((rows, out), 0.1, gen, pad), _wide((rows, hidden), 0.1, gen, pad)
    downs = [_wide((r, hidden), hidden ** -0.5, gen, pad) for r in ranks]
    ups = [_wide((out, r), 0.3, gen, pad) for r in ranks]
    d_downs = [torch.full((r, hidden), 7.0, dtype=gtype, device="cuda") for r in ranks]
    d_ups = [torch.full((out, r), 7.0, dtype=gtype, device="cuda") for r in ranks]
    scales = [0.5 + 0.25 * i for i in range(k)]
    s = bd.AdapterSet(downs, ups, scales, d_downs=d_downs, d_ups=d_ups)
    assert rows >= s._low_rows
    index = _index(rows, k, kind, rows).cuda()
    plan = bd.AdapterRows(index, k)
    low = torch.full((rows, s.rank), float("nan"), dtype=torch.bfloat16, device="cuda")
    y0, dx0, y2 = y.clone(), dx.clone(), y.clone()
    bd.adapter_forward(x, y, s, plan, low=low)
    bd.adapter_forward(x, y2, s, plan)            # (with a workspace of its own)
    bd.adapter_backward(x, dy, low, dx, s, plan)
    torch.cuda.synchronize()
    assert int(plan.status.item()) == bd.OK
    assert torch.equal(y, y2)
    none = index < 0
    assert torch.equal(y[none], y0[none]) and torch.equal(dx[none], dx0[none])
    assert torch.isnan(low[none]).all()
    gu = U if gtype == torch.bfloat16 else F
    for i, r in enumerate(ranks):
        m = (index == i).nonzero().squeeze(1)
        a, b, c = downs[i].double(), ups[i].double(), scales[i]
        xs, dys = x[m].double(), dy[m].double()
        wl, wd = c * xs @ a.T, c * dys @ b
        e_l = U * wl.abs() + (hidden * F + U * U) * c * xs.abs() @ a.abs().T
        e_d = U * wd.abs() + (out * F + U * U) * c * dys.abs() @ b.abs()
        got = low[m].double()
        assert bool(((got[:, :r] - wl).abs() <= e_l).all()) and not bool(got[:, r:].any())
        for res, base, p, e, f in ((y, y0, wl, e_l, b.T), (dx, dx0, wd, e_d, a)):
            want = base[m].double() + p @ f
            tol = (e @ f.abs() + r * F * p.abs() @ f.abs()) * (1 + U) + U * want.abs()
            assert bool(((res[m].double() - want).abs() <= tol).all())
            del want, tol
        t = m.numel()
        for res, p, e, q in ((d_downs[i], wd, e_d, xs), (d_ups[i].T, wl, e_l, dys)):
            want = p.T @ q
            tol = e.T @ q.abs() + t * F * (p.abs() + e).T @ q.abs()
            tol = tol * (1 + gu) + gu * want.abs()
            assert bool(((res.double() - want).abs() <= tol).all())
        if t == 0:
            assert not d_downs[i].any() and not d_ups[i].any()


def test_infinities_stay_in_their_rows():
    rows, hidden, out = 4500, 4104, 16392
    outs = []
    for bad in (False, True):
        gen = torch.Generator(device="cuda").manual_seed(1)
        x, y = _wide((rows, hidden), 1.0, gen, 0), _wide((rows, out), 1.0, gen, 0)
        dy, dx = _wide((rows, out), 0.1, gen, 0), _wide((rows, hidden), 0.1, gen, 0)
        downs = [_wide((r, hidden), 0.02, gen, 0).abs() + 0.01 for r in (20, 20)]
        ups = [_wide((out, r), 0.02, gen, 0).abs() + 0.01 for r in (20, 20)]
        grads = dict(d_downs=[torch.zeros_like(t) for t in downs], d_ups=[torch.zeros_like(t) for t in ups])
        index = (torch.arange(rows, device="cuda") % 300 < 150).int()
        if bad:
            x[7, 11], x[200, 0], dy[9, 3] = float("inf"), float("nan"), float("inf")
        s, plan = bd.AdapterSet(downs, ups, 1.0, **grads), bd.AdapterRows(index, 2)
        low = torch.empty(rows, s.rank, dtype=torch.bfloat16, device="cuda")
        bd.adapter_forward(x, y, s, plan, low=low)
        bd.adapter_backward(x, dy, low, dx, s, plan)
        torch.cuda.synchronize()
        outs.append((y, dx, grads))
    (y, dx, grads), (y2, dx2, grads2) = outs
    assert bool((y2[7] == float("inf")).all()) and bool(torch.isnan(y2[200]).all())
    assert bool((dx2[9] == float("inf")).all())
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[[7, 200]] = False
    assert torch.equal(y[keep], y2[keep])
    keep[[7, 200]] = True
    keep[9] = False
    assert torch.equal(dx[keep], dx2[keep])
    # row 200 is adapter 0's: its NaN reaches the first column of dA and no other; rows 7 and 9 are
    # adapter 1's
    assert torch.isnan(grads2["d_downs"][0][:, 0]).all() and torch.isfinite(grads2["d_downs"][0][:, 1:]).all()


def test_same_result_every_time():
    rows, hidden, out = 5000, 4096, 16384
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, y0 = _wide((rows, hidden), 1.0, gen, 0), _wide((rows, out), 1.0, gen, 0)
    dy, dx0 = _wide((rows, out), 0.1, gen, 0), _wide((rows, hidden), 0.1, gen, 0)
    downs, ups = [_wide((64, hidden), 0.02, gen, 0) for _ in range(3)], [_wide((out, 64), 0.02, gen, 0) for _ in range(3)]
    grads = dict(d_downs=[torch.zeros_like(t) for t in downs], d_ups=[torch.zeros_like(t) for t in ups])
    s, plan = bd.AdapterSet(downs, ups, 1.0, **grads), bd.AdapterRows(_index(rows, 3, "runs", 5).cuda(), 3)
    low = torch.empty(rows, s.rank, dtype=torch.bfloat16, device="cuda")
    first = None
    for _ in range(4):
        y, dx = y0.clone(), dx0.clone()
        bd.adapter_forward(x, y, s, plan, low=low)
        bd.adapter_backward(x, dy, low, dx, s, plan)
        torch.cuda.synchronize()
        now = [y, dx] + [g.clone() for v in grads.values() for g in v]
        if first is None:
            first = now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


def test_forward_without_low_is_refused_by_the_library():
    s = bd.AdapterSet([torch.zeros(8, 4096, dtype=torch.bfloat16, device="cuda")],
                      [torch.zeros(16384, 8, dtype=torch.bfloat16, device="cuda")], 1.0)
    n = s._low_rows
    assert 1 < n < 4096
    lib = bd._ops_lib.load()
    plan = bd.AdapterRows(torch.zeros(n, dtype=torch.int32, device="cuda"), 1)
    x = torch.zeros(n, 4096, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(n, 16384, dtype=torch.bfloat16, device="cuda")
    assert lib.bo_adapter_forward(s._ref, plan._ref, x.data_ptr(), 4096, y.data_ptr(), 16384, None,
                                  None) == bd.ERR_INVALID_ARG
