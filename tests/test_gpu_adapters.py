"""adapter_forward and adapter_backward against the formulas in 64 bits (GPU).

Bounds, with u = 2^-8 (half a unit of BF16 relative to a value) and f = 2^-24:
  low   its FP32 sum of K products is off by at most K f S, S the sum of the products' sizes, and
        it is rounded once to BF16: e_low = u |low| + (K f + u^2) S;
  y     sum over r of |B| e_low, the FP32 sum's own r f of its terms, and one rounding: u |y|;
  dx    the same with B and A in each other's place;
  dA    sum over the rows of |x| e_dlow, the sum's own T f, and one rounding of a BF16 gradient;
  dB    the same with dy and e_low.
"""
import numpy as np
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


def _normal(shape, scale, gen, pad=0, offset=0):
    """A BF16 matrix; pad: columns behind each row (a row stride), offset: elements before it
    (an address off the 16-byte boundary).  What lies around it is NaN."""
    rows, cols = shape
    buf = torch.full((rows * (cols + pad) + offset + 8,), float("nan"), dtype=torch.bfloat16, device="cuda")
    t = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    t.copy_(torch.randn(shape, generator=gen, device="cuda") * scale)
    return t


class Problem:
    def __init__(self, index, ranks, hidden, out, seed=0, pad=0, offset=0, gtype=torch.bfloat16,
                 train=True):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.index, self.ranks, t = np.asarray(index), ranks, len(index)
        self.x = _normal((t, hidden), 1.0, gen, pad, offset)
        self.y = _normal((t, out), 1.0, gen, pad, offset)
        self.dy = _normal((t, out), 0.1, gen, pad, offset)
        self.dx = _normal((t, hidden), 0.1, gen, pad, offset)
        self.downs = [_normal((r, hidden), hidden ** -0.5, gen, pad, offset) for r in ranks]
        self.ups = [_normal((out, r), 0.3, gen, pad, offset) for r in ranks]
        self.scales = [0.5 + 0.25 * i for i in range(len(ranks))]
        kw = {}
        if train:
            self.d_downs = [torch.full((r, hidden + pad), 7.0, dtype=gtype, device="cuda")[:, :hidden]
                            for r in ranks]
            self.d_ups = [torch.full((out, r + pad), 7.0, dtype=gtype, device="cuda")[:, :r]
                          for r in ranks]
            kw = dict(d_downs=self.d_downs, d_ups=self.d_ups)
        self.set = bd.AdapterSet(self.downs, self.ups, self.scales, **kw)
        self.rows = bd.AdapterRows(torch.tensor(index, dtype=torch.int32, device="cuda"), len(ranks))
        self.low = torch.full((t, self.set.rank), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.gtype = gtype

    def numpy(self):
        f = lambda v: v.double().cpu().numpy()  # noqa: E731
        return {n: f(getattr(self, n)) for n in ("x", "y", "dy", "dx")}

    def check_forward(self, before, y, low=None):
        y = y.double().cpu().numpy()
        for i, r in enumerate(self.ranks):
            rows = self.index == i
            a, b = self.downs[i].double().cpu().numpy(), self.ups[i].double().cpu().numpy()
            x, s = before["x"][rows], self.scales[i]
            want_low = s * x @ a.T
            e_low = U * np.abs(want_low) + (a.shape[1] * F + U * U) * s * np.abs(x) @ np.abs(a).T
            want = before["y"][rows] + want_low @ b.T
            tol = e_low @ np.abs(b).T + (r * F) * np.abs(want_low) @ np.abs(b).T
            tol = tol * (1 + U) + U * np.abs(want)
            assert np.all(np.abs(y[rows] - want) <= tol), (i, np.max(np.abs(y[rows] - want) / tol))
            if low is not None:
                got = low.double().cpu().numpy()[rows]
                assert np.all(np.abs(got[:, :r] - want_low) <= e_low)
                assert np.all(got[:, r:] == 0)
        none = (self.index < 0) | (self.index >= len(self.ranks))
        assert np.array_equal(y[none], before["y"][none])
        if low is not None:
            assert torch.isnan(low[torch.from_numpy(none).cuda()]).all()

    def check_backward(self, before, dx, accumulate=0.0):
        gu = U if self.gtype == torch.bfloat16 else F
        for i, r in enumerate(self.ranks):
            rows = self.index == i
            a, b = self.downs[i].double().cpu().numpy(), self.ups[i].double().cpu().numpy()
            x, dy, s = before["x"][rows], before["dy"][rows], self.scales[i]
            low, dlow = s * x @ a.T, s * dy @ b
            e_low = U * np.abs(low) + (a.shape[1] * F + U * U) * s * np.abs(x) @ np.abs(a).T
            e_dlow = U * np.abs(dlow) + (b.shape[0] * F + U * U) * s * np.abs(dy) @ np.abs(b)
            if dx is not None:
                want = before["dx"][rows] + dlow @ a
                tol = (e_dlow @ np.abs(a) + r * F * np.abs(dlow) @ np.abs(a)) * (1 + U) + U * np.abs(want)
                assert np.all(np.abs(dx.double().cpu().numpy()[rows] - want) <= tol)
            t = rows.sum()
            for got, p, e_p, q, flip in ((self.d_downs[i], dlow, e_dlow, x, False),
                                         (self.d_ups[i], low, e_low, dy, True)):
                want = p.T @ q
                tol = e_p.T @ np.abs(q) + t * F * (np.abs(p) + e_p).T @ np.abs(q)
                want, tol = (want.T, tol.T) if flip else (want, tol)
                want = want + accumulate
                tol = tol * (1 + gu) + gu * np.abs(want)
                g = got.double().cpu().numpy()
                assert np.all(np.abs(g - want) <= tol), (i, flip, np.max(np.abs(g - want) - tol))
        none = self.index < 0
        if dx is not None:
            assert np.array_equal(dx.double().cpu().numpy()[none], before["dx"][none])


def _index(rows, k, none, seed, runs=True):
    rng = np.random.default_rng(seed)
    if runs:   # contiguous requests
        cuts = np.sort(rng.integers(0, rows + 1, max(0, min(rows, 3 * k) - 1)))
        ids = rng.integers(0, k, len(cuts) + 1)
        ids[rng.random(len(ids)) < none] = -1
        return np.repeat(ids, np.diff(np.concatenate([[0], cuts, [rows]])))
    ids = rng.integers(0, k, rows)
    ids[rng.random(rows) < none] = -1
    return ids


CASES = [   # rows, ranks, hidden, out, none, runs
    (1, [16], 4096, 4096, 0.0, True),
    (1, [1], 8, 8, 0.0, True),
    (7, [8, 4, 16], 512, 264, 0.2, False),
    (16, [16], 256, 512, 0.0, True),
    (17, [64], 1024, 136, 0.0, True),
    (64, [16] * 40, 2048, 1024, 0.1, False),
    (100, [3, 128, 17, 40], 72, 40, 0.3, False),
    (129, [128, 100], 640, 520, 0.1, True),
    (300, [32, 8], 1096, 2056, 0.1, True),
    (513, [16], 4096, 1024, 0.0, True),
    (700, [64, 24, 64], 520, 1000, 0.4, False),
    (1000, [128], 512, 768, 0.0, True),
    (2500, [16, 8, 16, 16, 2], 264, 312, 0.2, False),
]
ODD = [     # widths, strides, addresses off the 16-byte boundary, odd ranks
    (1, [16], 33, 65, 0.0, True),
    (40, [5, 16], 77, 131, 0.1, False),
    (200, [7, 33], 1, 1, 0.1, False),
    (333, [9, 100], 203, 99, 0.2, True),
]


@pytest.mark.parametrize("rows,ranks,hidden,out,none,runs", CASES)
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 8)])
def test_forward_and_backward(rows, ranks, hidden, out, none, runs, pad, offset):
    _both(rows, ranks, hidden, out, none, runs, pad, offset, torch.bfloat16)


@pytest.mark.parametrize("rows,ranks,hidden,out,none,runs", ODD)
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1)])
def test_odd_sizes_strides_and_addresses(rows, ranks, hidden, out, none, runs, pad, offset):
    _both(rows, ranks, hidden, out, none, runs, pad, offset, torch.float32)


def _both(rows, ranks, hidden, out, none, runs, pad, offset, gtype):
    p = Problem(_index(rows, len(ranks), none, rows, runs), ranks, hidden, out, seed=rows, pad=pad,
                offset=offset, gtype=gtype)
    before = p.numpy()
    bd.adapter_forward(p.x, p.y, p.set, p.rows, low=p.low)
    bd.adapter_backward(p.x, p.dy, p.low, p.dx, p.set, p.rows)
    torch.cuda.synchronize()
    assert int(p.rows.status.item()) == bd.OK
    p.check_forward(before, p.y, p.low)
    p.check_backward(before, p.dx)


def test_gradients_add_up_and_dx_is_optional():
    p = Problem(_index(900, 3, 0.1, 4), [16, 8, 32], 264, 136, gtype=torch.float32)
    before = p.numpy()
    bd.adapter_forward(p.x, p.y, p.set, p.rows, low=p.low)
    for g in p.d_downs + p.d_ups:
        g.fill_(3.0)
    bd.adapter_backward(p.x, p.dy, p.low, None, p.set, p.rows, accumulate=True)
    torch.cuda.synchronize()
    p.check_backward(before, None, accumulate=3.0)


@pytest.mark.parametrize("index", [_index(150, 2, 0.1, 9), np.arange(150) % 3 - 1])
def test_gradients_against_differences(index):
    """The loss sum(w * y) as a function of one value of A, B or x: a difference of the formula
    in 64 bits over a step h has the slope that the backward pass gives, as y is linear in each.
    The bound is that of the gradient itself (check_backward), here with its sums written out by
    the difference instead of the formula's derivative."""
    p = Problem(index, [8, 16], 48, 40, gtype=torch.float32)
    before = p.numpy()
    w = before["dy"]
    dx0 = before["dx"]
    bd.adapter_forward(p.x, p.y, p.set, p.rows, low=p.low)
    bd.adapter_backward(p.x, p.dy, p.low, p.dx, p.set, p.rows)
    torch.cuda.synchronize()
    a = [t.double().cpu().numpy() for t in p.downs]
    b = [t.double().cpu().numpy() for t in p.ups]

    def loss(x, a, b):
        total = 0.0
        for i in range(2):
            r = p.index == i
            total += (w[r] * (p.scales[i] * x[r] @ a[i].T @ b[i].T)).sum()
        return total

    rng = np.random.default_rng(3)
    h = 2.0 ** -3
    for i in range(2):
        r = p.index == i
        if not r.any():
            continue
        x = before["x"][r]
        low, dlow = p.scales[i] * x @ a[i].T, p.scales[i] * w[r] @ b[i]
        for _ in range(6):
            j, c = rng.integers(0, a[i].shape[0]), rng.integers(0, 48)
            up = [m.copy() for m in a]
            up[i][j, c] += h
            slope = (loss(before["x"], up, b) - loss(before["x"], a, b)) / h
            tol = (2 * U * np.abs(dlow[:, j]) + 1e-4 * np.abs(dlow).max()) @ np.abs(x[:, c]) + 1e-9
            assert abs(float(p.d_downs[i][j, c]) - slope) <= tol
            o = rng.integers(0, 40)
            up = [m.copy() for m in b]
            up[i][o, j] += h
            slope = (loss(before["x"], a, up) - loss(before["x"], a, b)) / h
            tol = (2 * U * np.abs(low[:, j]) + 1e-4 * np.abs(low).max()) @ np.abs(w[r][:, o]) + 1e-9
            assert abs(float(p.d_ups[i][o, j]) - slope) <= tol
            t = rng.choice(np.flatnonzero(r))
            xs = before["x"].copy()
            xs[t, c] += h
            slope = (loss(xs, a, b) - loss(before["x"], a, b)) / h
            got = float(p.dx[t, c]) - dx0[t, c]
            tol = (2 * U * np.abs(p.scales[i] * w[t] @ b[i])) @ np.abs(a[i][:, c]) \
                + 1e-4 + U * abs(dx0[t, c] + slope)
            assert abs(got - slope) <= tol


def test_adapters_without_rows_and_rows_without_adapters():
    # adapter 1 has no rows: its gradients are 0 (or as they were); all rows without an adapter
    for index in ([0] * 70 + [-1] * 5 + [2] * 3, [-1] * 40):
        p = Problem(index, [16, 16, 8], 128, 64)
        before = p.numpy()
        bd.adapter_forward(p.x, p.y, p.set, p.rows, low=p.low)
        bd.adapter_backward(p.x, p.dy, p.low, p.dx, p.set, p.rows)
        torch.cuda.synchronize()
        p.check_forward(before, p.y, p.low)
        p.check_backward(before, p.dx)
        assert not p.d_downs[1].any() and not p.d_ups[1].any()
        p.d_downs[1].fill_(2.0)
        bd.adapter_backward(p.x, p.dy, p.low, p.dx, p.set, p.rows, accumulate=True)
        assert bool((p.d_downs[1] == 2.0).all())


def test_no_rows():
    p = Problem(np.zeros(0, dtype=np.int64), [16, 8], 128, 64)
    bd.adapter_forward(p.x, p.y, p.set, p.rows, low=p.low)
    bd.adapter_backward(p.x, p.dy, p.low, p.dx, p.set, p.rows)
    torch.cuda.synchronize()
    assert not any(g.any() for g in p.d_downs + p.d_ups)


def test_indices_out_of_range_count_as_none():
    p = Problem([0, 1, 2, -2, 1, 1 << 20, -(1 << 31), 0], [8, 8], 64, 64, train=False)
    before = p.numpy()
    bd.adapter_forward(p.x, p.y, p.set, p.rows)
    torch.cuda.synchronize()
    assert int(p.rows.status.item()) == bd.ERR_INVALID_ARG
    p.index = np.where((p.index < 0) | (p.index > 1), -1, p.index)
    p.check_forward(before, p.y)
    p.rows.update(torch.tensor([0, 1, -1, -1, 1, -1, -1, 0], dtype=torch.int32, device="cuda"))
    assert int(p.rows.status.item()) == bd.OK


@pytest.mark.parametrize("rows", [40, 400])
@pytest.mark.parametrize("rank", [5, 16, 24, 100])
def test_infinities_and_nans_stay_in_their_rows(rows, rank):
    """A row with an infinity or a NaN gives what the formula gives for it and touches no other
    row; other adapters' gradients do not see it."""
    index = np.arange(rows) % 2
    p = Problem(index, [rank, rank], 128, 64)
    q = Problem(index, [rank, rank], 128, 64)
    p.x[4, 3], p.x[6, 100], p.dy[8, 5] = float("inf"), float("nan"), float("-inf")
    with torch.no_grad():   # one sign in A's column 3 and B: the infinity keeps it
        for pr in (p, q):
            pr.downs[0][:, 3] = pr.downs[0][:, 3].abs() + 0.125
            pr.ups[0].copy_(pr.ups[0].abs() + 0.125)
    for pr in (p, q):
        bd.adapter_forward(pr.x, pr.y, pr.set, pr.rows, low=pr.low)
        bd.adapter_backward(pr.x, pr.dy, pr.low, pr.dx, pr.set, pr.rows)
    torch.cuda.synchronize()
    assert bool((p.y[4] == float("inf")).all()) and bool(torch.isnan(p.y[6]).all())
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[[4, 6]] = False
    assert torch.equal(p.y[keep], q.y[keep])
    keep[[4, 6]] = True
    keep[8] = False
    assert torch.equal(p.dx[keep], q.dx[keep]) and not torch.isfinite(p.dx[8]).any()
    assert torch.equal(p.d_downs[1], q.d_downs[1]) and torch.equal(p.d_ups[1], q.d_ups[1])


def test_a_row_does_not_depend_on_its_batch():
    """The same rows with others around them, in any order: the same values."""
    p = Problem(np.zeros(48, dtype=np.int64), [16], 1024, 512, seed=3, train=False)
    y0 = p.y.clone()
    bd.adapter_forward(p.x, p.y, p.set, p.rows)
    perm = torch.randperm(48, generator=torch.Generator().manual_seed(0)).cuda()
    y = y0[perm].contiguous()
    index = torch.zeros(48, dtype=torch.int32, device="cuda")
    bd.adapter_forward(p.x[perm].contiguous(), y, p.set, bd.AdapterRows(index, 1))
    assert torch.equal(y, p.y[perm])


def test_same_result_every_time_and_from_a_graph():
    p = Problem(_index(1500, 4, 0.1, 2), [64, 16, 8, 64], 1024, 768)
    y0, dx0 = p.y.clone(), p.dx.clone()
    ws = torch.empty(int(bd._ops_lib.load().bo_adapter_backward_workspace_size(
        p.set._ref, 1500)), dtype=torch.uint8, device="cuda")

    def go(stream=None):
        p.rows.update(p.rows.index, stream)
        bd.adapter_forward(p.x, p.y, p.set, p.rows, low=p.low, stream=stream)
        bd.adapter_backward(p.x, p.dy, p.low, p.dx, p.set, p.rows, workspace=ws, stream=stream)

    go()
    first = [t.clone() for t in [p.y, p.dx] + p.d_downs + p.d_ups]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        go(side)
    for _ in range(3):
        p.y.copy_(y0)
        p.dx.copy_(dx0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(first, [p.y, p.dx] + p.d_downs + p.d_ups):
            assert torch.equal(a, b)


def test_two_sets_on_two_streams():
    made = []
    for seed in (1, 2):
        p = Problem(_index(2000, 3, 0.1, seed), [16, 32, 16], 512, 512, seed=seed)
        made.append((p, p.numpy(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for p, _, s in made:
        bd.adapter_forward(p.x, p.y, p.set, p.rows, low=p.low, stream=s)
        bd.adapter_backward(p.x, p.dy, p.low, p.dx, p.set, p.rows, stream=s)
    torch.cuda.synchronize()
    for p, before, _ in made:
        p.check_forward(before, p.y, p.low)
        p.check_backward(before, p.dx)


def test_row_offsets_beyond_32_bits():
    """x and y whose last rows lie past 2^32 elements."""
    rows, width = 1030, 1 << 22
    x = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    for t in (0, 600, 1029):
        x[t].copy_(torch.randn(width, generator=gen, device="cuda"))
    down = (torch.randn(8, width, generator=gen, device="cuda") * width ** -0.5).bfloat16()
    up = (torch.randn(width, 8, generator=gen, device="cuda") * 0.3).bfloat16()
    s = bd.AdapterSet([down], [up], 2.0)
    rows_ = bd.AdapterRows(torch.zeros(rows, dtype=torch.int32, device="cuda"), 1)
    bd.adapter_forward(x, y, s, rows_)
    for t in (0, 600, 1029):
        low = 2.0 * (down.double() @ x[t].double())
        want = up.double() @ low
        size = 2.0 * (down.double().abs() @ x[t].double().abs())
        e_low = U * low.abs() + (width * F + U * U) * size
        tol = (up.double().abs() @ e_low) * (1 + U) + (8 * F + U) * (up.double().abs() @ low.abs())
        assert bool(((y[t].double() - want).abs() <= tol).all())
    assert not y[1:600].any() and not y[601:1029].any()
    del x, y
    torch.cuda.empty_cache()


def test_refusals():
    p = Problem([0, 0, 1, -1], [8, 16], 64, 32)
    x, y, low = p.x, p.y, p.low
    for bad in (x.float(), x[:, :32], x[:2], x.t()):
        with pytest.raises(ValueError):
            bd.adapter_forward(bad, y, p.set, p.rows)
    with pytest.raises(ValueError):
        bd.adapter_forward(x, y.cpu(), p.set, p.rows)
    with pytest.raises(ValueError):
        bd.adapter_forward(x, y, p.set, p.rows, low=low[:, :8])
    with pytest.raises(ValueError):
        bd.adapter_forward(x, y, p.set, bd.AdapterRows(p.rows.index, 3))
    with pytest.raises(ValueError):
        bd.AdapterRows(p.rows.index.long(), 2)
    with pytest.raises(ValueError):
        bd.AdapterRows(p.rows.index, 0)
    with pytest.raises(ValueError):
        p.rows.update(p.rows.index[:2])
    with pytest.raises(ValueError):
        bd.AdapterSet(p.downs, p.ups[:1])
    with pytest.raises(ValueError):
        bd.AdapterSet([torch.zeros(129, 64, dtype=torch.bfloat16, device="cuda")],
                      [torch.zeros(32, 129, dtype=torch.bfloat16, device="cuda")])
    with pytest.raises(ValueError):
        bd.AdapterSet([p.downs[0].t()], [p.ups[0]])
    with pytest.raises(ValueError):
        bd.AdapterSet(p.downs, p.ups, [1.0])
    with pytest.raises(ValueError):
        bd.AdapterSet(p.downs, p.ups, d_downs=p.d_downs)
    # refused by the library: outputs over inputs, a workspace too small
    square = Problem([0, 1], [8, 8], 64, 64)
    with pytest.raises(bd.OpsError):
        bd.adapter_forward(square.x, square.x, square.set, square.rows)
    with pytest.raises(bd.OpsError):
        bd.adapter_backward(square.x, square.dy, square.low, square.dy, square.set, square.rows)
    with pytest.raises(bd.OpsError):
        bd.adapter_backward(square.x, square.dy, square.low, square.dx, square.set, square.rows,
                            workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
