"""AdamWBatch against the formulas of include/ops/bf16ops.h in 64 bits (GPU).

Tolerances are bounds on the rounding of the FP32 computation, in units of u = 2^-24 (half a unit
in the last place): with A = |beta1 m| + |(1 - beta1) g'|,
  m   four roundings of its terms: 4 u A;
  v   the same: 6 u v (all terms have one sign); with clipping the factor's own error, at most
      16 u (a norm summed over at most 16 FP32 additions in a row), counts once in m, twice in v;
  p   the update is off by at most 64 u of A / (its denominator): m's and v's errors, two bias
      corrections (4 u each), an approximate root (2 u) and quotient (4 u), products (u each);
      p's own two roundings add 3 u |p|.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("lossless_bf16_weight_old_gb300")

U = 2.0 ** -24
BLOCK = 256
MASK = (1 << 64) - 1
GAMMA = 0x9E3779B97F4A7C15


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    bd._ops_lib.load()


# ------------------------------------------------------------------ the formulas in 64 bits

def _mix(z):
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & MASK
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & MASK
    return z ^ (z >> 31)


def _noise(seed, t, elements):
    """The 32 random bits of arena elements, one Python int at a time."""
    key = _mix((seed ^ (t * GAMMA)) & MASK)
    return np.array([(_mix((key + ((int(e) >> 1) + 1) * GAMMA) & MASK) >> (32 * (int(e) & 1)))
                     & 0xFFFFFFFF for e in elements], dtype=np.int64)


def _step(p, g, m, v, t, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, wd=0.0):
    b1, b2 = betas
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    den = np.sqrt(v / (1 - b2 ** t)) + eps
    return p * (1 - lr * wd) - lr * (m / (1 - b1 ** t)) / den, m, v, den


def _m_value(code, scale):
    code = code.astype(np.float64)
    return np.sign(code) * (code / 127) ** 2 * scale


def _v_value(code, scale):
    return (code.astype(np.float64) / 255) ** 4 * scale


def _np(t):
    return t.detach().double().cpu().numpy()


def _tensors(shapes, dtype, scale, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(s, generator=g, device="cuda") * scale).to(dtype) for s in shapes]


SHAPES = [(3, 700), (1,), (256,), (2048,), (2049,), (7,), (33, 129), (4096 * 3 + 255,)]
HYPER = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8)


def _check_p(got, p64, p0, m0, g, den, t, lr, b1):
    a = (np.abs(b1 * m0) + np.abs((1 - b1) * g)) / (1 - b1 ** t)
    tol = lr * 64 * U * a / den + 3 * U * np.abs(p64) + 3 * U * np.abs(p0)
    assert np.all(np.abs(got - p64) <= tol)


@pytest.mark.parametrize("wtype,master", [("bf16", True), ("bf16", False), ("fp32", False)])
@pytest.mark.parametrize("gtype", ["bf16", "fp32"])
@pytest.mark.parametrize("clip", [None, 0.5, float("inf")])
def test_step32(wtype, master, gtype, clip):
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32}
    ws = _tensors(SHAPES, dt[wtype], 0.02, 1)
    gs = _tensors(SHAPES, dt[gtype], 0.05, 2)
    wds = [0.1 * (i % 3) for i in range(len(SHAPES))]
    ad = bd.AdamWBatch(ws, gs, master=master, weight_decay=wds, max_norm=clip, step=4, **HYPER)
    ad.state["m"].normal_(0, 0.01, generator=torch.Generator(device="cuda").manual_seed(3))
    ad.state["v"].normal_(0, 0.01, generator=torch.Generator(device="cuda").manual_seed(4)).square_()
    if master:
        ad.state["master"].add_(1e-5)
    k = range(len(SHAPES))
    m0, v0 = [_np(ad.view("m", i)) for i in k], [_np(ad.view("v", i)) for i in k]
    p0 = [_np(ad.view("master", i) if master else ws[i]) for i in k]
    arena0 = {n: x.clone() for n, x in ad.state.items()}
    ad.run()
    torch.cuda.synchronize()
    assert int(ad.status.item()) == bd.OK and int(ad.steps.item()) == 5
    norm = np.sqrt(sum((_np(g) ** 2).sum() for g in gs))
    coef = 1.0
    if clip is not None:
        assert abs(float(ad.norm.item()) - norm) <= 16 * U * norm
        coef = min(1.0, clip / (norm + 1e-6))
    extra = 16 if clip is not None else 0
    for i in k:
        g = _np(gs[i]) * coef
        p, m, v, den = _step(p0[i], g, m0[i], v0[i], 5, wd=wds[i], **HYPER)
        a = np.abs(0.9 * m0[i]) + np.abs(0.1 * g)
        assert np.all(np.abs(_np(ad.view("m", i)) - m) <= (4 + extra) * U * a)
        assert np.all(np.abs(_np(ad.view("v", i)) - v) <= (6 + 2 * extra) * U * v)
        if master:
            mst = ad.view("master", i)
            _check_p(_np(mst), p, p0[i], m0[i], g, den, 5, HYPER["lr"], 0.9)
            assert torch.equal(ws[i].view(torch.int16), mst.bfloat16().view(torch.int16))
        elif wtype == "fp32":
            _check_p(_np(ws[i]), p, p0[i], m0[i], g, den, 5, HYPER["lr"], 0.9)
        else:   # half a unit of BF16 (2^-8 of the power of two below) and the FP32 error
            tol = 2.0 ** -8 * np.abs(p) * (1 + 1e-3) + HYPER["lr"] * 64 * U * a / (1 - 0.9 ** 5) / den
            assert np.all(np.abs(_np(ws[i]) - p) <= tol)
    # nothing between the tensors was written
    for n, x in ad.state.items():
        inside = torch.zeros(x.numel(), dtype=torch.bool, device="cuda")
        for i in k:
            b = ad.first_blocks[i] * BLOCK
            inside[b:b + ad.ns[i]] = True
        assert torch.equal(x[~inside], arena0[n][~inside])


def _state8(ad, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n, b = ad.blocks * BLOCK, ad.blocks
    ad.state["m"].copy_((torch.randn(n, generator=gen, device="cuda") * 40).clamp(-127, 127))
    ad.state["v"].copy_((torch.rand(n, generator=gen, device="cuda") * 255))
    ad.state["m_scale"].copy_(torch.rand(b, generator=gen, device="cuda") * 0.1 + 1e-3)
    ad.state["v_scale"].copy_(torch.rand(b, generator=gen, device="cuda") * 0.01 + 1e-4)
    ad.state["m_scale"][1::7] = 0   # blocks without a history
    ad.state["v_scale"][1::7] = 0


@pytest.mark.parametrize("wtype,master", [("bf16", True), ("bf16", False), ("fp32", False)])
@pytest.mark.parametrize("gtype", ["bf16", "fp32"])
@pytest.mark.parametrize("magnitude", [1.0, 1e-16, 1e16])
def test_step8(wtype, master, gtype, magnitude):
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32}
    ws = _tensors(SHAPES, dt[wtype], 0.02, 5)
    gs = _tensors(SHAPES, dt[gtype], 0.05 * magnitude, 6)
    for g in gs:
        g.view(-1)[::5] = 0
    gs[3].zero_()                   # a tensor without gradients
    ad = bd.AdamWBatch(ws, gs, master=master, state_bits=8, seed=77, step=9, **HYPER)
    _state8(ad, 7)
    ad.state["m_scale"].mul_(magnitude)
    ad.state["v_scale"].mul_(magnitude ** 2)
    before = {n: _np(x) for n, x in ad.state.items()}
    p0 = [_np(ad.view("master", i) if master else w) for i, w in enumerate(ws)]
    ad.run()
    torch.cuda.synchronize()
    assert int(ad.steps.item()) == 10
    for i, n in enumerate(ad.ns):
        b0, nb = ad.first_blocks[i], -(-n // BLOCK)
        pad = nb * BLOCK - n
        sl = slice(b0 * BLOCK, b0 * BLOCK + n)
        sms = np.repeat(before["m_scale"][b0:b0 + nb], BLOCK)[:n]
        svs = np.repeat(before["v_scale"][b0:b0 + nb], BLOCK)[:n]
        m0, v0 = _m_value(before["m"][sl], sms), _v_value(before["v"][sl], svs)
        g = _np(gs[i]).reshape(-1)
        p, m, v, den = _step(p0[i].reshape(-1), g, m0, v0, 10, **HYPER)
        got_p = _np(ad.view("master", i) if master else ws[i]).reshape(-1)
        a = (np.abs(0.9 * m0) + np.abs(0.1 * g)) / (1 - 0.9 ** 10)
        slack = HYPER["lr"] * 64 * U * a / den
        if wtype == "bf16" and not master:
            assert np.all(np.abs(got_p - p) <= 2.0 ** -8 * np.abs(p) * (1 + 1e-3) + slack)
        else:
            assert np.all(np.abs(got_p - p) <= slack + 3 * U * (np.abs(p) + np.abs(p0[i].reshape(-1))))
        # scales: the blocks' maxima
        grid_m = np.pad(np.abs(m), (0, pad)).reshape(nb, BLOCK).max(1)
        grid_v = np.pad(v, (0, pad)).reshape(nb, BLOCK).max(1)
        sm, sv = _np(ad.view("m_scale", i)), _np(ad.view("v_scale", i))
        grid_a = np.pad(a, (0, pad)).reshape(nb, BLOCK).max(1)
        assert np.all(np.abs(sm - grid_m) <= 8 * U * grid_a)
        # (denormal numbers: half their spacing for each of three roundings)
        assert np.all(np.abs(sv - grid_v) <= 8 * U * grid_v + 3 * 2.0 ** -149)
        cm = _np(ad.view("m", i)).reshape(-1)
        cv = _np(ad.view("v", i)).reshape(-1)
        rm, rv = np.repeat(grid_m, BLOCK)[:n], np.repeat(grid_v, BLOCK)[:n]
        # m: within half a code of 127 sqrt(|m| / sm).  The ratio is off by 16 u of a / sm at most
        # (a bounds m's terms), the root by half of that over its own size, and by 4 u relative
        ok = rm > 0
        ideal = 127 * np.sqrt(np.divide(np.abs(m), rm, where=ok, out=np.zeros(n)))
        off = 127 * np.sqrt(16 * U * np.divide(a, rm, where=ok, out=np.zeros(n)))
        tol = 0.5 + np.minimum(off, np.divide(off ** 2, ideal, where=ideal > 0, out=off.copy())) + 127 * 8 * U
        assert np.all(np.abs(np.abs(cm) - ideal) <= tol)
        sure = np.abs(m) > 16 * U * a
        assert np.all((cm == 0) | (np.sign(cm) == np.sign(m)) | ~sure)
        # v: the code that the random bits choose.  The chance is (x - lower) / (upper - lower)
        # with x off by 16 u relative and the code's spacing at least 4/255 of its value from
        # code 1 on: off by at most 64 * 16 u, plus the same for the values' own roundings
        if magnitude < 1:
            continue   # (v is denormal there: its relative error has no such bound)
        x = np.divide(v, rv, where=rv > 0, out=np.zeros(n))
        y = 255 * x ** 0.25
        low = np.minimum(np.floor(y), 254)
        lo, hi = (low / 255) ** 4, ((low + 1) / 255) ** 4
        u16 = (_noise(77, 10, range(b0 * BLOCK, b0 * BLOCK + n)) >> 16) / 65536
        chance = (x - lo) / (hi - lo)
        want = np.where(v > 0, np.maximum(low + (u16 < chance), 1), 0)
        near = (np.abs(u16 - chance) <= 2 * 64 * 16 * U) | (np.abs(y - np.round(y)) <= 255 * 8 * U)
        assert np.all((cv == want) | (near & (np.abs(cv - want) <= 1)))
        assert np.all(_np(ad.state["m"][(b0 * BLOCK + n):(b0 + nb) * BLOCK]) == 0)
        assert np.all(_np(ad.state["v"][(b0 * BLOCK + n):(b0 + nb) * BLOCK]) == 0)
    # the read-out: three products, and one rounding to BF16
    for dtype, u in ((torch.float32, 6 * U), (torch.bfloat16, 2.0 ** -8 * 1.01)):
        mv, vv = ad.moments(dtype=dtype)
        want_m = _m_value(_np(ad.state["m"]), np.repeat(_np(ad.state["m_scale"]), BLOCK))
        want_v = _v_value(_np(ad.state["v"]), np.repeat(_np(ad.state["v_scale"]), BLOCK))
        tiny = 4 * 2.0 ** (-133 if dtype == torch.bfloat16 else -149)
        assert np.all(np.abs(_np(mv) - want_m) <= u * np.abs(want_m) + tiny)
        assert np.all(np.abs(_np(vv) - want_v) <= u * want_v + tiny)


def test_stochastic_weights_follow_the_random_bits():
    n = 5000
    w = _tensors([(n,)], torch.bfloat16, 1.0, 8)[0]
    g = _tensors([(n,)], torch.float32, 1.0, 9)[0]
    for bits in (32, 8):
        w2 = w.clone()
        new = torch.empty_like(w)
        ad = bd.AdamWBatch([w2], [g], news=[new], master=False, stochastic=True, state_bits=bits,
                           seed=(1 << 64) - 3, lr=1e-3)
        ad.run()
        torch.cuda.synchronize()
        assert torch.equal(w2, w)       # out of place
        p, _, _, den = _step(_np(w), _np(g), 0.0, 0.0, 1, lr=1e-3)
        low16 = _noise((1 << 64) - 3, 1, range(n)) & 0xFFFF
        step = 2.0 ** (np.floor(np.log2(np.abs(p))) - 7)
        down = np.floor(np.abs(p) / step)
        cut = (np.abs(p) / step - down) * 65536
        want = np.sign(p) * (down + (np.floor(cut) + low16 >= 65536)) * step
        # p is off by at most 64 u lr + 3 u |p|: where that reaches the next 16-bit fraction,
        # the carry may differ
        err = (64 * U * 1e-3 + 6 * U * np.abs(p)) / step * 65536 + 1
        near = np.abs(cut + low16 - 65536) <= err + 1
        got = _np(new)
        assert np.all((got == want) | (near & (np.abs(got - want) <= step * 1.01)))
        assert near.mean() < 0.01
        # unbiased: the mean of n roundings, each within one step, off by less than 5 sigma
        assert abs(((got - p) / step).mean()) < 5 * 0.5 / np.sqrt(n)


def test_8bit_second_moment_does_not_freeze():
    """beta2 = 0.999 moves v by less than half a code step: v has to follow its recursion on
    average all the same.  After k steps of a constant g, v = g^2 + 0.999^k (v0 - g^2).  One code
    step is at most 13% of v for codes from 32 on, so a rounding's variance is at most
    0.13^2 / 4 of v^2 and the recursion's 500 times that at most (a factor of 3 in deviation);
    averaged over 2^18 independent elements that is 0.6%.  Tolerance: 3%."""
    n = 1 << 18
    g = torch.exp(torch.randn(n, generator=torch.Generator(device="cuda").manual_seed(1),
                              device="cuda") * 0.3).bfloat16()
    w = torch.zeros(n, dtype=torch.float32, device="cuda")
    ad = bd.AdamWBatch([w], [g], state_bits=8, betas=(0.9, 0.999), lr=0.0, seed=5)
    g2 = _np(g) ** 2
    # start at 4 g^2, coded to the nearest code
    v0 = torch.from_numpy(4 * g2).cuda().view(-1, BLOCK)
    sv = v0.amax(1)
    ad.state["v_scale"].copy_(sv)
    ad.state["v"].copy_(((v0 / sv[:, None]) ** 0.25 * 255).round().view(-1))
    start = _np(ad.moments()[1])
    for _ in range(600):
        ad.run()
    v = _np(ad.moments()[1])
    want = g2 + 0.999 ** 600 * (start - g2)
    assert abs((v / want).mean() - 1) < 0.03
    assert (want / start).mean() < 0.7     # (it has moved far)


def test_nonfinite_norm_skips_the_step():
    for bits in (32, 8):
        for bad in (float("nan"), float("inf")):
            ws = _tensors(SHAPES, torch.bfloat16, 0.02, 1)
            gs = _tensors(SHAPES, torch.bfloat16, 0.02, 2)
            gs[4].view(-1)[-1] = bad
            ad = bd.AdamWBatch(ws, gs, state_bits=bits, max_norm=float("inf"), step=3)
            w0 = [w.clone() for w in ws]
            s0 = {n: x.clone() for n, x in ad.state.items()}
            ad.run()
            torch.cuda.synchronize()
            assert int(ad.status.item()) == bd.SKIPPED_NONFINITE and int(ad.steps.item()) == 3
            assert all(torch.equal(a, b) for a, b in zip(ws, w0))
            assert all(torch.equal(ad.state[n], s0[n]) for n in s0)
            gs[4].view(-1)[-1] = 0.01
            ad.run()
            torch.cuda.synchronize()
            assert int(ad.status.item()) == bd.OK and int(ad.steps.item()) == 4
            assert not torch.equal(ws[0], w0[0])


def test_nonfinite_gradients_without_a_norm_stay_in_their_place():
    ws = _tensors([(1024,)], torch.float32, 0.02, 1)
    gs = _tensors([(1024,)], torch.float32, 0.02, 2)
    gs[0][300], gs[0][600] = float("nan"), float("inf")
    ad = bd.AdamWBatch(ws, gs)
    ad.run()
    bad = ~torch.isfinite(ws[0])
    assert bad.nonzero().squeeze(1).tolist() == [300, 600]
    ws = _tensors([(1024,)], torch.float32, 0.02, 1)
    ad = bd.AdamWBatch(ws, gs, state_bits=8)
    ad.run()
    m, v = ad.moments()
    assert (~torch.isfinite(ws[0])).nonzero().squeeze(1).tolist() == [300, 600]
    for x in (m, v):   # the blocks of 256 that hold them, and no others
        assert torch.isnan(x[256:768]).all() and torch.isfinite(x[:256]).all()
        assert torch.isfinite(x[768:]).all()


def test_zero_gradients_and_betas_of_zero():
    ws = _tensors([(700,)], torch.float32, 0.02, 1)
    w0 = ws[0].clone()
    g = torch.zeros(700, device="cuda")
    for bits in (32, 8):
        ad = bd.AdamWBatch(ws, [g], state_bits=bits, eps=1e-8)
        ad.run()
        assert torch.equal(ws[0], w0)
        assert not any(x.any() for n, x in ad.state.items())
    g.fill_(2.0)
    ad = bd.AdamWBatch(ws, [g], betas=(0.0, 0.0), lr=0.5, eps=0.0)
    ad.run()   # m = g, v = g^2: the sign of the gradient
    assert torch.allclose(ws[0], w0 - 0.5, atol=1e-6)


def test_learning_rate_from_the_device_and_graph_replay():
    ws = _tensors(SHAPES, torch.bfloat16, 0.02, 1)
    gs = _tensors(SHAPES, torch.bfloat16, 0.02, 2)
    ws2 = [w.clone() for w in ws]
    lr = torch.zeros(1, device="cuda")
    a = bd.AdamWBatch(ws, gs, max_norm=0.1, weight_decay=0.1)
    b = bd.AdamWBatch(ws2, gs, max_norm=0.1, weight_decay=0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        a.run(lr=lr, stream=side)
    for i in range(4):
        lr.fill_(1e-3 * (i + 1))
        graph.replay()
        b.run(lr=1e-3 * (i + 1))
    torch.cuda.synchronize()
    assert int(a.steps.item()) == int(b.steps.item()) == 4
    for x, y in zip(ws, ws2):
        assert torch.equal(x, y)
    for n in a.state:
        assert torch.equal(a.state[n], b.state[n])


def test_two_batches_on_two_streams():
    made = []
    for seed in (1, 2):
        ws = _tensors(SHAPES + [(1 << 20,)], torch.bfloat16, 0.02, seed)
        gs = _tensors(SHAPES + [(1 << 20,)], torch.bfloat16, 0.02, seed + 10)
        ws2 = [w.clone() for w in ws]
        made.append((bd.AdamWBatch(ws, gs, max_norm=1.0, state_bits=8),
                     bd.AdamWBatch(ws2, gs, max_norm=1.0, state_bits=8), ws, ws2,
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        for a, _, _, _, s in made:
            a.run(stream=s)
    torch.cuda.synchronize()
    for a, b, ws, ws2, _ in made:
        for _ in range(3):
            b.run()
        torch.cuda.synchronize()
        assert torch.equal(a.norm, b.norm)
        assert all(torch.equal(x, y) for x, y in zip(ws, ws2))
        assert all(torch.equal(a.state[n], b.state[n]) for n in a.state)


def test_offsets_beyond_32_bits():
    n = (1 << 32) + 1000
    w = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    places = [0, 12345, (1 << 31) + 7, (1 << 32) - 1, (1 << 32) + 3, n - 1]
    g[places] = 0.5
    ad = bd.AdamWBatch([w], [g], master=False, state_bits=8, lr=0.25, eps=0.0, max_norm=1e9)
    ad.run()
    torch.cuda.synchronize()
    assert abs(float(ad.norm.item()) - 0.5 * len(places) ** 0.5) < 1e-5
    assert w[places].tolist() == [-0.25] * len(places)     # a first step moves by lr
    assert int(torch.count_nonzero(w)) == len(places)
    assert int(torch.count_nonzero(ad.state["v"])) == len(places)
    del w, g, ad
    torch.cuda.empty_cache()


def test_refusals():
    w = torch.zeros(64, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(64, dtype=torch.bfloat16, device="cuda")
    f = w.float()
    new = torch.zeros(64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        bd.AdamWBatch([], [])
    with pytest.raises(ValueError):
        bd.AdamWBatch([w], [g, g])
    with pytest.raises(TypeError):
        bd.AdamWBatch([w.half()], [g])
    with pytest.raises(ValueError):
        bd.AdamWBatch([w], [g[:32]])
    with pytest.raises(ValueError):
        bd.AdamWBatch([w.cpu()], [g.cpu()])
    with pytest.raises(ValueError):
        bd.AdamWBatch([w.view(8, 8).t()], [g])
    with pytest.raises(ValueError):
        bd.AdamWBatch([w, f], [g, g])
    with pytest.raises(ValueError):
        bd.AdamWBatch([w], [g], state_bits=16)
    with pytest.raises(ValueError):
        bd.AdamWBatch([f], [g], master=True)
    with pytest.raises(ValueError):
        bd.AdamWBatch([w], [g], stochastic=True)
    with pytest.raises(ValueError):
        bd.AdamWBatch([w], [g], max_norm=0.0)
    with pytest.raises(ValueError):
        bd.AdamWBatch([w], [g], betas=(1.0, 0.9))
    with pytest.raises(ValueError):
        bd.AdamWBatch([w], [g], weight_decay=[0.1, 0.2])
    with pytest.raises(ValueError):
        bd.AdamWBatch([w], [g], state={"m": torch.zeros(64, device="cuda")})
    with pytest.raises(ValueError):
        bd.AdamWBatch([w], [g], state={"x": w})
    # refused by the library: pointers off their alignment, outputs over inputs
    big = torch.zeros(80, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(bd.OpsError):
        bd.AdamWBatch([big[1:65]], [g], master=False)
    with pytest.raises(bd.OpsError):
        bd.AdamWBatch([big[:64]], [g], news=[big[8:72]], master=False)
    with pytest.raises(bd.OpsError):
        bd.AdamWBatch([w], [g], news=[g])
    ad = bd.AdamWBatch([w], [g], news=[new])
    with pytest.raises(ValueError):
        ad.run(lr=torch.zeros(1))
    with pytest.raises(bd.OpsError):
        ad.run(lr=float("nan"))
