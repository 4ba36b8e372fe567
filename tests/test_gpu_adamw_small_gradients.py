"""AdamW with an eps of 0, or so small that the root of a denormal second moment counts beside it:
an element with a gradient of 1e-20 moves as far as one with 1 (GPU).

Against the formula in 64 bits from the state as it was.  With u = 2^-24 and d = 2^-150 (half the
spacing of denormal numbers): the corrected second moment vt goes through at most five products and
sums, each off by u of it or by d (and those before the bias correction grow with it), so
  |vt - exact| <= 6 (u vt + d / (1 - beta2^t)) = e
and the step, off by 64 u for all that tests/test_gpu_adamw.py counts, by as much of itself as
sqrt(vt) is: e / vt at most where e < vt / 2.  p starts at 0, so that nothing of the step is lost.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("lossless_bf16_weight_old_gb300")

U, D, BLOCK = 2.0 ** -24, 2.0 ** -150, 256
LR, B1, B2 = 1e-3, 0.9, 0.95


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    bd._ops_lib.load()


def _np(t):
    return t.detach().double().cpu().numpy()


def _moments(ad):
    m, v = _np(ad.state["m"]), _np(ad.state["v"])
    if ad.state_bits == 8:
        m = np.sign(m) * (m / 127) ** 2 * np.repeat(_np(ad.state["m_scale"]), BLOCK)
        v = (v / 255) ** 4 * np.repeat(_np(ad.state["v_scale"]), BLOCK)
    return m[:ad.ns[0]], v[:ad.ns[0]]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [0.0, 1e-21, 1e-17, 1e-13])
@pytest.mark.parametrize("n", [2048, 2300])
def test_small_gradients_take_the_formulas_step(bits, eps, n):
    rng = np.random.default_rng(n)
    g = torch.zeros(n, device="cuda")
    w = torch.zeros(n, device="cuda")
    ad = bd.AdamWBatch([w], [g], state_bits=bits, eps=eps, lr=LR, betas=(B1, B2))
    sizes = 10.0 ** rng.choice([-20.5, -20.0, -19.0, -17.0, -15.0], n)
    for t in (1, 2, 3):
        g.copy_(torch.from_numpy(sizes * rng.choice([-1, 1], n) * rng.uniform(0.5, 1, n)))
        m, v = _moments(ad)
        w.zero_()
        ad.run()
        x = _np(g)
        m, v = B1 * m + (1 - B1) * x, B2 * v + (1 - B2) * x * x
        mt, vt = m / (1 - B1 ** t), v / (1 - B2 ** t)
        want = -LR * mt / (np.sqrt(vt) + eps)
        size = LR * (np.abs(m) + 2 * (1 - B1) * np.abs(x)) / (1 - B1 ** t) / (np.sqrt(vt) + eps)
        e = 6 * (U * vt + D / (1 - B2 ** t))
        assert np.all(e < vt / 2)
        assert np.all(np.abs(_np(w) - want) <= size * (64 * U + e / vt))
        assert np.abs(want).max() < 10 * LR     # (and a step is of the size of lr)


@pytest.mark.parametrize("bits", [32, 8])
def test_an_underflowed_second_moment_makes_no_step(bits):
    w = torch.full((300,), 0.5, device="cuda")
    g = torch.full((300,), 1e-25, device="cuda")    # 0.05 g^2 is 0 in FP32
    g[7] = 0.25
    ad = bd.AdamWBatch([w], [g], state_bits=bits, eps=0.0, lr=0.125, betas=(B1, B2))
    ad.run()
    torch.cuda.synchronize()
    assert abs(float(w[7]) - 0.375) < 1e-6
    w[7] = 0.5
    assert bool((w == 0.5).all())
