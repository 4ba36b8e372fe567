"""The rate of a step is the one that it is given, or the batch's own (GPU).  A gradient of 1 whose
size never changes moves a weight by the rate in every step (m / (1 - b1^t) = v / (1 - b2^t) = 1, to
a few units of FP32; the sum of four steps to 1e-5)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("lossless_bf16_weight_old_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    bd._ops_lib.load()


def _moved(steps):
    w, g = torch.zeros(300, device="cuda"), torch.ones(300, device="cuda")
    ad = bd.AdamWBatch([w], [g], lr=0.125, betas=(0.9, 0.95))
    steps(ad)
    torch.cuda.synchronize()
    assert bool((w == w[0]).all())
    return -float(w[0])


def test_a_rate_from_the_device_is_one_steps():
    lr = torch.full((1,), 0.5, device="cuda")

    def steps(ad):
        ad.run(lr=lr)
        lr.fill_(2.0)
        ad.run()
        ad.run(lr=lr)
        ad.run()

    assert abs(_moved(steps) - (0.5 + 0.125 + 2.0 + 0.125)) < 1e-5


def test_a_number_is_one_steps():
    def steps(ad):
        ad.run(lr=1.0)
        ad.run()
        ad.lr = 0.25
        ad.run()

    assert abs(_moved(steps) - (1.0 + 0.125 + 0.25)) < 1e-5


def test_a_refused_rate_leaves_nothing_behind():
    def steps(ad):
        for bad in (float("nan"), float("inf")):
            with pytest.raises(bd.OpsError):
                ad.run(lr=bad)
        with pytest.raises(ValueError):
            ad.run(lr=torch.zeros(2, device="cuda"))
        ad.run()

    assert abs(_moved(steps) - 0.125) < 1e-5
