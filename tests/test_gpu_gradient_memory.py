"""The memory that a gradient of logits gets for itself, of logits whose rows lie far apart (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("lossless_bf16_weight_old_gb300")

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    bd._ops_lib.load()


def _views(rows, width, dtype):
    """The last position of sequences, every third row, columns of a wide buffer, a few columns of padding."""
    gen = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)
    return [normal(rows, 9, width)[:, -1], normal(3 * rows, width)[::3], normal(rows, 7 * width + 3)[:, 5:5 + width],
            normal(rows, width + 3)[:, :width], normal(rows, width), normal(1, 5, width)[:, 2]]


def _check(make, x, width):
    dx = make(x)
    assert dx.shape == x.shape and torch.equal(dx, make(x, out=torch.empty(x.shape, dtype=x.dtype, device="cuda")))
    words = 32 // dx.element_size()
    assert dx.untyped_storage().nbytes() <= dx.shape[0] * (width + words) * dx.element_size()
    if x.shape[0] > 1:      # (and its rows begin alike)
        assert dx.stride(0) >= width and (dx.stride(0) - x.stride(0)) % words == 0


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("width", [1, 17, 1000, 4101])
def test_of_log_probabilities(dtype, width):
    rows = 12
    tokens, g = torch.arange(rows, device="cuda") % width, torch.randn(rows, device="cuda")
    for x in _views(rows, width, dtype):
        n = x.shape[0]
        lp = bd.TokenLogprobs(n, width)

        def make(x, **kw):
            lp.run(x, tokens[:n])
            return lp.backward(x, g[:n], **kw)
        _check(make, x, width)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("width", [1, 17, 128, 1000])
def test_of_routing(dtype, width):
    rows = 12
    gw = torch.randn(rows, 1, device="cuda")
    for x in _views(rows, width, dtype):
        n = x.shape[0]
        a = bd.ExpertRouting(n, width, 1, normalize=False)

        def make(x, **kw):
            a.run(x)
            return a.backward(x, gw[:n], 0.5, **kw)
        _check(make, x, width)
