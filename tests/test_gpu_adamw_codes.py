"""An 8-bit AdamW step has one right result: its codes and scales equal a computation that rounds
every FP32 operation of include/ops/bf16ops.h's formulas once, in their order (GPU).

PyTorch's elementwise operations are such roundings (products, sums, quotients and roots of
IEEE 754), so the comparison is for equality; nothing is compared that an approximate root or
quotient enters (the weights).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("lossless_bf16_weight_old_gb300")

BLOCK = 256
GAMMA = 0x9E3779B97F4A7C15


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    bd._ops_lib.load()


def _signed(x):
    x &= (1 << 64) - 1
    return x - (1 << 64) if x >> 63 else x


def _mix(z):
    def shift(x, k):
        return (x >> k) & ((1 << (64 - k)) - 1)
    z = (z ^ shift(z, 30)) * _signed(0xBF58476D1CE4E5B9)
    z = (z ^ shift(z, 27)) * _signed(0x94D049BB133111EB)
    return z ^ shift(z, 31)


def _noise(count, seed, t):
    key = _mix(torch.tensor(_signed(seed ^ (t * GAMMA)), device="cuda"))
    r = _mix(key + torch.arange(1, count // 2 + 1, device="cuda") * _signed(GAMMA))
    return torch.stack([r & 0xFFFFFFFF, (r >> 32) & 0xFFFFFFFF], 1).view(-1)


def _ratio(x, scale):
    return torch.where(scale[:, None] > 0, x / scale[:, None], torch.zeros((), device="cuda"))


@pytest.mark.parametrize("size", [1.0, 1e-6])
@pytest.mark.parametrize("gtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("b1,b2", [(0.9, 0.95), (0.9, 0.999)])
def test_codes_are_exact(size, gtype, b1, b2):
    n, seed = BLOCK * 4096, 99
    gen = torch.Generator(device="cuda").manual_seed(7)
    spread = torch.exp(torch.randn(n // BLOCK, 1, generator=gen, device="cuda")) * size
    spread = spread * (torch.rand(n // BLOCK, 1, generator=gen, device="cuda") > 0.1)
    w = (torch.randn(n, generator=gen, device="cuda") * 0.02).bfloat16()
    g = torch.empty(n, dtype=gtype, device="cuda")
    adam = bd.AdamWBatch([w], [g], state_bits=8, betas=(b1, b2), seed=seed)
    st = adam.state
    cm, cv = torch.zeros(2, n // BLOCK, BLOCK, device="cuda")
    sm, sv = torch.zeros(2, n // BLOCK, device="cuda")
    for t in range(1, 5):
        g.copy_((torch.randn(n // BLOCK, BLOCK, generator=gen, device="cuda") * spread).view(-1))
        adam.run()
        x = g.float().view(-1, BLOCK)
        m = cm * cm.abs() * (1 / 127 ** 2) * sm[:, None]
        v = (cv * (1 / 255)).square().square() * sv[:, None]
        m = m * b1 + x * (1 - b1)
        v = v * b2 + x.square() * (1 - b2)
        sm, sv = m.abs().amax(1), v.amax(1)
        cm = (_ratio(m.abs(), sm).sqrt() * 127).round() * m.sign()
        q = _ratio(v, sv)
        low = (q.sqrt().sqrt() * 255).floor().clamp(max=254)
        a = (low * (1 / 255)).square().square()
        b = ((low + 1) * (1 / 255)).square().square()
        u = (_noise(n, seed, t) >> 16).float().view(-1, BLOCK) * (1 / 65536)
        cv = torch.where(v > 0, (low + (u * (b - a) < q - a)).clamp(min=1),
                         torch.zeros((), device="cuda"))
        assert torch.equal(st["m_scale"], sm) and torch.equal(st["v_scale"], sv)
        assert torch.equal(st["m"].float().view(-1, BLOCK), cm)
        assert torch.equal(st["v"].float().view(-1, BLOCK), cv)
