"""The example that trains a policy from its log probabilities and keeps a worker in step (GPU): it
runs, and its gradients are those of the loss."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    spec = importlib.util.spec_from_file_location("policy_step", os.path.join(ROOT, "examples", "policy_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_it_runs_and_the_worker_stays_in_step(example):
    assert len(example.main(4)) == 4     # (raises where a log probability differs in any bit)


def test_gradients(example):
    """Against automatic differentiation of the loss in 64 bits, with the chosen experts as they are.

    The gradients are chains of at most six FP32 products whose sums have at most L = 4099 terms: each
    is off by L u of the sum of its terms' sizes (u = 2^-24), which for signs at random is sqrt(L) of
    the sum.  6 L sqrt(L) u = 0.094 bounds the worst order of summation; in 2-norm, over many
    elements, the terms' errors are as random as their signs, sqrt(L) in place of L: 6 L u = 1.5e-3."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    params = example.weights(gen)
    policy = example.Policy(params)
    x = torch.randn(example.ROWS, example.HIDDEN, generator=gen, device="cuda")
    tokens = torch.randint(example.VOCAB, (example.ROWS,), generator=gen, device="cuda")
    tokens[::7] = -1                                     # rows that are left out
    advantage = torch.randn(example.ROWS, generator=gen, device="cuda")
    got = policy.gradients(policy.logits(x), tokens, advantage)

    leaves = [p.double().requires_grad_() for p in params]
    router, experts, head = leaves
    n, chosen = tokens.numel(), policy.routing.experts.long()
    p = torch.softmax(x.double() @ router.T, 1)
    w = p.gather(1, chosen)
    w = w / w.sum(1, keepdim=True)
    y = x.double() + (w[:, :, None] * torch.einsum("rkoi,ri->rko", experts[chosen], x.double())).sum(1)
    lp = torch.log_softmax(y @ head.T / example.TEMPERATURE, 1)
    counts = torch.bincount(chosen.reshape(-1), minlength=example.EXPERTS).double()
    balance = example.EXPERTS * (counts / counts.sum() * p.mean(0)).sum()
    real = tokens >= 0
    given = lp.gather(1, tokens.clamp(min=0)[:, None]).squeeze(1)
    entropy = -(lp.exp() * lp).sum(1)
    each = advantage.double() * given + example.ENTROPY * entropy
    (-(each * real).sum() / n + example.BALANCE * balance).backward()
    for name, a, leaf in zip(("router", "experts", "head"), got, leaves):
        off = float((a.double() - leaf.grad).norm() / leaf.grad.norm())
        assert off < 1.5e-3, (name, off)
