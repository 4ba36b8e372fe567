"""One policy in two places: a worker answers, a trainer learns from the answers and sends the update.

The policy is a small mixture of experts: a router, experts beside a residual stream, and a head over
the vocabulary.  A worker draws tokens and reports their log probabilities with the top alternatives
(TokenLogprobs).  The trainer runs the same tokens forward, takes the loss's gradient by hand (the log
probabilities' and entropies' by TokenLogprobs.backward, the router's with its balance loss by
ExpertRouting.backward), updates all weights at once (AdamWBatch) and encodes what changed
(CompressBatch).  The worker applies the update in place, verified bit for bit (DecompressBatch): from
then on its log probabilities are the trainer's, bit for bit.

    python examples/policy_step.py [steps]
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import lossless_bf16_weight_old_gb300 as bd  # noqa: E402

ROWS, HIDDEN, EXPERTS, CHOSEN, VOCAB = 512, 64, 16, 2, 4099
TOP, TEMPERATURE, ENTROPY, BALANCE = 5, 0.9, 1e-3, 1e-2


def weights(gen: torch.Generator) -> list[torch.Tensor]:
    """Router, experts and head, in BF16 as the sync takes them."""
    def normal(*shape):
        return (torch.randn(shape, generator=gen, device="cuda") * shape[-1] ** -0.5).bfloat16()
    return [normal(EXPERTS, HIDDEN), normal(EXPERTS, HIDDEN, HIDDEN), normal(VOCAB, HIDDEN)]


class Policy:
    """The forward pass in FP32 over BF16 weights, and its gradient."""

    def __init__(self, params: list[torch.Tensor], rows: int = ROWS):
        self.params = params
        self.routing = bd.ExpertRouting(rows, EXPERTS, CHOSEN)
        self.scores = bd.TokenLogprobs(rows, VOCAB, top=TOP, entropy=True)

    def logits(self, x: torch.Tensor) -> torch.Tensor:
        """x [rows, HIDDEN], float32; keeps what the gradient needs."""
        router, experts, head = (p.float() for p in self.params)
        self.x, self.router_logits = x, x @ router.T
        self.routing.run(self.router_logits)
        chosen = self.routing.experts[:x.shape[0]].long()
        self.each = torch.einsum("rkoi,ri->rko", experts[chosen], x)
        self.y = x + (self.routing.weights[:x.shape[0], :, None] * self.each).sum(1)
        return self.y @ head.T

    def gradients(self, logits: torch.Tensor, tokens: torch.Tensor, advantage: torch.Tensor):
        """Of -mean(advantage logprob + ENTROPY entropy) + BALANCE balance, by weight.  logits: of
        the last forward pass; their gradient takes their place."""
        n = tokens.numel()
        router, experts, head = (p.float() for p in self.params)
        self.scores.run(logits, tokens, TEMPERATURE)
        bonus = torch.full((1,), -ENTROPY / n, device="cuda").expand(n)
        d = self.scores.backward(logits, advantage * (-1.0 / n), bonus, out=logits)
        d_head, d_y = d.T @ self.y, d @ head
        chosen = self.routing.experts[:n].long()
        d_each = self.routing.weights[:n, :, None] * d_y[:, None, :]
        d_weights = (self.each * d_y[:, None, :]).sum(2)
        outer = torch.einsum("rko,ri->rkoi", d_each, self.x).reshape(-1, HIDDEN, HIDDEN)
        d_experts = torch.zeros(EXPERTS, HIDDEN, HIDDEN, device="cuda")
        for e in range(EXPERTS):   # (summed in a fixed order)
            d_experts[e] = outer[chosen.reshape(-1) == e].sum(0)
        d_router_logits = self.routing.backward(self.router_logits, d_weights, BALANCE)
        return [d_router_logits.T @ self.x, d_experts, d_head]


class Trainer:
    def __init__(self, params: list[torch.Tensor]):
        self.params = params
        self.policy = Policy(params)
        self.news = [torch.empty_like(p) for p in params]
        self.grads = [torch.zeros(p.shape, device="cuda") for p in params]
        self.adam = bd.AdamWBatch(params, self.grads, news=self.news, lr=2e-3, max_norm=1.0)
        self.delta = bd.CompressBatch(params, self.news)

    def step(self, x, tokens, advantage) -> bd.CompressBatch:
        logits = self.policy.logits(x)
        torch._foreach_copy_(self.grads, self.policy.gradients(logits, tokens, advantage))
        self.adam.run()            # (skips the step where a gradient is not finite)
        self.delta.run()
        return self.delta

    def commit(self) -> None:
        torch._foreach_copy_(self.params, self.news)


class Worker:
    def __init__(self, params: list[torch.Tensor]):
        self.params = [p.clone() for p in params]
        self.policy = Policy(self.params)

    def apply(self, delta: bd.CompressBatch) -> None:
        sizes = [int(n) for n in delta.sizes.tolist()]
        update = bd.DecompressBatch(self.params, delta.payloads, sizes, delta.checksums)
        update.run()
        if int(update.status.item()) != bd.OK:
            raise bd.DeltaError(int(update.status.item()), "update")

    def answer(self, x: torch.Tensor, gen: torch.Generator) -> torch.Tensor:
        """A token for each row; `policy.scores` has their log probabilities and alternatives."""
        logits = self.policy.logits(x)
        p = torch.softmax(logits / TEMPERATURE, 1)
        tokens = torch.multinomial(p, 1, generator=gen).squeeze(1)
        self.policy.scores.run(logits, tokens, TEMPERATURE)
        return tokens


def main(steps: int = 6) -> list[float]:
    gen = torch.Generator(device="cuda").manual_seed(0)
    trainer = Trainer(weights(gen))
    worker = Worker(trainer.params)
    liked = torch.rand(VOCAB, generator=gen, device="cuda") < 0.2    # tokens that are rewarded
    rewards = []
    for i in range(steps):
        x = torch.randn(ROWS, HIDDEN, generator=gen, device="cuda")
        tokens = worker.answer(x, gen)
        reported = worker.policy.scores.logprobs.clone()
        scores = bd.TokenLogprobs(ROWS, VOCAB, entropy=True)
        scores.run(trainer.policy.logits(x), tokens, TEMPERATURE)
        if not torch.equal(scores.logprobs, reported):
            raise RuntimeError("the worker's log probabilities are not the trainer's")
        reward = liked[tokens].float()
        worker.apply(trainer.step(x, tokens, reward - reward.mean()))
        trainer.commit()
        rewards.append(float(reward.mean()))
        print(f"step {i}: reward {rewards[-1]:.3f}, entropy {float(scores.entropy.mean()):.3f}, balance "
              f"{float(trainer.policy.routing.loss):.3f}, update {sum(trainer.delta.sizes.tolist())} bytes of "
              f"{sum(2 * p.numel() for p in trainer.params)}, log probabilities as the trainer's")
    return rewards


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 6)
