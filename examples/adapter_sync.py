"""Adapters trained in one place and served in another, in step.

A trainer holds a projection that stays as it is and a few low-rank adapters beside it, one per
policy.  Every step it runs a batch forward and backward (adapter_forward, adapter_backward),
updates all adapters at once (AdamWBatch) and encodes what changed (CompressBatch).  A worker that
serves the same adapters applies the update in place, verified bit for bit (DecompressBatch), and
answers the next requests with it: its adapters are read where they lie, so nothing is rebuilt.

    python examples/adapter_sync.py [steps]
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import lossless_bf16_weight_old_gb300 as bd  # noqa: E402

POLICIES, RANK, HIDDEN, OUT = 3, 16, 1024, 2048
ROWS, REQUESTS, SCALE = 1536, 40, 2.0


def _adapters(gen):
    downs = [(torch.randn(RANK, HIDDEN, generator=gen, device="cuda") * HIDDEN ** -0.5).bfloat16()
             for _ in range(POLICIES)]
    ups = [torch.zeros(OUT, RANK, dtype=torch.bfloat16, device="cuda") for _ in range(POLICIES)]
    return downs, ups


class Trainer:
    def __init__(self, shared: torch.Tensor, gen: torch.Generator):
        self.shared = shared
        downs, ups = _adapters(gen)
        self.weights = downs + ups
        self.news = [torch.empty_like(w) for w in self.weights]
        self.grads = [torch.zeros_like(w) for w in self.weights]
        self.set = bd.AdapterSet(downs, ups, SCALE, d_downs=self.grads[:POLICIES],
                                 d_ups=self.grads[POLICIES:])
        self.adam = bd.AdamWBatch(self.weights, self.grads, news=self.news, lr=4e-3,
                                  betas=(0.9, 0.95), max_norm=1.0)
        self.delta = bd.CompressBatch(self.weights, self.news)

    def step(self, x: torch.Tensor, target: torch.Tensor, policy: torch.Tensor):
        """One step; returns the loss and the update (payloads, sizes, checksums)."""
        rows = bd.AdapterRows(policy, POLICIES)
        low = torch.empty(x.shape[0], self.set.rank, dtype=torch.bfloat16, device="cuda")
        y = bd.adapter_forward(x, x @ self.shared.T, self.set, rows, low=low)
        error = y.float() - target.float()
        dy = (error * (2.0 / error.numel())).bfloat16()
        dx = dy @ self.shared          # the shared projection's part, for the layers below
        bd.adapter_backward(x, dy, low, dx, self.set, rows)
        self.adam.run()
        self.delta.run()
        return error.square().mean(), self.delta

    def commit(self) -> None:
        """The new adapters take the old ones' place (the update has left)."""
        torch._foreach_copy_(self.weights, self.news)


class Worker:
    def __init__(self, shared: torch.Tensor, weights):
        self.shared = shared
        self.weights = [w.clone() for w in weights]
        self.set = bd.AdapterSet(self.weights[:POLICIES], self.weights[POLICIES:], SCALE)

    def apply(self, delta: bd.CompressBatch) -> None:
        sizes = [int(n) for n in delta.sizes.tolist()]
        update = bd.DecompressBatch(self.weights, delta.payloads, sizes, delta.checksums)
        update.run()
        if int(update.status.item()) != bd.OK:
            raise bd.DeltaError(int(update.status.item()), "update")

    def answer(self, x: torch.Tensor, policy: torch.Tensor) -> torch.Tensor:
        """One token each of many requests, -1 for a request without an adapter."""
        return bd.adapter_forward(x, x @ self.shared.T, self.set, bd.AdapterRows(policy, POLICIES))


def main(steps: int = 8) -> list[float]:
    gen = torch.Generator(device="cuda").manual_seed(0)
    shared = (torch.randn(OUT, HIDDEN, generator=gen, device="cuda") * HIDDEN ** -0.5).bfloat16()
    trainer = Trainer(shared, gen)
    # what the policies are to learn: other second factors
    truth = bd.AdapterSet(
        [w.clone() for w in trainer.weights[:POLICIES]],
        [(torch.randn(OUT, RANK, generator=gen, device="cuda") * 0.05).bfloat16()
         for _ in range(POLICIES)], SCALE)
    worker = Worker(shared, trainer.weights)
    losses = []
    for i in range(steps):
        x = torch.randn(ROWS, HIDDEN, generator=gen, device="cuda").bfloat16()
        policy = (torch.arange(ROWS, device="cuda") * POLICIES // ROWS).int()
        target = bd.adapter_forward(x, x @ shared.T, truth, bd.AdapterRows(policy, POLICIES))
        loss, delta = trainer.step(x, target, policy)
        worker.apply(delta)
        trainer.commit()
        ask = torch.randint(-1, POLICIES, (REQUESTS,), generator=gen, device="cuda").int()
        q = torch.randn(REQUESTS, HIDDEN, generator=gen, device="cuda").bfloat16()
        answers = worker.answer(q, ask)
        here = bd.adapter_forward(q, q @ shared.T, trainer.set, bd.AdapterRows(ask, POLICIES))
        if not torch.equal(answers, here):
            raise RuntimeError("the worker's answers are not the trainer's")
        losses.append(float(loss))
        raw = sum(2 * w.numel() for w in trainer.weights)
        print(f"step {i}: loss {losses[-1]:.4f}, update {sum(delta.sizes.tolist())} bytes "
              f"of {raw}, {REQUESTS} answers as the trainer's")
    return losses


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 8)
