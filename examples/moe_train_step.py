"""A data-parallel training step of a small mixture of experts, on N logical ranks of one GPU.

    python examples/moe_train_step.py [--steps 200] [--state-bits 8]

Every rank has its own tokens and a bfloat16 working copy of all weights (a
router and E linear experts).  A step is

    route          top-2 experts per token, gate weights, counts, balance loss
    experts        y = sum_k weight_k x W_k, squared error against a teacher
    route_grad     gradient of the router's logits, balance loss included
    reduce_scatter each rank gets its shard of the gradients' sum
    AdamW          grad_norm clips the mean gradient, step updates the shards
                   (float32 weights, 32- or 8-bit states) and their copies
    allgather      the copies of all shards to every rank
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tree_allreduce_algorithms_amd as ar  # noqa: E402

RANKS, TOKENS, DIM, EXPERTS, TOP_K = 4, 256, 32, 8, 2
BALANCE = 0.01           # weight of the balance loss
SIZES = (DIM * EXPERTS, EXPERTS * DIM * DIM)


def split(flat):
    """The router's and the experts' weights in a flat buffer."""
    router, experts = flat[:sum(SIZES)].split(SIZES)
    return router.view(DIM, EXPERTS), experts.view(EXPERTS, DIM, DIM)


def expert_outputs(x, indices, experts):
    """x W_k of each token's chosen experts: [tokens, top_k, dim]."""
    return torch.matmul(x[:, None, None, :], experts[indices.long()])[:, :, 0]


class Trainer:
    def __init__(self, state_bits=32, seed=0, device="cuda"):
        torch.manual_seed(seed)
        # whole blocks of 256 for every rank's shard
        self.count = -(-sum(SIZES) // (RANKS * 256)) * RANKS * 256
        self.teacher = torch.randn(self.count, device=device) * 0.5
        start = torch.randn(self.count, device=device) * 0.1
        self.copies = [start.bfloat16() for _ in range(RANKS)]
        self.grads = [torch.zeros(self.count, device=device) for _ in range(RANKS)]
        spans = [ar.chunk_range(RANKS, self.count, r) for r in range(RANKS)]
        self.optimizer = ar.AdamW(
            params=[start[lo:hi].clone() for lo, hi in spans],
            grads=[g[lo:hi] for g, (lo, hi) in zip(self.grads, spans)],
            copies=[c[lo:hi] for c, (lo, hi) in zip(self.copies, spans)],
            state_bits=state_bits, weight_decay=0.0, grad_scale=1.0 / RANKS)
        self.balance = torch.full((), BALANCE, device=device)

    def step(self, lr):
        """One step on fresh tokens; (mean squared error, balance loss, gradient norm), on the GPU."""
        x = [torch.randn(TOKENS, DIM, device=self.teacher.device) for _ in range(RANKS)]
        weights = [split(c.float()) for c in self.copies]
        teacher_router, teacher_experts = split(self.teacher)
        truth = ar.route([t @ teacher_router for t in x], TOP_K, renormalize=True)

        logits = [t @ router for t, (router, _) in zip(x, weights)]
        routing = ar.route(logits, TOP_K, renormalize=True)
        errors, dweights, douts = [], [], []
        for r in range(RANKS):
            target = (truth.weights[r][:, :, None] *
                      expert_outputs(x[r], truth.indices[r], teacher_experts)).sum(1)
            out = expert_outputs(x[r], routing.indices[r], weights[r][1])
            error = (routing.weights[r][:, :, None] * out).sum(1) - target
            dy = error * (2.0 / error.numel())
            errors.append(error.square().mean())
            dweights.append((dy[:, None] * out).sum(-1))
            douts.append(routing.weights[r][:, :, None] * dy[:, None])
        dlogits = ar.route_grad(logits, routing, dweights=dweights, dloss=self.balance)
        for r in range(RANKS):
            drouter, dexperts = split(self.grads[r].zero_())
            torch.matmul(x[r].t(), dlogits[r], out=drouter)
            products = x[r][:, None, :, None] * douts[r][:, :, None, :]      # [tokens, top_k, dim, dim]
            dexperts.index_add_(0, routing.indices[r].flatten(), products.flatten(0, 1))

        ar.reduce_scatter(self.grads)
        norm = self.optimizer.grad_norm(max_norm=1.0)
        self.optimizer.step(lr, clip=True)
        ar.allgather(self.copies)
        return torch.stack(errors).mean(), routing.loss, norm


def main(steps=200, state_bits=32):
    trainer = Trainer(state_bits)
    for k in range(steps):
        error, balance, norm = trainer.step(lr=1e-2 * (1 - k / steps))
        if k % max(1, steps // 10) == 0 or k == steps - 1:
            print(f"step {k:4d}  error {float(error):.4f}  balance {float(balance):.3f}  "
                  f"gradient norm {float(norm):.4f}", flush=True)
    return float(error)


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    parser.add_argument("--steps", type=int, default=200)
    parser.add_argument("--state-bits", type=int, choices=(8, 32), default=32)
    args = parser.parse_args()
    main(args.steps, args.state_bits)
