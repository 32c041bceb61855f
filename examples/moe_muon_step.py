"""A data-parallel training step of a layer of experts on N logical ranks of one GPU, with Muon.

    python examples/moe_muon_step.py [--steps 100]

Every rank has its own tokens and a bfloat16 working copy of all weights: a
router, and E experts of two matrices with a ReLU between them.  A step is

    route, expert_order        top-2 experts per token, the pairs in order by expert
    expert_matmul (twice)      the experts' products, as many rows as chose each
    expert_combine             the tokens' weighted sums
    backward                   expert_combine_grad, expert_weight_grad, expert_matmul
                               with the transposed weights, route_grad
    reduce_scatter             each rank gets the sum of whole experts' gradients
    Muon, AdamW                Muon for the experts' matrices, AdamW for the router
    allgather                  the copies of all shards to every rank
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tree_allreduce_algorithms_amd as ar  # noqa: E402

RANKS, TOKENS, DIM, HIDDEN, EXPERTS, TOP_K = 4, 256, 64, 96, 8, 2
BALANCE = 0.01           # weight of the balance loss
OWN = EXPERTS // RANKS   # experts whose matrices a rank updates


def layer(x, routing, rank, order, w1, w2):
    """(hidden values, rows, sums) of one rank's tokens."""
    u = ar.expert_matmul(x, w1, order, gather=True)
    y = ar.expert_matmul(torch.relu(u), w2, order)
    return u, y, ar.expert_combine(y, order, routing.weights[rank])


def layer_grad(x, routing, rank, order, w1, w2, u, y, dout, dw1, dw2):
    """Gradient of the weights into dw1 and dw2; returns those of x and of the gate weights."""
    dy, dgate = ar.expert_combine_grad(dout, y, order, routing.weights[rank])
    ar.expert_weight_grad(torch.relu(u), dy, order, out=dw2)
    du = ar.expert_matmul(dy, w2.transpose(1, 2), order) * (u > 0)
    ar.expert_weight_grad(x, du, order, gather=True, out=dw1)
    return ar.expert_combine(ar.expert_matmul(du, w1.transpose(1, 2), order), order), dgate


class Trainer:
    def __init__(self, seed=0, device="cuda"):
        torch.manual_seed(seed)
        shapes = [(EXPERTS, DIM, HIDDEN), (EXPERTS, HIDDEN, DIM)]
        start = [torch.randn(s, device=device) * s[1] ** -0.5 for s in shapes]
        self.teacher = [torch.randn(s, device=device).bfloat16() * s[1] ** -0.5 for s in shapes]
        self.copies = [[w.bfloat16() for _ in range(RANKS)] for w in start]        # [matrix][rank]
        self.grads = [[torch.zeros_like(w) for _ in range(RANKS)] for w in start]
        own = [slice(r * OWN, (r + 1) * OWN) for r in range(RANKS)]
        shards = lambda ts: [t[s] for matrix in ts for t, s in zip(matrix, own)]  # noqa: E731
        # match_rms, since the matrices stand as [in, out]: the other scale is for [out, in]
        self.muon = ar.Muon([w[s].clone() for w in start for s in own], shards(self.grads), shards(self.copies),
                            momentum=0.9, match_rms=0.2, grad_scale=1.0 / RANKS)
        # the router is small: its gradient's sum is updated once and copied
        self.router = torch.randn(DIM, EXPERTS, device=device) * DIM ** -0.5
        self.router_grads = [torch.zeros_like(self.router) for _ in range(RANKS)]
        self.adamw = ar.AdamW([self.router], self.router_grads[:1], grad_scale=1.0 / RANKS, weight_decay=0.0)
        self.balance = torch.full((), BALANCE, device=device)

    def backward(self, x):
        """Gradients on these tokens [ranks][tokens, dim]; (mean squared error, balance loss)."""
        logits = [t.float() @ self.router for t in x]
        routing = ar.route(logits, TOP_K, renormalize=True)
        errors, dgates = [], []
        for r in range(RANKS):
            order = ar.expert_order(routing.indices[r], EXPERTS)
            w1, w2 = (c[r] for c in self.copies)
            target = layer(x[r], routing, r, order, *self.teacher)[2]
            u, y, out = layer(x[r], routing, r, order, w1, w2)
            error = out.float() - target.float()
            dout = (error * (2.0 / error.numel())).bfloat16()
            _, dgate = layer_grad(x[r], routing, r, order, w1, w2, u, y, dout, self.grads[0][r], self.grads[1][r])
            errors.append(error.square().mean())
            dgates.append(dgate)
        dlogits = ar.route_grad(logits, routing, dweights=dgates, dloss=self.balance)
        for r in range(RANKS):
            torch.matmul(x[r].float().t(), dlogits[r], out=self.router_grads[r])
        return torch.stack(errors).mean(), routing.loss

    def step(self, lr):
        """One step on fresh tokens; (mean squared error, balance loss), on the GPU."""
        x = [torch.randn(TOKENS, DIM, device=self.router.device).bfloat16() for _ in range(RANKS)]
        losses = self.backward(x)
        for grads in self.grads:
            ar.reduce_scatter(grads)
        ar.ring_allreduce(self.router_grads)
        self.muon.step(lr)
        self.adamw.step(0.1 * lr)
        for copies in self.copies:
            ar.allgather(copies)
        return losses


def main(steps=100):
    trainer = Trainer()
    for k in range(steps):
        error, balance = trainer.step(lr=0.03 * (1 - k / steps))
        if k % max(1, steps // 10) == 0 or k == steps - 1:
            print(f"step {k:4d}  error {float(error):.4f}  balance {float(balance):.3f}", flush=True)
    return float(error)


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    parser.add_argument("--steps", type=int, default=100)
    main(parser.parse_args().steps)
