"""Training steps of a small mixture-of-experts layer on the MXFP8 cast.

    python examples/moe_training_step.py [--steps 20]

Token ids go through an embedding table, a router with its balance loss and one
linear layer per expert, whose products run in MXFP8 on what the dual-axis cast
gives: the row-wise bytes forward, the column-wise ones for the weights' gradients,
all experts in one call each.  Experts' weights move by orthogonalised momentum, the
table and the router by AdamW with moments in 8 bits.  The data is synthetic: each
token id has a fixed target.
"""
from __future__ import annotations

import argparse
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parent.parent))
import mx_block_quantization_gb300 as mxq  # noqa: E402


class MoeLayer:
    """embedding -> router -> k of E linear experts, with its gradients.  D is a
    multiple of 128."""

    def __init__(self, vocabulary: int, D: int, experts: int, k: int, seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        self.D, self.E, self.k = D, experts, k
        self.table = torch.randn(vocabulary, D, generator=g).to(torch.bfloat16).cuda()
        self.router = (torch.randn(experts, D, generator=g) / D**0.5).cuda()
        self.experts = (torch.randn(experts, D, D, generator=g) / D**0.5).to(torch.bfloat16).cuda()
        self.momentum = torch.zeros(experts, D, D, device="cuda")
        self.moments = mxq.adamw_moments([self.table, self.router], bits=8)
        self.steps = 0
        # the experts' weights are cast as one matrix: a group of rows for each
        self.each = torch.arange(1, experts + 1, dtype=torch.int32, device="cuda") * D

    def forward(self, ids):
        """Layer output [T, D] and the balance loss; keeps what backward needs."""
        D, E = self.D, self.E
        self.ids, self.x = ids, mxq.embedding(ids, self.table)
        self.logits = self.x.float() @ self.router.t()
        self.routing = mxq.moe_route(self.logits, self.k)
        self.plan = mxq.moe_plan(self.routing.ids, E)
        self.cast = mxq.quantize_2d_dual(mxq.moe_dispatch(self.x, self.plan), self.plan.offs)
        self.w = mxq.quantize_2d_dual(self.experts.view(E * D, D), self.each)
        self.rows = mxq.moe_linear(self.cast.q_row, self.cast.s_row, self.w.q_row.view(E, D, D), self.w.s_row, self.plan.offs)
        return mxq.moe_combine(self.rows, self.plan, self.routing.weights), self.routing.loss

    def backward(self, dy, dloss):
        """Gradients of the table, the router and the experts."""
        D, E, offs = self.D, self.E, self.plan.offs
        drows, dweights = mxq.moe_combine_backward(dy, self.rows, self.plan, self.routing.weights)
        cast = mxq.quantize_2d_dual(drows, offs)
        by_output = self.w.q_col.view(D, E, D).transpose(0, 1)      # blocks along the output, transposed
        dx_rows = mxq.moe_linear(cast.q_row, cast.s_row, by_output, self.w.s_col, offs)
        dexperts = mxq.moe_weight_gradient(cast.q_col, cast.s_col, self.cast.q_col, self.cast.s_col, offs)
        dlogits = mxq.moe_route_backward(self.logits, self.routing, dweights, dloss)
        dx = mxq.moe_combine(dx_rows, self.plan).float() + dlogits @ self.router
        dtable = mxq.embedding_backward(self.ids, dx, self.table.shape[0])
        return dtable, dlogits.t() @ self.x.float(), dexperts

    def update(self, gradients, lr: float, lr_experts: float, beta: float = 0.9):
        dtable, drouter, dexperts = gradients
        self.steps += 1
        mxq.adamw_step([self.table, self.router], [dtable, drouter], self.moments, self.steps, lr=lr, betas=(beta, 0.95),
                       weight_decay=0.0)
        self.momentum.mul_(beta).add_(dexperts)
        self.experts -= mxq.orthogonalize(self.momentum, scale=lr_experts)


def train(steps: int, tokens: int = 4096, vocabulary: int = 1000, D: int = 256, experts: int = 8, k: int = 2):
    """The mean squared error and the balance loss of each step."""
    layer = MoeLayer(vocabulary, D, experts, k)
    g = torch.Generator().manual_seed(1)
    target = torch.randn(vocabulary, D, generator=g).cuda()
    history = []
    for _ in range(steps):
        ids = torch.randint(0, vocabulary, (tokens,), generator=g).cuda()
        y, balance = layer.forward(ids)
        off = y.float() - target[ids]
        gradients = layer.backward((off * (2 / tokens)).to(torch.bfloat16), torch.tensor(0.01, device="cuda"))
        layer.update(gradients, lr=0.02, lr_experts=0.05)
        history.append((float(off.square().mean()), float(balance)))
    status = mxq.device_status()
    if status:
        raise RuntimeError(f"device status {status:#x}")
    return history


def main():
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=20)
    for i, (error, balance) in enumerate(train(parser.parse_args().steps)):
        print(f"step {i:3d}  error {error:.4f}  balance loss {balance:.4f}")


if __name__ == "__main__":
    main()
