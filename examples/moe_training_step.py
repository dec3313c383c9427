"""Training steps of a small mixture-of-experts layer on the MXFP8 cast.

    python examples/moe_training_step.py [--steps 20]

Token ids go through an embedding table, a router with its balance loss and one
linear layer per expert, whose products run in MXFP8 on what the dual-axis cast
gives: the row-wise bytes forward, the column-wise ones for the weights' gradients.
Experts' weights move by orthogonalised momentum, the table and the router by
their gradients.  The data is synthetic: each token id has a fixed target.
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

    def _product(self, q, s, at, w, e):
        """Rows `at` of the cast (q, s), times expert e of the cast w: [rows, D] fp32."""
        (lo, hi), D = at, self.D
        wq, ws = w
        return mxq.mxfp8_scaled_mm(q[lo:hi], s[lo * D // 32:hi * D // 32], wq[e], ws[e])

    def forward(self, ids):
        """Layer output [T, D] and the balance loss; keeps what backward needs."""
        D, E = self.D, self.E
        self.ids, self.x = ids, mxq.embedding(ids, self.table)
        self.logits = self.x.float() @ self.router.t()
        self.routing = mxq.moe_route(self.logits, self.k)
        self.plan = mxq.moe_plan(self.routing.ids, E)
        ends = self.plan.offs.tolist()
        self.groups = [(e, (lo, hi)) for e, (lo, hi) in enumerate(zip([0] + ends, ends)) if hi > lo]
        self.cast = mxq.quantize_2d_dual(mxq.moe_dispatch(self.x, self.plan), self.plan.offs)
        w = [mxq.quantize_2d_dual(self.experts[e]) for e in range(E)]
        self.w_rows = [c.q_row for c in w], [c.s_row for c in w]      # blocks along the input
        self.w_cols = [c.q_col for c in w], [c.s_col for c in w]      # transposed, along the output
        self.rows = torch.zeros(self.plan.source.numel(), D, dtype=torch.bfloat16, device="cuda")
        for e, at in self.groups:
            self.rows[slice(*at)] = self._product(self.cast.q_row, self.cast.s_row, at, self.w_rows, e)
        return mxq.moe_combine(self.rows, self.plan, self.routing.weights), self.routing.loss

    def backward(self, dy, dloss):
        """Gradients of the table, the router and the experts."""
        D = self.D
        drows, dweights = mxq.moe_combine_backward(dy, self.rows, self.plan, self.routing.weights)
        cast = mxq.quantize_2d_dual(drows, self.plan.offs)
        dx_rows = torch.zeros_like(self.rows)
        dexperts = torch.zeros_like(self.momentum)
        for e, at in self.groups:
            lo, hi = at
            slab = slice(D * lo // 32, D * hi // 32)
            dx_rows[lo:hi] = self._product(cast.q_row, cast.s_row, at, self.w_cols, e)
            mxq.mxfp8_scaled_mm(cast.q_col[:, lo:hi], cast.s_col[slab], self.cast.q_col[:, lo:hi], self.cast.s_col[slab],
                                out=dexperts[e])
        dlogits = mxq.moe_route_backward(self.logits, self.routing, dweights, dloss)
        dx = mxq.moe_combine(dx_rows, self.plan).float() + dlogits @ self.router
        dtable = mxq.embedding_backward(self.ids, dx, self.table.shape[0])
        return dtable, dlogits.t() @ self.x.float(), dexperts

    def update(self, gradients, lr: float, lr_router: float, lr_experts: float, beta: float = 0.9):
        dtable, drouter, dexperts = gradients
        self.table -= (lr * dtable).to(torch.bfloat16)
        self.router -= lr_router * drouter
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
        layer.update(gradients, lr=1.0, lr_router=0.05, lr_experts=0.05)
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
