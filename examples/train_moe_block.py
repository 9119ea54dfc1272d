"""Trains one small mixture-of-experts block with libmuon's operators and Muon.

    python examples/train_moe_block.py [--steps N]

The block is y = x + sum over the k experts taken of w_e W2_e relu(W1_e n(x)),
with a layer norm n and a router over n(x).  Its activations are kept in 8
bits: one checkpoint of the normalised rows serves the norm's backward pass
and the gradients of the router's and the experts' first matrices, one of the
hidden activations the gradients of their second matrices.  The experts'
gradients are taken over their own tokens and written into the tensors that
Muon steps with.  The products of activations with weights are torch's.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import newton_schulz_06_gb300 as ns  # noqa: E402


class Block:
    def __init__(self, hidden: int, inner: int, experts: int, k: int, device="cuda", seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            return (torch.randn(shape, generator=g, device=device) * shape[-1] ** -0.5).bfloat16()

        self.k, self.experts = k, experts
        self.router, self.w1, self.w2 = (weight(experts, hidden), weight(experts, inner, hidden),
                                         weight(experts, hidden, inner))
        self.gain = torch.ones(hidden, device=device)
        self.shift = torch.zeros(hidden, device=device)
        self.g_router, self.g_w1, self.g_w2 = (torch.zeros_like(w) for w in
                                               (self.router, self.w1, self.w2))
        # every matrix of the block in one grouped Muon step
        pairs = [(self.router, self.g_router), *zip(self.w1, self.g_w1), *zip(self.w2, self.g_w2)]
        self.muon = ns.Muon([(w, grad, torch.zeros(w.shape, device=device)) for w, grad in pairs])

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        y, rstd, saved = ns.layer_norm_checkpoint(x, self.gain, self.shift)
        logits = y @ self.router.t()
        r = ns.route(logits, self.k)
        # rows by expert: the token of each, in the order of the offsets
        order = torch.argsort(r.indices.flatten(), stable=True)
        token = order // self.k
        ends = r.offsets.tolist()
        spans = list(zip(ends, ends[1:]))
        rows = y[token]
        inner = torch.cat([rows[a:b] @ w.t() for (a, b), w in zip(spans, self.w1)]).relu()
        result = torch.cat([inner[a:b] @ w.t() for (a, b), w in zip(spans, self.w2)])
        w = r.weights.flatten()[order][:, None]
        out = x.float().index_add(0, token, result.float() * w)
        self.kept = (rstd, saved, logits, r, order, token, spans, ns.checkpoint8(inner), inner > 0,
                     result, w)
        return out

    def backward(self, dout: torch.Tensor) -> torch.Tensor:
        """Fills the gradients of every matrix; returns that of x."""
        rstd, saved, logits, r, order, token, spans, inner8, active, result, w = self.kept
        rows = dout[token]
        dweights = torch.empty_like(r.weights)
        dweights.view(-1)[order] = (rows * result.float()).sum(-1)
        dresult = (rows * w).bfloat16()
        ns.weight_grad(dresult, inner8, offsets=r.offsets, out=self.g_w2)
        dinner = torch.cat([dresult[a:b] @ m for (a, b), m in zip(spans, self.w2)]) * active
        rows8 = ns.Checkpoint8(saved.q[token], saved.e[token], saved.cols)
        ns.weight_grad(dinner, rows8, weight=self.gain, bias=self.shift, offsets=r.offsets,
                       out=self.g_w1)
        drows = torch.cat([dinner[a:b] @ m for (a, b), m in zip(spans, self.w1)])
        dy = torch.zeros_like(dout).index_add_(0, token, drows.float())
        dlogits = ns.route_backward(logits, r, dloss=torch.ones((), device=dout.device),
                                    dweights=dweights)
        ns.weight_grad(dlogits, saved, weight=self.gain, bias=self.shift, out=self.g_router)
        dy = (dy + dlogits.float() @ self.router.float()).bfloat16()
        dx, self.d_gain, self.d_shift = ns.layer_norm_backward(dy, saved, None, rstd, self.gain,
                                                               self.shift)
        return dx.float() + dout

    def step(self, lr: float) -> None:
        self.muon.step(lr=lr, beta=0.9)
        self.gain -= lr * self.d_gain
        self.shift -= lr * self.d_shift


def train(steps: int = 30, tokens: int = 2048, hidden: int = 256, inner: int = 128, experts: int = 16,
          k: int = 2, lr: float = 0.02, device="cuda"):
    """Fits the block to a fixed random map; the loss of every step."""
    g = torch.Generator(device=device).manual_seed(1)
    block = Block(hidden, inner, experts, k, device)
    target = torch.randn(hidden, hidden, generator=g, device=device) * hidden ** -0.5
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, hidden, generator=g, device=device).bfloat16()
        out = block.forward(x)
        diff = out - (x.float() + torch.relu(x.float() @ target))
        balance = block.kept[3].loss
        losses.append((diff.square().mean() + balance).item())
        block.backward(diff * (2.0 / diff.numel()))
        block.step(lr)
    block.muon.sync()
    ns.ops_sync()
    block.muon.close()
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=30)
    for i, loss in enumerate(train(ap.parse_args().steps)):
        print(f"step {i:3d}  loss {loss:.4f}")
