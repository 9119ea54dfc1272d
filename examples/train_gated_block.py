"""Trains one small transformer block with libmuon's operators and Muon.

    python examples/train_gated_block.py [--steps N]

    x1 = x + dropout(attention(norm(x)) Wo^T)
    out = x1 + dropout(sum over the k experts taken of w_e ffn_e(norm(x1)))

with rotary positions on queries and keys, fewer key than query heads, and gated
experts ffn_e(y) = (silu(y Wg_e^T) * (y Wu_e^T)) Wd_e^T.  No dropout mask is
kept: the backward pass makes it again from the step's number.  The norms'
rows are kept in 8 bits and serve the gradients of every matrix that reads
them.  The weight gradients are written into the tensors that Muon steps
with.  The projections and the attention's softmax are torch's.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import newton_schulz_06_gb300 as ns  # noqa: E402

MATRICES = ("wq", "wk", "wv", "wo", "router", "w_gate", "w_up", "w_down")


def attention(q, k, v):
    """Causal attention of tokens x heads x head, keys and values of fewer heads."""
    group = q.shape[1] // k.shape[1]
    k, v = (t.repeat_interleave(group, 1) for t in (k, v))
    s = torch.einsum("qhd,khd->hqk", q, k) * q.shape[-1] ** -0.5
    s = s.masked_fill(torch.ones(s.shape[1:], dtype=torch.bool, device=s.device).triu(1), float("-inf"))
    return torch.einsum("hqk,khd->qhd", torch.softmax(s, -1), v).flatten(1)


class Block:
    def __init__(self, hidden: int, heads: int, kv_heads: int, head: int, inner: int, experts: int, k: int,
                 p: float = 0.1, device="cuda", seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            return (torch.randn(shape, generator=g, device=device) * shape[-1] ** -0.5).bfloat16()

        self.k, self.p, self.seed, self.head = k, p, seed + 12345, head
        self.plan = ns.RotaryPlan(head)
        self.wq, self.wo = weight(heads * head, hidden), weight(hidden, heads * head)
        self.wk, self.wv = weight(kv_heads * head, hidden), weight(kv_heads * head, hidden)
        self.router = weight(experts, hidden)
        self.w_gate, self.w_up = weight(experts, inner, hidden), weight(experts, inner, hidden)
        self.w_down = weight(experts, hidden, inner)
        self.gain1, self.gain2 = (torch.ones(hidden, device=device) for _ in range(2))
        self.shift1, self.shift2 = (torch.zeros(hidden, device=device) for _ in range(2))
        self.grads = {n: torch.zeros_like(getattr(self, n)) for n in MATRICES}
        # every matrix of the block in one grouped Muon step
        pairs = []
        for n in MATRICES:
            w, grad = getattr(self, n), self.grads[n]
            pairs += [(w, grad)] if w.dim() == 2 else list(zip(w, grad))
        self.muon = ns.Muon([(w, grad, torch.zeros(w.shape, device=device)) for w, grad in pairs])

    def forward(self, x: torch.Tensor, step: int) -> torch.Tensor:
        y, rstd1, saved1 = ns.layer_norm_checkpoint(x, self.gain1, self.shift1)
        q, k, v = ((y @ w.t()).unflatten(-1, (-1, self.head)) for w in (self.wq, self.wk, self.wv))
        q, k = ns.rotary(q, k, self.plan, out_q=q, out_k=k)
        leaves = [t.float().requires_grad_() for t in (q, k, v)]
        with torch.enable_grad():
            attended = attention(*leaves)
        a = attended.detach().bfloat16()
        x1 = ns.dropout(a @ self.wo.t(), self.p, self.seed, 2 * step, residual=x)

        y, rstd2, saved2 = ns.layer_norm_checkpoint(x1, self.gain2, self.shift2)
        logits = y @ self.router.t()
        r = ns.route(logits, self.k)
        order = torch.argsort(r.indices.flatten(), stable=True)
        token = order // self.k
        f, gates = ns.gated_ffn(y[token], self.w_gate, self.w_up, self.w_down, offsets=r.offsets)
        w = r.weights.flatten()[order][:, None]
        mixed = torch.zeros(x.shape, device=x.device).index_add_(0, token, f.float() * w)
        out = ns.dropout(mixed.bfloat16(), self.p, self.seed, 2 * step + 1, residual=x1)
        self.kept = dict(step=step, rstd1=rstd1, saved1=saved1, leaves=leaves, attended=attended, a=a,
                         rstd2=rstd2, saved2=saved2, logits=logits, routing=r, order=order, token=token, f=f,
                         gates=gates, w=w)
        return out

    def backward(self, dout: torch.Tensor) -> torch.Tensor:
        """Fills the gradients of every matrix, gain and shift; returns that of x."""
        c, grads = self.kept, self.grads
        r, order, token = c["routing"], c["order"], c["token"]
        rows = ns.dropout_backward(dout, self.p, self.seed, 2 * c["step"] + 1)[token]
        dweights = torch.empty_like(r.weights)
        dweights.view(-1)[order] = (rows.float() * c["f"].float()).sum(-1)
        saved = c["saved2"]
        rows8 = ns.Checkpoint8(saved.q[token], saved.e[token], saved.cols)
        drows = ns.gated_ffn_backward((rows * c["w"]).bfloat16(), rows8, c["gates"], self.w_gate, self.w_up,
                                      self.w_down, offsets=r.offsets, weight=self.gain2, bias=self.shift2,
                                      grads=[grads[n] for n in ("w_gate", "w_up", "w_down")])[0]
        dlogits = ns.route_backward(c["logits"], r, dloss=torch.ones((), device=dout.device), dweights=dweights)
        ns.weight_grad(dlogits, saved, weight=self.gain2, bias=self.shift2, out=grads["router"])
        dy = (dlogits.float() @ self.router.float()).index_add_(0, token, drows.float())
        d, grads["gain2"], grads["shift2"] = ns.layer_norm_backward(dy.bfloat16(), saved, None, c["rstd2"],
                                                                    self.gain2, self.shift2)
        dx1 = d + dout

        do = ns.dropout_backward(dx1, self.p, self.seed, 2 * c["step"])
        ns.weight_grad(do, ns.checkpoint8(c["a"]), out=grads["wo"])
        dq, dk, dv = (t.bfloat16() for t in
                      torch.autograd.grad(c["attended"], c["leaves"], (do @ self.wo).float()))
        dq, dk = ns.rotary_backward(dq, dk, self.plan, out_q=dq, out_k=dk)
        dy = 0
        for n, d in (("wq", dq), ("wk", dk), ("wv", dv)):
            d = d.flatten(1)
            ns.weight_grad(d, c["saved1"], weight=self.gain1, bias=self.shift1, out=grads[n])
            dy = dy + (d @ getattr(self, n)).float()
        d, grads["gain1"], grads["shift1"] = ns.layer_norm_backward(dy.bfloat16(), c["saved1"], None, c["rstd1"],
                                                                    self.gain1, self.shift1)
        return d + dx1

    def step(self, lr: float) -> None:
        self.muon.step(lr=lr, beta=0.9)
        for n in ("gain1", "shift1", "gain2", "shift2"):
            getattr(self, n).sub_(lr * self.grads[n])


def train(steps: int = 30, tokens: int = 512, hidden: int = 256, inner: int = 128, experts: int = 16, k: int = 2,
          lr: float = 0.02, device="cuda"):
    """Fits the block to a fixed random map of the tokens' running mean; the
    loss of every step."""
    g = torch.Generator(device=device).manual_seed(1)
    block = Block(hidden, 4, 2, max(16, hidden // 4), inner, experts, k, device=device)
    target = torch.randn(hidden, hidden, generator=g, device=device) * hidden ** -0.5
    count = torch.arange(1, tokens + 1, device=device)[:, None]
    losses = []
    for i in range(steps):
        x = torch.randn(tokens, hidden, generator=g, device=device).bfloat16()
        out = block.forward(x, i)
        diff = out.float() - (x.float() + torch.tanh((x.float().cumsum(0) / count.sqrt()) @ target))
        losses.append((diff.square().mean() + block.kept["routing"].loss).item())
        block.backward((diff * (2.0 / diff.numel())).bfloat16())
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
