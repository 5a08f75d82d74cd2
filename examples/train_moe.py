"""A block of SwiGLU experts trained by Muon, its gradients clipped by their global norm.

    p = softmax(x Wr^T);  each token goes to the k experts of largest p
    y = x + sum over its experts of p_e ((silu(gate) up) Wd_e^T),  [gate | up] = x Wgu_e^T

Tokens are put in their experts' order once; the products, the activation and the weight
gradients then work on ragged ranges of rows, and the weighted sum brings them back.  The
experts' activations are kept in 8 bits between the passes.  Weight gradients are summed in
fp32 over the micro-batches, clipped together with the router's, and go to the optimizer step
in bf16.  The router itself (one small product and its softmax) is torch's.

    python examples/train_moe.py [--tokens 4096] [--hidden 1024] [--ffn 704] [--experts 16] [--choices 4] [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matrix_orthogonalising_optimizer_muon_gb300 as muon  # noqa: E402


class MoEBlock:
    """Weights, buffers and the two passes of one block for a fixed number of tokens."""

    def __init__(self, tokens, hidden, ffn, experts, choices, fmt="int8", seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.tokens, self.hidden, self.ffn, self.experts, self.choices = tokens, hidden, ffn, experts, choices
        self.router = torch.randn((experts, hidden), generator=g, device="cuda") * 0.02
        # fp32 master weights, which Muon steps one by one, and their bf16 copies for the products
        shapes = ((experts, 2 * ffn, hidden), (experts, hidden, ffn))
        self.weights = [torch.randn(s, generator=g, device="cuda") * 0.02 for s in shapes]
        self.momentum = [torch.zeros_like(w) for w in self.weights]
        self.low = [w.bfloat16() for w in self.weights]
        self.sums = [torch.zeros_like(w) for w in self.weights]                  # fp32, over micro-batches
        self.grads = [torch.empty_like(w, dtype=torch.bfloat16) for w in self.weights]   # clipped, for the step
        self.drouter = torch.zeros_like(self.router)
        rows = tokens * choices

        def new(n, cols, dtype=torch.bfloat16):
            return torch.empty((n, cols), dtype=dtype, device="cuda")
        self.offsets = torch.empty(experts + 1, dtype=torch.int32, device="cuda")
        self.slots = new(tokens, choices, torch.int32)
        # rows behind the last expert are no expert's: zero, so that 8-bit copies of them are, too
        self.xs, self.gu, self.a, self.ys = (new(rows, c).zero_() for c in (hidden, 2 * ffn, ffn, hidden))
        self.dys, self.da, self.dgu, self.dxs = (new(rows, c).zero_() for c in (hidden, ffn, 2 * ffn, hidden))
        self.y, self.dx = new(tokens, hidden), new(tokens, hidden)
        self.dp = new(tokens, choices, torch.float32)
        # what lives from the forward to the backward pass, beside ys
        self.x8, (self.gate8, self.up8, self.a8) = muon.Act8.empty(rows, hidden, fmt), \
            (muon.Act8.empty(rows, ffn, fmt) for _ in range(3))
        self.norm = torch.zeros(1, device="cuda")
        self.grad_plan = muon.GradPlan()
        self.plan = muon.MuonPlan([(2 * ffn, hidden)] * experts + [(hidden, ffn)] * experts, "bf16")
        self.clip_in = muon.GradList(self.sums + [self.drouter])
        self.clip_out = muon.GradList(self.grads + [self.drouter])

    def forward(self, x):
        f, p = self.ffn, self.grad_plan
        self.probs = torch.softmax(x.float() @ self.router.t(), 1)
        self.ids = self.probs.topk(self.choices, 1).indices.to(torch.int32)
        self.weights_of = self.probs.gather(1, self.ids.long())
        muon.expert_order(self.ids, self.offsets, self.slots)
        muon.expert_dispatch(x, self.slots, self.xs)
        muon.act_pack(self.xs, self.x8)
        p.product(self.xs, self.low[0], self.gu, offsets=self.offsets)
        muon.swiglu_forward(self.gu[:, :f], self.gu[:, f:], self.a, saved_gate=self.gate8, saved_up=self.up8)
        p.product(self.a, self.low[1], self.ys, offsets=self.offsets)
        muon.expert_combine(self.ys, self.slots, self.y, weights=self.weights_of)
        self.x = x
        return x + self.y

    def backward(self, dy):
        """Adds to sums and drouter from dy (tokens, hidden) bf16; returns the gradient of x."""
        f, p = self.ffn, self.grad_plan
        muon.expert_combine_backward(dy, self.slots, self.weights_of, rows=self.ys, drows=self.dys, dweights=self.dp)
        p.dgrad(self.dys, self.low[1], self.da, offsets=self.offsets)
        muon.swiglu_backward(self.da, self.gate8, self.up8, self.dgu[:, :f], self.dgu[:, f:], saved_out=self.a8)
        p.wgrad(self.dys, self.a8, self.sums[1], offsets=self.offsets, accumulate=True)
        p.wgrad(self.dgu, self.x8, self.sums[0], offsets=self.offsets, accumulate=True)
        p.dgrad(self.dgu, self.low[0], self.dxs, offsets=self.offsets)
        muon.expert_combine(self.dxs, self.slots, self.dx)
        dp = torch.zeros_like(self.probs).scatter_(1, self.ids.long(), self.dp)
        dlogits = self.probs * (dp - (self.probs * dp).sum(1, keepdim=True))
        self.drouter += dlogits.t() @ self.x.float()
        return (self.dx.float() + dy.float() + dlogits @ self.router).bfloat16()

    def step(self, lr, wd=0.0, max_norm=1.0):
        p = self.grad_plan
        p.grad_norm(self.clip_in, self.norm)
        p.grad_clip(self.clip_in, self.norm, max_norm, out=self.clip_out)
        self.plan.step(*([t for w in ws for t in w] for ws in (self.weights, self.grads, self.momentum)), lr, wd)
        self.router -= lr * self.drouter
        for low, w, s in zip(self.low, self.weights, self.sums):
            low.copy_(w)
            s.zero_()
        self.drouter.zero_()

    def sync(self):
        self.grad_plan.sync()
        self.plan.sync()


def train(tokens=4096, hidden=1024, ffn=704, experts=16, choices=4, steps=20, lr=5e-3, micro=2):
    """Fits a fixed random block's outputs, `micro` micro-batches a step; returns losses, norms and the block."""
    g = torch.Generator(device="cuda").manual_seed(1)
    xs = [torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16() for _ in range(micro)]
    target = MoEBlock(tokens, hidden, ffn, experts, choices, seed=2)
    for w, low in zip(target.weights, target.low):
        low.copy_(w * 2)
    want = [target.forward(x).float() for x in xs]
    block, losses, norms = MoEBlock(tokens, hidden, ffn, experts, choices), [], []
    for _ in range(steps):
        total = 0.0
        for x, y in zip(xs, want):
            diff = block.forward(x).float() - y
            total = total + diff.square().mean() / micro
            block.backward((diff * (2 / (micro * diff.numel()))).bfloat16())
        block.step(lr)
        losses.append(total)
        norms.append(block.norm.clone())
    block.sync()
    return [float(v) for v in losses], [float(v) for v in norms], block


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("tokens", 4096), ("hidden", 1024), ("ffn", 704), ("experts", 16), ("choices", 4), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=default)
    ap.add_argument("--lr", type=float, default=5e-3)
    a = ap.parse_args()
    losses, norms, _ = train(a.tokens, a.hidden, a.ffn, a.experts, a.choices, a.steps, a.lr)
    for i, (v, n) in enumerate(zip(losses, norms)):
        print("step %3d  loss %.6f  gradient norm %.4f" % (i, v, n))


if __name__ == "__main__":
    main()
