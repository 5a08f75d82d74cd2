"""A pre-norm SwiGLU FFN block trained by Muon, its activations held in 8 bits.

    h = x;  n = rmsnorm(h) g;  [gate | up] = n Wgu^T;  a = silu(gate) up;  y = h + a Wd^T

Between the forward and the backward pass the block keeps the unweighted norm, gate and up
in 8 bits and one fp32 per token, 3 bytes per FFN value instead of 6 (and one instead of
four per hidden value).  The weight gradients come from the 8-bit copies in the layout and
type that the optimizer step reads.  Dense products of bf16 tensors are torch's.

    python examples/train_ffn.py [--tokens 4096] [--hidden 1024] [--ffn 2816] [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matrix_orthogonalising_optimizer_muon_gb300 as muon  # noqa: E402

EPS = 1e-6


class FFNBlock:
    """Weights, buffers and the two passes of one block for a fixed number of tokens."""

    def __init__(self, tokens, hidden, ffn, fmt="int8", seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.tokens, self.hidden, self.ffn = tokens, hidden, ffn
        # fp32 master weights, which Muon steps, and their bf16 copies for the products
        self.weights = [torch.randn(s, generator=g, device="cuda") * 0.02 for s in ((2 * ffn, hidden), (hidden, ffn))]
        self.momentum = [torch.zeros_like(w) for w in self.weights]
        self.grads = [torch.empty_like(w, dtype=torch.bfloat16) for w in self.weights]
        self.gain, self.dgain = torch.ones(hidden, device="cuda"), torch.empty(hidden, device="cuda")
        self.low = [w.bfloat16() for w in self.weights]

        def new(cols):
            return torch.empty((tokens, cols), dtype=torch.bfloat16, device="cuda")
        self.n, self.gu, self.a = new(hidden), new(2 * ffn), new(ffn)
        self.dgu, self.dx = new(2 * ffn), new(hidden)
        self.rstd = torch.empty(tokens, device="cuda")
        # what lives from the forward to the backward pass
        self.norm8 = muon.Act8.empty(tokens, hidden, fmt)
        self.gate8, self.up8, self.a8 = (muon.Act8.empty(tokens, ffn, fmt) for _ in range(3))
        self.grad_plan = muon.GradPlan()
        self.plan = muon.MuonPlan([tuple(w.shape) for w in self.weights], "bf16")

    def forward(self, x):
        f = self.ffn
        muon.rmsnorm_forward(x, self.gain, EPS, y=self.n, saved=self.norm8, rstd=self.rstd)
        torch.matmul(self.n, self.low[0].t(), out=self.gu)
        muon.swiglu_forward(self.gu[:, :f], self.gu[:, f:], self.a, saved_gate=self.gate8, saved_up=self.up8)
        return torch.addmm(x, self.a, self.low[1].t())

    def backward(self, dy):
        """Fills grads and dgain from dy (tokens, hidden) bf16; returns the gradient of x."""
        f, p = self.ffn, self.grad_plan
        da = dy @ self.low[1]
        muon.swiglu_backward(da, self.gate8, self.up8, self.dgu[:, :f], self.dgu[:, f:], saved_out=self.a8)
        p.wgrad(dy, self.a8, self.grads[1])
        # the product read norm * gain: the gain goes onto the gradient's columns
        p.wgrad(self.dgu, self.norm8, self.grads[0], col_scale=self.gain)
        dn = self.dgu @ self.low[0]
        p.rmsnorm_backward(dn, self.gain, self.rstd, self.dx, self.dgain, saved=self.norm8, dres=dy)
        return self.dx

    def step(self, lr, wd=0.0):
        self.plan.step(self.weights, self.grads, self.momentum, lr, wd)
        self.gain -= lr * self.dgain
        for low, w in zip(self.low, self.weights):
            low.copy_(w)

    def sync(self):
        self.grad_plan.sync()
        self.plan.sync()

    def saved_bytes(self):
        return self.norm8.nbytes + self.gate8.nbytes + self.up8.nbytes + 4 * self.tokens


def train(tokens=4096, hidden=1024, ffn=2816, steps=20, lr=2e-2, fmt="int8"):
    """Fits a fixed random block's outputs; returns the losses (mean squared error per value)."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16()
    target = FFNBlock(tokens, hidden, ffn, fmt, seed=2)
    for w, low in zip(target.weights, target.low):
        low.copy_(w * 2)
    want = target.forward(x).float()
    block, losses = FFNBlock(tokens, hidden, ffn, fmt), []
    for _ in range(steps):
        diff = block.forward(x).float() - want
        losses.append(diff.square().mean())
        block.backward((diff * (2 / diff.numel())).bfloat16())
        block.step(lr)
    block.sync()
    return [float(v) for v in losses], block


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("tokens", 4096), ("hidden", 1024), ("ffn", 2816), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=default)
    ap.add_argument("--lr", type=float, default=2e-2)
    ap.add_argument("--fmt", choices=("int8", "e4m3"), default="int8")
    a = ap.parse_args()
    losses, block = train(a.tokens, a.hidden, a.ffn, a.steps, a.lr, a.fmt)
    full = a.tokens * (2 * a.hidden * 2 + 3 * a.ffn * 2)
    for i, v in enumerate(losses):
        print("step %3d  loss %.6f" % (i, v))
    print("kept between the passes: %.1f MB (bf16 h, norm, gate, up and their product: %.1f MB)"
          % (block.saved_bytes() / 1e6, full / 1e6))


if __name__ == "__main__":
    main()
