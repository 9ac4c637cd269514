"""Training a small residual network whose activations are kept in 8 bits,
with Muon on its matrices.

    python examples/train_block8.py [--steps 40] [--hidden 512] [--ffn 2048]

A block is  h = x + r,  out = W2 relu(W1 norm(h))^2.  What a block keeps from
its forward for its backward pass is 8 bits per value: the norm's output, the
norm's input h and the activation between the matrices (relu(u) is its square
root, so u itself is not kept).  The 8-bit rows that feed a product are the
checkpoint its weight gradient reads.  Data and target are synthetic: a fixed
random linear map of the input.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from matrix_aware_optimizer_muon_amd import linear8 as l8  # noqa: E402
from matrix_aware_optimizer_muon_amd.optim import MuonMI355X  # noqa: E402


class Block:
    def __init__(self, hidden: int, ffn: int, gen: torch.Generator):
        def matrix(n, k):
            return torch.randn(n, k, generator=gen, device="cuda") / k ** 0.5

        self.norm = torch.ones(hidden, device="cuda")
        self.w1, self.w2 = matrix(ffn, hidden), matrix(hidden, ffn)

    def pack(self):
        """The 8-bit form of the weights, once per optimizer step."""
        self.w1q, self.w2q = l8.quantize(self.w1), l8.quantize(self.w2)

    def forward(self, x: torch.Tensor, residual: torch.Tensor):
        """(out, h), keeping y8, h8, a8 and rstd."""
        self.y8, h, self.rstd = l8.rmsnorm(x, self.norm, residual=residual, q8=True)
        u = l8.matmul(self.y8, self.w1q)
        self.a8 = l8.quantize(torch.relu(u).square_())
        self.h8 = l8.quantize(h)
        return l8.matmul(self.a8, self.w2q), h

    def backward(self, dout: torch.Tensor, dh: torch.Tensor):
        """The gradient of x (and of the residual); sets dw1, dw2, dnorm."""
        da = l8.grad_input(dout, self.w2q)
        self.dw2 = l8.grad_weight(dout, self.a8)
        du = da * (2.0 * l8.dequantize(self.a8).sqrt())
        dy = l8.grad_input(du, self.w1q)
        self.dw1 = l8.grad_weight(du, self.y8)
        dx, self.dnorm = l8.rmsnorm_backward(dy, self.h8, self.rstd, self.norm, dh=dh)
        return dx


class Net:
    def __init__(self, hidden: int, ffn: int, blocks: int, seed: int = 0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.blocks = [Block(hidden, ffn, gen) for _ in range(blocks)]
        self.matrices = [w for b in self.blocks for w in (b.w1, b.w2)]

    def loss_and_gradients(self, x: torch.Tensor, target: torch.Tensor) -> torch.Tensor:
        """Mean squared error of the stream after the last block; every
        block's gradients are set."""
        for b in self.blocks:
            b.pack()
        out, h = torch.zeros_like(x), x
        for b in self.blocks:
            out, h = b.forward(out, h)
        diff = h.float() + out.float() - target
        grad = (diff * (2.0 / diff.numel())).to(torch.bfloat16)
        dout = dh = grad
        for b in reversed(self.blocks):
            dout = dh = b.backward(dout, dh)
        return diff.square().mean()


def train(steps: int = 40, tokens: int = 1024, hidden: int = 512, ffn: int = 2048, blocks: int = 2,
          lr: float = 0.02, refresh_period: int = 0, log=None):
    """The losses, one per step."""
    net = Net(hidden, ffn, blocks)
    opt = MuonMI355X(net.matrices, grad_dtype="f32", ns_dtype="bf16", refresh_period=refresh_period)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x = torch.randn(tokens, hidden, generator=gen, device="cuda")
    target = x + x @ (torch.randn(hidden, hidden, generator=gen, device="cuda") / hidden ** 0.5)
    x = x.to(torch.bfloat16)
    losses = []
    for i in range(steps):
        loss = net.loss_and_gradients(x, target)
        opt.step([g for b in net.blocks for g in (b.dw1, b.dw2)], lr * (1 - i / steps), 0.0)
        for b in net.blocks:
            b.norm -= lr * b.dnorm
        losses.append(loss)
        if log:
            log(f"step {i:3d}  loss {float(loss):.5f}")
    return [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("steps", 40), ("tokens", 1024), ("hidden", 512), ("ffn", 2048), ("blocks", 2),
                        ("refresh-period", 0)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    began = time.perf_counter()
    losses = train(a.steps, a.tokens, a.hidden, a.ffn, a.blocks, refresh_period=a.refresh_period,
                   log=lambda s: print(s, flush=True))
    print(f"loss {losses[0]:.5f} -> {losses[-1]:.5f} in {time.perf_counter() - began:.2f} s")


if __name__ == "__main__":
    main()
