"""A tensor-parallel gated MLP block's training step on the 8-bit operators, emulated on one GPU.

    h = x + sum over ranks of down_r(silu(gate_r(norm(x))) * up_r(norm(x)))

Each rank holds a slice of the inner width.  What is kept for the backward pass
is in 8 bits: the norm's quantised output, the gated unit's output and its
inputs.  The products run in FP8; the ranks' partial sums meet in the library's
compressed two-shot all-reduce, forward and backward, as they would between
GPUs.  Master weights and their gradients are fp32, activations bf16.

Usage: python examples/mlp_step.py [--tokens 4096] [--hidden 4096] [--inner 8192] [--ranks 2] [--steps 4]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_compression_tensor_taco_amd as taco  # noqa: E402

COMPRESSION_BLOCK = 64


class Linear:
    """An fp32 master weight [outputs, inputs], its 8-bit forms of this step, and its gradient."""

    def __init__(self, weight: torch.Tensor):
        self.weight = weight
        self.grad = torch.zeros_like(weight)
        self.quantize()

    def quantize(self) -> None:
        self.q, self.scale, self.qt, self.scale_t = taco.quantize_weight(self.weight.to(torch.bfloat16))

    def forward(self, q, scale):
        return taco.matmul_fp8(q, scale, self.q, self.scale)

    def backward(self, dy, dq, dscale, xq, xscale):
        """dx for the bf16 gradient dy and its quantised form; adds to grad, from the 8-bit input."""
        taco.wgrad_fp8(dy, xq, xscale, self.weight.shape[1], dw=self.grad, accumulate=True)
        return taco.matmul_fp8(dq, dscale, self.qt, self.scale_t)


class MlpBlock:
    def __init__(self, norm: torch.Tensor, gate_up: list[torch.Tensor], down: list[torch.Tensor], eps: float = 1e-5):
        """norm [hidden]; per rank gate_up [2 * inner / ranks, hidden] (gate rows, then up) and down [hidden, inner / ranks]."""
        self.norm, self.eps = norm, eps
        self.norm_grad = torch.zeros_like(norm)
        self.gate_up = [Linear(w) for w in gate_up]
        self.down = [Linear(w) for w in down]

    def _sum(self, parts):
        return parts[0] if len(parts) == 1 else taco.two_shot_allreduce(parts, COMPRESSION_BLOCK)

    def forward(self, x: torch.Tensor, residual: torch.Tensor):
        """x + residual is the block's input; returns (the MLP's output, that input z), to be added by the next norm."""
        z, rstd, q, scale = taco.rmsnorm_quantize(x, self.norm.to(torch.bfloat16), self.eps, residual=residual)
        self.kept = [z, rstd, q, scale]
        partial = []
        for up, down in zip(self.gate_up, self.down):
            hq, hs, cq, cs = taco.swiglu_quantize(up.forward(q, scale))
            self.kept.append((hq, hs, cq, cs))
            partial.append(down.forward(hq, hs))
        return self._sum(partial), z

    def backward(self, dy: torch.Tensor, dz: torch.Tensor) -> torch.Tensor:
        """dy, dz: gradients of the two outputs.  Returns the gradient of x (and of residual)."""
        z, rstd, q, scale, *ranks = self.kept
        dq, ds = taco.quantize_rows(dy)
        partial = []
        for up, down, (hq, hs, cq, cs) in zip(self.gate_up, self.down, ranks):
            dh = down.backward(dy, dq, ds, hq, hs)
            partial.append(up.backward(*taco.swiglu_backward(dh, cq, cs), q, scale))
        dx, dw = taco.rmsnorm_backward(self._sum(partial), z, rstd, self.norm.to(torch.bfloat16), dz=dz)
        self.norm_grad += dw
        return dx

    def step(self, rate: float) -> None:
        """Plain gradient descent on the master weights, then their 8-bit forms anew."""
        self.norm -= rate * self.norm_grad
        self.norm_grad.zero_()
        for layer in (*self.gate_up, *self.down):
            layer.weight -= rate * layer.grad
            layer.grad.zero_()
            layer.quantize()


def make_block(hidden: int, inner: int, ranks: int, seed: int = 0, device="cuda") -> MlpBlock:
    if inner % ranks:
        raise ValueError("the inner width must split evenly over the ranks")
    g = torch.Generator(device=device).manual_seed(seed)
    width = inner // ranks

    def weight(rows, cols, fan):
        return torch.randn(rows, cols, device=device, generator=g) * fan ** -0.5

    return MlpBlock(torch.ones(hidden, device=device), [weight(2 * width, hidden, hidden) for _ in range(ranks)],
                    [weight(hidden, width, inner) for _ in range(ranks)])


def main() -> None:
    a = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    a.add_argument("--tokens", type=int, default=4096)
    a.add_argument("--hidden", type=int, default=4096)
    a.add_argument("--inner", type=int, default=8192)
    a.add_argument("--ranks", type=int, default=2)
    a.add_argument("--steps", type=int, default=4)
    args = a.parse_args()
    block = make_block(args.hidden, args.inner, args.ranks)
    g = torch.Generator(device="cuda").manual_seed(1)

    def draw():
        return torch.randn(args.tokens, args.hidden, device="cuda", generator=g).to(torch.bfloat16)

    x, residual, target = draw(), draw(), draw()
    for k in range(args.steps):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        y, z = block.forward(x, residual)
        error = y.float() - target.float()
        block.backward((error * (2 / error.numel())).to(torch.bfloat16), torch.zeros_like(z))
        block.step(0.05 * args.hidden)
        end.record()
        torch.cuda.synchronize()
        print(f"step {k}: loss {float(error.square().mean()):.5f}, {begin.elapsed_time(end):.3f} ms", flush=True)


if __name__ == "__main__":
    main()
