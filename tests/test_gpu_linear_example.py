"""examples/mlp_step.py on the GPU: its forward and backward pass against the same block in fp32.

Every product's operands are rounded to E4M3 (relative error at most 2^-4 and about 0.026 in the mean square), so a
result three or four products deep is off by a few times that in the mean: 0.15 of its norm bounds it, and a wrong
transpose, scale or term would be off by its whole norm."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("mlp_step", os.path.join(ROOT, "examples", "mlp_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def off(got, want):
    return float((got.float().cpu() - want.float().cpu()).norm() / want.float().cpu().norm())


def plain(z, norm, ups, downs, eps):
    n = z * torch.rsqrt(z.square().mean(1, keepdim=True) + eps) * norm
    total = 0
    for up, down in zip(ups, downs):
        g, u = (n @ up.t()).chunk(2, 1)
        total = total + (torch.nn.functional.silu(g) * u) @ down.t()
    return total


@pytest.mark.parametrize("tokens,hidden,inner,ranks", [(96, 320, 512, 2), (64, 256, 300, 1), (256, 1024, 1536, 4)])
def test_block_against_fp32(tokens, hidden, inner, ranks):
    mlp = example()
    block = mlp.make_block(hidden, inner, ranks)
    x, r, dy, dz = (torch.randn(tokens, hidden, device="cuda").to(torch.bfloat16) for _ in range(4))
    y, z = block.forward(x, r)
    dx = block.backward(dy, dz)

    leaves = [x.float().cpu().requires_grad_(), block.norm.cpu().requires_grad_()]
    ups = [l.weight.cpu().requires_grad_() for l in block.gate_up]
    downs = [l.weight.cpu().requires_grad_() for l in block.down]
    zz = leaves[0] + r.float().cpu()
    want = plain(zz, leaves[1], ups, downs, block.eps)
    ((want * dy.float().cpu()).sum() + (zz * dz.float().cpu()).sum()).backward()
    assert off(z, zz) < 2 ** -8 and off(y, want) < 0.15 and off(dx, leaves[0].grad) < 0.15
    assert off(block.norm_grad, leaves[1].grad) < 0.15
    for layer, w in zip((*block.gate_up, *block.down), (*ups, *downs)):
        assert off(layer.grad, w.grad) < 0.15


def test_training_follows_fp32():
    """Eight steps of gradient descent beside the same in fp32: the losses stay within a fifth of each other (the
    gradients are within 0.15 of their norm, see above) and fall."""
    mlp = example()
    block = mlp.make_block(256, 512, 2)
    x, r, target = (torch.randn(128, 256, device="cuda").to(torch.bfloat16) for _ in range(3))
    leaves = [block.norm.cpu(), *(l.weight.cpu().clone() for l in (*block.gate_up, *block.down))]
    rate, losses, plain_losses = 0.05 * 256, [], []
    for _ in range(8):
        y, z = block.forward(x, r)
        error = y.float() - target.float()
        losses.append(float(error.square().mean()))
        block.backward((error * (2 / error.numel())).to(torch.bfloat16), torch.zeros_like(z))
        block.step(rate)
        leaves = [w.detach().requires_grad_() for w in leaves]
        out = plain(x.float().cpu() + r.float().cpu(), leaves[0], leaves[1:3], leaves[3:], block.eps)
        loss = (out - target.float().cpu()).square().mean()
        loss.backward()
        plain_losses.append(loss.item())
        leaves = [w.detach() - rate * w.grad for w in leaves]
    assert all(abs(a - b) <= 0.2 * b for a, b in zip(losses, plain_losses)), (losses, plain_losses)
    assert losses[-1] < 0.5 * losses[0]
