"""The weight gradient's largest tiles: exact sums over every start and end of their pipeline."""
import numpy as np
import pytest
import torch

import fp8_compression_tensor_taco_amd as taco

pytestmark = pytest.mark.gpu

CODES = torch.tensor([0x00, 0x38, 0x3C, 0x40, 0xB8, 0xBC, 0xC0], dtype=torch.uint8)        # 0, +-1, +-1.5, +-2
VALUES = torch.tensor([0.0, 1.0, 1.5, 2.0, -1.0, -1.5, -2.0])


def operands(t, n, k):
    """dy, the block format of x, and x in fp32: products are multiples of 1/4 and every sum is exact in fp32."""
    gen = torch.Generator(device="cuda").manual_seed(t + n)
    pick = torch.randint(0, 7, (t, taco.fp8_cols(k)), generator=gen, device="cuda")
    scale = torch.randint(127, 129, (t, taco.fp8_scale_cols(k)), generator=gen, device="cuda").to(torch.uint8)
    x = VALUES.cuda()[pick] * torch.exp2(scale.float() - 127).repeat_interleave(128, 1)[:, :pick.shape[1]]
    dy = VALUES.cuda()[torch.randint(0, 7, (t, n), generator=gen, device="cuda")].to(torch.bfloat16)
    return dy, CODES.cuda()[pick], scale, x[:, :k].contiguous()


# 16-byte aligned rows of dy and others; fewer rows than a step, one step, and rows left over
@pytest.mark.parametrize("n,k", [(16000, 16100), (15999, 16100)])
@pytest.mark.parametrize("t", [1, 40, 63, 64, 65, 100, 128, 192, 230, 256, 453, 512, 575, 640, 705, 768, 961])
def test_wgrad_exact_sums(t, n, k):
    dy, q, scale, x = operands(t, n, k)
    want = dy.float().t().contiguous() @ x
    whole = torch.full((n * k + 4096,), 7.0, device="cuda")
    dw = whole[2048:2048 + n * k].view(n, k)
    taco.wgrad_fp8(dy, q, scale, k, dw=dw)
    assert torch.equal(dw, want)
    taco.wgrad_fp8(dy, q, scale, k, dw=dw, accumulate=True)
    assert torch.equal(dw, 2 * want)
    assert (whole[:2048] == 7).all() and (whole[2048 + n * k:] == 7).all()


@pytest.mark.parametrize("t,row", [(100, 99), (100, 5), (128, 127), (30, 29), (800, 799), (800, 5)])
@pytest.mark.parametrize("n,k", [(16000, 16100), (15999, 16100)])
def test_wgrad_non_finite_stays_in_its_line(t, row, n, k):
    dy, q, scale, x = operands(t, n, k)
    clean = taco.wgrad_fp8(dy, q, scale, k)
    dy[row, 3] = float("inf")
    x = x[row]
    dw = taco.wgrad_fp8(dy, q, scale, k)
    assert torch.isnan(dw[3][x == 0]).all() and (dw[3][x != 0] == torch.sign(x[x != 0]) * float("inf")).all()
    keep = torch.arange(n, device="cuda") != 3
    assert torch.equal(dw[keep], clean[keep])
    dy[row, 3] = 0.0
    q[row, 256:384], scale[row, 2] = 0x7F, 255
    nan = torch.isnan(taco.wgrad_fp8(dy, q, scale, k))
    assert nan[:, 256:384].all() and not nan[:, :256].any() and not nan[:, 384:].any()
