"""How the 8-bit linear layer's operators are called: what they return, and the layouts they take."""
import pytest
import torch

import fp8_compression_tensor_taco_amd as taco

pytestmark = pytest.mark.gpu


def test_norm_without_a_residual_returns_x_itself():
    wide = torch.randn(9, 512, device="cuda").to(torch.bfloat16)
    weight = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    flat = torch.randn(4 * 256 + 1, device="cuda").to(torch.bfloat16)
    for x in (wide[:, :256].contiguous(), wide[:, 128:384], wide[:, ::2], flat[1:].view(4, 256)):
        z, rstd, q, scale = taco.rmsnorm_quantize(x, weight)
        assert z is x
        for a, b in zip((rstd, q, scale), taco.rmsnorm_quantize(x.contiguous().clone(), weight)[1:]):
            assert torch.equal(a, b)
