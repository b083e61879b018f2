"""Scale byte 255 and codes 0x7F and 0xFF read as NaN in every call that takes the block format, whatever stands beside
them: also over codes of zero, and against operands of zero."""
import pytest
import torch

import fp8_compression_tensor_taco_amd as taco

pytestmark = pytest.mark.gpu


def block(rows, cols, seed, code=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(0x20, 0x60, (rows, taco.fp8_cols(cols)), device="cuda", generator=gen, dtype=torch.uint8)
    if code is not None:
        q.fill_(code)
    return q, torch.full((rows, taco.fp8_scale_cols(cols)), 127, dtype=torch.uint8, device="cuda")


# each kernel of the product: few rows, split, 64 x 64, 128 x 128 (two and one group of wavefronts), 256 x 256
PRODUCTS = [(3, 300, 512), (30, 300, 512), (300, 512, 8192), (70, 300, 512), (450, 3000, 512), (1900, 1980, 512),
            (2100, 2203, 512), (3700, 3901, 512)]


@pytest.mark.parametrize("codes", [0x00, 0x38])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(m, n, k, codes):
    (qa, sa), (qb, _) = block(m, k, 0, codes), block(n, k, 1, codes)
    sb = torch.full((-(-n // 128), taco.fp8_scale_cols(k)), 127, dtype=torch.uint8, device="cuda")
    sa[1, 2] = 255
    nan = torch.isnan(taco.matmul_fp8(qa, sa, qb, sb))
    assert nan[1].all() and not nan[0].any() and not nan[2:].any()
    sa[1, 2] = 127
    sb[1, 3] = 255
    nan = torch.isnan(taco.matmul_fp8(qa, sa, qb, sb))
    assert nan[:, 128:256].all() and not nan[:, :128].any() and not nan[:, 256:].any()
    sb[1, 3] = 127
    for code in (0x7F, 0xFF):
        qa[2, 300] = code
        nan = torch.isnan(taco.matmul_fp8(qa, sa, qb, sb))
        assert nan[2].all() and not nan[:2].any() and not nan[3:].any()


# 64 x 64 tiles, 128 x 128, split tokens, short rows of dy, both 256 x 256 kernels and their rows left over
GRADIENTS = [(70, 100, 300, 5), (1021, 1601, 1600, 3), (8192, 200, 300, 4000), (700, 5, 300, 600), (700, 4096, 4090, 5),
             (700, 4096, 4090, 699), (700, 4095, 4090, 5), (700, 4095, 4090, 699)]


@pytest.mark.parametrize("codes", [0x00, 0x38])
@pytest.mark.parametrize("gradient", [0.0, 1.0])
@pytest.mark.parametrize("t,n,k,row", GRADIENTS)
def test_weight_gradient(t, n, k, row, codes, gradient):
    q, s = block(t, k, 2, codes)
    dy = torch.full((t, n), gradient, device="cuda").to(torch.bfloat16)
    s[row, 1] = 255
    nan = torch.isnan(taco.wgrad_fp8(dy, q, s, k))
    assert nan[:, 128:256].all() and not nan[:, :128].any() and not nan[:, 256:].any()
    s[row, 1] = 127
    for code in (0x7F, 0xFF):
        q[row, 2] = code
        nan = torch.isnan(taco.wgrad_fp8(dy, q, s, k))
        assert nan[:, 2].all() and not nan[:, :2].any() and not nan[:, 3:].any()


@pytest.mark.parametrize("inner", [256, 300])
@pytest.mark.parametrize("codes", [0x00, 0x38])
def test_gate_gradient(inner, codes):
    wide = taco.fp8_cols(inner)
    cq, cs = block(4, 2 * wide, 3, codes)
    dh = torch.ones(4, inner, device="cuda").to(torch.bfloat16)
    for part, byte in (("gate", 1), ("up", wide // 128 + 1)):
        cs[2, byte] = 255
        dgu, dq, ds = taco.swiglu_backward(dh, cq, cs)
        cs[2, byte] = 127
        nan = torch.isnan(dgu)
        assert not nan[[0, 1, 3]].any()
        assert nan[2, 128:256].all() and not nan[2, :128].any() and not nan[2, 256:inner].any()      # dg holds both
        if part == "gate":                                                                             # du only the gate
            assert nan[2, inner + 128:inner + 256].all()
            assert not nan[2, inner:inner + 128].any() and not nan[2, inner + 256:].any()
        else:
            assert not nan[2, inner:].any()
        held = ds[2, :taco.fp8_cols(2 * inner) // 128] == 255
        blocks = torch.zeros(taco.fp8_cols(2 * inner), dtype=torch.bool, device="cuda")
        blocks[:2 * inner] = nan[2]
        assert torch.equal(held, blocks.view(-1, 128).any(1))
        assert (dq[2].view(-1, 128)[held] == 0x7F).all()
