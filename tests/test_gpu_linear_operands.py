"""The FP8 product with an operand of more than 2^32 bytes of codes, as a and as b: every element, bit for bit, of
products whose sums are exact (0, +-1, +-1.5 and +-2 with scales 1 and 2: multiples of 1/4 below 2^22, exact in fp32)."""
import pytest
import torch

import fp8_compression_tensor_taco_amd as taco

pytestmark = pytest.mark.gpu

CODES = torch.tensor([0x00, 0x38, 0x3C, 0x40, 0xB8, 0xBC, 0xC0], dtype=torch.uint8)
VALUES = torch.tensor([0.0, 1.0, 1.5, 2.0, -1.0, -1.5, -2.0])


def operand(rows, k, scale_rows, gen, often=7):
    """Codes and scale bytes; `often` above 7 makes the others zeros, for sums over a long k."""
    q = torch.empty(rows, k, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // k)
    codes = torch.cat([CODES, CODES.new_zeros(often - 7)]).cuda()
    for i in range(0, rows, step):
        n = min(step, rows - i)
        q[i:i + n] = codes[torch.randint(0, often, (n, k), device="cuda", generator=gen, dtype=torch.int32)]
    scale = torch.randint(127, 129, (scale_rows, taco.fp8_scale_cols(k)), device="cuda", generator=gen)
    return q, scale.to(torch.uint8)


def values(q, scale):
    """fp32 values of rows of codes; scale has a row for each of them."""
    table = torch.zeros(256, device="cuda")
    table[CODES.cuda().long()] = VALUES.cuda()
    v = table[q.int()].view(q.shape[0], -1, 128)
    return (v * torch.exp2(scale[:, :v.shape[1], None].float() - 127)).view(q.shape)


def weight_values(q, scale):
    return values(q, scale.repeat_interleave(128, 0)[:q.shape[0]])


# 256 x 256 tiles; the first rows of the large operand are 2^32 bytes and a part of a tile from its end, and a tile
# further in: 1048700 * 4096, 1200000 * 3584
@pytest.mark.parametrize("rows,k", [(1048700, 4096), (1200000, 3584)])
@pytest.mark.parametrize("as_a", [True, False])
def test_large_operand(rows, k, as_a):
    gen = torch.Generator(device="cuda").manual_seed(k)
    few = 256
    m, n = (rows, few) if as_a else (few, rows)
    qa, sa = operand(m, k, m, gen)
    qb, sb = operand(n, k, -(-n // 128), gen)
    y = taco.matmul_fp8(qa, sa, qb, sb)
    step = 1 << 15
    if as_a:
        b = weight_values(qb, sb).t().contiguous()
        for i in range(0, rows, step):
            assert torch.equal(y[i:i + step], (values(qa[i:i + step], sa[i:i + step]) @ b).to(torch.bfloat16)), i
    else:
        a = values(qa, sa)
        for i in range(0, rows, step):
            b = weight_values(qb[i:i + step], sb[i // 128:(i + step) // 128]).t().contiguous()
            assert torch.equal(y[:, i:i + step], (a @ b).to(torch.bfloat16)), i


# the kernels for few rows and few tiles: 1030 rows of 2^22 columns
@pytest.mark.parametrize("m", [3, 40])
def test_long_rows(m):
    gen = torch.Generator(device="cuda").manual_seed(m)
    n, k = 1030, 1 << 22
    qa, sa = operand(m, k, m, gen, often=64)
    qb, sb = operand(n, k, -(-n // 128), gen, often=64)
    y = taco.matmul_fp8(qa, sa, qb, sb)
    want = torch.zeros(m, n, device="cuda")
    step = 1 << 15
    for i in range(0, k, step):
        blocks = slice(i // 128, (i + step) // 128)
        b = weight_values(qb[:, i:i + step], sb[:, blocks]).t().contiguous()
        want += values(qa[:, i:i + step], sa[:, blocks]) @ b
    assert torch.equal(y, want.to(torch.bfloat16))


# x of more than 2^32 codes in the weight gradient
def test_weight_gradient():
    gen = torch.Generator(device="cuda").manual_seed(1)
    t, n, k = 1048700, 72, 4096
    q, scale = operand(t, k, t, gen, often=64)
    dy = VALUES.cuda()[torch.randint(0, 7, (t, n), device="cuda", generator=gen)].to(torch.bfloat16)
    dw = taco.wgrad_fp8(dy, q, scale, k)
    want = torch.zeros(n, k, device="cuda")
    step = 1 << 15
    for i in range(0, t, step):
        want += dy[i:i + step].float().t().contiguous() @ values(q[i:i + step], scale[i:i + step])
    assert torch.equal(dw, want)
