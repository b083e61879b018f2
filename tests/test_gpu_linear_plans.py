"""The weight gradient's and the product's kernels at sizes that choose them: exact sums, bit for bit, and scale bytes
over their whole range.

256 x 256 tiles are taken from 7 or 8 steps of 64 tokens on (a last one begun counts) where dy's rows are 16-byte
aligned, from 9 on otherwise, and 128 x 128 or 64 x 64 tiles below; the workspace tells the first (the widened x) and
split runs of tokens."""
import pytest
import torch

import fp8_compression_tensor_taco_amd as taco
from test_gpu_linear_tiles import CODES, VALUES, operands

pytestmark = pytest.mark.gpu


def exact(t, n, k):
    dy, q, scale, x = operands(t, n, k)
    want = dy.float().t().contiguous() @ x
    whole = torch.full((n * k + 4096,), 7.0, device="cuda")
    dw = whole[2048:2048 + n * k].view(n, k)
    taco.wgrad_fp8(dy, q, scale, k, dw=dw)
    assert torch.equal(dw, want)
    taco.wgrad_fp8(dy, q, scale, k, dw=dw, accumulate=True)
    assert torch.equal(dw, 2 * want)
    assert (whole[:2048] == 7).all() and (whole[2048 + n * k:] == 7).all()


# 256 tiles of 256 x 256, from the fewest steps on: none, some, half a step and more of rows left over
@pytest.mark.parametrize("t,n,k", [(385, 65536, 250), (416, 65536, 250), (448, 65536, 250), (449, 4096, 4090)] +
                         [(t, 4096, 4090) for t in (460, 479, 480, 481, 511, 512, 577, 640, 1023)])
def test_wgrad_of_widened_rows(t, n, k):
    assert taco.wgrad_fp8_workspace_bytes(t, n, k) == 2 * (t // 64 * 64) * taco.fp8_cols(k)
    exact(t, n, k)


@pytest.mark.parametrize("t", [513, 544, 545, 575, 576, 577, 608, 639, 640, 1023])
def test_wgrad_of_odd_rows(t):
    exact(t, 4095, 4090)


# runs of tokens over workgroups: 128 x 128 tiles, 64 x 64, rows of dy shorter than eight columns
@pytest.mark.parametrize("t,n,k", [(8192, 1600, 1600), (8191, 1599, 1600), (8192, 200, 300), (8192, 7, 4096), (4097, 1, 500)])
def test_wgrad_of_split_tokens(t, n, k):
    need = taco.wgrad_fp8_workspace_bytes(t, n, k)
    assert need > 0 and need % (4 * n * k) == 0 and need // (4 * n * k) >= 2
    exact(t, n, k)


@pytest.mark.parametrize("t,n,k", [(1, 5, 300), (63, 7, 128), (130, 5, 300), (130, 3, 1)])
def test_wgrad_of_short_rows(t, n, k):
    exact(t, n, k)


# one code and one byte per row, so that every sum is a small multiple of a power of two
POWERS = torch.tensor([2.0 ** e for e in range(-254, 255)], dtype=torch.float64)
BYTES = torch.tensor([0, 1, 2, 31, 64, 100, 126, 127, 128, 150, 190, 230, 252, 253, 254])


@pytest.mark.parametrize("m,n,k", [(5, 2000, 256), (30, 2000, 300), (70, 2000, 300), (300, 512, 8192), (450, 3000, 300),
                                   (1900, 1980, 300), (2100, 2203, 300), (3700, 3901, 300)])
def test_product_of_every_scale_byte(m, n, k):
    """Scales from 2^-127 to 2^127 against each other, where every product (a multiple of 1/4, times the scales) and
    every sum (below 4 k of them) is a normal number."""
    gen = torch.Generator(device="cuda").manual_seed(m)
    wide, sc, blocks = taco.fp8_cols(k), taco.fp8_scale_cols(k), -(-n // 128)
    pa, pb = (torch.randint(0, 7, (r, wide), generator=gen, device="cuda") for r in (m, n))
    ba = BYTES.cuda()[torch.arange(m, device="cuda") % len(BYTES)]
    bb = BYTES.flip(0).cuda()[torch.arange(blocks, device="cuda") % len(BYTES)]
    y = taco.matmul_fp8(CODES.cuda()[pa], ba.to(torch.uint8)[:, None].expand(m, sc).contiguous(),
                        CODES.cuda()[pb], bb.to(torch.uint8)[:, None].expand(blocks, sc).contiguous())
    sums = VALUES.cuda()[pa] @ VALUES.cuda()[pb].t().contiguous()
    power = (ba[:, None] - 127) + (bb - 127).repeat_interleave(128)[None, :n]
    normal = (power >= -124) & (power <= 110)
    assert normal.float().mean() > 0.3
    want = sums.to(torch.bfloat16).double() * POWERS.cuda()[power + 254]      # sums are exact: multiples of 1/4 below 2^16
    assert torch.equal(y.double()[normal], want[normal])


@pytest.mark.parametrize("t,n,k", [(140, 140, 300), (640, 4096, 4090), (640, 4095, 4090)])
def test_weight_gradient_of_every_scale_byte(t, n, k):
    """Row t of x meets column t of dy alone: products of one bf16 value and one power of two, both normal."""
    gen = torch.Generator(device="cuda").manual_seed(t)
    pick = torch.randint(0, 7, (t, taco.fp8_cols(k)), generator=gen, device="cuda")
    byte = 1 + torch.arange(t, device="cuda") % 253                     # 2^-126 .. 2^126, times at most 2
    scale = byte.to(torch.uint8)[:, None].expand(t, taco.fp8_scale_cols(k)).contiguous()
    dy = torch.zeros(t, n, dtype=torch.bfloat16, device="cuda")
    rows = torch.arange(min(t, n), device="cuda")
    dy[rows, rows] = torch.ldexp(torch.ones(len(rows), device="cuda"), 127 - byte[:len(rows)]).to(torch.bfloat16)
    dw = taco.wgrad_fp8(dy, CODES.cuda()[pick], scale, k)
    want = torch.zeros(n, k, device="cuda")
    want[rows] = VALUES.cuda()[pick][:len(rows), :k]
    assert torch.equal(dw, want)
