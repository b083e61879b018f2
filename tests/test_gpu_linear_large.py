"""The 8-bit linear layer's operators past 2^32 elements (offsets that need 64 bits): a few rows of a large call
against the same rows in a call of their own, which tests/test_gpu_linear.py holds to the oracle."""
import pytest
import torch

import fp8_compression_tensor_taco_amd as taco

pytestmark = pytest.mark.gpu


def rows_of(total):
    return [0, 1, total // 2, total - 1] + [int(2 ** 32 * f) for f in (0.5, 1.0) if 2 ** 32 * f < total]


def fill(rows, cols, seed):
    """bf16 rows that differ, without a second large tensor."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(1024, cols, device="cuda", generator=g).to(torch.bfloat16)
    out = torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16)
    for i in range(0, rows, 1024):
        n = min(1024, rows - i)
        out[i:i + n] = x[:n].roll(i // 1024, 0)
    return out


def test_row_operators():
    rows, cols = 540000, 8192                         # 4.4e9 elements
    x = fill(rows, cols, 0)
    picks = torch.tensor([0, 1, 262143, 262144, 524287, 524288, rows - 1], device="cuda")     # 2^31 / cols, 2^32 / cols
    w = torch.ones(cols, device="cuda", dtype=torch.bfloat16)
    q, s = taco.quantize_rows(x)
    rq, rs = taco.quantize_rows(x[picks])
    assert torch.equal(q[picks], rq) and torch.equal(s[picks], rs)
    z, rstd, q, s = taco.rmsnorm_quantize(x, w, q=q, scale=s)
    _, rr, rq, rs = taco.rmsnorm_quantize(x[picks], w)
    assert torch.equal(q[picks], rq) and torch.equal(s[picks], rs) and torch.equal(rstd[picks], rr)
    del q, s
    dx, _ = taco.rmsnorm_backward(x, x, rstd, w)
    assert torch.equal(dx[picks], taco.rmsnorm_backward(x[picks], x[picks], rr, w)[0])
    del dx
    hq, hs, cq, cs = taco.swiglu_quantize(x)
    want = taco.swiglu_quantize(x[picks])
    assert all(torch.equal(a[picks], b) for a, b in zip((hq, hs, cq, cs), want))
    del hq, hs
    dh = x.view(-1)[:rows * cols // 2].view(rows, cols // 2)
    dgu, dq, ds = taco.swiglu_backward(dh, cq, cs)
    want = taco.swiglu_backward(dh[picks], cq[picks], cs[picks])
    assert all(torch.equal(a[picks], b) for a, b in zip((dgu, dq, ds), want))


def test_products():
    m, n, k = 70000, 65536, 256                       # y: 4.6e9 elements
    x, w = fill(m, k, 1), fill(n, k, 2)
    q, s = taco.quantize_rows(x)
    wq, ws, _, _ = taco.quantize_weight(w, transposed=False)
    y = taco.matmul_fp8(q, s, wq, ws)
    for at in (0, 32768, 65536, m - 300):             # 2^31 / n and 2^32 / n rows
        assert torch.equal(y[at:at + 300], taco.matmul_fp8(q[at:at + 300], s[at:at + 300], wq, ws))
    # y as dy [tokens, n]: its first rows past 2^32 elements alone, by zeros elsewhere
    y[:65536] = 0
    dw = taco.wgrad_fp8(y, q, s, k)
    alone = taco.wgrad_fp8(y[65536:], q[65536:], s[65536:], k)
    assert float((dw - alone).norm() / alone.norm()) < 1e-5
    # a gradient of more than 2^31 elements
    dy, xs = fill(64, 70000, 3), fill(64, 40000, 4)
    xq, xsc = taco.quantize_rows(xs)
    dw = taco.wgrad_fp8(dy, xq, xsc, 40000)
    for at in (0, 53687, 69900):                      # 2^31 / 40000
        part = taco.wgrad_fp8(dy[:, at:at + 64].contiguous(), xq, xsc, 40000)
        assert float((dw[at:at + 64] - part).abs().max()) <= 2e-5 * float(part.abs().max())
