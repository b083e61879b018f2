"""The product with a bias, a nonlinearity and a residual, its quantised form, and the nonlinearity's gradient, on the GPU
against oracle/linear.py (fp64).

Tolerances, from the arithmetic (u = 2^-24, one fp32 rounding):
* t = a b^T + bias: the product's error (see test_gpu_linear.py) and one rounding, E.
* act(t): no nonlinearity steepens by more than 1.13, so 1.13 E; and with w the exponential's argument, P or the sigmoid
  at -|t| is off by (4 w + 24) u of itself (the roundings of the argument and of its constants are each at most u w, and
  there are four; the exponential, the sum, the reciprocal and the polynomial are below 24 u), with two more roundings on
  the positive side.  Values under 2^-100 may flush.  gelu's own P is a polynomial's exponential, fitted to 1.52 times
  that with a factor 2^(|t| - 1) beyond |t| = 1 and evaluated to 1.65 times (over a grid of 3e6 values in fp32), the
  exponential besides: twice that.
* y: one more rounding for the residual, and half a step of bf16, 2^-8 |y|.
* act'(t): the same factor, times (1 + |t|) for the term that t multiplies and its derivative's factor, at most 2 + w.
* dbias: at most (rows + 64) roundings of the terms' sum of magnitudes, and the terms' own errors.
* Sums of operands 0, 1, 1.5 and 2 with scales 1 and 2 are exact, and so are quarters added to them: bit for bit.
"""
import numpy as np
import pytest
import torch

import fp8_compression_tensor_taco_amd as taco
import oracle
from oracle import linear as ol
from test_gpu_linear import U, activations, bf16, check_codes, f64, guarded, operands, survived

pytestmark = pytest.mark.gpu
ACTS = ol.ACTIVATIONS


def product_error(a, b):
    k = a.shape[1]
    eights = np.abs(a).reshape(-1, k // 8, 8).max(2) @ np.abs(b).reshape(-1, k // 8, 8).max(2).T
    return 7 * 2.0 ** -13 * eights + k / 8 * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)


def factor_error(t, name):
    """Of P or the sigmoid at -|t|, absolutely; and w."""
    if name in (None, "relu"):
        return np.zeros_like(t), np.zeros_like(t)
    if name == "gelu":
        w, tail = t * t / 2, ol._normal(-np.abs(t))
    else:
        w = np.abs(t if name == "silu" else ol._tanh_argument(t))
        tail = ol.sigmoid(-w)
    return (4 * w + 24) * U * tail, w


def act_error(t, err, name):
    factor = factor_error(t, name)[0]
    if name == "gelu":
        factor = 2 * factor * np.exp2(np.clip(np.abs(t) - 1, 0, 200))
    return 1.13 * err + np.abs(t) * (factor + (t > 0) * 2 * U) + 2.0 ** -100


def vectors(rng, m, n, with_bias=True, with_residual=True):
    return (bf16(0.3 * rng.standard_normal(n)) if with_bias else None,
            bf16(rng.standard_normal((m, n))) if with_residual else None)


def cuda(t):
    return None if t is None else t.cuda()


# For quantised outputs: 16 x 128 tiles (one and two rows of them), few rows and a second kernel (up to 8, 16 and 32 rows, one
# workgroup to a CU and two), k split, 32 x 128, 64 x 128, 128 x 128 with two groups of wavefronts and with one, 256 x 256.
# For the others: few rows, k split, 64 x 64 with two groups and with one, 128 x 128, 256 x 256; and 16 x 128 tiles.
KERNELS = [(3, 300, 512), (30, 300, 512), (5, 300, 2000), (12, 300, 2000), (25, 300, 2000), (300, 512, 8192), (70, 300, 512),
           (450, 3000, 512), (1900, 1980, 512), (2100, 2203, 512), (3700, 3901, 512), (7, 4200, 1700), (14, 4200, 1700),
           (29, 4200, 1700), (20, 12300, 300)]
SMALLER = [s for s in KERNELS if s[0] < 3000]
SHAPES = [(1, 1, 1), (1, 128, 128), (4, 256, 512), (3, 100, 1600), (16, 1601, 300), (17, 130, 2000), (33, 512, 4096),
          (65, 1000, 1000), (100, 257, 129), (257, 260, 1600), (777, 1601, 1600), (1, 3000, 14336), (20, 5, 8200)]


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("m,n,k", SHAPES + SMALLER)
def test_linear_fp8(m, n, k, name):
    rng = np.random.default_rng(m * n + k)
    (qa, sa), (qb, sb, _, _) = operands(rng, m, n, k)
    a, b = ol.row_values(qa.cpu().numpy(), sa.cpu().numpy()), ol.weight_values(qb.cpu().numpy(), sb.cpu().numpy())
    product, err = a @ b.T, product_error(a, b)
    for with_bias, with_residual in ((True, True), (False, True), (True, False), (False, False)):
        bias, residual = vectors(rng, m, n, with_bias, with_residual)
        y = taco.linear_fp8(qa, sa, qb, sb, bias=cuda(bias), activation=name, residual=cuda(residual))
        assert y.shape == (m, n) and y.dtype == torch.bfloat16
        t = product + (f64(bias) if with_bias else 0)
        want = ol.activation(t, name) + (f64(residual) if with_residual else 0)
        e = act_error(t, err + U * np.abs(t), name) + 2 * U * np.abs(want)
        assert (np.abs(f64(y) - want) <= 2.0 ** -8 * np.abs(want) + 1.01 * e).all()
        assert torch.equal(y, taco.linear_fp8(qa, sa, qb, sb, bias=cuda(bias), activation=name, residual=cuda(residual)))
    assert name or torch.equal(y, taco.matmul_fp8(qa, sa, qb, sb))


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("m,n,k", SHAPES + SMALLER)
def test_linear_quantize(m, n, k, name):
    rng = np.random.default_rng(m + n * k)
    (qa, sa), (qb, sb, _, _) = operands(rng, m, n, k)
    a, b = ol.row_values(qa.cpu().numpy(), sa.cpu().numpy()), ol.weight_values(qb.cpu().numpy(), sb.cpu().numpy())
    for with_bias in (True, False):
        bias, _ = vectors(rng, m, n, with_bias, False)
        hq, hs, cq, cs = taco.linear_quantize(qa, sa, qb, sb, bias=cuda(bias), activation=name)
        t, h = ol.linear(a, b, f64(bias) if with_bias else None, name)
        err = product_error(a, b) + U * np.abs(t)
        check_codes(hq, hs, h, 1.01 * act_error(t, err, name))
        if name is None:
            assert cq is None and cs is None
        else:
            check_codes(cq, cs, t, 1.01 * err)
        again = taco.linear_quantize(qa, sa, qb, sb, bias=cuda(bias), activation=name, checkpoint=False)
        assert again[2] is None and again[3] is None and torch.equal(again[0], hq) and torch.equal(again[1], hs)


def exact_operands(rng, m, n, k):
    wide, sc = ol.padded(k), ol.scale_cols(k)
    values = np.array([0x00, 0x38, 0x3C, 0x40, 0xB8, 0xBC, 0xC0], np.uint8)          # 0, +-1, +-1.5, +-2
    qa, qb = (values[rng.integers(0, 7, (r, wide))] for r in (m, n))
    sa, sb = rng.integers(127, 129, (m, sc)).astype(np.uint8), rng.integers(127, 129, (-(-n // 128), sc)).astype(np.uint8)
    product = torch.from_numpy(ol.row_values(qa, sa)).float() @ torch.from_numpy(ol.weight_values(qb, sb)).float().t()
    return [torch.from_numpy(t).cuda() for t in (qa, sa, qb, sb)], product            # exact: quarters below 2^18


# every kernel, and every start and end of their pipelines
@pytest.mark.parametrize("m,n,k", KERNELS + [(m, n, k) for m, n in ((40, 130), (450, 3000), (1900, 1980), (2100, 2203), (3700, 3901))
                                               for k in (100, 256, 300, 1100)])
def test_exact_sums(m, n, k):
    rng = np.random.default_rng(m + k)
    given, product = exact_operands(rng, m, n, k)
    bias = torch.from_numpy(rng.integers(-64, 65, n) / 4).to(torch.bfloat16)
    residual = torch.from_numpy(rng.integers(-64, 65, (m, n)) / 4).to(torch.bfloat16)
    t = product + bias.float()
    whole, out = guarded((m, n), torch.bfloat16)
    assert torch.equal(taco.matmul_fp8(*given, out=out).cpu(), product.to(torch.bfloat16)) and survived(whole)
    for name, h in ((None, t), ("relu", t.clamp(min=0))):
        whole, out = guarded((m, n), torch.bfloat16)
        y = taco.linear_fp8(*given, bias=bias.cuda(), activation=name, residual=residual.cuda(), out=out)
        assert torch.equal(y.cpu(), (h + residual.float()).to(torch.bfloat16)) and survived(whole)
        held = [guarded((m, c), torch.uint8) for c in (taco.fp8_cols(n), taco.fp8_scale_cols(n)) * 2]
        outs = dict(zip(("hq", "hs", "cq", "cs") if name else ("hq", "hs"), (v for _, v in held)))
        got = taco.linear_quantize(*given, bias=bias.cuda(), activation=name, **outs)
        for x, (q, s) in ((h, got[:2]), (t, got[2:]))[:2 if name else 1]:
            # a value times a power of two has at most 24 bits: the conversion is the only rounding on either side
            want_q, want_s = ol.quantize_rows(x.double().numpy())
            assert (s.cpu().numpy() == want_s).all() and (q.cpu().numpy() == want_q).all()
        assert all(survived(w) for w, _ in held)


def every_bf16():
    return torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("m", [2, 40, 200])
def test_every_value_of_t(m, name):
    """Rows of zeros: t is the bias, here every bf16 value, NaN and the infinities among them."""
    bias = every_bf16()
    n = bias.numel()
    qa, sa = torch.zeros(m, 128, dtype=torch.uint8).cuda(), torch.full((m, 4), 127, dtype=torch.uint8).cuda()
    qb, sb = torch.full((n, 128), 0x38, dtype=torch.uint8).cuda(), torch.full((n // 128, 4), 127, dtype=torch.uint8).cuda()
    y = taco.linear_fp8(qa, sa, qb, sb, bias=bias.cuda(), activation=name)
    assert (y.view(torch.int16) == y[:1].view(torch.int16)).all()
    got, t = f64(y[0]), f64(bias)
    want = ol.activation(t, name)
    fine = np.isfinite(want)
    assert (np.isnan(got) == np.isnan(t)).all() and (got[np.isinf(want)] == want[np.isinf(want)]).all()
    top = float(torch.finfo(torch.bfloat16).max)
    with np.errstate(over="ignore", invalid="ignore"):
        e = act_error(np.where(np.isfinite(t), t, 0), 0.0, name) + 2.0 ** -8 * np.abs(want) + 2.0 ** -133
    assert (np.abs(got - want)[fine] <= e[fine]).all() and (np.abs(got[fine]) <= top).all()
    hq, hs, cq, cs = taco.linear_quantize(qa, sa, qb, sb, bias=bias.cuda(), activation=name)
    if name:
        rq, rs = taco.quantize_rows((bias.float() + 0.0).to(torch.bfloat16)[None].cuda())           # 0 + -0 is 0
        assert torch.equal(cq, rq.expand(m, -1)) and torch.equal(cs, rs.expand(m, -1))
    finite = np.repeat(np.isfinite(t).reshape(-1, 128).all(1), 128)
    assert (hq[0].cpu().numpy()[~finite] == 0x7F).all()
    assert ((hs[0].cpu().numpy() == 255) == ~finite[::128]).all()
    t0 = np.where(finite, t, 0)
    assert (hq == hq[:1]).all() and (hs == hs[:1]).all()
    keep = finite.reshape(-1, 128)[:, 0]
    v, err = ol.activation(t0, name).reshape(-1, 128)[keep], act_error(t0, 0.0, name).reshape(-1, 128)[keep]
    scale = torch.full((int(keep.sum()), 4), 127, dtype=torch.uint8)
    scale[:, 0] = hs[0].cpu()[torch.from_numpy(keep)]
    check_codes(hq[0].cpu().view(-1, 128)[torch.from_numpy(keep)], scale, v, err)


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("m,n,k", KERNELS)
def test_nan_rows_and_columns_stay_apart(m, n, k, name):
    (qa, sa), (qb, sb, _, _) = operands(np.random.default_rng(n), m, n, k)
    bias, residual = (cuda(v) for v in vectors(np.random.default_rng(1), m, n))
    sa[1, 1] = 255
    nan = torch.isnan(taco.linear_fp8(qa, sa, qb, sb, bias=bias, activation=name, residual=residual))
    assert nan[1].all() and not nan[0].any() and not nan[2:].any()
    hq, hs, cq, cs = taco.linear_quantize(qa, sa, qb, sb, bias=bias, activation=name)
    blocks = ol.padded(n) // 128
    for q, s in ((hq, hs), (cq, cs))[:2 if name else 1]:
        assert (q[1] == 0x7F).all() and (s[1, :blocks] == 255).all() and (s[1, blocks:] == 127).all()
        assert not (s[0] == 255).any() and not (s[2:] == 255).any()
    sa[1, 1] = 127
    bias[130] = float("nan")
    residual[2, 5] = float("nan")
    nan = torch.isnan(taco.linear_fp8(qa, sa, qb, sb, bias=bias, activation=name, residual=residual))
    assert nan[:, 130].all() and nan[2, 5] and int(nan.sum()) == m + 1
    hs = taco.linear_quantize(qa, sa, qb, sb, bias=bias, activation=name)[1]
    assert (hs[:, 1] == 255).all() and int((hs == 255).sum()) == m


# ------------------------------------------------------------------------------- the gradient

GRADIENT_SHAPES = [(1, 1), (3, 100), (16, 128), (17, 129), (5, 1600), (64, 512), (300, 2049), (1021, 1601), (33, 4104),
                   (700, 513), (4100, 72), (2, 40001)]


def slope_error(t, name):
    e, w = factor_error(t, name)
    return (2 + w) * (1 + np.abs(t)) * (e + 8 * U * (name not in (None, "relu"))) + 2.0 ** -100


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("rows,cols", GRADIENT_SHAPES)
def test_activation_backward(rows, cols, name):
    rng = np.random.default_rng(rows + cols)
    dh = bf16(rng.standard_normal((rows, cols)) * 1e-3 * np.exp(rng.standard_normal((rows, 1)))).cuda()
    cq, cs = taco.quantize_rows(bf16(1.5 * rng.standard_normal((rows, cols))).cuda()) if name else (None, None)
    t = ol.row_values(cq.cpu().numpy(), cs.cpu().numpy(), cols) if name else np.zeros((rows, cols))
    got, dq, ds, dbias = taco.activation_backward(dh, cq, cs, name)
    dt, want = ol.activation_backward(f64(dh), t, name)
    err = np.abs(f64(dh)) * slope_error(t, name) * (name is not None) + 2 * U * np.abs(dt)
    if name is None:
        assert got is dh
        assert all(torch.equal(a, b) for a, b in zip((dq, ds), taco.quantize_rows(dh)))
    else:
        assert (np.abs(f64(got) - dt) <= 2.0 ** -8 * np.abs(dt) + 1.01 * err + 2.0 ** -133).all()
    check_codes(dq, ds, dt, 1.01 * err)
    assert dbias.shape == (cols,) and dbias.dtype == torch.float32
    assert (np.abs(f64(dbias) - want) <= (rows + 64) * U * np.abs(dt).sum(0) + err.sum(0)).all()
    # parts of the call give the same, and so does a second one
    alone = taco.activation_backward(dh, cq, cs, name, quantize=False)
    assert alone[1] is None and alone[2] is None and torch.equal(alone[3], dbias) and torch.equal(alone[0], got)
    codes = taco.activation_backward(dh, cq, cs, name, bias=False)
    assert codes[3] is None and torch.equal(codes[1], dq) and torch.equal(codes[2], ds) and torch.equal(codes[0], got)


@pytest.mark.parametrize("name", ACTS[1:])
def test_every_code_and_scale_of_t(name):
    """Every code with scale bytes over their whole range: far values of t, infinities and NaN."""
    cols = 256
    cq = torch.arange(256, dtype=torch.int32).to(torch.uint8).expand(256, cols).contiguous()
    cs = torch.full((256, 4), 127, dtype=torch.uint8)
    cs[:, 0] = cs[:, 1] = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    with np.errstate(over="ignore"):
        t = ol.row_values(cq.numpy(), cs.numpy()).astype(np.float32).astype(np.float64)
        want = ol.activation_slope(np.where(np.isfinite(t), t, 0), name)
        want = np.where(np.isinf(t), (t > 0).astype(float), np.where(np.isnan(t), np.nan, want))
        want = np.where(np.abs(t) > 200, (t > 0).astype(float), want)        # its limits, without their formulas' 0 times infinity
        err = np.where(np.isfinite(t) & (np.abs(t) < 200), slope_error(np.clip(np.nan_to_num(t), -200, 200), name), 2.0 ** -100)
    dt = f64(taco.activation_backward(torch.ones(256, cols, dtype=torch.bfloat16).cuda(), cq.cuda(), cs.cuda(), name)[0])
    assert (np.isnan(dt) == np.isnan(want)).all()
    fine = ~np.isnan(want)
    assert (np.abs(dt - want)[fine] <= (2.0 ** -8 * np.abs(want) + 1.01 * err)[fine]).all()


@pytest.mark.parametrize("name", ACTS)
def test_gradient_nan_stays_in_its_block(name):
    rng = np.random.default_rng(3)
    dh = bf16(rng.standard_normal((40, 700))).cuda()
    cq, cs = taco.quantize_rows(bf16(rng.standard_normal((40, 700))).cuda()) if name else (None, None)
    clean = taco.activation_backward(dh, cq, cs, name)
    dh[7, 300] = float("nan")
    if name:
        cs[9, 1] = 255
    dt, dq, ds, dbias = taco.activation_backward(dh, cq, cs, name)
    want = torch.zeros(40, 700, dtype=torch.bool).cuda()
    want[7, 300] = True
    if name:
        want[9, 128:256] = True
    assert torch.equal(torch.isnan(dt), want) and torch.equal(torch.isnan(dbias), want.any(0))
    assert torch.equal(dbias[~want.any(0)], clean[3][~want.any(0)])
    assert ds[7, 2] == 255 and (not name or ds[9, 1] == 255) and int((ds == 255).sum()) == (2 if name else 1)


@pytest.mark.parametrize("name", ["gelu", None])
@pytest.mark.parametrize("rows,cols", GRADIENT_SHAPES)
def test_gradient_writes_only_its_outputs(rows, cols, name):
    dh = activations(np.random.default_rng(rows), rows, cols).cuda()
    cq, cs = taco.quantize_rows(dh) if name else (None, None)
    want = taco.activation_backward(dh, cq, cs, name)
    held = [guarded((rows, cols), torch.bfloat16), guarded((rows, taco.fp8_cols(cols)), torch.uint8),
            guarded((rows, taco.fp8_scale_cols(cols)), torch.uint8), guarded((cols,), torch.float32)]
    outs = {k: v for k, (_, v) in zip(("dt", "dq", "ds", "dbias"), held) if name or k != "dt"}
    need = taco.activation_backward_workspace_bytes(rows, cols)
    whole, ws = guarded((need,), torch.uint8)
    got = taco.activation_backward(dh, cq, cs, name, workspace=ws if need else None, **outs)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert survived(whole) and all(survived(w) for w, _ in held)
