"""Pins of oracle/linear.py (CPU): the block format against its definition and
torch's casts, the gradients against central differences in fp64."""
import numpy as np
import pytest
import torch

import oracle
from oracle import linear as ol


def test_scale_bytes_at_the_borders():
    for e in (-126, -60, -1, 0, 1, 60, 119):
        top = 448.0 * 2.0 ** e
        assert ol.scale_bytes(np.array([top])) == e + 127
        assert ol.scale_bytes(np.array([np.nextafter(top, np.inf)])) == e + 128
    assert ol.scale_bytes(np.array([0.0])) == 127
    assert ol.scale_bytes(np.array([2.0 ** -133])) == 1
    assert (ol.scale_bytes(np.array([np.inf, np.nan])) == 255).all()
    v = ol.scale_values(np.array([0, 1, 127, 254, 255], np.uint8))
    assert v[:4].tolist() == [2.0 ** -127, 2.0 ** -126, 1.0, 2.0 ** 127] and np.isnan(v[4])
    t = torch.tensor([0, 1, 127, 254], dtype=torch.uint8).view(torch.float8_e8m0fnu).double().numpy()
    assert (t == v[:4]).all()


@pytest.mark.parametrize("cols", [1, 127, 128, 129, 700])
def test_rows_round_trip(cols):
    rng = np.random.default_rng(cols)
    x = rng.standard_normal((5, cols)) * np.exp(rng.standard_normal((5, cols)) * 3)
    x[3] = 0
    q, s = ol.quantize_rows(x)
    assert q.shape == (5, ol.padded(cols)) and s.shape == (5, ol.scale_cols(cols))
    assert (q[:, cols:] == 0).all() and (s[:, ol.padded(cols) // 128:] == 127).all() and (s[3] == 127).all()
    v = ol.row_values(q, s, cols)
    step = np.repeat(ol.scale_values(s[:, :ol.padded(cols) // 128]), 128, 1)[:, :cols]
    assert (np.abs(v - x) <= np.maximum(np.abs(x) / 16, step * 2.0 ** -10)).all()      # half a step
    # a largest magnitude that rounded down to 448 may take the next smaller scale, which holds the same values
    assert (ol.row_values(*ol.quantize_rows(v), cols) == v).all()


def test_weight_and_transpose_agree():
    w = np.random.default_rng(0).standard_normal((200, 333))
    q, s, qt, st = ol.quantize_weight(w)
    assert (ol.weight_values(q, s)[:, :333].T == ol.weight_values(qt, st)[:, :200]).all()
    assert q.shape == (200, 384) and s.shape == (2, 4) and qt.shape == (333, 256) and st.shape == (3, 4)


def test_codes_match_torch_cast():
    x = torch.randn(64, 128, dtype=torch.float64) * 50
    q, s = ol.quantize_rows(x.numpy())
    cast = (x / torch.from_numpy(ol.scale_values(s[:, :1]))).float().to(torch.float8_e4m3fn).view(torch.uint8)
    assert (cast.numpy() == q).mean() > 0.999          # fp32 in between may tie


def test_non_finite_block():
    x = np.ones((2, 256))
    x[0, 5], x[1, 200] = np.inf, np.nan
    q, s = ol.quantize_rows(x)
    assert s[:, :2].tolist() == [[255, 119], [119, 255]] and (q[0, :128] == 0x7F).all() and (q[1, :128] != 0x7F).all()


def _difference(f, x, d, h=1e-5):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 5), (4, 130)])
def test_norm_gradient_against_differences(rows, cols):
    rng = np.random.default_rng(rows)
    z, w, dy, dz = (rng.standard_normal(s) for s in ((rows, cols), (cols,), (rows, cols), (rows, cols)))

    def loss_z(v):
        rstd = 1 / np.sqrt((v * v).mean(1) + 1e-3)
        return (dy * v * rstd[:, None] * w).sum() + (dz * v).sum()

    rstd = 1 / np.sqrt((z * z).mean(1) + 1e-3)
    dx, dw = ol.rmsnorm_backward(dy, z, rstd, w, dz)
    d = rng.standard_normal(z.shape)
    assert abs(_difference(loss_z, z, d) - (dx * d).sum()) <= 1e-7 * (1 + np.abs(dx * d).sum())
    dwdir = rng.standard_normal(cols)
    want = _difference(lambda v: (dy * z * rstd[:, None] * v).sum(), w, dwdir)
    assert abs(want - (dw * dwdir).sum()) <= 1e-7 * (1 + np.abs(dw * dwdir).sum())


def test_swiglu_gradient_against_differences():
    rng = np.random.default_rng(1)
    g, u, dh, d = (rng.standard_normal((4, 9)) * 3 for _ in range(4))
    dg, du = ol.swiglu_backward(dh, g, u)
    for grad, f in ((dg, lambda v: (dh * ol.swiglu(v, u)).sum()), (du, lambda v: (dh * ol.swiglu(g, v)).sum())):
        at = g if grad is dg else u
        assert abs(_difference(f, at, d) - (grad * d).sum()) <= 1e-6 * (1 + np.abs(grad * d).sum())
    assert ol.sigmoid(np.array([-800.0, 800.0])).tolist() == [0.0, 1.0]


def test_bf16_sum_of_the_residual():
    x, r = np.array([[1.0, 1.0]]), np.array([[2.0 ** -9, 3 * 2.0 ** -9]])
    z, _, _ = ol.rmsnorm(x, np.ones(2), 0.0, r)
    assert z.tolist() == [[1.0, 1.0 + 2.0 ** -7]]
    assert oracle.Q_MAX == 448.0
