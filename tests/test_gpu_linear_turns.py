"""The norm's gradient where a workgroup takes several turns over the rows (512 workgroups of two rows up to 8192
columns, of one beyond, 64 above 16384) and the last turn is not full: every training size.  Bounds as in
tests/test_gpu_linear.py."""
import numpy as np
import pytest
import torch

import fp8_compression_tensor_taco_amd as taco
from oracle import linear as ol
from test_gpu_linear import U, activations, bf16, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_dz", [False, True])
@pytest.mark.parametrize("rows,cols", [(9001, 300), (5003, 1000), (2501, 1600), (1099, 4104), (1500, 8192), (600, 8193),
                                       (201, 16392)])
def test_several_turns(rows, cols, with_dz):
    rng = np.random.default_rng(rows)
    z = activations(rng, rows, cols)
    dy, dz = (bf16(rng.standard_normal((rows, cols)) * 1e-3) for _ in range(2))
    w = bf16(1 + 0.1 * rng.standard_normal(cols))
    rstd = torch.from_numpy(1 / np.sqrt((f64(z) ** 2).mean(1) + 1e-5)).float()
    got = taco.rmsnorm_backward(dy.cuda(), z.cuda(), rstd.cuda(), w.cuda(), dz=dz.cuda() if with_dz else None)
    r = f64(rstd)
    rx, rw = ol.rmsnorm_backward(f64(dy), f64(z), r, f64(w), f64(dz) if with_dz else None)
    xhat, g = f64(z) * r[:, None], f64(dy) * f64(w)
    e = 8 * U * np.abs(g) + np.abs(xhat) * (128 + 8) * U * np.abs(g * xhat).mean(1, keepdims=True)
    e = r[:, None] * e + (2 * U * np.abs(f64(dz)) if with_dz else 0)
    assert (np.abs(f64(got[0]) - rx) <= 2.0 ** -8 * np.abs(rx) + 1.01 * e + 2.0 ** -133).all()
    assert (np.abs(f64(got[1]) - rw) <= (rows + 64) * U * np.abs(f64(dy) * xhat).sum(0)).all()
    again = taco.rmsnorm_backward(dy.cuda(), z.cuda(), rstd.cuda(), w.cuda(), dz=dz.cuda() if with_dz else None)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
