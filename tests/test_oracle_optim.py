"""Pins of oracle/optim.py (CPU): its generator against the published known answers, the update against torch's AdamW in
fp64, the stochastic rounding against its definition by search and in the mean."""
import numpy as np
import pytest
import torch

from oracle import linear as ol
from oracle import optim as oo
from oracle.taco_oracle import e4m3_decode


def test_generator_known_answers():
    """Zero, all ones, and digits of pi as counter and key, with ten rounds."""
    ones = 0xFFFFFFFF
    pi = (0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)
    for counter, key, want in (((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
                               ((ones,) * 4, (ones,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
                               (*pi, (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        assert tuple(int(w) for w in oo.philox([counter], key, rounds=10)[0]) == want


def test_random_halves_are_even():
    n = 80000
    for half in oo.random_halves(n, 3, 17, 12345678901234):
        assert half.min() >= 0 and half.max() <= 65535
        assert abs(half.mean() - 32767.5) < 5 * 65536 / np.sqrt(12 * n)
        for bit in range(16):
            assert abs((half >> bit & 1).mean() - 0.5) < 5 * 0.5 / np.sqrt(n)
    a, b, c = oo.random_halves(n, 3, 17, 1)
    for x, y in ((a, b), (a, c), (b, c), (a[1:], a[:-1]), (a, oo.random_halves(n, 4, 17, 1)[0]), (a, oo.random_halves(n, 3, 18, 1)[0])):
        assert abs(np.corrcoef(x, y)[0, 1]) < 5 / np.sqrt(n)


def test_stochastic_codes_by_search():
    """The upper neighbour exactly where the fraction and the bits carry over, on every code's interval."""
    grid = e4m3_decode(np.arange(0x7F, dtype=np.uint8))                 # 0 .. 448
    rng = np.random.default_rng(0)
    low = rng.integers(0, 126, 4000)
    f = rng.random(4000)
    half = rng.integers(0, 65536, 4000)
    x = grid[low] + f * (grid[low + 1] - grid[low])
    f = (x - grid[low]) / (grid[low + 1] - grid[low])                   # exact: a difference of close numbers over a power of two
    want = np.where(f + (half + 0.5) / 65536 >= 1, grid[low + 1], grid[low])
    assert (oo.stochastic(x, 3, -6, half) == want).all()
    assert (oo.stochastic(grid, 3, -6, np.full(127, 65535)) == grid).all()       # a code stays


def test_states_are_unbiased():
    x = np.float32(np.random.default_rng(1).standard_normal(256) * 1e-5)
    total = np.zeros(256)
    for seed in range(4000):
        total += oo.decode_state(oo.encode_state(x, oo.random_halves(256, 0, 1, seed)[0]), 256)
    step = 2.0 ** -3 * np.abs(x) + 2.0 ** -9 * np.repeat(ol.scale_values(oo.encode_state(x, 0)[1][:2]), 128)
    assert (np.abs(total / 4000 - x) <= 5 * step / 2 / np.sqrt(4000)).all()


def test_root_above_zero_stays_so():
    x = np.zeros(128, np.float32)
    x[0], x[1], x[2] = 1.0, 1e-30, 1e-44
    q, _ = oo.encode_state(x, 0, True)
    assert q[1] == q[2] == 1 and (q[3:] == 0).all()
    q, _ = oo.encode_state(x, 0)
    assert q[1] == q[2] == 0


def test_non_finite_block():
    x = np.ones(300, np.float32)
    x[130] = np.inf
    q, s = oo.encode_state(x, np.zeros(300))
    assert s.tolist() == [119, 255, 119, 127] and (q[128:256] == 0x7F).all() and (q[:128] == 0x78).all()          # 1 = 256 * 2^(119 - 127)
    assert (q[300:] == 0).all()


@pytest.mark.parametrize("steps,decay", [(1, 0.0), (5, 0.1)])
def test_update_against_torch(steps, decay):
    rng = np.random.default_rng(2)
    p = torch.from_numpy(rng.standard_normal(50)).requires_grad_()
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.8, 0.95), eps=1e-6, weight_decay=decay)
    q, m, v = p.detach().numpy().copy(), np.zeros(50, np.float32), np.zeros(50, np.float32)
    for step in range(1, steps + 1):
        g = rng.standard_normal(50).astype(np.float32)
        p.grad = torch.from_numpy(g.astype(np.float64))
        opt.step()
        q, m, v = oo.adamw(q, g, m, v, lr=1e-2, step=step, betas=(0.8, 0.95), eps=1e-6, decay=decay)
    # m and v carry fp32 roundings: the update, at most lr, is off by a few 2^-24 of itself a step
    assert np.abs(q - p.detach().numpy()).max() <= 1e-2 * steps * 20 * 2.0 ** -24
