"""Oracle of the training step's update (include/taco_optim.h).

Numpy from the definitions.  The moments are defined with each product and sum
rounded to fp32, so they are computed so, in fp32; the parameters in fp64, with no
rounding but bf16's stochastic one.  8-bit states round stochastically: a magnitude
over its block's scale is k steps of its binade's eighth (of 2^-9 below 2^-6), and
floor(k + (u + 1/2) / 2^16) is kept.  Test infrastructure: product code never
imports it.
"""
from __future__ import annotations

import numpy as np

from . import linear as ol
from .taco_oracle import e4m3_decode, e4m3_encode

F = np.float32


def philox(counter, key, rounds=7):
    """Philox4x32: counter [n, 4] and key (2 words) -> [n, 4] words."""
    x = [np.asarray(counter, dtype=np.uint64)[:, i] for i in range(4)]
    k0, k1 = (np.uint64(k) for k in key)
    low = np.uint64(0xFFFFFFFF)
    for r in range(rounds):
        a, b = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)          # below 2^64
        x = [(b >> np.uint64(32)) ^ x[1] ^ k0, b & low, (a >> np.uint64(32)) ^ x[3] ^ k1, a & low]
        k0, k1 = (k0 + np.uint64(0x9E3779B9)) & low, (k1 + np.uint64(0xBB67AE85)) & low
    return np.stack(x, 1)


def random_halves(n, index, step, seed, first=0):
    """16 bits of each element, from `first` on, for m, for sqrt(v) and for a bf16 parameter."""
    at = np.arange(n)
    e = at + first
    key = (seed & 0xFFFFFFFF, seed >> 32)

    def words(call):
        c = np.stack([e // 8, call, np.full(n, index), np.full(n, step & 0xFFFFFFFF)], 1)
        return philox(c, key)

    w = words(e % 8 // 4)[at, e % 4].astype(np.int64)
    p = words(np.full(n, 2))[at, e % 8 // 2].astype(np.int64)
    return w & 0xFFFF, w >> 16, np.where(e % 2 == 0, p & 0xFFFF, p >> 16)


def stochastic(size, mantissa, least, half):
    """Magnitudes on a grid of `mantissa` bits, exponents from `least` on."""
    e = np.maximum(np.frexp(np.where(size > 0, size, 1.0))[1] - 1, least) - mantissa
    return np.ldexp(np.floor(np.ldexp(size, -e) + (half + 0.5) / 65536), e)


def encode_state(x, half, root=False):
    """fp32 row -> (codes, scale bytes), padded."""
    n = len(x)
    wide = np.zeros(ol.padded(n))
    wide[:n] = x
    blocks = wide.reshape(-1, 128)
    byte = ol.scale_bytes(ol._largest(blocks, 1))
    bad = np.repeat(byte == ol.NAN_BYTE, 128)
    size = np.where(bad, 0.0, np.abs(wide)) / np.repeat(np.where(byte == ol.NAN_BYTE, 1.0, ol.scale_values(byte)), 128)
    halves = np.zeros(len(wide))
    halves[:n] = half
    size = np.where(size > 0, stochastic(size, 3, -6, halves), 0.0)
    if root:
        size = np.where(wide > 0, np.maximum(size, 2.0 ** -9), size)
    q = np.where(bad, ol.NAN_CODE, e4m3_encode(np.copysign(size, np.where(bad, 0.0, wide))))
    return q.astype(np.uint8), ol._pad_scales(byte[None], n)[0]


def decode_state(state, n):
    q, s = state
    return (e4m3_decode(q) * np.repeat(ol.scale_values(s[:len(q) // 128]), 128))[:n]


def adamw(p, grad, m, v, *, lr, step, betas, eps, decay, factor=1.0, index=0, seed=0, bf16=False, first=0):
    """(p', m', v') of one tensor, or of its elements from `first` on, a multiple of 128; m, v fp32 arrays or pairs of codes and scale bytes (then pairs come back).

    p' in fp64, with the stochastic rounding for bf16."""
    n = len(p)
    bits8 = isinstance(m, tuple)
    half_m, half_v, half_p = random_halves(n, index, step, seed, first)
    g = np.asarray(grad, F) * F(factor)
    m_, r_ = (decode_state(m, n).astype(F), decode_state(v, n).astype(F)) if bits8 else (np.asarray(m, F), None)
    v_ = r_ * r_ if bits8 else np.asarray(v, F)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        m_ = m_ * F(betas[0]) + g * F(1 - betas[0])
        v_ = v_ * F(betas[1]) + g * g * F(1 - betas[1])
        root = np.sqrt(v_)
        hat = (m_.astype(float) / (1 - betas[0] ** step)) / (root.astype(float) / np.sqrt(1 - betas[1] ** step) + eps)
        new = np.asarray(p, float) * (1 - lr * decay) - lr * hat
    if bf16:
        new = np.copysign(stochastic(np.abs(new), 7, -126, half_p), new)
    if bits8:
        return new, encode_state(m_, half_m), encode_state(root, half_v, True)
    return new, m_, v_
