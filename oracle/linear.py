"""Plain fp64 oracle of the 8-bit linear layer's operators (include/taco_linear.h).

Numpy, element by element from the definitions: a block of 128 columns shares
one power-of-two scale, the smallest (from 2^-126) that brings its largest
magnitude to 448 or less; 1 for a block of zeros; NaN, with NaN codes, for a
block that holds a non-finite value.  Nothing is rounded but the codes, and z,
which is stored in bf16.  Test infrastructure: product code never imports it.
"""
from __future__ import annotations

import math

import numpy as np

from .taco_oracle import bf16_bits_to_f64, e4m3_decode, e4m3_encode, f64_to_bf16_bits

BLOCK = 128
NAN_CODE, NAN_BYTE, ONE_BYTE = 0x7F, 255, 127


def padded(cols: int) -> int:
    return (cols + BLOCK - 1) // BLOCK * BLOCK


def scale_cols(cols: int) -> int:
    return (padded(cols) // BLOCK + 3) // 4 * 4


def scale_bytes(amax: np.ndarray) -> np.ndarray:
    """E8M0 byte for each largest magnitude, by search: the first e in 1..254
    with amax <= 448 * 2^(e - 127)."""
    amax = np.asarray(amax, dtype=np.float64)
    limits = 448.0 * np.exp2(np.arange(1, 255) - 127.0)
    byte = np.searchsorted(limits, amax, side="left") + 1      # limits[i] belongs to byte i + 1
    byte = np.where(amax == 0, ONE_BYTE, byte)
    return np.where(np.isfinite(amax), byte, NAN_BYTE).astype(np.uint8)


def scale_values(byte: np.ndarray) -> np.ndarray:
    b = np.asarray(byte, dtype=np.uint8)
    return np.where(b == NAN_BYTE, np.nan, np.exp2(b.astype(np.float64) - 127.0))


def _encode(v: np.ndarray, byte: np.ndarray) -> np.ndarray:
    """Codes of v for scale bytes that broadcast against it."""
    bad = np.broadcast_to(byte == NAN_BYTE, v.shape)
    scaled = np.where(bad, 0.0, v) / np.where(byte == NAN_BYTE, 1.0, scale_values(byte))
    return np.where(bad, NAN_CODE, e4m3_encode(scaled)).astype(np.uint8)


def _largest(v: np.ndarray, axis) -> np.ndarray:
    return np.where(np.isfinite(v).all(axis=axis), np.abs(np.where(np.isfinite(v), v, 0)).max(axis=axis), np.nan)


def _pad_scales(byte: np.ndarray, cols: int) -> np.ndarray:
    out = np.full((byte.shape[0], scale_cols(cols)), ONE_BYTE, dtype=np.uint8)
    out[:, :byte.shape[1]] = byte
    return out


def quantize_rows(v: np.ndarray):
    """fp64 [rows, cols] -> (codes [rows, padded], bytes [rows, scale_cols])."""
    rows, cols = v.shape
    wide = np.zeros((rows, padded(cols)))
    wide[:, :cols] = v
    blocks = wide.reshape(rows, -1, BLOCK)
    byte = scale_bytes(_largest(blocks, 2))
    return _encode(blocks, byte[:, :, None]).reshape(wide.shape), _pad_scales(byte, cols)


def quantize_weight(w: np.ndarray):
    """fp64 [rows, cols] -> (q, scale, qt, scale_t)."""
    n, k = w.shape
    wide = np.zeros((padded(n), padded(k)))
    wide[:n, :k] = w
    blocks = wide.reshape(padded(n) // BLOCK, BLOCK, padded(k) // BLOCK, BLOCK)
    byte = scale_bytes(_largest(blocks, (1, 3)))
    codes = _encode(blocks, byte[:, None, :, None]).reshape(wide.shape)
    return codes[:n], _pad_scales(byte, k), np.ascontiguousarray(codes[:, :k].T), _pad_scales(byte.T, n)


def row_values(q: np.ndarray, scale: np.ndarray, cols: int | None = None) -> np.ndarray:
    """fp64 values of codes in the block format (the first `cols` columns)."""
    s = scale_values(scale[:, :q.shape[1] // BLOCK])
    return (e4m3_decode(q) * np.repeat(s, BLOCK, axis=1))[:, :cols]


def weight_values(q: np.ndarray, scale: np.ndarray) -> np.ndarray:
    s = scale_values(scale[:, :q.shape[1] // BLOCK])
    return e4m3_decode(q) * np.repeat(np.repeat(s, BLOCK, axis=0)[:q.shape[0]], BLOCK, axis=1)


def rmsnorm(x: np.ndarray, weight: np.ndarray, eps: float, residual: np.ndarray | None = None):
    """(z, rstd, y): z rounded to bf16, the rest in fp64."""
    z = x if residual is None else bf16_bits_to_f64(f64_to_bf16_bits(x + residual))
    rstd = 1.0 / np.sqrt((z * z).mean(axis=1) + eps)
    return z, rstd, z * rstd[:, None] * weight


def rmsnorm_backward(dy, z, rstd, weight, dz=None):
    """(dx, dweight) for z's own rstd given."""
    xhat = z * rstd[:, None]
    g = dy * weight
    dx = rstd[:, None] * (g - xhat * (g * xhat).mean(axis=1, keepdims=True))
    return (dx if dz is None else dx + dz), (dy * xhat).sum(axis=0)


def sigmoid(g: np.ndarray) -> np.ndarray:
    e = np.exp(-np.abs(g))                         # no overflow on either side
    return np.where(g >= 0, 1.0, e) / (1.0 + e)


def swiglu(g: np.ndarray, u: np.ndarray) -> np.ndarray:
    return g * sigmoid(g) * u


def swiglu_backward(dh, g, u):
    s = sigmoid(g)
    return dh * u * s * (1.0 + g * (1.0 - s)), dh * g * s


ACTIVATIONS = (None, "relu", "gelu", "gelu_tanh", "silu")


def _normal(t: np.ndarray) -> np.ndarray:
    """The normal distribution function; its tail from erfc, which does not cancel."""
    return 0.5 * np.vectorize(math.erfc, otypes=[float])(-t / math.sqrt(2))


def _tanh_argument(t: np.ndarray) -> np.ndarray:
    return 2 * math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3)


def activation(t: np.ndarray, name: str | None) -> np.ndarray:
    """act(t); the limits at the infinities."""
    with np.errstate(invalid="ignore", over="ignore"):
        if name == "relu":
            v = np.maximum(t, 0)
        elif name == "gelu":
            v = t * _normal(t)
        elif name == "gelu_tanh":
            v = t * sigmoid(_tanh_argument(t))
        else:
            v = t * sigmoid(t) if name == "silu" else t
    return v if name is None else np.where(t == -np.inf, 0.0, v)


def activation_slope(t: np.ndarray, name: str | None) -> np.ndarray:
    """act'(t); 0 for relu at 0."""
    if name is None:
        return np.ones_like(t)
    if name == "relu":
        return np.where(np.isnan(t), t, (t > 0).astype(float))
    if name == "gelu":
        return _normal(t) + t * np.exp(-t * t / 2) / math.sqrt(2 * math.pi)
    z, dz = (t, 1.0) if name == "silu" else (_tanh_argument(t), 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * t * t))
    return sigmoid(z) + t * dz * sigmoid(z) * sigmoid(-z)


def linear(a, b, bias=None, name=None, residual=None):
    """(t, act(t) + residual), t = a b^T + bias."""
    t = a @ b.T + (0 if bias is None else bias)
    h = activation(t, name)
    return t, h if residual is None else h + residual


def activation_backward(dh, t, name):
    """(dt, dbias)."""
    dt = dh * activation_slope(t, name)
    return dt, dt.sum(axis=0)


def checkpoint(g: np.ndarray, u: np.ndarray):
    """Codes and bytes of gate and up side by side."""
    inner = g.shape[1]
    (gq, gs), (uq, us) = quantize_rows(g), quantize_rows(u)
    blocks = padded(inner) // BLOCK
    return np.concatenate([gq, uq], 1), _pad_scales(np.concatenate([gs[:, :blocks], us[:, :blocks]], 1),
                                                    2 * padded(inner))


def checkpoint_values(cq: np.ndarray, cs: np.ndarray, inner: int):
    v = row_values(cq, cs)
    return v[:, :inner], v[:, padded(inner):padded(inner) + inner]
