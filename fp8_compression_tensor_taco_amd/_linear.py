"""The 8-bit linear layer's operators (include/taco_linear.h) on torch tensors.

The operators run in the HIP kernels of libtaco.so; the arguments go there
through csrc/linear_binding.cpp, which checks them, allocates outputs that are
not passed in, and raises ValueError or TacoError.  There is no CPU fallback.
Matrices are 2-D; an input that is not contiguous is copied.  A call runs on
`stream`, or on the current stream of the tensors' device, which must be the
current device.

Codes and scales are uint8 tensors.  ``q.view(torch.float8_e4m3fn)`` and
``scale.view(torch.float8_e8m0fnu)`` give their values.
"""
from __future__ import annotations

import ctypes
import os

import torch

from ._binding import _on, load
from .build import BINDING_PATH

BLOCK = 128

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_size = ctypes.c_size_t
_SIGNATURES = {
    "taco_fp8_cols": (_i64, [_i64]),
    "taco_fp8_scale_cols": (_i64, [_i64]),
    "taco_quantize_rows": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _vp]),
    "taco_quantize_weight": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
    "taco_rmsnorm_quantize": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, ctypes.c_float, _vp, _vp, _vp, _vp, _vp]),
    "taco_rmsnorm_backward_workspace_bytes": (_size, [_i64, _i64]),
    "taco_rmsnorm_backward": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _size, _vp]),
    "taco_matmul_fp8_workspace_bytes": (_size, [_i64, _i64, _i64]),
    "taco_matmul_fp8": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _size, _vp]),
    "taco_wgrad_fp8_workspace_bytes": (_size, [_i64, _i64, _i64]),
    "taco_wgrad_fp8": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _i64, _vp, ctypes.c_int32, _vp, _size, _vp]),
    "taco_swiglu_quantize": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
    "taco_swiglu_backward": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp]),
    "taco_linear_fp8_workspace_bytes": (_size, [_i64, _i64, _i64]),
    "taco_linear_fp8": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int32, _i64, _i64, _i64, _vp, _vp, _size, _vp]),
    "taco_linear_quantize_workspace_bytes": (_size, [_i64, _i64, _i64]),
    "taco_linear_quantize": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, ctypes.c_int32, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp,
                                            _size, _vp]),
    "taco_activation_backward_workspace_bytes": (_size, [_i64, _i64]),
    "taco_activation_backward": (ctypes.c_int, [_vp, _vp, _vp, ctypes.c_int32, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _size, _vp]),
}
_typed = None
_native = None


def _lib():
    """The C ABI with its argument types, for callers with pointers."""
    global _typed
    if _typed is None:
        lib = load()
        for name, (restype, argtypes) in _SIGNATURES.items():
            f = getattr(lib, name)
            f.restype, f.argtypes = restype, argtypes
        _typed = lib
    return _typed


def fp8_cols(cols: int) -> int:
    """Codes in a row of ``cols`` columns: rounded up to whole blocks of 128."""
    if cols < 1:
        raise ValueError("cols must be at least 1")
    return -(-cols // BLOCK) * BLOCK


def fp8_scale_cols(cols: int) -> int:
    """Scale bytes in a row of ``cols`` columns: one per 128, rounded up to 4."""
    return -(-fp8_cols(cols) // (4 * BLOCK)) * 4


def _binding():
    global _native
    if _native is None:
        load()
        try:
            from . import _linear_binding
        except ImportError as e:
            what = ("does not load, it may be of another Python or torch" if os.path.exists(BINDING_PATH)
                    else "is not built")
            raise ImportError(f"the binding of the 8-bit linear layer {what}: build it with `python -m "
                              f"fp8_compression_tensor_taco_amd.build` (no CPU fallback exists); {e}") from e
        _native = _linear_binding
    return _native


def _current(t: torch.Tensor) -> int:
    """Handle of the current stream; the library launches on the current device.  (The binding refuses CPU tensors.)"""
    if not t.is_cuda:
        return 0
    index = t.get_device()
    if torch._C._cuda_getDevice() != index:
        raise ValueError(f"the tensors are on cuda:{index}, the current device is cuda:{torch._C._cuda_getDevice()}")
    return torch._C._cuda_getCurrentRawStream(index)


def rmsnorm_backward_workspace_bytes(tokens: int, hidden: int) -> int:
    return int(_lib().taco_rmsnorm_backward_workspace_bytes(tokens, hidden))


def matmul_fp8_workspace_bytes(m: int, n: int, k: int) -> int:
    return int(_lib().taco_matmul_fp8_workspace_bytes(m, n, k))


def wgrad_fp8_workspace_bytes(tokens: int, n: int, cols: int) -> int:
    return int(_lib().taco_wgrad_fp8_workspace_bytes(tokens, n, cols))


def linear_fp8_workspace_bytes(m: int, n: int, k: int) -> int:
    return int(_lib().taco_linear_fp8_workspace_bytes(m, n, k))


def linear_quantize_workspace_bytes(m: int, n: int, k: int) -> int:
    return int(_lib().taco_linear_quantize_workspace_bytes(m, n, k))


def activation_backward_workspace_bytes(tokens: int, cols: int) -> int:
    return int(_lib().taco_activation_backward_workspace_bytes(tokens, cols))


# Every call with a stream makes it current and calls itself: outputs, copies of
# inputs and the launch then belong to that stream (see _binding._on).


def quantize_rows(x: torch.Tensor, *, q: torch.Tensor | None = None, scale: torch.Tensor | None = None, stream=None):
    """Quantise bf16 [rows, cols] into the block format.

    Returns (q uint8 [rows, fp8_cols(cols)], scale uint8 [rows, fp8_scale_cols(cols)])."""
    if stream is not None:
        with _on(stream):
            return quantize_rows(x, q=q, scale=scale)
    return _binding().quantize_rows(x, q, scale, _current(x))


def quantize_weight(w: torch.Tensor, *, transposed: bool = True, q: torch.Tensor | None = None,
                    scale: torch.Tensor | None = None, qt: torch.Tensor | None = None,
                    scale_t: torch.Tensor | None = None, stream=None):
    """Quantise a bf16 weight [rows, cols], one scale per 128 x 128 block.

    Returns (q, scale, qt, scale_t): the weight [rows, cols] and the same codes
    of its transpose [cols, rows], both in the weight format, for the forward
    product and the input's gradient.  transposed=False gives None for the last two."""
    if stream is not None:
        with _on(stream):
            return quantize_weight(w, transposed=transposed, q=q, scale=scale, qt=qt, scale_t=scale_t)
    return _binding().quantize_weight(w, transposed, q, scale, qt, scale_t, _current(w))


def rmsnorm_quantize(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5, *,
                     residual: torch.Tensor | None = None, z: torch.Tensor | None = None,
                     rstd: torch.Tensor | None = None, q: torch.Tensor | None = None,
                     scale: torch.Tensor | None = None, stream=None):
    """Root-mean-square norm of bf16 x (+ residual), quantised.

    Returns (z, rstd, q, scale): z = bf16(x + residual), the new residual
    stream (x itself without a residual); rstd fp32 [tokens]; and
    z * rstd * weight in the block format."""
    if stream is not None:
        with _on(stream):
            return rmsnorm_quantize(x, weight, eps, residual=residual, z=z, rstd=rstd, q=q, scale=scale)
    return _binding().rmsnorm_quantize(x, weight, eps, residual, z, rstd, q, scale, _current(x))


def rmsnorm_backward(dy: torch.Tensor, z: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor, *,
                     dz: torch.Tensor | None = None, dx: torch.Tensor | None = None,
                     dweight: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Gradient of rmsnorm_quantize for dy, the gradient of its (unquantised) output.

    dz is the gradient that reached z by the residual path.  Returns (dx bf16,
    the gradient of x and of the residual; dweight fp32 [hidden])."""
    if stream is not None:
        with _on(stream):
            return rmsnorm_backward(dy, z, rstd, weight, dz=dz, dx=dx, dweight=dweight, workspace=workspace)
    return _binding().rmsnorm_backward(dy, z, rstd, weight, dz, dx, dweight, workspace, _current(dy))


def matmul_fp8(qa: torch.Tensor, sa: torch.Tensor, qb: torch.Tensor, sb: torch.Tensor, *,
               out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """bf16 [m, n] = a b^T of a [m, k] in the block format and b [n, k] in the weight format.

    With a = x and b = w a linear layer's output; with a = dy and b the
    transposed weight, the gradient of its input.

    The matrix cores align the products of each eight consecutive columns to the
    largest of them and cut the others below 2^-13 of it, and cut instead of
    rounding where they add to the fp32 sum: a relative error near 3e-5 on
    ordinary data, beside the 2^-9 of the output's rounding (bound in taco_linear.h)."""
    if stream is not None:
        with _on(stream):
            return matmul_fp8(qa, sa, qb, sb, out=out, workspace=workspace)
    return _binding().matmul_fp8(qa, sa, qb, sb, out, workspace, _current(qa))


def wgrad_fp8(dy: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, cols: int, *, dw: torch.Tensor | None = None,
              accumulate: bool = False, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """fp32 [n, cols] = dy^T x of bf16 dy [tokens, n] and x [tokens, cols] in the block format.

    x is a linear layer's input as it was kept in 8 bits.  accumulate=True adds
    to dw, which must then be given."""
    if stream is not None:
        with _on(stream):
            return wgrad_fp8(dy, q, scale, cols, dw=dw, accumulate=accumulate, workspace=workspace)
    return _binding().wgrad_fp8(dy, q, scale, cols, dw, accumulate, workspace, _current(dy))


def swiglu_quantize(gu: torch.Tensor, *, checkpoint: bool = True, hq: torch.Tensor | None = None,
                    hs: torch.Tensor | None = None, cq: torch.Tensor | None = None, cs: torch.Tensor | None = None,
                    stream=None):
    """SiLU-gated unit of bf16 gu [tokens, 2 * inner] (gate, then up), quantised.

    Returns (hq, hs, cq, cs): silu(gate) * up in the block format, and gate and
    up in 8 bits for swiglu_backward (checkpoint=False gives None for those)."""
    if stream is not None:
        with _on(stream):
            return swiglu_quantize(gu, checkpoint=checkpoint, hq=hq, hs=hs, cq=cq, cs=cs)
    return _binding().swiglu_quantize(gu, checkpoint, hq, hs, cq, cs, _current(gu))


def swiglu_backward(dh: torch.Tensor, cq: torch.Tensor, cs: torch.Tensor, *, quantize: bool = True,
                    dgu: torch.Tensor | None = None, dq: torch.Tensor | None = None, ds: torch.Tensor | None = None,
                    stream=None):
    """Gradient of swiglu_quantize for dh bf16 [tokens, inner], at the checkpoint's gate and up.

    Returns (dgu bf16 [tokens, 2 * inner], dq, ds): the gradient of gu, and the
    same in the block format (quantize=False gives None for those)."""
    if stream is not None:
        with _on(stream):
            return swiglu_backward(dh, cq, cs, quantize=quantize, dgu=dgu, dq=dq, ds=ds)
    return _binding().swiglu_backward(dh, cq, cs, quantize, dgu, dq, ds, _current(dh))


def linear_fp8(qa: torch.Tensor, sa: torch.Tensor, qb: torch.Tensor, sb: torch.Tensor, *, bias: torch.Tensor | None = None,
               activation: str | None = None, residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """bf16 [m, n] = act(a b^T + bias) + residual, with matmul_fp8's operands and sums and one rounding at the end.

    bias bf16 [n] and residual bf16 [m, n] may be left out; activation is None, 'relu', 'gelu' (through the normal
    distribution function), 'gelu_tanh' or 'silu'."""
    if stream is not None:
        with _on(stream):
            return linear_fp8(qa, sa, qb, sb, bias=bias, activation=activation, residual=residual, out=out, workspace=workspace)
    return _binding().linear_fp8(qa, sa, qb, sb, bias, activation, residual, out, workspace, _current(qa))


def linear_quantize(qa: torch.Tensor, sa: torch.Tensor, qb: torch.Tensor, sb: torch.Tensor, *, bias: torch.Tensor | None = None,
                    activation: str | None = None, checkpoint: bool = True, hq: torch.Tensor | None = None,
                    hs: torch.Tensor | None = None, cq: torch.Tensor | None = None, cs: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None):
    """linear_fp8 without a residual, quantised: h = act(t), t = a b^T + bias.

    Returns (hq, hs, cq, cs): h in the block format, and t in 8 bits for activation_backward (None for those with
    checkpoint=False, and without an activation, whose gradient needs no t)."""
    if stream is not None:
        with _on(stream):
            return linear_quantize(qa, sa, qb, sb, bias=bias, activation=activation, checkpoint=checkpoint, hq=hq, hs=hs,
                                   cq=cq, cs=cs, workspace=workspace)
    return _binding().linear_quantize(qa, sa, qb, sb, bias, activation, checkpoint, hq, hs, cq, cs, workspace, _current(qa))


def activation_backward(dh: torch.Tensor, cq: torch.Tensor | None, cs: torch.Tensor | None, activation: str | None, *,
                        quantize: bool = True, bias: bool = True, dt: torch.Tensor | None = None,
                        dq: torch.Tensor | None = None, ds: torch.Tensor | None = None, dbias: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, stream=None):
    """Gradient of linear_quantize's nonlinearity and bias for dh bf16 [tokens, cols], at the checkpoint's t.

    Returns (dt, dq, ds, dbias): dt = dh act'(t) in bf16 (dh itself without an activation, whose checkpoint is None),
    the same in the block format for the gradients of the product (None with quantize=False), and its sums over tokens
    in fp32, the bias's gradient (None with bias=False)."""
    if stream is not None:
        with _on(stream):
            return activation_backward(dh, cq, cs, activation, quantize=quantize, bias=bias, dt=dt, dq=dq, ds=ds,
                                       dbias=dbias, workspace=workspace)
    return _binding().activation_backward(dh, cq, cs, activation, quantize, bias, dt, dq, ds, dbias, workspace, _current(dh))
