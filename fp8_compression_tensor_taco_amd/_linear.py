"""ctypes binding over the 8-bit linear layer's C ABI (include/taco_linear.h).

Argument marshalling only, as in _binding: the operators run in the HIP kernels
of libtaco.so, there is no CPU fallback, and outputs may be passed in to avoid
allocation.  Matrices are 2-D; an input that is not contiguous is copied.

Codes and scales are uint8 tensors.  ``q.view(torch.float8_e4m3fn)`` and
``scale.view(torch.float8_e8m0fnu)`` give their values.
"""
from __future__ import annotations

import ctypes

import torch

from ._binding import _check, _on, load

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
}
_typed = None


def _lib():
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


def _input(t, name, dtype, dims=2):
    """The tensor as the kernels take it: on a GPU, contiguous, 16-byte aligned."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError("libtaco works on GPU tensors only (no CPU fallback)")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    if not t.is_contiguous():
        return t.contiguous()
    return t if t.data_ptr() & 15 == 0 else t.clone()


def _shaped(t, name, dtype, shape, device):
    """The same, of a given shape and on the call's device."""
    t = _input(t, name, dtype, len(shape))
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError("all tensors must be on the same device")
    return t


def _output(t, name, dtype, shape, device):
    if t is None:          # with strides: quicker than torch.empty, and small calls are bound by the host
        return torch.empty_strided(shape, (shape[1], 1) if len(shape) == 2 else (1,), dtype=dtype, device=device)
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on {device}")
    return t


def _current(device):
    """Handle of the device's current stream; the library launches on the current device."""
    if torch._C._cuda_getDevice() != device.index:
        raise ValueError(f"the tensors are on {device}, the current device is {torch._C._cuda_getDevice()}")
    return torch._C._cuda_getCurrentRawStream(device.index)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _scratch(workspace, device, nbytes):
    """(the given workspace or a new one, its address, its bytes).

    A new one per call: torch's allocator hands it out again in the stream's
    order, and a captured graph keeps its own."""
    if workspace is None:
        if nbytes == 0:
            return None, None, 0
        workspace = torch.empty_strided((nbytes,), (1,), dtype=torch.uint8, device=device)
    elif not workspace.is_contiguous() or workspace.device != device:
        raise ValueError(f"workspace must be contiguous and on {device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


# Every call with a stream makes it current and calls itself: outputs, copies of
# inputs and the launch then belong to that stream (see _binding._on).

def quantize_rows(x: torch.Tensor, *, q: torch.Tensor | None = None, scale: torch.Tensor | None = None, stream=None):
    """Quantise bf16 [rows, cols] into the block format.

    Returns (q uint8 [rows, fp8_cols(cols)], scale uint8 [rows, fp8_scale_cols(cols)])."""
    if stream is not None:
        with _on(stream):
            return quantize_rows(x, q=q, scale=scale)
    x = _input(x, "x", torch.bfloat16)
    rows, cols = x.shape
    dev = x.device
    q = _output(q, "q", torch.uint8, (rows, fp8_cols(cols)), dev)
    scale = _output(scale, "scale", torch.uint8, (rows, fp8_scale_cols(cols)), dev)
    _check(_lib().taco_quantize_rows(x.data_ptr(), rows, cols, q.data_ptr(), scale.data_ptr(), _current(dev)))
    return q, scale


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
    w = _input(w, "w", torch.bfloat16)
    rows, cols = w.shape
    dev = w.device
    q = _output(q, "q", torch.uint8, (rows, fp8_cols(cols)), dev)
    scale = _output(scale, "scale", torch.uint8, (fp8_cols(rows) // BLOCK, fp8_scale_cols(cols)), dev)
    if transposed:
        qt = _output(qt, "qt", torch.uint8, (cols, fp8_cols(rows)), dev)
        scale_t = _output(scale_t, "scale_t", torch.uint8, (fp8_cols(cols) // BLOCK, fp8_scale_cols(rows)), dev)
    elif qt is not None or scale_t is not None:
        raise ValueError("qt and scale_t are outputs of transposed=True")
    _check(_lib().taco_quantize_weight(w.data_ptr(), rows, cols, q.data_ptr(), scale.data_ptr(), _ptr(qt),
                                       _ptr(scale_t), _current(dev)))
    return q, scale, qt, scale_t


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
    x = _input(x, "x", torch.bfloat16)
    tokens, hidden = x.shape
    dev = x.device
    weight = _shaped(weight, "weight", torch.bfloat16, (hidden,), dev)
    if residual is not None:
        residual = _shaped(residual, "residual", torch.bfloat16, (tokens, hidden), dev)
        z = _output(z, "z", torch.bfloat16, (tokens, hidden), dev)
    elif z is not None:
        raise ValueError("z is an output of the call with a residual")
    rstd = _output(rstd, "rstd", torch.float32, (tokens,), dev)
    q = _output(q, "q", torch.uint8, (tokens, fp8_cols(hidden)), dev)
    scale = _output(scale, "scale", torch.uint8, (tokens, fp8_scale_cols(hidden)), dev)
    _check(_lib().taco_rmsnorm_quantize(x.data_ptr(), _ptr(residual), weight.data_ptr(), tokens, hidden, eps,
                                        _ptr(z), rstd.data_ptr(), q.data_ptr(), scale.data_ptr(),
                                        _current(dev)))
    return x if z is None else z, rstd, q, scale


def rmsnorm_backward(dy: torch.Tensor, z: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor, *,
                     dz: torch.Tensor | None = None, dx: torch.Tensor | None = None,
                     dweight: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Gradient of rmsnorm_quantize for dy, the gradient of its (unquantised) output.

    dz is the gradient that reached z by the residual path.  Returns (dx bf16,
    the gradient of x and of the residual; dweight fp32 [hidden])."""
    if stream is not None:
        with _on(stream):
            return rmsnorm_backward(dy, z, rstd, weight, dz=dz, dx=dx, dweight=dweight, workspace=workspace)
    dy = _input(dy, "dy", torch.bfloat16)
    tokens, hidden = dy.shape
    dev = dy.device
    z = _shaped(z, "z", torch.bfloat16, (tokens, hidden), dev)
    rstd = _shaped(rstd, "rstd", torch.float32, (tokens,), dev)
    weight = _shaped(weight, "weight", torch.bfloat16, (hidden,), dev)
    if dz is not None:
        dz = _shaped(dz, "dz", torch.bfloat16, (tokens, hidden), dev)
    dx = _output(dx, "dx", torch.bfloat16, (tokens, hidden), dev)
    dweight = _output(dweight, "dweight", torch.float32, (hidden,), dev)
    lib = _lib()
    workspace, at, size = _scratch(workspace, dev, lib.taco_rmsnorm_backward_workspace_bytes(tokens, hidden))
    _check(lib.taco_rmsnorm_backward(dy.data_ptr(), z.data_ptr(), rstd.data_ptr(), weight.data_ptr(), _ptr(dz),
                                     tokens, hidden, dx.data_ptr(), dweight.data_ptr(), at, size, _current(dev)))
    return dx, dweight


def matmul_fp8(qa: torch.Tensor, sa: torch.Tensor, qb: torch.Tensor, sb: torch.Tensor, *,
               out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """bf16 [m, n] = a b^T of a [m, k] in the block format and b [n, k] in the weight format.

    With a = x and b = w a linear layer's output; with a = dy and b the
    transposed weight, the gradient of its input."""
    if stream is not None:
        with _on(stream):
            return matmul_fp8(qa, sa, qb, sb, out=out, workspace=workspace)
    qa, qb = _input(qa, "qa", torch.uint8), _input(qb, "qb", torch.uint8)
    (m, k), n = qa.shape, qb.shape[0]
    if k == 0 or k % BLOCK or qb.shape[1] != k:
        raise ValueError(f"qa and qb must have the same number of columns, a multiple of {BLOCK}: "
                         f"got {k} and {qb.shape[1]}")
    dev = qa.device
    sa = _shaped(sa, "sa", torch.uint8, (m, fp8_scale_cols(k)), dev)
    sb = _shaped(sb, "sb", torch.uint8, (-(-n // BLOCK), fp8_scale_cols(k)), dev)
    if qb.device != dev:
        raise ValueError("all tensors must be on the same device")
    out = _output(out, "out", torch.bfloat16, (m, n), dev)
    lib = _lib()
    workspace, at, size = _scratch(workspace, dev, lib.taco_matmul_fp8_workspace_bytes(m, n, k))
    _check(lib.taco_matmul_fp8(qa.data_ptr(), sa.data_ptr(), qb.data_ptr(), sb.data_ptr(), m, n, k,
                               out.data_ptr(), at, size, _current(dev)))
    return out


def wgrad_fp8(dy: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, cols: int, *, dw: torch.Tensor | None = None,
              accumulate: bool = False, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """fp32 [n, cols] = dy^T x of bf16 dy [tokens, n] and x [tokens, cols] in the block format.

    x is a linear layer's input as it was kept in 8 bits.  accumulate=True adds
    to dw, which must then be given."""
    if stream is not None:
        with _on(stream):
            return wgrad_fp8(dy, q, scale, cols, dw=dw, accumulate=accumulate, workspace=workspace)
    dy = _input(dy, "dy", torch.bfloat16)
    tokens, n = dy.shape
    dev = dy.device
    q = _shaped(q, "q", torch.uint8, (tokens, fp8_cols(cols)), dev)
    scale = _shaped(scale, "scale", torch.uint8, (tokens, fp8_scale_cols(cols)), dev)
    if accumulate and dw is None:
        raise ValueError("accumulate=True adds to dw: pass it")
    dw = _output(dw, "dw", torch.float32, (n, cols), dev)
    lib = _lib()
    workspace, at, size = _scratch(workspace, dev, lib.taco_wgrad_fp8_workspace_bytes(tokens, n, cols))
    _check(lib.taco_wgrad_fp8(dy.data_ptr(), q.data_ptr(), scale.data_ptr(), tokens, n, cols, dw.data_ptr(),
                              int(bool(accumulate)), at, size, _current(dev)))
    return dw


def swiglu_quantize(gu: torch.Tensor, *, checkpoint: bool = True, hq: torch.Tensor | None = None,
                    hs: torch.Tensor | None = None, cq: torch.Tensor | None = None, cs: torch.Tensor | None = None,
                    stream=None):
    """SiLU-gated unit of bf16 gu [tokens, 2 * inner] (gate, then up), quantised.

    Returns (hq, hs, cq, cs): silu(gate) * up in the block format, and gate and
    up in 8 bits for swiglu_backward (checkpoint=False gives None for those)."""
    if stream is not None:
        with _on(stream):
            return swiglu_quantize(gu, checkpoint=checkpoint, hq=hq, hs=hs, cq=cq, cs=cs)
    gu = _input(gu, "gu", torch.bfloat16)
    tokens, both = gu.shape
    if both == 0 or both % 2:
        raise ValueError("gu must have an even number of columns: gate, then up")
    inner = both // 2
    dev, wide = gu.device, fp8_cols(inner)
    hq = _output(hq, "hq", torch.uint8, (tokens, wide), dev)
    hs = _output(hs, "hs", torch.uint8, (tokens, fp8_scale_cols(inner)), dev)
    if checkpoint:
        cq = _output(cq, "cq", torch.uint8, (tokens, 2 * wide), dev)
        cs = _output(cs, "cs", torch.uint8, (tokens, fp8_scale_cols(2 * wide)), dev)
    elif cq is not None or cs is not None:
        raise ValueError("cq and cs are outputs of checkpoint=True")
    _check(_lib().taco_swiglu_quantize(gu.data_ptr(), tokens, inner, hq.data_ptr(), hs.data_ptr(), _ptr(cq),
                                       _ptr(cs), _current(dev)))
    return hq, hs, cq, cs


def swiglu_backward(dh: torch.Tensor, cq: torch.Tensor, cs: torch.Tensor, *, quantize: bool = True,
                    dgu: torch.Tensor | None = None, dq: torch.Tensor | None = None, ds: torch.Tensor | None = None,
                    stream=None):
    """Gradient of swiglu_quantize for dh bf16 [tokens, inner], at the checkpoint's gate and up.

    Returns (dgu bf16 [tokens, 2 * inner], dq, ds): the gradient of gu, and the
    same in the block format (quantize=False gives None for those)."""
    if stream is not None:
        with _on(stream):
            return swiglu_backward(dh, cq, cs, quantize=quantize, dgu=dgu, dq=dq, ds=ds)
    dh = _input(dh, "dh", torch.bfloat16)
    tokens, inner = dh.shape
    wide = fp8_cols(inner)
    dev = dh.device
    cq = _shaped(cq, "cq", torch.uint8, (tokens, 2 * wide), dev)
    cs = _shaped(cs, "cs", torch.uint8, (tokens, fp8_scale_cols(2 * wide)), dev)
    dgu = _output(dgu, "dgu", torch.bfloat16, (tokens, 2 * inner), dev)
    if quantize:
        dq = _output(dq, "dq", torch.uint8, (tokens, fp8_cols(2 * inner)), dev)
        ds = _output(ds, "ds", torch.uint8, (tokens, fp8_scale_cols(2 * inner)), dev)
    elif dq is not None or ds is not None:
        raise ValueError("dq and ds are outputs of quantize=True")
    _check(_lib().taco_swiglu_backward(dh.data_ptr(), cq.data_ptr(), cs.data_ptr(), tokens, inner,
                                       dgu.data_ptr(), _ptr(dq), _ptr(ds), _current(dev)))
    return dgu, dq, ds
