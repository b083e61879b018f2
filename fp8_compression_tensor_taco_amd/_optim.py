"""The update of a training step (include/taco_optim.h) on lists of torch tensors.

Adam with decoupled weight decay, its states in fp32 or in 8 bits, and the global
norm of the gradients.  The work is done by the HIP kernels of libtaco.so; lists
go there through csrc/optim_binding.cpp, which raises ValueError or TacoError.
There is no CPU fallback.  A call runs on `stream`, or on the current stream of
the tensors' device, which must be the current device.
"""
from __future__ import annotations

import ctypes
import math

import torch

from ._binding import _on, load
from ._linear import _binding, _current, fp8_cols, fp8_scale_cols

TACO_TYPE_FP32, TACO_TYPE_BF16 = 0, 1

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64


class AdamwTensor(ctypes.Structure):
    """taco_adamw_tensor_t, for callers with pointers."""
    _fields_ = [("param", _vp), ("grad", _vp), ("m", _vp), ("v", _vp), ("m_scale", _vp), ("v_scale", _vp), ("copy", _vp),
                ("count", _i64), ("param_type", ctypes.c_int32), ("grad_type", ctypes.c_int32)]


class AdamwOptions(ctypes.Structure):
    """taco_adamw_options_t."""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("weight_decay", ctypes.c_double), ("step", _i64), ("seed", ctypes.c_uint64), ("lr_device", _vp),
                ("step_device", _vp), ("grad_scale", _vp)]


class NormTensor(ctypes.Structure):
    """taco_norm_tensor_t."""
    _fields_ = [("data", _vp), ("count", _i64), ("type", ctypes.c_int32)]


_SIGNATURES = {
    "taco_adamw_step": (ctypes.c_int, [ctypes.POINTER(AdamwTensor), _i64, ctypes.POINTER(AdamwOptions), _vp]),
    "taco_gradient_norm_workspace_bytes": (ctypes.c_size_t, [_i64]),
    "taco_gradient_norm": (ctypes.c_int, [ctypes.POINTER(NormTensor), _i64, ctypes.c_double, _vp, _vp, ctypes.c_size_t, _vp]),
}
_typed = None


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


def adamw_state(param: torch.Tensor, bits: int = 32):
    """(m, v) of a parameter before its first step, for adamw_step: fp32 tensors, or with bits=8 a pair (q, scale) each,
    one row of the block format that holds m and sqrt(v)."""
    if bits == 32:
        return tuple(torch.zeros(param.shape, dtype=torch.float32, device=param.device) for _ in range(2))
    if bits != 8:
        raise ValueError("bits must be 32 or 8")
    n = param.numel()
    if n == 0:
        raise ValueError("a parameter of no elements has no 8-bit states")
    return tuple((torch.zeros(fp8_cols(n), dtype=torch.uint8, device=param.device),
                  torch.full((fp8_scale_cols(n),), 127, dtype=torch.uint8, device=param.device)) for _ in range(2))


def _stream_of(tensors, name: str) -> int:
    """Handle of the current stream of a list's device."""
    if not isinstance(tensors, (list, tuple)):
        raise ValueError(f"{name} must be a list or tuple")
    if not tensors:
        return 0
    if not isinstance(tensors[0], torch.Tensor):
        raise ValueError(f"{name}[0] must be a tensor")
    return _current(tensors[0])


def adamw_step(params, grads, m, v, *, lr, step, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
               grad_scale: torch.Tensor | None = None, copies=None, seed: int = 0, stream=None) -> None:
    """One step of Adam with decoupled weight decay, in place, for all tensors of a list.

    params are fp32 or bf16, grads fp32 or bf16 of the same shapes; m[i] and v[i] are what adamw_state gives, and change
    with them.  8-bit states and bf16 parameters are rounded stochastically, with random bits that seed, step and the
    tensor's place in the list determine (taco_optim.h has the formulas); everything else is fp32.

    copies: bf16 tensors (or None) that receive the new fp32 parameters, as quantize_weight takes them.  lr and step
    (from 1 on) are numbers, or tensors of one element on the device (float32, int64), so that a captured graph can be
    replayed with others.  grad_scale: a float32 tensor of one element that multiplies the gradients, such as
    gradient_norm's factor; where it is not finite the step is left out."""
    if stream is not None:
        with _on(stream):
            return adamw_step(params, grads, m, v, lr=lr, step=step, betas=betas, eps=eps, weight_decay=weight_decay,
                              grad_scale=grad_scale, copies=copies, seed=seed)
    return _binding().adamw_step(params, grads, m, v, lr, step, betas[0], betas[1], eps, weight_decay, grad_scale, copies,
                                 seed, _stream_of(params, "params"))


def gradient_norm_workspace_bytes(tensors: int) -> int:
    return int(_lib().taco_gradient_norm_workspace_bytes(tensors))


def gradient_norm(grads, max_norm: float | None = None, *, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """fp32 [2]: the global norm of a list of fp32 or bf16 tensors, and the factor that clips it to max_norm.

    The factor is max_norm / norm where that is below 1, otherwise 1, and NaN where the norm is not finite;
    ``grad_scale=gradient_norm(grads, max_norm)[1:]`` clips adamw_step's gradients without the host."""
    if stream is not None:
        with _on(stream):
            return gradient_norm(grads, max_norm, out=out, workspace=workspace)
    return _binding().gradient_norm(grads, math.inf if max_norm is None else max_norm, out, workspace,
                                    _stream_of(grads, "grads"))
