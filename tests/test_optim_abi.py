"""The training step's update: the C ABI's exports, structures and argument checks, and the binding's refusals (CPU; all
fail before any HIP call, so made-up pointers are never used), and the generated code."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import fp8_compression_tensor_taco_amd as taco
from fp8_compression_tensor_taco_amd import _optim, build
from fp8_compression_tensor_taco_amd._optim import AdamwOptions, AdamwTensor, NormTensor

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "taco_optim.h")
A, B, C, D, E, F, G, H = (0x40000000 * k for k in range(1, 9))     # far apart: no two ranges meet
NULL, ALIGN, SHAPE, WORKSPACE, FLAGS, ALIAS = 1, 2, 3, 6, 9, 10


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(build.LIB_PATH):
        build.build_library(verbose=False)
    return _optim._lib()


def test_header_library_and_binding_agree(lib, tmp_path):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(taco_[a-z_0-9]+)\s*\(", text))
    assert names == set(_optim._SIGNATURES)
    for name in names:
        assert hasattr(lib, name), name
    source = tmp_path / "sizes.c"
    source.write_text('#include <stdio.h>\n#include "taco_optim.h"\nint main(void) { printf("%zu %zu %zu %zu %zu", '
                      "sizeof(taco_adamw_tensor_t), sizeof(taco_adamw_options_t), sizeof(taco_norm_tensor_t), "
                      "offsetof(taco_adamw_tensor_t, grad_type), offsetof(taco_adamw_options_t, grad_scale)); return 0; }\n")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", f"-I{os.path.dirname(HEADER)}", str(source), "-o",
                    str(tmp_path / "sizes")], check=True)
    got = subprocess.run([str(tmp_path / "sizes")], check=True, capture_output=True, text=True).stdout.split()
    assert [int(v) for v in got] == [ctypes.sizeof(AdamwTensor), ctypes.sizeof(AdamwOptions), ctypes.sizeof(NormTensor),
                                     AdamwTensor.grad_type.offset, AdamwOptions.grad_scale.offset]


def adamw(lib, tensors, **over):
    o = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1, seed=0)
    o.update(over)
    array = (AdamwTensor * max(1, len(tensors)))(*tensors)
    return lib.taco_adamw_step(array, len(tensors), ctypes.byref(AdamwOptions(**o)), None)


def tensor(**over):
    t = dict(param=A, grad=B, m=C, v=D, m_scale=None, v_scale=None, copy=E, count=1000, param_type=0, grad_type=0)
    t.update(over)
    return AdamwTensor(**t)


def test_adamw_checks(lib):
    assert lib.taco_adamw_step(None, 1, ctypes.byref(AdamwOptions(step=1)), None) == NULL
    assert lib.taco_adamw_step((AdamwTensor * 1)(tensor()), 1, None, None) == NULL
    for name in ("param", "grad", "m", "v"):
        assert adamw(lib, [tensor(**{name: None})]) == NULL
    assert adamw(lib, [tensor(m_scale=F)]) == adamw(lib, [tensor(v_scale=F)]) == NULL
    assert adamw(lib, [tensor(param_type=1)]) == NULL                   # no copy of a bf16 parameter
    for count in (-1, (1 << 34) + 1):
        assert adamw(lib, [tensor(count=count)]) == SHAPE
    for bad in (dict(lr=float("nan")), dict(lr=float("inf")), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0),
                dict(beta2=float("nan")), dict(eps=-1e-8), dict(eps=float("inf")), dict(weight_decay=float("nan")),
                dict(step=0), dict(step=-5)):
        assert adamw(lib, [tensor()], **bad) == SHAPE
    for bad in (dict(param_type=2), dict(grad_type=-1)):
        assert adamw(lib, [tensor(**bad)]) == FLAGS
    for name, p in (("param", A + 2), ("grad", B + 1), ("m", C + 2), ("v", D + 1), ("copy", E + 1)):
        assert adamw(lib, [tensor(**{name: p})]) == ALIGN
    for name, p in (("m", C + 8), ("v", D + 4), ("m_scale", F + 2), ("v_scale", G + 1)):
        assert adamw(lib, [tensor(**{"m_scale": F, "v_scale": G, name: p})]) == ALIGN
    assert adamw(lib, [tensor()], lr_device=H + 2) == adamw(lib, [tensor()], step_device=H + 4) == ALIGN
    assert adamw(lib, [tensor()], grad_scale=H + 1) == ALIGN
    assert lib.taco_adamw_step((AdamwTensor * 1)(tensor()), (1 << 20) + 1, ctypes.byref(AdamwOptions(step=1)), None) == SHAPE


def test_adamw_aliases(lib):
    for over in (dict(param=B), dict(m=A), dict(v=C + 3996), dict(copy=A + 3998), dict(copy=B), dict(m=B - 3996),
                 dict(m_scale=F, v_scale=F), dict(m_scale=F, v_scale=C + 1020), dict(grad=D)):
        assert adamw(lib, [tensor(**over)]) == ALIAS, over
    second = dict(param=A + 0x100000, m=C + 0x100000, v=D + 0x100000, copy=E + 0x100000)
    for over in (dict(param=A), dict(m=C + 3996), dict(v=A + 2000), dict(copy=B), dict(grad=E), dict(grad=C + 3996)):
        assert adamw(lib, [tensor(), tensor(**{**second, **over})]) == ALIAS, over
        assert adamw(lib, [tensor(**{**second, **over}), tensor()]) == ALIAS, over
    for name in ("lr_device", "step_device", "grad_scale"):
        assert adamw(lib, [tensor()], **{name: A + 8}) == adamw(lib, [tensor()], **{name: D}) == ALIAS


def test_norm_checks(lib):
    assert lib.taco_gradient_norm_workspace_bytes(0) == 0 and lib.taco_gradient_norm_workspace_bytes(-1) == 0
    assert lib.taco_gradient_norm_workspace_bytes(64) == 8192 and taco.gradient_norm_workspace_bytes(65) == 16384

    def f(tensors=None, count=1, max_norm=1.0, out=C, ws=D, size=8192):
        array = (NormTensor * 1)(NormTensor(**{"data": A, "count": 1000, "type": 0, **(tensors or {})}))
        return lib.taco_gradient_norm(array, count, max_norm, out, ws, size, None)
    assert f(out=None) == f(ws=None) == f(dict(data=None)) == NULL
    assert lib.taco_gradient_norm(None, 1, 1.0, C, D, 8192, None) == NULL
    assert f(count=-1) == f(dict(count=-1)) == f(dict(count=(1 << 34) + 1)) == SHAPE
    assert f(max_norm=0.0) == f(max_norm=-1.0) == f(max_norm=float("nan")) == SHAPE
    assert f(dict(type=3)) == FLAGS
    assert f(dict(data=A + 2)) == f(dict(data=A + 1, type=1)) == f(out=C + 2) == f(ws=D + 128) == ALIGN
    assert f(size=8191) == WORKSPACE
    assert f(out=A + 3996) == f(ws=A) == f(out=D + 8) == ALIAS


def test_binding_refusals():
    p = torch.zeros(4)
    m, v = taco.adamw_state(p)
    for bad in (lambda: taco.adamw_step([p], [p], [m], [v], lr=0.1, step=1), lambda: taco.gradient_norm([p])):
        with pytest.raises(ValueError, match="GPU"):
            bad()
    for bad in (lambda: taco.adamw_step(p, [p], [m], [v], lr=0.1, step=1), lambda: taco.adamw_step([1], [p], [m], [v], lr=0.1, step=1),
                lambda: taco.adamw_step([p], [], [m], [v], lr=0.1, step=1), lambda: taco.gradient_norm([]),
                lambda: taco.gradient_norm(p), lambda: taco.gradient_norm([None]), lambda: taco.adamw_state(p, 16),
                lambda: taco.adamw_state(p[:0], 8)):
        with pytest.raises(ValueError):
            bad()
    assert taco.adamw_step([], [], [], [], lr=0.1, step=1) is None


def test_states():
    p = torch.zeros(3, 100, dtype=torch.bfloat16)
    m, v = taco.adamw_state(p)
    assert m.shape == v.shape == (3, 100) and m.dtype == v.dtype == torch.float32 and m.data_ptr() != v.data_ptr()
    (mq, ms), (vq, vs) = taco.adamw_state(p, 8)
    assert mq.shape == vq.shape == (384,) and ms.shape == vs.shape == (4,) and (ms == 127).all() and not mq.any()


def test_generated_code(tmp_path):
    out = tmp_path / "optim.s"
    res = subprocess.run([build.hipcc(), *build.compile_flags(), "--cuda-device-only", "-S", *build.OPTIM_SOURCES, "-o", str(out),
                          "-Rpass-analysis=kernel-resource-usage"], capture_output=True, text=True, check=True)
    lines = [line.split(";")[0] for line in out.read_text().splitlines()]
    for bad in (r"s_swappc_b64", r"s_setpc_b64", r"\bflat_(load|store)", r"v_pk_(add|mul|fma)_f32", r"\bscratch_(load|store)"):
        assert not any(re.search(bad, line) for line in lines), bad
    assert re.findall(r"VGPRs Spill: (\d+)", res.stderr) and not any(int(n) for n in re.findall(r"VGPRs Spill: (\d+)", res.stderr))
