"""The product with an epilogue and the nonlinearity's gradient: sizes and argument checks of the C ABI and the binding
(CPU), all of which fail before any HIP call, so made-up pointers are never used; and the generated code of the large
product's kernels, which write their matrix instructions as inline assembly."""
import os
import re
import subprocess

import pytest
import torch

import fp8_compression_tensor_taco_amd as taco
from fp8_compression_tensor_taco_amd import _linear, build
from test_linear_matrix_asm import asm, instructions, operands, registers  # noqa: F401

A, B, C, D, E, F, G, H, I = (0x40000000 * k for k in range(1, 10))     # far apart: no two ranges meet
W = 0x400000000
OK, NULL, ALIGN, SHAPE, WORKSPACE, FLAGS, ALIAS = 0, 1, 2, 3, 6, 9, 10


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(build.LIB_PATH):
        build.build_library(verbose=False)
    return _linear._lib()


def test_workspace_sizes(lib):
    for m, n, k in ((4, 64, 128), (300, 512, 8192), (777, 1601, 1600), (4096, 4096, 4096)):
        assert lib.taco_linear_fp8_workspace_bytes(m, n, k) == lib.taco_matmul_fp8_workspace_bytes(m, n, k)
    assert lib.taco_linear_quantize_workspace_bytes(4, 64, 4096) == 4 * 4 * 64      # the sums of few rows and columns
    for m, n, k in ((4, 64, 128), (8, 16384, 4096), (777, 1601, 1600), (4096, 4096, 4096)):
        assert lib.taco_linear_quantize_workspace_bytes(m, n, k) == 0
    assert lib.taco_linear_quantize_workspace_bytes(300, 512, 8192) == lib.taco_matmul_fp8_workspace_bytes(300, 512, 8192)
    assert lib.taco_linear_quantize_workspace_bytes(0, 64, 128) == lib.taco_linear_fp8_workspace_bytes(4, 0, 128) == 0
    assert lib.taco_activation_backward_workspace_bytes(16, 4096) == 0
    assert lib.taco_activation_backward_workspace_bytes(17, 4096) == 2 * 4096 * 4       # groups of sixteen rows
    assert lib.taco_activation_backward_workspace_bytes(0, 5) == 0
    assert taco.linear_quantize_workspace_bytes(4, 64, 4096) == 1024
    assert taco.linear_fp8_workspace_bytes(4, 64, 128) == 0 and taco.activation_backward_workspace_bytes(17, 4096) == 32768


def test_linear_checks(lib):
    def f(qa=A, sa=B, qb=C, sb=D, bias=E, residual=F, act=2, m=4, n=64, k=128, y=G, ws=W, size=1 << 20):
        return lib.taco_linear_fp8(qa, sa, qb, sb, bias, residual, act, m, n, k, y, ws, size, None)
    for name in ("qa", "sa", "qb", "sb", "y"):
        assert f(**{name: None}) == NULL
    for m, n, k in ((0, 64, 128), (4, 0, 128), (4, 64, 0), (1 << 24, 1 << 11, 128), (4, 64, (1 << 22) + 1)):
        assert f(m=m, n=n, k=k) == SHAPE
    assert f(act=-1) == f(act=5) == FLAGS
    for name, p in (("qa", A + 8), ("sa", B + 1), ("qb", C + 8), ("sb", D + 2), ("bias", E + 2), ("residual", F + 8), ("y", G + 2),
                    ("ws", W + 16)):
        assert f(**{name: p}) == ALIGN
    assert f(m=300, n=512, k=8192, ws=None, size=0) == f(m=300, n=512, k=8192, size=1000) == WORKSPACE
    for y in (A, B, C, D, E, F, F + 496, E + 112, W):
        assert f(y=y) == ALIAS
    assert f(ws=F) == f(ws=E) == f(ws=A) == ALIAS


def test_quantize_checks(lib):
    def f(qa=A, sa=B, qb=C, sb=D, bias=E, act=2, m=4, n=64, k=128, hq=F, hs=G, cq=H, cs=I, ws=W, size=1 << 20):
        return lib.taco_linear_quantize(qa, sa, qb, sb, bias, act, m, n, k, hq, hs, cq, cs, ws, size, None)
    for name in ("qa", "sa", "qb", "sb", "hq", "hs", "cq", "cs"):
        assert f(**{name: None}) == NULL
    for m, n, k in ((0, 64, 128), (4, 0, 128), (4, 64, 0), (1 << 24, 1 << 10, 1 << 11), (4, 64, (1 << 22) + 1),
                    (1 << 24, 1025, 128)):                        # 2^24 x 1152 padded codes
        assert f(m=m, n=n, k=k) == SHAPE
    assert f(act=-1) == f(act=5) == FLAGS
    for name, p in (("qa", A + 8), ("sa", B + 1), ("qb", C + 8), ("sb", D + 2), ("bias", E + 2), ("hq", F + 8), ("hs", G + 2),
                    ("cq", H + 4), ("cs", I + 1), ("ws", W + 16)):
        assert f(**{name: p}) == ALIGN
    assert f(k=4096, ws=None, size=0) == f(k=4096, size=1023) == WORKSPACE
    for name in ("hq", "hs", "cq", "cs", "ws"):
        for p in (A, B, C, D, E):
            assert f(**{name: p}) == ALIAS
    assert f(hs=F) == f(cq=F + 384) == f(cs=G) == f(ws=H) == f(ws=I) == ALIAS


def test_gradient_checks(lib):
    def f(dh=A, cq=B, cs=C, act=2, tokens=40, cols=128, dt=D, dq=E, ds=F, dbias=G, ws=W, size=1 << 20):
        return lib.taco_activation_backward(dh, cq, cs, act, tokens, cols, dt, dq, ds, dbias, ws, size, None)
    for name in ("dh", "cq", "cs", "dt", "dq", "ds"):
        assert f(**{name: None}) == NULL
    assert f(act=0) == f(act=0, cq=None) == f(act=0, cq=None, cs=None) == NULL         # dt is dh
    assert f(act=0, cq=None, cs=None, dt=None, dq=None, ds=None, dbias=None) == NULL   # nothing to do
    for tokens, cols in ((0, 128), (40, 0), ((1 << 24) + 1, 1), (1, (1 << 22) + 1), (1 << 24, 1 << 12)):
        assert f(tokens=tokens, cols=cols) == SHAPE
    assert f(act=-1) == f(act=5) == FLAGS
    for name, p in (("dh", A + 2), ("cq", B + 8), ("cs", C + 2), ("dt", D + 8), ("dq", E + 8), ("ds", F + 1), ("dbias", G + 2),
                    ("ws", W + 128)):
        assert f(**{name: p}) == ALIGN
    assert f(ws=None, size=0) == f(size=1000) == WORKSPACE
    for name in ("dt", "dq", "ds", "dbias", "ws"):
        for p in (A, B, C):
            assert f(**{name: p}) == ALIAS
    assert f(dq=D) == f(ds=E) == f(dbias=F) == f(ws=G) == ALIAS


def test_binding_refusals():
    q, s = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8)
    dh = torch.zeros(4, 128, dtype=torch.bfloat16)
    for call in (lambda **k: taco.linear_fp8(q, s, q, s, **k), lambda **k: taco.linear_quantize(q, s, q, s, **k),
                 lambda activation: taco.activation_backward(dh, q, s, activation)):
        with pytest.raises(ValueError, match="GPU"):
            call(activation="gelu")
        for name in ("tanh", "", "GELU", "none"):
            with pytest.raises(ValueError, match="activation must be"):
                call(activation=name)
    with pytest.raises(ValueError, match="uint8"):
        taco.linear_fp8(dh, s, q, s)
    with pytest.raises(ValueError, match="bfloat16"):
        taco.activation_backward(q, q, s, "relu")


def test_no_scratch(tmp_path):
    """No kernel keeps anything in scratch memory: accumulators there would be read and written around each instruction."""
    for source in (s for s in build.LINEAR_SOURCES if s.endswith("matmul.hip")):
        res = subprocess.run([build.hipcc(), *build.compile_flags(), "--cuda-device-only", "-S", source, "-o", str(tmp_path / "x.s"),
                              "-Rpass-analysis=kernel-resource-usage"], capture_output=True, text=True, check=True)
        sizes = re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", res.stderr)
        assert len(sizes) >= 10 and not any(int(n) for n in sizes)


LARGE = [f"matmul_large_kernelINS_{kind}" for kind in ("9LinearOut", "9BlocksOut")]


@pytest.mark.parametrize("kernel", LARGE)
def test_operands_and_sums_of_the_large_product(asm, kernel):  # noqa: F811
    """As of the plain one: operands from LDS reads, sums in the accumulation registers and read after the wait."""
    code = instructions(asm, kernel, every=True)
    at = [i for i, line in enumerate(code) if line.startswith("v_mfma")]
    assert len(at) >= 128
    for i in at:
        assert registers(operands(code[i])[0], "a"), code[i]
        reads = set().union(*(registers(o, "v") for o in operands(code[i])[1:]))
        for line in code[max(0, i - 4):i]:
            if line.startswith("v_") and not line.startswith("v_mfma"):
                assert not reads & registers(operands(line)[0], "v"), (line, code[i])
    waited, reads = False, 0
    for line in code[at[-1] + 1:]:
        waited = waited or line == "s_nop 15"
        if not line.startswith("v_mfma") and any(registers(o, "a") for o in operands(line)[1:]):
            reads += 1
            assert waited, line
    assert reads >= 64
