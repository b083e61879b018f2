"""The two kernels that write their matrix instructions as inline assembly, which the compiler takes for ordinary
code: it must neither write an operand with a vector instruction beside them nor read a sum before it is there."""
import re
import subprocess

import pytest

from fp8_compression_tensor_taco_amd import build

KERNELS = {"matmul_large_kernel": "v_mfma_scale_f32_16x16x128_f8f6f4", "wgrad_copies_kernel": "v_mfma_f32_16x16x32_bf16"}


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    out = tmp_path_factory.mktemp("asm") / "matmul.s"
    source = [s for s in build.LINEAR_SOURCES if s.endswith("matmul.hip")]
    subprocess.run([build.hipcc(), *build.compile_flags(), "--cuda-device-only", "-S", *source, "-o", str(out)], check=True,
                   capture_output=True)
    return out.read_text()


def instructions(asm, kernel, every=False):
    body = re.search(rf"^_ZN\w*{kernel}\w*:(.*?)^\.Lfunc_end", asm, re.M | re.S).group(1)
    lines = (line.split(";")[0].strip() for line in body.splitlines())
    return [line for line in lines if re.match(r"[vsdgb]\w*_\w+", line) or every and re.match(r"\.LBB\w+:", line)]


def registers(operand, bank):
    m = re.fullmatch(rf"{bank}(?:(\d+)|\[(\d+):(\d+)\])", operand.strip())
    if not m:
        return set()
    return {int(m[1])} if m[1] else set(range(int(m[2]), int(m[3]) + 1))


def operands(line):
    return re.sub(r"op_sel\S*|offset\S*", "", line.split(None, 1)[1]).split(",") if " " in line or "\t" in line else []


@pytest.mark.parametrize("kernel", KERNELS)
def test_operands_come_from_lds_reads(asm, kernel):
    """No vector instruction among the matrix instructions, or up to four before one, writes what it reads."""
    code = instructions(asm, kernel)
    at = [i for i, line in enumerate(code) if line.startswith(KERNELS[kernel])]
    assert len(at) >= 128
    for i in at:
        assert registers(operands(code[i])[0], "a"), code[i]               # sums in the accumulation registers
        reads = set().union(*(registers(o, "v") for o in operands(code[i])[1:]))
        for line in code[max(0, i - 4):i]:
            if line.startswith("v_") and not line.startswith("v_mfma"):
                assert not reads & registers(operands(line)[0], "v"), (line, code[i])


@pytest.mark.parametrize("kernel", KERNELS)
def test_sums_are_read_after_the_wait(asm, kernel):
    code = instructions(asm, kernel, every=True)
    last = max(i for i, line in enumerate(code) if line.startswith(KERNELS[kernel]))
    waited, reads = False, 0
    for line in code[last + 1:]:
        waited = waited or line == "s_nop 15"
        if not line.startswith("v_mfma") and any(registers(o, "a") for o in operands(line)[1:]):
            reads += 1
            assert waited, line
    assert reads >= 64


@pytest.mark.parametrize("kernel", KERNELS)
def test_nothing_reads_sums_in_the_loops(asm, kernel):
    """A basic block with matrix instructions touches the accumulation registers with nothing else."""
    block, matrix, other = [], 0, 0
    for line in instructions(asm, kernel, every=True) + ["label:"]:
        if line.endswith(":"):
            if matrix >= 64:
                assert not other, block
            block, matrix, other = [], 0, 0
        elif line.startswith("v_mfma"):
            matrix += 1
        elif matrix and not line.startswith("v_accvgpr_write") and any(registers(o, "a") for o in operands(line)):
            other += 1
            block.append(line)
