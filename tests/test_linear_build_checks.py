"""Checks on the generated gfx950 code of the 8-bit linear layer (CPU: hipcc
cross-compiles the device code here; nothing runs on a GPU).

* m0 is written only by the direct-to-LDS copies' inline assembly, whose m0
  clobber clang may not honour.
* No kernel calls a function, and none loads through flat addresses: those
  count as LDS operations too, and every wait for LDS reads would wait for
  them.
* The product kernels spill nothing: a reload from scratch waits for every
  load in flight.
* No packed fp32 instruction.
"""
import os
import re
import subprocess

import pytest

from fp8_compression_tensor_taco_amd import build


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    try:
        hipcc = build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    found = {}
    for source in build.LINEAR_SOURCES:
        out = str(tmp_path_factory.mktemp("asm") / "code.s")
        res = subprocess.run([hipcc, *build.compile_flags(), "--cuda-device-only", "-S", source, "-o", out,
                              "-Rpass-analysis=kernel-resource-usage"], capture_output=True, text=True, timeout=600)
        assert res.returncode == 0, res.stderr[-2000:]
        found[os.path.basename(source)] = (open(out).read(), res.stderr)
    return found


def test_m0_is_only_written_by_the_copy_asm(code):
    for name, (asm, _) in code.items():
        inside, outside = False, []
        for line in asm.splitlines():
            if "ASMSTART" in line:
                inside = True
            elif "ASMEND" in line:
                inside = False
            elif not inside and re.search(r"\bm0\b", line.split(";")[0]):
                outside.append(line.strip())
        assert not outside, (name, outside[:5])
    assert "global_load_lds_dwordx4" in code["matmul.hip"][0]
    assert "v_mfma_scale_f32_16x16x128_f8f6f4" in code["matmul.hip"][0]
    assert "ds_read_b64_tr_b16" in code["matmul.hip"][0]


def test_no_calls_no_flat_loads_no_packed_fp32(code):
    for name, (asm, _) in code.items():
        lines = [line.split(";")[0] for line in asm.splitlines()]
        for bad in (r"s_swappc_b64", r"s_setpc_b64", r"\bflat_(load|store)", r"v_pk_(add|mul|fma)_f32"):
            assert not any(re.search(bad, line) for line in lines), (name, bad)


def test_product_kernels_do_not_spill(code):
    name, spills = None, {}
    for line in code["matmul.hip"][1].splitlines():
        m = re.search(r"Function Name: (\S+)", line)
        name = m.group(1) if m else name
        m = re.search(r"VGPRs Spill: (\d+)", line)
        if m and name:
            spills[name] = int(m.group(1))
    assert sum("matmul_" in k for k in spills) >= 7 and sum("wgrad_" in k for k in spills) >= 8, sorted(spills)
    assert not any(spills.values()), {k: v for k, v in spills.items() if v}
