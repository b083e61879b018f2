"""Build libtaco.so (HIP, gfx950) in-tree with hipcc, and the torch binding of its 8-bit linear layer.

Usage: ``python -m fp8_compression_tensor_taco_amd.build`` or ``build_library()``.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import warnings

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libtaco.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
SOURCES = [os.path.join(CSRC, "taco.hip")]                  # the compression calls (include/taco.h)
LINEAR_SOURCES = [os.path.join(CSRC, "rowops.hip"),         # the 8-bit linear layer (include/taco_linear.h)
                  os.path.join(CSRC, "matmul.hip")]
BINDING_SOURCE = os.path.join(CSRC, "linear_binding.cpp")   # host code only
BINDING_PATH = os.path.join(PKG_DIR, "_linear_binding.so")
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (set HIPCC or install ROCm)")


def compile_flags() -> list[str]:
    return [
        f"--offload-arch={ARCH}",
        "-O3",
        "-std=c++17",
        "-fPIC",
        "-Wall",
        # packed fp32 VALU ops stay off on this target
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        # MFMA results in VGPRs (no v_accvgpr_read copies before the VALU epilogue)
        "-mllvm", "-amdgpu-mfma-vgpr-form=1",
        f"-I{INCLUDE}",
    ]


def build_library(verbose: bool = True, binding_required: bool = False) -> str:
    """Compile every HIP source into ``libtaco.so`` next to this file, and the binding; returns the library's path.

    The binding needs a host compiler and the headers of Python and torch, which
    the library and the compression calls do without.  Where it cannot be built a
    warning says why, and an older one, which may not fit the new library, is
    removed; with ``binding_required`` the error is raised."""
    tmp = LIB_PATH + ".tmp"
    cmd = [hipcc(), *compile_flags(), "-shared", "-parallel-jobs=3", *SOURCES, *LINEAR_SOURCES, "-o", tmp]
    _run(cmd, verbose)
    os.replace(tmp, LIB_PATH)
    try:
        build_binding(verbose)
    except (ImportError, OSError, RuntimeError) as e:
        if os.path.exists(BINDING_PATH):
            os.remove(BINDING_PATH)
        if binding_required:
            raise
        warnings.warn(f"the binding of the 8-bit linear layer was not built ({e}); the compression calls work without it")
    return LIB_PATH


def build_binding(verbose: bool = True) -> str:
    """Compile ``_linear_binding.so`` against torch and the library beside it; returns its path."""
    import sysconfig

    from torch.utils import cpp_extension

    tmp = BINDING_PATH + ".tmp"
    includes = [INCLUDE, sysconfig.get_paths()["include"], *cpp_extension.include_paths()]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-Wall",
           *(f"-I{i}" for i in includes), BINDING_SOURCE, "-o", tmp, f"-L{PKG_DIR}", f"-l:{LIB_NAME}",
           "-Wl,-rpath,$ORIGIN", *(f"-L{i}" for i in cpp_extension.library_paths()), "-ltorch_python", "-ltorch_cpu",
           "-lc10"]
    _run(cmd, verbose)
    os.replace(tmp, BINDING_PATH)
    return BINDING_PATH


def _run(cmd: list[str], verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed with exit code {res.returncode}")


def build_asm(out_path: str) -> None:
    """Device assembly of the library (for inspection of the generated gfx950 code)."""
    cmd = [hipcc(), *compile_flags(), "--cuda-device-only", "-S", *SOURCES, "-o", out_path]
    subprocess.run(cmd, check=True)


if __name__ == "__main__":
    print(build_library())
