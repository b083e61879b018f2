"""The weight gradient's choice of kernel (CPU), as its workspace tells it: the 256 x 256 kernel widens whole steps of 64
tokens into it, and is never chosen for so few tokens that it would have none."""
import os

import pytest

import fp8_compression_tensor_taco_amd as taco
from fp8_compression_tensor_taco_amd import build


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(build.LIB_PATH):
        build.build_library(verbose=False)


def widens(t, n, k):
    need = taco.wgrad_fp8_workspace_bytes(t, n, k)
    return need > 0 and need == 2 * (t // 64 * 64) * taco.fp8_cols(k)


@pytest.mark.parametrize("n,k", [(4096, 4096), (65536, 250), (256, 65536), (16000, 16100), (40000, 30000), (65536, 65536)])
def test_few_tokens_take_smaller_tiles(n, k):
    assert not any(widens(t, n, k) for t in range(1, 385))
    assert taco.wgrad_fp8_workspace_bytes(60, n, k) == 0       # 128 x 128 tiles, unsplit: no other takes none


@pytest.mark.parametrize("n,k", [(4096, 4096), (65536, 250), (16000, 16100), (40000, 30000), (65536, 65536)])
def test_many_tokens_are_widened(n, k):
    assert widens(1023, n, k) and widens(1024, n, k)
