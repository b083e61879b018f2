"""What a call of the 8-bit linear layer says where its binding is missing or does not load (CPU)."""
import importlib.abc
import os
import sys

import pytest
import torch

import fp8_compression_tensor_taco_amd as taco
from fp8_compression_tensor_taco_amd import _linear, build


class Refusing(importlib.abc.MetaPathFinder):
    def find_spec(self, name, path, target=None):
        if name.endswith("._linear_binding"):
            raise ImportError("Python version mismatch")
        return None


@pytest.fixture
def unloadable(monkeypatch):
    if not os.path.exists(build.LIB_PATH):
        build.build_library(verbose=False)
    monkeypatch.setattr(_linear, "_native", None)
    monkeypatch.delattr(taco, "_linear_binding", raising=False)
    monkeypatch.delitem(sys.modules, f"{taco.__name__}._linear_binding", raising=False)
    monkeypatch.setattr(sys, "meta_path", [Refusing(), *sys.meta_path])


def call():
    taco.quantize_rows(torch.zeros(1, 128, dtype=torch.bfloat16))


def test_a_binding_that_does_not_load(unloadable, tmp_path, monkeypatch):
    there = tmp_path / "_linear_binding.so"
    there.write_text("")
    monkeypatch.setattr(_linear, "BINDING_PATH", str(there), raising=False)
    with pytest.raises(ImportError, match="another Python or torch.*Python version mismatch") as e:
        call()
    assert "not built" not in str(e.value)


def test_a_binding_that_is_not_there(unloadable, tmp_path, monkeypatch):
    monkeypatch.setattr(_linear, "BINDING_PATH", str(tmp_path / "absent.so"), raising=False)
    with pytest.raises(ImportError, match="not built"):
        call()
