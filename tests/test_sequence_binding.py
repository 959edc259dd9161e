"""The sequence operators' compiled binding stands apart from the library."""
import os
import subprocess
import sys

import pytest

import sparse_spd_selected_amd as ssa
from conftest import ROOT
from sparse_spd_selected_amd import buildlib, sequence


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssa.LIB_PATH):
        ssa.build()
    return ssa.lib()


def test_the_library_loads_without_the_binding(lib):
    """Everything else of the package needs ctypes alone."""
    code = """
import sys
sys.modules["sparse_spd_selected_amd._seqbind"] = None  # importing it fails
import torch
import sparse_spd_selected_amd as ssa
assert ssa.lib().selinv_strerror(0)
try:
    ssa.short_conv(torch.zeros(1, 1, 4), torch.zeros(4, 4))
except ImportError as e:
    print("refused:", e)
"""
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert out.returncode == 0, out.stderr
    assert "refused: the binding of the sequence operators" in out.stdout


def test_a_binding_that_does_not_compile(tmp_path, monkeypatch):
    """It is reported, and the library is there all the same."""
    out = str(tmp_path / "lib.so")

    def fails():
        raise RuntimeError("compile failed: binding")

    monkeypatch.setattr(buildlib, "LIB", out)
    monkeypatch.setattr(buildlib, "SOURCES", ["seq_abi.cpp"])
    monkeypatch.setattr(buildlib, "build_binding", fails)
    with pytest.raises(RuntimeError, match="binding"):
        buildlib.build(out=out, build_dir=str(tmp_path))
    assert os.path.exists(out)


def test_a_new_library_is_bound_anew(lib, monkeypatch):
    assert sequence._binding() is sequence._bound
    monkeypatch.setattr(buildlib, "build", lambda: ssa.LIB_PATH)
    ssa.build()
    assert sequence._bound is None
    assert sequence._binding() is sequence._bound
