"""The compiled calls belong to the Python and torch they were built against (host only)."""

import pytest
import torch

from block_diffusion_speculative_gemm_b200 import build as B
from block_diffusion_speculative_gemm_b200 import dflash as D


def test_the_built_module_is_of_this_python_and_torch(monkeypatch):
    runs = []
    monkeypatch.setattr(B, "_run", lambda cmd, verbose: runs.append(cmd))
    assert B.build_binding() == B.BINDING and not runs
    assert B.binding_current()


def test_another_torch_means_another_build(monkeypatch, tmp_path):
    runs = []

    def run(cmd, verbose):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "wb").close()

    lib = tmp_path / "_calls.so"
    lib.write_bytes(open(B.BINDING, "rb").read())
    monkeypatch.setattr(B, "_run", run)
    monkeypatch.setattr(B, "BINDING", str(lib))
    assert B.build_binding() == str(lib) and not runs
    monkeypatch.setattr(torch, "__version__", "2.99.0+cu999")
    assert not B.binding_current()
    B.build_binding()
    assert len(runs) == 1


def test_a_module_of_another_torch_is_not_loaded(monkeypatch):
    monkeypatch.setattr(torch, "__version__", "2.99.0+cu999")
    monkeypatch.setattr(D, "_calls", None)
    with pytest.raises(RuntimeError, match="built"):
        D.calls()
