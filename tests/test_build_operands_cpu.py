"""The Python module of the binding's quick argument check: built for the torch and the Python at hand."""
import os
import subprocess
import sysconfig

import pytest
import torch

from mixture_experts_ffn_gemm_gb300 import binding as B
from mixture_experts_ffn_gemm_gb300 import build


def test_the_module_s_name_holds_the_versions_it_was_built_with(moelib):
    path = build.operands_path()
    assert os.path.exists(path) and build.build_operands() == path
    assert torch.__version__ in os.path.basename(path)
    assert sysconfig.get_config_var("SOABI") in os.path.basename(path)
    assert os.path.samefile(B._operands_module().__file__, path)


@pytest.mark.parametrize("what", ["torch", "python"])
def test_another_version_s_module_is_neither_taken_nor_up_to_date(moelib, monkeypatch, what):
    ours = build.operands_path()
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "0.0.1+none")
    else:
        config = sysconfig.get_config_var
        monkeypatch.setattr(sysconfig, "get_config_var", lambda n: "cpython-000" if n == "SOABI" else config(n))
    assert build.operands_path() != ours
    compiled = []

    def run(cmd, **_):
        compiled.append(cmd)
        return subprocess.CompletedProcess(cmd, 1, "", "a stand-in for the compiler")

    monkeypatch.setattr(subprocess, "run", run)
    with pytest.raises(RuntimeError, match="operands"):
        build.build_operands()
    assert len(compiled) == 1 and os.path.exists(ours)
