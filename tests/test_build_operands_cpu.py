"""The Python module of the binding's quick argument check: built for the torch and the Python at hand."""
import os
import subprocess
import sysconfig

import pytest
import torch

from mixture_experts_ffn_gemm_gb300 import binding as B
from mixture_experts_ffn_gemm_gb300 import build
from test_products_cpu import OnDevice


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


@pytest.mark.parametrize("failure", ["no compiler", "no headers"])
def test_the_library_is_built_without_a_cpp_compiler(moelib, monkeypatch, tmp_path, failure):
    """Without g++ (or torch's or Python's headers) the build warns, an older module goes, and the binding makes
    the same checks by itself."""
    old = tmp_path / "_operands.old.so"
    old.write_bytes(b"of older sources")
    os.utime(old, (1, 1))
    monkeypatch.setattr(build, "operands_path", lambda: str(old))

    def run(cmd, **_):
        if failure == "no compiler":
            raise FileNotFoundError("g++")
        return subprocess.CompletedProcess(cmd, 1, "", "Python.h: No such file or directory")

    monkeypatch.setattr(subprocess, "run", run)
    with pytest.warns(RuntimeWarning, match="quick argument check"):
        assert build.build() == build.LIB
    assert not old.exists()
    B._operands_module.cache_clear()
    try:
        assert B._operands_module() is None
        made = []

        class Library:
            def __getattr__(self, name):
                return lambda *a: made.append(name) or B.MOE_OK

        monkeypatch.setattr(B, "_lib", Library())
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
        z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype).as_subclass(OnDevice)  # noqa: E731
        cfg = B.make_product_config(4, 2, 8, 16)
        good = [z(3, dtype=torch.int32), z(4, 16), z(2, 8, 16), z(4, 8), z(256, dtype=torch.uint8)]
        B.moe_grouped_product(cfg, *good, stream=0)
        assert made == ["moe_grouped_product"]
        for i in range(4):
            with pytest.raises(ValueError):
                B.moe_grouped_product(cfg, *good[:i], z(1), *good[i + 1:], stream=0)
        assert len(made) == 1
    finally:
        B._operands_module.cache_clear()
