"""The build and the import: both libraries from one call, and the package
without the native binding."""
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "sparse_moe_layer_expert_b200")


@pytest.fixture
def build(monkeypatch, tmp_path):
    """build.py with the native binding's place under tmp_path and a compiler that only writes its output."""
    spec = importlib.util.spec_from_file_location("_moe_build_test", os.path.join(PKG, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.NATIVE = str(tmp_path / "_native.so")
    mod.runs = []

    def run(cmd, check):
        mod.runs.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "wb") as f:
            f.write(b"".join(c.encode() + b"\0" for c in cmd))

    monkeypatch.setattr(mod.subprocess, "run", run)
    return mod


def test_one_call_builds_both(build):
    build.build()
    assert os.path.exists(build.NATIVE) and len(build.runs) == 1
    build.build()
    assert len(build.runs) == 1  # up to date


def test_binding_is_made_anew_for_another_torch_or_python(build, monkeypatch):
    import importlib.metadata
    import sysconfig
    build.build()
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "9.9.9")
    build.build()
    build.build()
    assert len(build.runs) == 2
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-999")
    build.build()
    assert len(build.runs) == 3


def test_the_built_binding_says_what_it_is_for():
    import torch
    from sparse_moe_layer_expert_b200 import _native
    assert _native.__doc__ and torch.__version__.split("+")[0] in _native.__doc__


CALLS = """
import sys, torch
import sparse_moe_layer_expert_b200 as m
assert m.__file__.startswith(sys.argv[1])
cfg = m.config(512, 256, 16, 4)
assert m.moe_router_splits(cfg, 64) >= 1 and m.moe_workspace_size(cfg, 64) > 0
x = torch.zeros((2, 256), dtype=torch.bfloat16)
for call in (lambda: m.fp8_add_rmsnorm_quant_1x128(x), lambda: m.add_rmsnorm_backward(x, x, x),
             lambda: m.moe_balance_loss(cfg, x, x, x), lambda: m.moe_router_backward(cfg, x, x)):
    try:
        call()
    except ImportError as e:
        assert "build.py" in str(e), e
    else:
        raise AssertionError("no ImportError")
"""


@pytest.mark.parametrize("native", [None, b"not a library"])
def test_package_without_the_native_binding(tmp_path, native):
    """Older calls do not need it; the operators that do say how to build it."""
    dst = tmp_path / "sparse_moe_layer_expert_b200"
    dst.mkdir()
    for f in os.listdir(PKG):
        if f.endswith(".py") or f == "libmoefp8.so":
            shutil.copy2(os.path.join(PKG, f), dst / f)
    if native is not None:
        (dst / "_native.so").write_bytes(native)
    r = subprocess.run([sys.executable, "-c", CALLS, str(tmp_path)], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-1500:]
