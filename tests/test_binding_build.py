"""The package without its PyTorch binding, and when that binding is built again (host only)."""
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAME = "mixed_precision_residual_gb300"


@pytest.fixture(scope="module")
def built():
    import __graft_entry__

    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("_far_build_under_test", os.path.join(ROOT, NAME, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("binding", ["missing", "broken"])
def test_the_other_operators_do_not_need_the_binding(built, tmp_path, binding):
    """Only libfar.so beside the Python files, or a binding that cannot be loaded: the package is imported, its ctypes
    entry points work, and a call that needs the binding fails with what to do, each time."""
    there = tmp_path / NAME
    (there / "_build").mkdir(parents=True)
    for f in os.listdir(os.path.join(ROOT, NAME)):
        if f.endswith(".py"):
            shutil.copy(os.path.join(ROOT, NAME, f), there / f)
    shutil.copy(built.LIB, there / "_build" / "libfar.so")
    if binding == "broken":
        (there / "_build" / "_far_torch.so").write_bytes(b"not a shared library")
    program = f"""
import sys
sys.path.insert(0, {str(tmp_path)!r})
import torch
import {NAME} as far
assert far.__file__.startswith({str(tmp_path)!r})
assert far.plan_for_sms(64, 4096, torch.bfloat16, torch.bfloat16, True, 152)["grid"] >= 1
assert far.lib.fused_add_rmsnorm(None, None, None, 1e-6, None, None, 4, 512, 0x22, None) == 3
assert far.lib.gemm_fp8_block(None, 128, None, None, 128, None, 1, None, 128, 0, 128, 128, 2, None) == 0
assert len(far.rope_frequencies(64)[0]) == 32
x = torch.zeros(4, 256)
for _ in range(2):
    try:
        far.quant_block_fp8(x)
    except ImportError as e:
        assert "_far_torch.so" in str(e) and "build" in str(e), e
    else:
        raise AssertionError("a call went through without the binding")
print("fine")
"""
    r = subprocess.run([sys.executable, "-c", program], capture_output=True, text=True, cwd=str(tmp_path))
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr[-2000:]


def test_a_binding_for_another_pytorch_is_built_again(built, tmp_path, monkeypatch):
    """File times alone do not tell: the binding's symbols are those of the PyTorch it was built for."""
    assert not built._binding_stale() and not built._library_stale()
    stamp = tmp_path / "built_for"
    monkeypatch.setattr(built, "BINDING_STAMP", str(stamp))
    assert built._binding_stale() and built._stale()  # nothing known
    stamp.write_text(built._built_for())
    assert not built._stale()
    stamp.write_text(built._built_for().replace("torch ", "torch 0."))
    assert built._binding_stale() and not built._library_stale()
    stamp.write_text(built._built_for().replace("python ", "python 9."))
    assert built._binding_stale()


def test_only_the_binding_is_built_again(built, tmp_path, monkeypatch):
    """A PyTorch upgrade compiles one file; the library is left as it is."""
    ran = []

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def fake(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return Done

    monkeypatch.setattr(built, "BINDING_STAMP", str(tmp_path / "built_for"))
    monkeypatch.setattr(built, "BUILD", str(tmp_path))
    monkeypatch.setattr(built, "BINDING", str(tmp_path / "_far_torch.so"))
    monkeypatch.setattr(built, "_library_stale", lambda: False)
    monkeypatch.setattr(built.subprocess, "run", fake)
    before = os.path.getmtime(built.LIB)
    built.build()
    assert [c[0] for c in ran] == ["g++", "g++"] and os.path.getmtime(built.LIB) == before
    assert not built._binding_stale()
