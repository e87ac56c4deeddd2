"""The package and its build without PyTorch, and a binding that no longer fits the PyTorch that runs."""
import os
import subprocess
import sys

import pytest

from int8_row_absmax_b200 import attn
from int8_row_absmax_b200 import build as blbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


def test_the_package_is_imported_without_pytorch():
    blbuild.build()
    r = python("import sys; sys.modules['torch'] = None\n"
               "import int8_row_absmax_b200 as bl\n"
               "lib = bl.load()\n"
               "assert lib.bl_pack5_ldp(5) == 16 and lib.bl_attention_backward_workspace_size(None) == 0")
    assert r.returncode == 0, r.stderr
    r = python("import sys, int8_row_absmax_b200\nassert 'torch' not in sys.modules")
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("lacking", ["torch", "header"])
def test_the_library_is_built_without_pytorch_or_its_headers(monkeypatch, capsys, lacking):
    if lacking == "torch":
        monkeypatch.setattr(blbuild.importlib.util, "find_spec", lambda name: None)
    else:
        monkeypatch.setattr(blbuild.sysconfig, "get_paths", lambda: {"include": "/nowhere"})
    ran = []
    monkeypatch.setattr(blbuild, "run", lambda cmd, verbose=False: ran.append(cmd))
    monkeypatch.setattr(blbuild.os, "replace", lambda a, b: None)
    assert blbuild.build(force=True) == blbuild.OUT
    assert len(ran) == 1 and "nvcc" in ran[0][0]
    assert "not built" in capsys.readouterr().err


def test_a_binding_that_fails_to_build_says_that_the_library_is_there(monkeypatch):
    def run(cmd, verbose=False):
        if "nvcc" not in cmd[0]:
            raise RuntimeError("g++ failed")
    monkeypatch.setattr(blbuild, "run", run)
    monkeypatch.setattr(blbuild.os, "replace", lambda a, b: None)
    with pytest.raises(RuntimeError, match="is built, its tensor binding is not: g"):
        blbuild.build(force=True)


def test_a_binding_for_another_pytorch_is_built_again_and_not_loaded(monkeypatch):
    blbuild.build()
    assert blbuild.binding_fits() and blbuild.up_to_date(blbuild.BINDING, blbuild.binding_sources())
    real = blbuild.importlib.metadata.version
    monkeypatch.setattr(blbuild.importlib.metadata, "version", lambda name: real(name) + ".1")
    assert not blbuild.binding_fits()
    ran = []
    monkeypatch.setattr(blbuild, "run", lambda cmd, verbose=False: ran.append(cmd))
    monkeypatch.setattr(blbuild.os, "replace", lambda a, b: None)
    blbuild.build()
    assert len(ran) == 1 and "nvcc" not in ran[0][0]                     # the binding alone
    monkeypatch.setattr(attn, "_binding", None)
    monkeypatch.setattr(attn, "_torch", lambda: None)
    with pytest.raises(RuntimeError, match="another PyTorch"):
        attn._native()


def test_the_binding_calls_the_library_that_was_loaded(tmp_path):
    """A copy under another path: no second library beside it, whose status word nobody would read."""
    import shutil
    blbuild.build()
    copy = shutil.copy(blbuild.OUT, tmp_path / "libother.so")
    r = python("import torch, int8_row_absmax_b200 as bl\n"
               "from int8_row_absmax_b200 import attn\n"
               "attn._torch = lambda: torch\n"
               f"bl.load({str(copy)!r})\n"
               "attn._native()\n"
               "maps = open('/proc/self/maps').read()\n"
               "assert 'libother.so' in maps and 'libbitlinear.so' not in maps")
    assert r.returncode == 0, r.stderr
