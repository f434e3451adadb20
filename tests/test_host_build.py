"""The build's order and freshness, with its commands replaced (CPU, nothing is compiled)."""
import os
import subprocess
import sys
import types

import pytest

from gemv_dg_bf16_gb300 import build as bld
from tests._helpers import ROOT


@pytest.fixture
def sandbox(tmp_path, monkeypatch):
    """Outputs under tmp_path; `commands` lists what ran, `fail` names a compiler that does not work."""
    box = types.SimpleNamespace(commands=[], fail=None, dir=tmp_path)
    for name, at in (("LIB", "libdecodegemm.so"), ("PYMOD", "_marshal.so"), ("OBJ", "_build")):
        monkeypatch.setattr(bld, name, str(tmp_path / at))

    def run(cmd, **kw):
        if "--version" in cmd:
            return subprocess.CompletedProcess(cmd, 0, "", "")
        box.commands.append(cmd)
        if cmd[0] == box.fail:
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(bld.subprocess, "run", run)
    return box


def test_library_is_linked_even_if_the_python_module_does_not_compile(sandbox):
    sandbox.fail = "g++"
    with pytest.raises(RuntimeError) as e:
        bld.build()
    assert "_marshal.cpp" in str(e.value) and "no such header" in str(e.value)
    assert os.path.exists(bld.LIB) and not os.path.exists(bld.PYMOD)
    sandbox.fail, n = None, len(sandbox.commands)
    bld.build()                                                # what is left: the module alone
    assert [c[0] for c in sandbox.commands[n:]] == ["g++"] and os.path.exists(bld.PYMOD)
    assert bld.build() == bld.LIB and len(sandbox.commands) == n + 1


def test_python_module_is_built_again_for_another_torch_or_python(sandbox, monkeypatch):
    bld.build()
    n = len(sandbox.commands)
    bld.build()
    assert len(sandbox.commands) == n
    import torch
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    bld.build()
    assert [c[0] for c in sandbox.commands[n:]] == ["g++"]
    monkeypatch.setattr(sys, "version", "4.0")
    bld.build()
    bld.build()
    assert [c[0] for c in sandbox.commands[n:]] == ["g++"] * 2


@pytest.mark.parametrize("module,needle", [(None, "is not built"), ("not a shared object", "cannot be loaded")])
def test_message_tells_a_missing_module_from_one_that_does_not_load(tmp_path, module, needle):
    bld.build()
    pkg = tmp_path / "gemv_dg_bf16_gb300"
    pkg.mkdir()
    for f in ("__init__.py", "_binding.py", "csrc", "libdecodegemm.so"):
        (pkg / f).symlink_to(os.path.join(ROOT, "gemv_dg_bf16_gb300", f))
    if module:
        (pkg / "_marshal.so").write_text(module)
    r = subprocess.run([sys.executable, "-c", "from gemv_dg_bf16_gb300 import _binding as b; b._load_marshal()"],
                       cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert r.returncode != 0 and "ImportError" in r.stderr and needle in r.stderr.splitlines()[-1], r.stderr[-600:]
