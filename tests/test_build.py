"""What the package builds and loads (CPU)."""
import os
import shutil
import subprocess
import sys

import pytest

import speculative_decoding_draft_rmsnorm_gb300 as D
from speculative_decoding_draft_rmsnorm_gb300 import _build


@pytest.fixture
def copy(tmp_path):
    """The package with its product libraries, without the marshalling module."""
    D.load()
    name = os.path.basename(_build.PKG)
    shutil.copytree(_build.PKG, tmp_path / name, ignore=shutil.ignore_patterns("_build", "_decode_bind*", "__pycache__"))
    shutil.copytree(os.path.join(_build.ROOT, "include"), tmp_path / "include")
    return tmp_path


def python(where, code):
    r = subprocess.run([sys.executable, "-c", f"import sys; sys.path.insert(0, {str(where)!r})\n" + code], cwd=where, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    return r.stdout


def test_the_library_loads_without_torch_or_the_marshalling_module(copy):
    out = python(copy, """
sys.modules["torch"] = None
import speculative_decoding_draft_rmsnorm_gb300 as D
print(D.__file__, D.load(build_if_missing=False).dflash_version())
""")
    assert out.startswith(str(copy))


def test_a_failing_marshalling_module_leaves_the_libraries_built(copy):
    out = python(copy, """
import os
from speculative_decoding_draft_rmsnorm_gb300 import _build
os.makedirs(_build.OBJ_DIR, exist_ok=True)
open(_build.BIND_SOURCE, "w").write("#error no headers here")
_build.SOURCES = ["draft_step.cu"]
_build.TARGETS = [(os.path.join(_build.LIB_DIR, "small.so"), [], _build.OBJ_DIR)]
try:
    _build.build()
except RuntimeError as e:
    print("raised", "bind.cpp" in str(e), os.path.exists(_build.TARGETS[0][0]))
""")
    assert out.split() == ["raised", "True", "True"]


def test_a_marshalling_module_of_another_torch_is_not_taken(monkeypatch):
    import torch
    _build.build()
    assert _build.up_to_date(_build.bind_path())
    monkeypatch.setattr(torch, "__version__", "2.0.1+other")
    assert not _build.up_to_date(_build.bind_path())
    monkeypatch.undo()
    assert _build.up_to_date(_build.bind_path())
