"""The binding's C++ half is compiled against torch's and Python's headers: it is built for, and loaded
by, the pair of them that it was compiled with, and no other."""
from __future__ import annotations

import os
import sysconfig

import pytest
import torch

from paged_kv_cache_173_gb300 import _lib, build


@pytest.fixture
def other_torch(monkeypatch):
    """The tree as a torch of another version finds it."""
    build.build_library()
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    monkeypatch.setattr(_lib, "_fast", None)


def test_the_file_is_named_by_torch_and_python(monkeypatch):
    here = build.fast_path()
    assert torch.__version__ in here and here.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    monkeypatch.setattr(torch, "compiled_with_cxx11_abi", lambda was=torch.compiled_with_cxx11_abi(): not was)
    assert build.fast_path() != here
    monkeypatch.undo()
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: ".cpython-399-elsewhere.so")
    assert build.fast_path() != here


def test_another_torch_does_not_load_it(other_torch):
    with pytest.raises(RuntimeError, match="build it first"):
        _lib.fast()


def test_another_torch_builds_its_own(other_torch, monkeypatch, tmp_path):
    ran = []

    def compiler(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        ran.append(out)
        open(out, "wb").close()
        return type("Done", (), {"returncode": 0, "stdout": "", "stderr": ""})

    monkeypatch.setattr(build, "PKG", str(tmp_path))
    monkeypatch.setattr(build.subprocess, "run", compiler)
    path = build.build_fast()
    assert len(ran) == 1 and os.path.dirname(path) == str(tmp_path) and "0.0.1+other" in path
    assert build.build_fast() == path and len(ran) == 1  # up to date


def test_this_torch_loads_its_own():
    build.build_library()
    assert os.path.exists(build.fast_path())
    assert _lib.fast().__file__ == build.fast_path()
