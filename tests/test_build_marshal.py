"""The marshalling module belongs to one interpreter and one PyTorch: its name
carries the interpreter's suffix, and it is built again when either changes."""
import os
import sysconfig

import pytest
import torch

from paged_kv_cache_141_gb300 import build


@pytest.fixture
def compiled(monkeypatch, tmp_path):
    """build_marshal into a folder of its own, with a compiler that only leaves a file; the list of its runs."""
    runs = []

    class Done:
        returncode, stderr = 0, ""

    def run(cmd, **kw):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return Done()

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / os.path.basename(build.MARSHAL)))
    return runs


def test_no_other_interpreter_imports_it(compiled, tmp_path):
    assert build.MARSHAL.endswith(sysconfig.get_config_var("EXT_SUFFIX")) and sysconfig.get_config_var("SOABI") in build.MARSHAL
    (tmp_path / "_marshal.so").touch()                  # an earlier build's, without a tag
    build.build_marshal()
    assert sorted(f for f in os.listdir(tmp_path) if f.startswith("_marshal")) == [os.path.basename(build.MARSHAL)]


def test_built_again_for_another_interpreter_or_pytorch(compiled, monkeypatch):
    build.build_marshal()
    build.build_marshal()
    assert len(compiled) == 1
    real = sysconfig.get_config_var
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda n: "cpython-311-other" if n == "SOABI" else real(n))
        build.build_marshal()
        assert len(compiled) == 2
    build.build_marshal()
    assert len(compiled) == 3
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "2.0.0")
        build.build_marshal()
        assert len(compiled) == 4
    with monkeypatch.context() as m:                    # the same version in another place: the rpath names it
        m.setattr(torch, "__file__", "/elsewhere" + torch.__file__)
        m.setattr(torch, "compiled_with_cxx11_abi", lambda: True)
        build.build_marshal()
        assert len(compiled) == 5
