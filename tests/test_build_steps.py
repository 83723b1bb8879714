"""The steps of the build, without running a compiler: what needs torch does not keep the
library and the oracle from being built where torch is missing."""
import importlib.util
import os

import pytest

import __graft_entry__
from expert_ffn_amd import _build


@pytest.fixture
def steps(monkeypatch):
    """The build's steps as they were taken; no compiler runs, and torch cannot be found."""
    import expert_ffn_amd
    import oracle
    done = []
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))

    class Done:
        returncode, stderr = 0, ""

    monkeypatch.setattr(_build.subprocess, "run", lambda cmd, **kw: done.append(cmd) or Done())
    monkeypatch.setattr(_build.os, "replace", lambda a, b: done.append(b))
    monkeypatch.setattr(oracle, "build", lambda force=False: done.append("oracle"))
    monkeypatch.setattr(expert_ffn_amd, "lib", lambda: done.append("loaded"))
    return done


def test_library_and_oracle_are_built_without_torch(steps, capsys):
    __graft_entry__.build()
    assert _build.LIB in steps and _build.PEAKS_LIB in steps and "oracle" in steps and steps[-1] == "loaded"
    assert _build.BINDING not in steps
    assert "torch is not installed" in capsys.readouterr().out


def test_binding_needs_a_host_compiler(monkeypatch):
    monkeypatch.setattr(_build.shutil, "which", lambda name, *a: None)
    with pytest.raises(RuntimeError, match="g\\+\\+"):
        _build.build_binding()


def test_headers_belong_to_the_compiler(monkeypatch, tmp_path):
    """The HIP headers are those beside hipcc, wherever the path finds it."""
    (tmp_path / "bin").mkdir()
    (tmp_path / "bin" / "hipcc").write_text("")
    (tmp_path / "bin" / "hipcc").chmod(0o755)
    monkeypatch.setattr(_build, "HIPCC", str(tmp_path / "bin" / "hipcc"))
    assert _build.rocm_include() == os.path.join(os.path.realpath(tmp_path), "include")
