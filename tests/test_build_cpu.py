"""The build's care for _marshal.so, which depends on the installed torch and Python: built again when
either changes, refused until then, left out where torch is missing.  Commands are recorded, not
run."""
import os
import subprocess
import sys

import pytest

import speculative_decoding_verification_59_gb300 as sv
from speculative_decoding_verification_59_gb300 import _build


class Done:
    returncode = 0

    def communicate(self):
        return "", None


@pytest.fixture
def built(monkeypatch, tmp_path):
    """A finished build in a folder of its own; returns the commands that build() runs after that."""
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        out = cmd[cmd.index("-o") + 1]
        with open(out, "w"):
            pass
        return Done()
    monkeypatch.setattr(_build, "BUILD", str(tmp_path))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libspecverify.so"))
    monkeypatch.setattr(_build, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(_build, "MARSHAL_STAMP", str(tmp_path / "sv_torch.stamp"))
    monkeypatch.setattr(_build, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(subprocess, "Popen", run)
    monkeypatch.setattr(subprocess, "run", run)
    _build.build()
    assert len(ran) == len(_build.sources()) + 3               # a unit each, sv_torch.cpp, two links
    ran.clear()
    return ran


def of_torch(cmd):
    return any(x.endswith(("sv_torch.cpp", "sv_torch.o")) for x in cmd)


def test_nothing_to_do_after_a_build(built):
    _build.build()
    assert built == []


@pytest.mark.parametrize("change", ["version", "place", "python"])
def test_another_torch_or_python_builds_the_module_again(built, monkeypatch, tmp_path, change):
    if change == "python":
        get = _build.sysconfig.get_config_var
        monkeypatch.setattr(_build.sysconfig, "get_config_var", lambda n: ".other.so" if n == "EXT_SUFFIX" else get(n))
    else:
        other = tmp_path / "elsewhere"
        other.mkdir()
        if change == "version":
            (other / "version.py").write_text("__version__ = '0.0'\n")
        monkeypatch.setattr(_build, "_torch_dir", lambda: str(other))
    assert not _build.marshal_matches(_build._torch_dir())
    _build.build()
    assert len(built) == 2 and all(of_torch(c) for c in built)
    built.clear()
    assert _build.marshal_matches(_build._torch_dir())
    _build.build()
    assert built == []


def test_a_failed_link_is_tried_again(built, monkeypatch, tmp_path):
    def fails(cmd, **kw):
        built.append(cmd)
        raise subprocess.CalledProcessError(1, cmd)
    os.remove(tmp_path / "sv_torch.stamp")
    run = subprocess.run
    monkeypatch.setattr(subprocess, "run", fails)
    with pytest.raises(subprocess.CalledProcessError):
        _build.build()
    monkeypatch.setattr(subprocess, "run", run)
    built.clear()
    _build.build()
    assert len(built) == 2 and all(of_torch(c) for c in built)


def test_without_torch_the_library_is_built(built, monkeypatch, tmp_path, capsys):
    monkeypatch.setattr(_build.importlib.util, "find_spec", lambda name: None)
    os.remove(tmp_path / "libspecverify.so")
    os.remove(tmp_path / "sv_torch.stamp")
    _build.build()
    assert len(built) == 1 and not of_torch(built[0])
    assert "torch is not installed" in capsys.readouterr().err


def test_a_module_of_another_torch_is_not_loaded(monkeypatch):
    pytest.importorskip("torch")
    if not os.path.exists(sv.lib_path()):
        import __graft_entry__
        __graft_entry__.build()
    monkeypatch.setattr(sv, "_marshal_module", None)
    monkeypatch.setattr(_build, "marshal_matches", lambda d: False)
    with pytest.raises(ImportError, match="not built for this torch"):
        sv._load_marshal()
    monkeypatch.undo()
    assert sv._load_marshal() is sys.modules[sv.__name__ + "._marshal"]


def test_two_threads_load_the_module_at_once(monkeypatch):
    """Another thread that finds the module imported, but not yet noted, loads it too."""
    torch = pytest.importorskip("torch")
    module = sv._load_marshal()
    monkeypatch.setattr(sv, "_marshal_module", None)
    with pytest.raises(ValueError, match="CUDA"):
        sv.token_logprobs(torch.zeros((2, 10)), torch.zeros(2, dtype=torch.int32))
    assert sv._marshal_module is module
