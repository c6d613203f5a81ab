"""The build without torch, and of the module that depends on it, with the compilers
replaced by a recorder (nothing is compiled here)."""
import os
import subprocess

import pytest


@pytest.fixture
def recorder(tmp_path, monkeypatch):
    """The build module on an empty output directory; compiler calls are recorded, and
    make their output file."""
    from dense_gemm_row_gb300 import build as b
    calls = []

    def run(cmd, **kw):
        calls.append(cmd)
        out = cmd[cmd.index("-o") + 1]
        bad = fail and any(fail[0] in part for part in cmd)
        if not bad:
            open(out, "w").close()
        return subprocess.CompletedProcess(cmd, int(bool(bad)), "", "refused" if bad else "")

    fail = []
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "LIB_PATH", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "LAYERS_PATH", str(tmp_path / "_layers.so"))
    monkeypatch.setattr(b, "nvcc", lambda: "nvcc")
    monkeypatch.setattr(b.subprocess, "run", run)
    return b, calls, fail


def no_torch(monkeypatch):
    import importlib.util
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else find(name, *a))


def test_c_library_builds_without_torch(recorder, monkeypatch, capfd):
    b, calls, _ = recorder
    no_torch(monkeypatch)
    assert b.build() == b.LIB_PATH and os.path.exists(b.LIB_PATH)
    assert not os.path.exists(b.LAYERS_PATH) and not any("py_layers.cpp" in c for c in sum(calls, []))
    assert "torch not found" in capfd.readouterr().err


def test_module_is_rebuilt_for_another_torch(recorder, monkeypatch):
    b, calls, _ = recorder
    b.build(quiet=True)
    assert os.path.exists(b.LAYERS_PATH)
    calls.clear()
    b.build(quiet=True)
    assert not calls  # nothing changed
    made_for = b._layers_made_for
    monkeypatch.setattr(b, "_layers_made_for", lambda d: made_for(d) + "another version")
    b.build(quiet=True)
    assert [os.path.basename(c[0]) for c in calls] == ["g++"]
    calls.clear()
    b.build(quiet=True)
    assert not calls


def test_c_library_stays_when_the_module_fails(recorder):
    b, _, fail = recorder
    fail.append("py_layers.cpp")
    with pytest.raises(RuntimeError, match="refused"):
        b.build(quiet=True)
    assert os.path.exists(b.LIB_PATH) and not os.path.exists(b.LAYERS_PATH)
    fail.clear()
    b.build(quiet=True)
    assert os.path.exists(b.LAYERS_PATH)
