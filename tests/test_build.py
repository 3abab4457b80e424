"""When the compiled binding is built: against the torch that is there, again when that
changes, and not at all where there is none (the C library needs no torch)."""
import importlib.metadata
import importlib.util
import os
import types

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def script(tmp_path, monkeypatch):
    """The build script with outputs of its own and a compiler that only writes its output file."""
    spec = importlib.util.spec_from_file_location("pa_b200_build_test", os.path.join(ROOT, "paged_kv_cache_389_b200", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.STEP, mod.OBJ, mod.made = str(tmp_path / "_step.so"), str(tmp_path / "obj"), []

    def run(cmd, **kw):
        mod.made.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(mod, "subprocess", types.SimpleNamespace(run=run))
    return mod


def hide_torch(mod, monkeypatch):
    util = types.SimpleNamespace(find_spec=lambda name: None if name == "torch" else importlib.util.find_spec(name))
    monkeypatch.setattr(mod, "importlib", types.SimpleNamespace(util=util, metadata=importlib.metadata), raising=False)
    real = __import__

    def no_torch(name, *a, **kw):
        if name.split(".")[0] == "torch":
            raise ImportError("no torch here")
        return real(name, *a, **kw)

    monkeypatch.setattr("builtins.__import__", no_torch)


def test_without_torch_the_library_is_built_alone(script, monkeypatch, capsys):
    hide_torch(script, monkeypatch)
    monkeypatch.setattr(script, "_stale", lambda: False)
    assert script.build() == script.LIB and not script.made
    monkeypatch.setattr(script, "_stale", lambda: True)
    monkeypatch.setattr(script, "_compile", lambda src, extra: src + ".o")
    monkeypatch.setattr(script, "LIB", os.path.join(os.path.dirname(script.STEP), "lib.so"))
    assert script.build() == script.LIB and len(script.made) == 1 and os.path.exists(script.LIB)
    assert "no torch" in capsys.readouterr().err and not os.path.exists(script.STEP)


def test_the_binding_is_built_again_for_another_torch(script, monkeypatch):
    assert script.build_binding() == script.STEP and len(script.made) == 1
    assert script.build_binding() == script.STEP and len(script.made) == 1      # up to date
    version = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "99.0" if name == "torch" else version(name))
    assert script.build_binding() == script.STEP and len(script.made) == 2
    assert script.build_binding() == script.STEP and len(script.made) == 2
    monkeypatch.undo()


def test_a_failed_compile_says_so(script, monkeypatch):
    failed = lambda cmd, **kw: types.SimpleNamespace(returncode=1, stdout="", stderr="no such header")
    monkeypatch.setattr(script, "subprocess", types.SimpleNamespace(run=failed))
    with pytest.raises(RuntimeError, match="no such header"):
        script.build_binding()
