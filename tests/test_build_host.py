"""What building needs: the C library stands on its own."""

import os
import subprocess
import sys
import sysconfig

import pytest

from forward_mode_flash_gb300 import build


def test_the_library_is_built_without_pytorch():
    build.build()
    code = (f"import sys; sys.modules['torch'] = None; sys.path.insert(0, {build.PKG!r}); "
            "import build; print(build.build(), build.build_bind())")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == [build.LIB, "None"]


def test_the_library_is_built_though_the_binding_is_not(tmp_path, monkeypatch):
    src = tmp_path / "csrc"
    src.mkdir()
    (src / "one.cu").write_text('extern "C" int jvp_attn_version() { return 1; }\n')
    (src / "exports.map").write_text("{ global: jvp_attn_*; local: *; };\n")
    monkeypatch.setattr(build, "CSRC", str(src))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "out"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "out" / "lib.so"))

    def no_headers():
        raise RuntimeError("no headers")

    monkeypatch.setattr(build, "build_bind", no_headers)
    with pytest.raises(RuntimeError, match="no headers"):
        build.build()
    assert os.path.exists(build.LIB)


def test_the_binding_is_built_for_this_interpreter():
    """(Another one with the same PyTorch must not load it.)"""
    assert sysconfig.get_config_var("SOABI") in os.path.basename(build.bind_path())


def test_the_binding_is_built_again_for_other_flags(tmp_path, monkeypatch):
    out = build.build_bind()
    before = os.path.getmtime(out)
    recipe = tmp_path / "build.py"
    recipe.write_text("")
    os.utime(recipe, (before - 10, before - 10))
    monkeypatch.setattr(build, "__file__", str(recipe))
    calls = []

    def compiler(cmd, **kw):
        calls.append(cmd)
        return subprocess.CompletedProcess(cmd, 1, "", "not run")

    monkeypatch.setattr(build.subprocess, "run", compiler)
    assert build.build_bind() == out and not calls
    os.utime(recipe, (before + 10, before + 10))
    with pytest.raises(RuntimeError, match="not run"):
        build.build_bind()
    assert len(calls) == 1
