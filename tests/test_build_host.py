"""What building needs: the C library stands on its own."""

import os
import subprocess
import sys

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
