"""The C library needs neither PyTorch nor the extension module of the Python
calls: what keeps that from being built does not keep the library from it."""
import os
import stat

import pytest

from weight_streaming_expert_gb300 import build_lib, native


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """An empty build folder, and a compiler that only writes its output file."""
    monkeypatch.setattr(build_lib, "BUILD", str(tmp_path / "build"))
    monkeypatch.setattr(build_lib, "LIB", str(tmp_path / "build" / "libwse.so"))
    monkeypatch.setattr(build_lib, "CALLS", str(tmp_path / "build" / "wse_calls.so"))
    fake = tmp_path / "nvcc"
    fake.write_text('#!/bin/sh\nwhile [ $# -gt 0 ]; do [ "$1" = -o ] && echo built > "$2"; shift; done\n')
    fake.chmod(fake.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("NVCC", str(fake))
    return tmp_path


def test_the_library_is_built_where_the_calls_cannot_be(elsewhere, monkeypatch):
    def fails(*_):
        raise RuntimeError("no headers")

    monkeypatch.setattr(build_lib, "_compile_calls", fails)
    with pytest.raises(RuntimeError, match="no headers"):
        build_lib.build()
    assert os.path.exists(build_lib.LIB) and not os.path.exists(build_lib.CALLS)


def test_the_library_is_built_without_pytorch(elsewhere, monkeypatch, capsys):
    monkeypatch.setattr(build_lib.importlib.util, "find_spec", lambda name: None)
    assert build_lib.build() == build_lib.LIB
    assert os.path.exists(build_lib.LIB) and not os.path.exists(build_lib.CALLS)
    assert "PyTorch" in capsys.readouterr().err


def test_the_library_is_loaded_without_the_calls(tmp_path, monkeypatch):
    native.lib()
    monkeypatch.setattr(native, "_lib", None)
    monkeypatch.setattr(build_lib, "CALLS", str(tmp_path / "none.so"))
    for name in [n for n in dir(build_lib) if n.startswith("build")]:
        monkeypatch.setattr(build_lib, name, lambda *a, **k: pytest.fail("the library is there"))
    assert native.lib().moe_last_error is not None


def test_a_newer_source_of_the_calls_leaves_the_library_alone(elsewhere, monkeypatch):
    build_lib.os.makedirs(build_lib.BUILD)
    newest = max(os.path.getmtime(p) for p in build_lib._inputs())
    for path, age in ((build_lib.LIB, 10), (build_lib.CALLS, -10 ** 9)):
        with open(path, "w") as f:
            f.write("old")
        os.utime(path, (newest + age, newest + age))
    made = []
    monkeypatch.setattr(build_lib, "_compile_calls", lambda: made.append(1) or "calls.o")
    monkeypatch.setattr(build_lib, "_run", lambda cmd, what: made.append(what) or open(cmd[cmd.index("-o") + 1], "w"))
    build_lib.build()
    assert made and open(build_lib.LIB).read() == "old"
