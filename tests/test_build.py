"""What the build needs: the library nvcc alone, the binding's native half a
host compiler and Python's headers.  CPU only; a stand-in takes nvcc's place."""
import os
import shutil
import stat

import pytest


@pytest.fixture
def b(tmp_path, monkeypatch):
    from mmvq_q2_gb300 import build as b
    fake = tmp_path / "nvcc"
    fake.write_text('#!/bin/sh\necho x >> "$0.log"\nwhile [ "$1" != -o ]; do shift; done\n: > "$2"\n')
    fake.chmod(fake.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(b, "nvcc", lambda: str(fake))
    monkeypatch.setattr(b, "OUT", str(tmp_path / "lib"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib" / "libq2k.so"))
    monkeypatch.setattr(b, "CALLS", str(tmp_path / "lib" / os.path.basename(b.CALLS)))
    b.runs = lambda: len((tmp_path / "nvcc.log").read_text().split())
    yield b
    del b.runs


def test_library_builds_without_python_headers(b, tmp_path, monkeypatch, capsys):
    paths = dict(b.sysconfig.get_paths(), include=str(tmp_path / "nowhere"))
    monkeypatch.setattr(b.sysconfig, "get_paths", lambda *a, **k: paths)
    assert b.build() == b.LIB and os.path.exists(b.LIB) and not os.path.exists(b.CALLS)
    assert "Python.h" in capsys.readouterr().err
    runs = b.runs()
    b.build()  # nothing to do: the part that cannot be built does not make the rest stale
    assert b.runs() == runs
    # a native half of older sources is not left beside a newer library
    open(b.CALLS, "w").close()
    os.utime(b.CALLS, (1, 1))
    b.build()
    assert not os.path.exists(b.CALLS)


def test_library_is_linked_before_a_failure_of_the_native_half(b, monkeypatch):
    monkeypatch.setattr(b, "CALLS_SOURCE", "no_such_file.c")
    with pytest.raises(RuntimeError, match="no_such_file"):
        b.build()
    assert os.path.exists(b.LIB)


def test_host_compiler_with_arguments(b, monkeypatch):
    monkeypatch.setenv("CC", f"{shutil.which('gcc') or shutil.which('cc')} -pipe")
    b.build()
    assert os.path.exists(b.LIB) and os.path.exists(b.CALLS)
    runs = b.runs()
    b.build()
    assert b.runs() == runs


def test_calls_say_what_is_missing(b, monkeypatch):
    import mmvq_q2_gb300 as q
    q.lib()
    native = q._native
    monkeypatch.setattr(q, "_native", None)
    monkeypatch.setattr(q, "LIB_PATH", b.LIB)
    with pytest.raises(RuntimeError, match="Python.h"):
        q._calls()
    q._native = native
