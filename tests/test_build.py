"""When the Python extension is built again (no GPU, no compiler run)."""
import os
import subprocess

import pytest

from paged_kv_cache_429_b200 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """An extension with its source in a folder of their own, and the
    commands that a build would run."""
    src, so = tmp_path / "binding.cpp", tmp_path / "_binding.so"
    src.write_text("")
    monkeypatch.setattr(build, "BINDING", str(so))
    monkeypatch.setattr(build, "BINDING_DEPS", [str(src)])
    monkeypatch.setattr(build, "BINDING_STAMP", str(tmp_path / "_build" / "binding.txt"))
    runs = []

    def run(cmd, check):
        runs.append(cmd)
        so.write_text("")
    monkeypatch.setattr(subprocess, "run", run)
    return src, so, runs


def test_the_extension_is_built_once(tree):
    src, so, runs = tree
    build.build_binding()
    build.build_binding()
    assert len(runs) == 1
    os.utime(src, ns=(so.stat().st_mtime_ns + 10**9,) * 2)
    build.build_binding()
    assert len(runs) == 2
    build.build_binding(force=True)
    assert len(runs) == 3


def test_another_torch_builds_the_extension_again(tree, monkeypatch):
    src, so, runs = tree
    build.build_binding()
    monkeypatch.setattr("torch.__version__", "0.0.0+other")
    build.build_binding()
    assert len(runs) == 2
    build.build_binding()
    assert len(runs) == 2


def test_a_build_that_fails_leaves_no_mark(tree, monkeypatch):
    src, so, runs = tree
    build.build_binding()

    def fails(cmd, check):
        raise subprocess.CalledProcessError(1, cmd)
    with monkeypatch.context() as m:
        m.setattr(subprocess, "run", fails)
        with pytest.raises(subprocess.CalledProcessError):
            build.build_binding(force=True)
    build.build_binding()
    assert len(runs) == 2


def test_the_library_alone_needs_no_extension(tree, tmp_path, monkeypatch):
    src, so, runs = tree
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libpa.so"))
    build.build(force=True, binding=False)
    assert len(runs) == 1 and not any("binding.cpp" in a for a in runs[0])
    monkeypatch.setattr(build, "up_to_date", lambda: True)
    build.build(binding=False)
    assert len(runs) == 1
    build.build()
    assert len(runs) == 2
