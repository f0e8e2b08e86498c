"""The build's steps on the CPU, with compilers that only leave the file they are
asked for: the C library stands whatever becomes of the marshalling module."""
import importlib.util
import os
import shutil
import stat
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "block_sparse_attention_slice_gb300")


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A copy of the sources, its _build module, and the log of what was run."""
    pkg = tmp_path / "pkg"
    pkg.mkdir()
    shutil.copy(os.path.join(PACKAGE, "_build.py"), pkg)
    shutil.copytree(os.path.join(PACKAGE, "csrc"), pkg / "csrc", ignore=shutil.ignore_patterns("__pycache__"))
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    for name, last in (("nvcc", ""), ("cxx", ""), ("broken", "exit 1\n")):
        f = tmp_path / name
        f.write_text(f"#!/bin/sh\necho {name} >> {tmp_path}/ran\n{last}"
                     'while [ $# -gt 0 ]; do if [ "$1" = -o ]; then echo > "$2"; fi; shift; done\n')
        f.chmod(f.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("NVCC", str(tmp_path / "nvcc"))
    monkeypatch.setenv("CXX", str(tmp_path / "cxx"))
    spec = importlib.util.spec_from_file_location("_build_of_a_copy", pkg / "_build.py")
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)

    def ran():
        log = tmp_path / "ran"
        names = log.read_text().split() if log.exists() else []
        log.write_text("")
        return names

    return m, tmp_path, ran


def test_builds_once_and_again_only_what_changed(tree):
    m, tmp, ran = tree
    assert m.build() == m.LIB and os.path.exists(m.LIB) and os.path.exists(m.MODULE)
    assert sorted(set(ran())) == ["cxx", "nvcc"] and m.up_to_date()
    m.build()
    assert ran() == []
    os.utime(m.MODULE, (1, 1))           # older than its sources
    assert not m.up_to_date() and m.library_up_to_date()
    m.build()
    assert ran() == ["cxx", "cxx"]
    os.utime(m.LIB, (1, 1))
    assert not m.up_to_date() and m.module_up_to_date()
    m.build()
    assert set(ran()) == {"nvcc"}
    m.build(force=True)
    assert set(ran()) == {"nvcc", "cxx"}


@pytest.mark.parametrize("cxx", ["broken", "nowhere"])
def test_the_library_stands_where_the_module_does_not_compile(tree, monkeypatch, cxx):
    m, tmp, ran = tree
    monkeypatch.setenv("CXX", str(tmp / cxx))
    with pytest.raises(RuntimeError, match="paging_module.cpp"):
        m.build()
    assert os.path.exists(m.LIB) and not os.path.exists(m.MODULE)
    assert m.library_up_to_date() and not m.up_to_date()
    ran()
    assert m.build_library() == m.LIB and ran() == []
    with pytest.raises(RuntimeError):
        m.build()                        # said again, and the library is not built again
    assert "nvcc" not in ran()


def test_the_library_is_built_without_torch(tree):
    m, tmp, ran = tree
    code = f"import sys; sys.modules['torch'] = None; sys.path.insert(0, {str(tmp / 'pkg')!r}); import _build; print(_build.build())"
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert done.returncode == 0, done.stderr
    assert done.stdout.split() == [m.LIB] and os.path.exists(m.LIB) and not os.path.exists(m.MODULE)
    assert set(ran()) == {"nvcc"}
