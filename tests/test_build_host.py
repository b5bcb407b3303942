"""The build with compilers that only write their output file: the library
does not depend on torch, and what is out of date is built again."""
import os
import stat
import subprocess
import sys

import pytest

from nvfp4_weight_only_rows_gb300 import _build

STUB = '''#!/bin/sh
echo "$(basename "$0") $*" >> "{log}"
[ -e "{fail}/$(basename "$0")" ] && exit 1
while [ $# -gt 1 ]; do
  if [ "$1" = -o ]; then echo built > "$2"; fi
  shift
done
'''


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A copy of the sources with stubs for nvcc and g++ on PATH."""
    pkg = tmp_path / "pkg"
    (pkg / "csrc").mkdir(parents=True)
    (tmp_path / "include").mkdir()
    (tmp_path / "include" / "nvfp4_lm_head.h").write_text("")
    for f in os.listdir(_build.CSRC):
        (pkg / "csrc" / f).write_text("")
    bin_dir, fail = tmp_path / "bin", tmp_path / "fail"
    bin_dir.mkdir()
    fail.mkdir()
    log = tmp_path / "log"
    log.write_text("")
    for name in ("nvcc", "g++"):
        f = bin_dir / name
        f.write_text(STUB.format(log=log, fail=fail))
        f.chmod(f.stat().st_mode | stat.S_IEXEC)
    monkeypatch.setenv("PATH", f"{bin_dir}:{os.environ['PATH']}")
    for name, path in (("HERE", pkg), ("CSRC", pkg / "csrc"), ("LIB", pkg / "libnvfp4_lm_head.so"),
                       ("CALLS", pkg / "_calls.so")):
        monkeypatch.setattr(_build, name, str(path))

    class Tree:
        lib, calls, csrc = pkg / "libnvfp4_lm_head.so", pkg / "_calls.so", pkg / "csrc"

        def break_(self, compiler):
            (fail / compiler).write_text("")

        def mend(self, compiler):
            (fail / compiler).unlink()

        def ran(self):
            """The compilers run since the last look."""
            lines = log.read_text().splitlines()
            log.write_text("")
            return [line.split()[0] for line in lines]

    return Tree()


def test_a_failure_of_the_python_side_leaves_the_library(tree):
    tree.break_("g++")
    with pytest.raises(RuntimeError, match="calls.cpp"):
        _build.build()
    assert tree.lib.exists() and not tree.calls.exists()


def test_the_library_without_torch(tree, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch fails
    assert _build.build_library() == str(tree.lib) and tree.lib.exists()
    assert "g++" not in tree.ran()
    tree.lib.unlink()
    with pytest.raises(ImportError):
        _build.build()
    assert tree.lib.exists()


def test_the_file_runs_alone():
    """... without the package, whose import needs torch."""
    code = ("import sys, runpy; sys.modules['torch'] = None; "
            f"m = runpy.run_path({_build.__file__!r}); assert callable(m['build_library'])")
    subprocess.run([sys.executable, "-c", code], check=True)


def test_what_is_built_again(tree, monkeypatch):
    def later(path):  # a source edited after the last build
        os.utime(path, (os.path.getmtime(path) + 1e6,) * 2)

    _build.build()
    assert {"nvcc", "g++"} == set(tree.ran())
    _build.build()
    assert tree.ran() == []
    monkeypatch.setattr("torch.__version__", "2.0.1+another")
    _build.build()
    assert set(tree.ran()) == {"g++"}  # against the torch there is now
    _build.build()
    assert tree.ran() == []
    later(tree.csrc / "calls.cpp")
    _build.build()
    assert set(tree.ran()) == {"g++"}
    os.utime(tree.csrc / "calls.cpp", (0, 0))
    later(tree.csrc / "moe.cu")
    _build.build_library()
    assert set(tree.ran()) == {"nvcc"}
    os.utime(tree.csrc / "moe.cu", (0, 0))
    later(tree.csrc / "common.cuh")
    _build.build_library()
    assert set(tree.ran()) == {"nvcc"}


def test_the_python_side_after_a_failed_build(tree):
    tree.break_("g++")
    with pytest.raises(RuntimeError):
        _build.build()
    tree.ran()
    tree.mend("g++")
    _build.build()
    assert set(tree.ran()) == {"g++"} and tree.calls.exists()
