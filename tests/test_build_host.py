"""What the build makes, and when, with stand-ins for the compilers: the library
needs nvcc alone, and the marshalling module is built for the torch and Python
that use it."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

COMPILER = """#!/bin/sh
echo "$(basename "$0") $*" >> "$BUILD_LOG"
case "$(basename "$0")" in *bad*) echo "no such header"; exit 1;; esac
out=""
while [ $# -gt 0 ]; do if [ "$1" = "-o" ]; then out="$2"; fi; shift; done
echo built > "$out"
"""


class Tree:
    """A copy of the sources, built by their script with the stand-ins."""

    def __init__(self, tmp):
        self.pkg = tmp / "softmax_tree_reduction_gb300"
        shutil.copytree(os.path.join(ROOT, "softmax_tree_reduction_gb300", "csrc"), self.pkg / "csrc")
        shutil.copy(os.path.join(ROOT, "softmax_tree_reduction_gb300", "build.py"), self.pkg / "build.py")
        shutil.copytree(os.path.join(ROOT, "include"), tmp / "include")
        self.bin, self.log, self.mods = tmp / "bin", tmp / "log", tmp / "mods"
        self.bin.mkdir()
        self.mods.mkdir()
        for name in ("nvcc", "cxx", "badcxx"):
            (self.bin / name).write_text(COMPILER)
            (self.bin / name).chmod(0o755)

    def torch(self, version):
        """The torch that the build finds (None: there is none)."""
        body = "raise ImportError('no torch here')" if version is None else f"__version__ = {version!r}"
        (self.mods / "torch.py").write_text(body + "\n")
        shutil.rmtree(self.mods / "__pycache__", ignore_errors=True)

    def build(self, cxx="cxx"):
        """(exit status, output, compiler calls) of one run."""
        self.log.write_text("")
        env = dict(os.environ, PATH=f"{self.bin}:/usr/bin:/bin", CXX=str(self.bin / cxx) if "/" not in cxx else cxx, BUILD_LOG=str(self.log),
                   PYTHONPATH=str(self.mods))
        r = subprocess.run([sys.executable, str(self.pkg / "build.py")], env=env, capture_output=True, text=True, timeout=120)
        return r.returncode, r.stdout + r.stderr, [line.split()[0] for line in self.log.read_text().splitlines()]

    def has(self, name):
        return (self.pkg / name).exists()


@pytest.fixture
def tree(tmp_path):
    return Tree(tmp_path)


def test_the_library_is_built_without_torch(tree):
    tree.torch(None)
    rc, out, calls = tree.build()
    assert rc == 0, out
    assert tree.has("libtreeattn.so") and not tree.has("_serving_calls.so") and set(calls) == {"nvcc"}
    assert tree.build()[2] == []                           # up to date
    tree.torch("2.9.0")                                    # torch arrives: its module is missing, the library is not
    rc, out, calls = tree.build()
    assert rc == 0 and calls == ["cxx"] and tree.has("_serving_calls.so"), out


def test_the_module_is_built_again_for_another_torch(tree):
    tree.torch("2.9.0")
    rc, out, calls = tree.build()
    assert rc == 0 and calls.count("cxx") == 1 and calls.count("nvcc") > 1, out
    assert tree.build()[2] == []
    tree.torch("2.11.0+cu130")
    assert tree.build()[::2] == (0, ["cxx"])
    assert tree.build()[2] == []


def test_a_compiler_that_fails_is_named_and_the_library_stays(tree):
    tree.torch("2.9.0")
    for cxx, why in (("badcxx", "no such header"), ("/nowhere/g++", "/nowhere/g++")):
        rc, out, calls = tree.build(cxx)
        assert rc != 0 and cxx in out and "serving_calls.cpp" in out and why in out and "nvcc failed" not in out
        assert tree.has("libtreeattn.so") and not tree.has("_serving_calls.so")
    rc, out, calls = tree.build()
    assert rc == 0 and calls == ["cxx"], out
