"""What build() makes where something is missing or has changed (no GPU, no
compiler: nvcc, g++ and torch are stand-ins that write their output files)."""

import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

from mhc_pre_gb300 import build as mbuild

TOOL = """#!/bin/sh
echo "$0 $*" >> "$BUILD_TEST_LOG"
while [ $# -gt 0 ]; do
    if [ "$1" = -o ]; then echo made > "$2"; fi
    shift
done
"""


class Tree:
    """A copy of the package's sources, and stand-ins of the tools on the path."""

    def __init__(self, tmp):
        self.root, self.bin, self.torch = tmp / "tree", tmp / "bin", tmp / "site" / "torch"
        shutil.copytree(mbuild.HERE, self.root / "mhc_pre_gb300",
                        ignore=shutil.ignore_patterns("_build", "__pycache__", "*.so"))
        shutil.copytree(mbuild.INCLUDE, self.root / "include")
        self.bin.mkdir()
        self.log = tmp / "log"
        for tool in ("nvcc", "g++"):
            path = self.bin / tool
            path.write_text(TOOL)
            path.chmod(0o755)

    def have_torch(self, version, headers=True):
        parts = ["include/torch/csrc/autograd/python_variable.h", "lib/libc10_cuda.so"] if headers else []
        for part in parts:
            (self.torch / part).parent.mkdir(parents=True, exist_ok=True)
            (self.torch / part).write_text("")
        self.torch.mkdir(parents=True, exist_ok=True)
        (self.torch / "__init__.py").write_text(
            f"__version__ = {version!r}\ndef compiled_with_cxx11_abi(): return True\n")

    def build(self, path=None):
        """Runs build.py by itself, as one without torch would; what it said, and which tools ran."""
        self.log.write_text("")
        env = dict(os.environ, PATH=path or f"{self.bin}:{os.environ['PATH']}", NVCC=str(self.bin / "nvcc"),
                   BUILD_TEST_LOG=str(self.log), PYTHONPATH=str(self.torch.parent), PYTHONDONTWRITEBYTECODE="1")
        script = self.root / "mhc_pre_gb300" / "build.py"
        # -S: no site-packages, so that only the stand-in of torch can be there
        r = subprocess.run([sys.executable, "-S", str(script)], env=env, capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stderr
        ran = [os.path.basename(line.split()[0]) for line in self.log.read_text().splitlines()]
        return r.stderr, {t: ran.count(t) for t in ("nvcc", "g++")}

    def made(self, name):
        return (self.root / "mhc_pre_gb300" / name).exists()


@pytest.fixture
def tree(tmp_path):
    return Tree(tmp_path)


LIBRARY = len(mbuild.SOURCES) + 1


def test_the_library_needs_no_torch(tree):
    said, ran = tree.build()
    assert "torch is missing" in said and ran == {"nvcc": LIBRARY, "g++": 0}
    assert tree.made("libmhc_gb300.so") and not tree.made("_attn_calls.so")
    assert tree.build()[1] == {"nvcc": 0, "g++": 0}


def test_the_library_needs_no_headers_of_torch(tree):
    tree.have_torch("9.9.0", headers=False)
    said, ran = tree.build()
    assert "python_variable.h is missing" in said and ran == {"nvcc": LIBRARY, "g++": 0}
    assert tree.made("libmhc_gb300.so") and not tree.made("_attn_calls.so")


def test_the_library_needs_no_gxx(tree):
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        pytest.skip("Python's headers are missing: that would be said first")
    tree.have_torch("9.9.0")
    (tree.bin / "g++").unlink()
    said, ran = tree.build(path=str(tree.bin))
    assert "g++ is missing" in said and tree.made("libmhc_gb300.so") and not tree.made("_attn_calls.so")


def test_another_torch_gets_another_module(tree):
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        pytest.skip("Python's headers are missing")
    tree.have_torch("9.9.0")
    said, ran = tree.build()
    assert said == "" and ran == {"nvcc": LIBRARY, "g++": 2} and tree.made("_attn_calls.so")
    assert tree.build()[1] == {"nvcc": 0, "g++": 0}
    tree.have_torch("9.9.1")
    assert tree.build()[1] == {"nvcc": 0, "g++": 2}
    assert tree.build()[1] == {"nvcc": 0, "g++": 0}
    assert "9.9.1" in (tree.root / "mhc_pre_gb300" / "_build" / "py_attn.for").read_text()


def test_a_module_for_another_torch_is_refused(monkeypatch):
    from mhc_pre_gb300 import binding as B
    mbuild.build()
    monkeypatch.setattr(B, "_calls_module", None)
    monkeypatch.setattr(mbuild, "calls_made_for", lambda: "torch 0.1, cpython-27")
    with pytest.raises(RuntimeError, match="was built for torch"):
        B._calls()
