"""The package works from wherever it lies (no GPU): one library per package,
for the ctypes calls and for the module of the attention sublayer's calls."""

import os
import shutil
import subprocess
import sys

import pytest

from mhc_pre_gb300 import build as mbuild

SCRIPT = """
import os
from mhc_pre_gb300 import binding as B
B.lib()
calls = B._calls()
print(os.path.dirname(B.__file__))
print(calls.__file__)
for line in sorted({l.split(None, 5)[5].strip() for l in open('/proc/self/maps') if 'libmhc_gb300.so' in l}):
    print(line)
import torch
q, w = torch.zeros(2, 4, 64), torch.ones(64)
try:
    B.mhc_qk_norm_rope(q, q, w, w)
except ValueError as e:
    print(e)
"""


def _moved(tmp_path):
    mbuild.build()
    where = tmp_path / "elsewhere" / "mhc_pre_gb300"
    shutil.copytree(mbuild.HERE, where, ignore=shutil.ignore_patterns("_build", "__pycache__"))
    return where


def _run(where, script=SCRIPT):
    env = dict(os.environ, PYTHONPATH=str(where.parent))
    r = subprocess.run([sys.executable, "-c", script], cwd=where.parent, env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr
    return r.stdout.splitlines()


def test_a_moved_package_has_one_library(tmp_path):
    where = _moved(tmp_path)
    home, calls, *rest = _run(where)
    assert home == str(where) and os.path.dirname(calls) == str(where)
    assert rest == [str(where / "libmhc_gb300.so"), "the mHC library takes CUDA tensors only"]


def test_two_packages_in_one_process_keep_their_own(tmp_path):
    """Under another name, beside this one."""
    where = _moved(tmp_path)
    shutil.move(where, where.parent / "mhc_other")
    where = where.parent / "mhc_other"
    lines = _run(where, f"""
import sys
sys.path.append({os.path.dirname(mbuild.HERE)!r})
import mhc_pre_gb300.binding as A
import mhc_other.binding as B
A._calls(), B._calls()
assert A._calls() is not B._calls()
for line in sorted({{l.split(None, 5)[5].strip() for l in open('/proc/self/maps') if 'libmhc_gb300.so' in l}}):
    print(line)
""")
    assert sorted(lines) == sorted([mbuild.LIB, str(where / "libmhc_gb300.so")])


def test_the_calls_refuse_to_run_without_a_library(tmp_path):
    where = _moved(tmp_path)
    lines = _run(where, """
from mhc_pre_gb300 import binding as B
import torch
from mhc_pre_gb300 import _attn_calls as calls
q, w = torch.zeros(2, 4, 64), torch.ones(64)
try:
    calls.qk_norm_rope(None, q, q, w, w, None, None, 1e-6, 0)
except RuntimeError as e:
    print(type(e).__name__)
""")
    assert lines == ["RuntimeError"]
