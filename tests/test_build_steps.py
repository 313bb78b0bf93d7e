"""The build step: what it needs, and when it builds again.  Compilers are stand-ins here: nothing is compiled."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

_SCRIPT = r"""
import sys, warnings
sys.path.insert(0, sys.argv[1])
if sys.argv[2] == "no torch":
    sys.modules["torch"] = None      # an import of it fails
from exact_io_aware_85_b200 import build
assert build.__file__.startswith(sys.argv[1])
with warnings.catch_warnings(record=True) as said:
    warnings.simplefilter("always")
    out = build.build_library()
assert open(out).read() == "library"
assert any("_fa_call.so" in str(w.message) for w in said), [str(w.message) for w in said]
try:
    build.build_call()
except Exception as e:
    print("refused", type(e).__name__)
"""


def _package(tmp_path):
    """A copy of the package's sources without anything built, and a compiler of the library that writes a word."""
    pkg = tmp_path / "exact_io_aware_85_b200"
    shutil.copytree(os.path.join(ROOT, "exact_io_aware_85_b200"), pkg, ignore=shutil.ignore_patterns("*.so*", "*.stamp", "__pycache__"))
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    bin_ = tmp_path / "bin"
    bin_.mkdir()
    for name, body in (("nvcc", 'while [ "$1" != -o ]; do shift; done; printf library > "$2"'),
                       ("g++", "echo 'fatal error: Python.h: No such file or directory' >&2; exit 1")):
        (bin_ / name).write_text(f"#!/bin/sh\n{body}\n")
        (bin_ / name).chmod(0o755)
    return dict(os.environ, PATH=f"{bin_}:{os.environ['PATH']}")


@pytest.mark.parametrize("lacks", ["no torch", "no headers"])
def test_the_library_needs_nvcc_alone(tmp_path, lacks):
    env = _package(tmp_path)
    r = subprocess.run([sys.executable, "-c", _SCRIPT, str(tmp_path), lacks], env=env, cwd=str(tmp_path), capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "refused" in r.stdout, r.stderr[-2000:]
