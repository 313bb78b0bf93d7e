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


@pytest.fixture
def step(tmp_path, monkeypatch):
    """The build step of a copy whose module compiler writes a word; `step()` tells whether it was called."""
    import importlib.util
    _package(tmp_path)
    spec = importlib.util.spec_from_file_location("build_copy", tmp_path / "exact_io_aware_85_b200" / "build.py")
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    calls, ok = [], [True]

    def run(cmd, check):
        calls.append(cmd)
        if not ok[0]:
            raise subprocess.CalledProcessError(1, cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("module")

    monkeypatch.setattr(build.subprocess, "run", run)

    def go():
        n = len(calls)
        build.build_call()
        return len(calls) > n

    go.build, go.ok = build, ok
    return go


def _older(path, than):
    t = os.path.getmtime(than) - 10
    os.utime(path, (t, t))


def test_the_module_follows_what_it_is_made_of(step):
    """It is called by hand-made signatures and linked against torch: built again when its source, the header or
    the build step are newer, and under another torch or Python."""
    import torch
    build = step.build
    assert step() and not step()
    for path in (os.path.join(build.CSRC, "call.cpp"), build.HEADER, build.__file__):
        _older(build.CALL, path)
        assert step() and not step(), path
    for name in ("torch.__version__", "sys.version"):
        with pytest.MonkeyPatch.context() as m:
            if name == "sys.version":
                m.setattr(sys, "version", "4.0.0 of another day")
            else:
                m.setattr(torch, "__version__", "3.0.0+of_another_day")
            assert step() and not step(), name
        assert step() and not step(), name


def test_a_module_that_could_not_be_built_again_is_gone(step):
    """The one from before would be called with arguments in other places."""
    build = step.build
    assert step()
    _older(build.CALL, build.HEADER)
    step.ok[0] = False
    with pytest.raises(subprocess.CalledProcessError):
        step()
    assert not os.path.exists(build.CALL)
    step.ok[0] = True
    assert step() and not step()


def test_the_module_is_compiled_against_the_prototypes(tmp_path):
    """A header that asks for one more argument: the module's six calls do not compile."""
    import re

    from exact_io_aware_85_b200 import build
    (tmp_path / "pkg" / "csrc").mkdir(parents=True)
    (tmp_path / "include").mkdir()
    shutil.copy(os.path.join(build.CSRC, "call.cpp"), tmp_path / "pkg" / "csrc")
    header = open(build.HEADER).read()
    for f in ("fa_key_weights", "fa_evict_keep", "fa_evict_slots", "fa_kv4_append", "fa_kv4_read", "fa_decode_kv4"):
        header, n = re.subn(rf"(int {f}\([^)]*)\)", r"\1, int more)", header)
        assert n == 1, f
    (tmp_path / "include" / "fa.h").write_text(header)
    cmd = build.call_command(str(tmp_path / "out.so"))
    cmd[cmd.index(os.path.join(build.CSRC, "call.cpp"))] = str(tmp_path / "pkg" / "csrc" / "call.cpp")
    r = subprocess.run([*cmd, "-fsyntax-only"], capture_output=True, text=True, timeout=300)
    assert r.returncode != 0 and r.stderr.count("too few arguments") == 6, r.stderr[-2000:]
