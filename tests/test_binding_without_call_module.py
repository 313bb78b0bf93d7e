"""The package without the cache operators' marshalling module (_fa_call.so): everything else works, and those
operators say what is missing and why."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

_SCRIPT = r"""
import sys
sys.path.insert(0, sys.argv[1])
import torch
from exact_io_aware_85_b200 import fa
assert fa.__file__.startswith(sys.argv[1])
assert fa.fa_status_string(0) == "FA_OK"
assert fa.fa_decode_workspace_bytes(1, 8, 2, 1000, 128) > 0
assert fa.fa_key_weights_workspace_bytes(1, 8, 2, 1000, 128, 64) > 0
q = torch.zeros((1, 2, 8, 64), dtype=torch.bfloat16)
lse = torch.zeros((1, 2, 8))
for call in (lambda: fa.fa_fwd(q, q, q, q, lse, False, 0.125),
             lambda: fa.fa_decode(q[:, :, 0], q, q, q[:, :, 0], lse[:, :, 0], 0.125, torch.zeros(256, dtype=torch.uint8))):
    try:
        call()
    except fa.FAError as e:      # host tensors: the ordinary refusal
        assert e.status == fa.FA_ERR_INVALID_ARG
    else:
        raise SystemExit("host tensors were taken")
i32 = dict(dtype=torch.int32)
cache = (torch.zeros((1, 1, 128, 32), dtype=torch.uint8), torch.zeros((1, 1, 128), dtype=torch.bfloat16)) * 2
for call in (lambda: fa.fa_evict_keep(torch.zeros(1, 1, 8), torch.zeros(1, 1, 4, **i32), torch.zeros(1, 1, **i32), 0, 0),
             lambda: fa.fa_evict_slots(*[None] * 5, 4, 0, 0), lambda: fa.fa_kv4_append(q, q, *cache),
             lambda: fa.fa_kv4_read(*cache, q, q), lambda: fa.fa_key_weights(q, q, lse, lse, True, 0.125, None),
             lambda: fa.fa_decode_kv4(q[:, :, 0], *cache, None, None, None, 0.125, None)):
    try:
        call()
    except ImportError as e:
        assert "_fa_call.so" in str(e) and sys.argv[2] in str(e) and "exact_io_aware_85_b200.build" in str(e), str(e)
    else:
        raise SystemExit("ran without its module")
print("done")
"""


@pytest.mark.parametrize("how,said", [("missing", "No module named"), ("broken", "file too short")])
def test_only_the_cache_operators_need_the_module(tmp_path, how, said):
    from exact_io_aware_85_b200 import build
    build.build_library()
    pkg = tmp_path / "exact_io_aware_85_b200"
    pkg.mkdir()
    for f in ("__init__.py", "build.py", "fa.py", "synth.py", "libfa.so"):
        shutil.copy2(os.path.join(build.PKG, f), pkg / f)
    if how == "broken":       # such as one of another Python or torch: the loader's own words have to come through
        (pkg / "_fa_call.so").write_bytes(b"")
    env = dict(os.environ, FA_DEBUG="0")
    r = subprocess.run([sys.executable, "-c", _SCRIPT, str(tmp_path), said], env=env, cwd=str(tmp_path),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-2000:]
