"""How the cache operators' marshalling module calls the library, seen with stand-ins in the library's place."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

_SCRIPT = r"""
import ctypes, sys, torch
sys.path.insert(0, sys.argv[1])
from exact_io_aware_85_b200 import fa
# a function that tells whether its thread holds the interpreter's lock, as each entry point
held = ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value
fa._fa_call.bind(*[held] * 6)
bf, f32, i32, u8 = ({"dtype": t, "device": "cuda"} for t in (torch.bfloat16, torch.float32, torch.int32, torch.uint8))
B, H, Hkv, N, C, d = 1, 2, 1, 8, 128, 64
q, k, w, acc = torch.zeros(B, H, N, d, **bf), torch.zeros(B, Hkv, N, d, **bf), torch.zeros(B, Hkv, N, **f32), torch.zeros(B, Hkv, C, **f32)
cache = (torch.zeros(B, Hkv, C, d // 2, **u8), torch.zeros(B, Hkv, C, **bf)) * 2
n, pos, seen, ws = torch.zeros(B, Hkv, **i32), torch.zeros(B, Hkv, C, **i32), torch.zeros(B, **i32), torch.zeros(256, **u8)
rows = torch.zeros(B, Hkv, 4, **i32)
# status 0 where the lock was let go, FA_ERR_INVALID_ARG (1) where it was held
fa.fa_key_weights(q, k, torch.zeros(B, H, N, **f32), w, True, 0.1, ws)
fa.fa_evict_keep(w, rows, n, 0, 0)
fa.fa_evict_slots(acc, pos, n, seen, rows, C, 0, 0)
fa.fa_kv4_append(k, k, *cache)
fa.fa_kv4_read(*cache, k, k)
fa.fa_decode_kv4(q[:, :, 0].contiguous(), *cache, n, q[:, :, 1].contiguous(), torch.zeros(B, H, **f32), 0.1, ws)
print("done")
"""


@pytest.mark.gpu
def test_other_threads_run_while_the_library_does():
    """A launch blocks while the stream's queue is full; work that is queued before it may need a Python thread."""
    r = subprocess.run([sys.executable, "-c", _SCRIPT, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-2000:]
