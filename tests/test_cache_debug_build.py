"""The cache operators in the FA_DEBUG build (device-side argument checks on every TMA copy, tensor-memory access
and MMA): no check fails, and the outputs are the release build's bits."""
import os
import subprocess
import sys

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

_SCRIPT = r"""
import math, sys, numpy as np, torch
sys.path.insert(0, sys.argv[1])
from exact_io_aware_85_b200 import fa
assert fa._DEBUG == (sys.argv[2] == "debug")
out, i32 = {}, dict(dtype=torch.int32, device="cuda")
for d, H, Hkv, N, rot in ((64, 3, 3, 333, False), (128, 8, 2, 600, True), (256, 6, 1, 257, True)):
    g = torch.Generator().manual_seed(d)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()
    q, k, v, qt = rnd(1, H, N, d), rnd(1, Hkv, N, d), rnd(1, Hkv, N, d), rnd(1, H, d)
    signs = (torch.randint(0, 2, (d,), generator=g) * 2 - 1).float().cuda() if rot else None
    o, lse = torch.empty_like(q), torch.empty((1, H, N), device="cuda")
    fa.fa_fwd_gqa(q, k, v, o, lse, True, 1 / math.sqrt(d))
    w = torch.empty((1, Hkv, N), device="cuda")
    ws = torch.empty(fa.fa_key_weights_workspace_bytes(1, H, Hkv, N, d, 100), dtype=torch.uint8, device="cuda")
    fa.fa_key_weights(q, k, lse, w, True, 1 / math.sqrt(d), ws, window=100)
    idx, lens = torch.empty((1, Hkv, 200), **i32), torch.empty((1, Hkv), **i32)
    fa.fa_evict_keep(w, idx, lens, 20, 4)
    C = 256
    cache = [torch.zeros((1, Hkv, C, d // 2), dtype=torch.uint8, device="cuda"), torch.zeros((1, Hkv, C), dtype=torch.bfloat16, device="cuda")]
    cache += [t.clone() for t in cache]
    acc, pos = torch.zeros((1, Hkv, C), device="cuda"), torch.zeros((1, Hkv, C), **i32)
    fa.fa_kv4_append(k, v, *cache, signs=signs, rows=idx, w=w, acc=acc, pos=pos)
    ot, lt = torch.empty_like(qt), torch.empty((1, H), device="cuda")
    wsd = torch.empty(fa.fa_decode_kv4_workspace_bytes(1, H, Hkv, C, d, True), dtype=torch.uint8, device="cuda")
    fa.fa_decode_kv4(qt, *cache, lens, ot, lt, 1 / math.sqrt(d), wsd, signs=signs, acc=acc)
    slots = torch.empty((1, Hkv, 3), **i32)
    fa.fa_evict_slots(acc, pos, lens, torch.full((1,), N, **i32), slots, 201, 20, 4)
    kr, vr = rnd(1, Hkv, 3, d), rnd(1, Hkv, 3, d)
    fa.fa_kv4_read(*cache, kr, vr, signs=signs, slots=slots)
    torch.cuda.synchronize()
    assert fa.fa_check_status() == 0, ("status", d)
    for n, t in (("w", w), ("idx", idx), ("o", ot), ("lse", lt), ("acc", acc), ("slots", slots), ("k", kr), ("v", vr)):
        out[f"{n}{d}"] = t.float().cpu().numpy()
np.savez(sys.argv[3], **out)
"""


@pytest.mark.gpu
def test_cache_operators_pass_the_device_checks(tmp_path):
    from exact_io_aware_85_b200 import build
    build.build_library(debug=True)
    res = {}
    for mode in ("release", "debug"):
        env = dict(os.environ, FA_DEBUG="1" if mode == "debug" else "0")
        path = str(tmp_path / f"{mode}.npz")
        r = subprocess.run([sys.executable, "-c", _SCRIPT, ROOT, mode, path], env=env, capture_output=True, text=True,
                           timeout=600)
        assert r.returncode == 0, r.stderr[-2000:]
        res[mode] = dict(np.load(path))
    for key, a in res["release"].items():
        assert np.array_equal(a, res["debug"][key]), key
