"""Queries of the 4-bit decoding step that are far from ordinary: zeros and tiny numbers at tiny softmax scales,
elements that dwarf the others of their head.  Against 64-bit references (helpers, tolerances: test_kv4_cache)."""
import math

import pytest
import torch

import cache_ref as R
from test_kv4_cache import DEV, _bounds, _cache, _randn, _signs

pytestmark = pytest.mark.gpu

# every variant of the kernel: 1 to 4, 5 to 8 and 9 to 16 query heads of a key/value head, plain and rotated
VARIANTS = [(d, g, rot) for d in (64, 128, 256) for g in (1, 3, 4, 6, 8, 12, 16) for rot in (False, True)]


def _decode(q, k, v, lens, scale, signs, weights, C):
    """Outputs of the kernel, and what they should be from the rows that the cache holds."""
    from exact_io_aware_85_b200 import fa
    B, H, d = q.shape
    Hkv = k.shape[1]
    cache = _cache(B, Hkv, C, d)
    n = torch.full((B, Hkv), lens, dtype=torch.int32, device=DEV)
    fa.fa_kv4_append(k, v, *cache, signs=signs)
    o, lse = torch.full((B, H, d), float("nan"), dtype=torch.bfloat16, device=DEV), torch.full((B, H), float("nan"), device=DEV)
    acc = torch.zeros((B, Hkv, C), device=DEV) if weights else None
    ws = torch.full((fa.fa_decode_kv4_workspace_bytes(B, H, Hkv, C, d, weights),), 255, dtype=torch.uint8, device=DEV)
    fa.fa_decode_kv4(q, *cache, n, o, lse, scale, ws, signs=signs, acc=acc)
    torch.cuda.synchronize()
    assert fa.fa_check_status() == fa.FA_OK
    kc = cache[1].cpu().float().nan_to_num(0)
    kr = R.values(cache[0].cpu(), kc, None if signs is None else signs.cpu())
    vr = R.values(cache[2].cpu(), cache[3].cpu().float().nan_to_num(0))
    return o, lse, acc, R.decode(q.cpu().double(), kr, vr, n.cpu(), scale), kc.double()[:, :, :lens].amax(-1)


@pytest.mark.parametrize("d,g,rot", VARIANTS)
def test_queries_of_zeros_and_tiny_numbers_at_tiny_scales(d, g, rot):
    """Scores that are zero, or too small to tell from it: every row in use gets the same weight, at lengths that end
    inside a block of rows, whatever the rows behind hold."""
    C, signs = 512, _signs(d, 7) if rot else None
    for scale in (1e-20, 1e-38, 2.0 ** -149):
        for lens in (1, 33, 511):
            for weights in (False, True):
                q, k, v = _randn(1, 1, 2 * g, d), _randn(2, 1, 2, lens, d), _randn(3, 1, 2, lens, d)
                q[0, 0] = 0                                   # a head of zeros, beside tiny and ordinary ones
                q[0, -1] = 0
                if g > 1:
                    q[0, 1] *= 2.0 ** -115
                o, lse, acc, (ro, rl, rw, pv, terms), _ = _decode(q, k, v, lens, scale, signs, weights, C)
                t_o, t_lse, t_w = _bounds(d, C, terms, rl, pv, ro)
                where = (scale, lens, weights)
                assert ((o.cpu().double() - ro).abs() <= t_o).all(), where
                assert ((lse.cpu().double() - rl).abs() <= t_lse).all(), where
                if weights:
                    assert ((acc.cpu().double() - rw).abs() <= t_w.amax() * rw + 2.0 ** -22 * (1 + rw)).all(), where
                    assert (acc[:, :, lens:] == 0).all(), where
