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


# (rotated, the element's product with the keys' own rounding makes scores that a larger one would only drown)
@pytest.mark.parametrize("d,g,rot,power", [(*v, p) for v in VARIANTS if v[1] in (1, 4, 8, 16) for p in ((8,) if v[2] else (8, 14))])
def test_a_large_element_that_meets_zeros(d, g, rot, power):
    """One element of the query 2^power times the others, where every key holds zero: it takes no part in a score, but
    its products with the codes, held as c + 8, do, until 8 sum(q) leaves again.

    Tolerance.  A score is scale ks (sum q_i n_i - 8 sum q_i), n_i = c_i + 8 <= 15, in the basis of the codes: an fp32
    accumulator that starts at -8 sum q (d / 32 + 5 additions, each rounded to 2^-24 of 8 sum|q| at most) and takes
    d / 16 products of 16 elements (twice that where q is held as two numbers), its contents at most 23 sum|q|.  Of the
    17 numbers that such a step adds up, each may be cut at 2^-24 of the largest:
    (d / 16 17 23 + (d / 32 + 5) 8) 2^-24 < d 2^-19 (d 2^-18 where held as two), times scale ks sum|q|."""
    C, lens, signs = 512, 500, _signs(d, 7) if rot else None
    q, k, v = _randn(1, 1, 2 * g, d), _randn(2, 1, 2, lens, d), _randn(3, 1, 2, lens, d)
    q[..., 5] = 2.0 ** power
    k[..., 5] = 0
    scale = 1 / math.sqrt(d)
    o, lse, acc, (ro, rl, rw, pv, terms), ks = _decode(q, k, v, lens, scale, signs, True, C)
    qh = q.cpu().double() if signs is None else R.rotate(q.cpu().double(), signs.cpu()) / d
    size = scale * ks.repeat_interleave(g, 1) * qh.abs().sum(-1)
    es = d * 2.0 ** (-18 if rot else -19) * size
    # terms of the scores in the codes' basis: at most 7 scale ks sum|q|
    t_o, t_lse, t_w = _bounds(d, C, 7 * size if rot else terms, rl, pv, ro)
    assert ((o.cpu().double() - ro).abs() <= t_o + 2 * es[..., None] * pv).all()
    assert ((lse.cpu().double() - rl).abs() <= t_lse + es).all()
    assert ((acc.cpu().double() - rw).abs() <= (t_w + 2 * es).amax() * rw + 2.0 ** -22 * (1 + rw)).all()


@pytest.mark.parametrize("power", [-110, -100, -60, 60, 100])
@pytest.mark.parametrize("rot", [False, True])
def test_keys_of_any_size(rot, power):
    """Keys far from one, with a softmax scale that brings the scores back."""
    d, g, C, lens = 128, 4, 256, 200
    signs = _signs(d, 4) if rot else None
    k = (_randn(2, 1, 2, lens, d).float() * 2.0 ** power).to(torch.bfloat16)
    q, v = _randn(1, 1, 2 * g, d), _randn(3, 1, 2, lens, d)
    scale = 2.0 ** -power / math.sqrt(d)
    o, lse, acc, (ro, rl, rw, pv, terms), ks = _decode(q, k, v, lens, scale, signs, True, C)
    qh = q.cpu().double() if signs is None else R.rotate(q.cpu().double(), signs.cpu()) / d
    size = scale * ks.repeat_interleave(g, 1) * qh.abs().sum(-1)       # see above
    es = d * 2.0 ** (-18 if rot else -19) * size
    t_o, t_lse, t_w = _bounds(d, C, 7 * size if rot else terms, rl, pv, ro)
    assert ((o.cpu().double() - ro).abs() <= t_o + 2 * es[..., None] * pv).all()
    assert ((lse.cpu().double() - rl).abs() <= t_lse + es).all()
    assert ((acc.cpu().double() - rw).abs() <= (t_w + 2 * es).amax() * rw + 2.0 ** -22 * (1 + rw)).all()
