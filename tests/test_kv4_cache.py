"""Rows into and out of the 4-bit cache, and the decoding step over it, against 64-bit references.

Tolerances (eps/2 = half a step relative: bf16 2^-8, fp16 2^-11, fp32 2^-24):
* codes: a value goes to the nearest code; the kernel forms a rotated value in fp32 by log2(d) additions, so it
  may be off by log2(d) 2^-24 sum|x|, and only a code whose border lies that near may differ, by one.
* read rows: one rounding to bf16 of an exact value: 2^-8 relative.
* decode O: the rounding of O (2^-8 |o|), of the weights before P V (at most a bf16 rounding, 2^-8 sum p|v|), and
  fp32 arithmetic (2^-16 sum p|v| covers 2^8 additions in a row).
* decode LSE, weights: scores are sums of d products of exact codes with q, which is held with at least 16 bits
  (2^-17): (2^-17 + d 2^-24) times the sum of the terms' magnitudes; exponent and logarithm arguments are rounded
  in fp32 (|x| 2^-22 with x in log2 units), sums of N terms in chains of at most N/128 + 64.
"""
import math

import pytest
import torch

import cache_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _cache(B, Hkv, C, d, fill=True):
    """A cache whose unused rows hold what must not matter: NaN scales, random codes."""
    kc, vc = (torch.randint(0, 256, (B, Hkv, C, d // 2), dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((B, Hkv, C), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    return [kc, ks, vc, vs]


def _signs(d, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randint(0, 2, (d,), generator=g) * 2 - 1).float().to(DEV)


def _randn(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16).to(DEV)


def _check_rows(packed, scale, x, signs):
    """Codes and scales written for rows x (bf16 on the GPU)."""
    x = x.cpu().double()
    c, s, y = R.quantise(x, None if signs is None else signs.cpu())
    got_s, got_c = scale.cpu().double(), R.unpack(packed.cpu())
    near = 0.0 if signs is None else math.log2(x.shape[-1]) * 2.0 ** -24
    size = x.abs().sum(-1)
    assert ((got_s - s).abs() <= (near * size / 7 + 0) * 2 + (0 if signs is None else 1) * s * 2.0 ** -7).all()
    same = got_s == s
    if signs is None:
        assert same.all()
    assert same.float().mean() > 0.99
    t = y / torch.where(s > 0, s, torch.ones_like(s))[..., None]
    border = (t - torch.floor(t) - 0.5).abs() * s[..., None]
    wrong = (got_c != c) & same[..., None]
    assert (border[wrong] <= (near * size)[..., None].expand_as(border)[wrong]).all()
    assert ((got_c - c).abs()[same] <= 1).all()


@pytest.mark.parametrize("B,Hkv,N,C,d,rot", [(1, 1, 1, 128, 64, False), (2, 3, 130, 256, 64, True),
                                             (2, 2, 77, 128, 128, True), (1, 2, 300, 384, 128, False),
                                             (1, 2, 129, 256, 256, True), (3, 1, 5, 128, 256, False)])
def test_append_and_read(B, Hkv, N, C, d, rot):
    from exact_io_aware_85_b200 import fa
    k, v = _randn(N + d, B, Hkv, N, d), _randn(N + d + 1, B, Hkv, N, d)
    k[..., 3] *= 20  # a channel of outliers
    signs = _signs(d, 5) if rot else None
    cache = _cache(B, Hkv, C, d)
    before = [t.clone() for t in cache]
    fa.fa_kv4_append(k, v, *cache, signs=signs)
    torch.cuda.synchronize()
    _check_rows(cache[0][:, :, :N], cache[1][:, :, :N], k, signs)
    _check_rows(cache[2][:, :, :N], cache[3][:, :, :N], v, None)
    for t, b in zip(cache, before):  # rows behind stay as they were
        assert torch.equal(t[:, :, N:].view(torch.uint8), b[:, :, N:].view(torch.uint8))
    ko, vo = torch.empty((B, Hkv, C, d), dtype=torch.bfloat16, device=DEV), torch.empty((B, Hkv, C, d), dtype=torch.bfloat16, device=DEV)
    lens = torch.full((B, Hkv), N, dtype=torch.int32, device=DEV)
    fa.fa_kv4_read(*cache, ko, vo, signs=signs, lens=lens)
    for got, at, sg in ((ko, 0, signs), (vo, 2, None)):
        want = R.values(cache[at][:, :, :N].cpu(), cache[at + 1][:, :, :N].cpu(), None if sg is None else sg.cpu())
        assert ((got[:, :, :N].cpu().double() - want).abs() <= 2.0 ** -8 * want.abs()).all()
        assert (got[:, :, N:] == 0).all()


def test_append_rows_slots_start_and_counts():
    """Gathered source rows, scattered cache rows, offsets, ragged counts, rows out of range on either side."""
    from exact_io_aware_85_b200 import fa
    B, Hkv, N, C, d = 2, 2, 40, 256, 64
    k, v = _randn(1, B, Hkv, N, d), _randn(2, B, Hkv, N, d)
    w = torch.rand((B, Hkv, N + 3), device=DEV)
    base = torch.tensor([100, 7], dtype=torch.int32, device=DEV)
    whole = _cache(B, Hkv, 128, d)
    fa.fa_kv4_append(k, v, *whole)
    rows = torch.tensor([5, -1, 39, 40, 0, 5], dtype=torch.int32, device=DEV).expand(B, Hkv, 6).contiguous()
    slots = torch.tensor([255, 3, 17, 18, -1, 256], dtype=torch.int32, device=DEV).expand(B, Hkv, 6).contiguous()
    cache = _cache(B, Hkv, C, d)
    before = [t.clone() for t in cache]
    acc, pos = torch.full((B, Hkv, C), -1.0, device=DEV), torch.full((B, Hkv, C), -1, dtype=torch.int32, device=DEV)
    fa.fa_kv4_append(k, v, *cache, rows=rows, slots=slots, w=w, acc=acc, pos=pos, base=base)
    written = {255: 5, 17: 39}  # the others name no source or no cache row
    for b in range(B):
        for h in range(Hkv):
            for r in range(C):
                if r in written:
                    for t, s in zip(cache, whole):
                        assert torch.equal(t[b, h, r], s[b, h, written[r]])
                    assert acc[b, h, r] == w[b, h, written[r]] and pos[b, h, r] == base[b] + written[r]
    keep = torch.ones(C, dtype=torch.bool, device=DEV)
    keep[[255, 17]] = False
    for t, s in zip(cache, before):
        assert torch.equal(t[:, :, keep].view(torch.uint8), s[:, :, keep].view(torch.uint8))
    assert (acc[:, :, keep] == -1).all() and (pos[:, :, keep] == -1).all()
    # an offset per head and ragged counts; without w the weight starts at zero
    start = torch.tensor([[0, 230], [-3, 9]], dtype=torch.int32, device=DEV)
    n_new = torch.tensor([[40, 40], [10, 0]], dtype=torch.int32, device=DEV)
    cache = _cache(B, Hkv, C, d)
    pos.fill_(-1)
    fa.fa_kv4_append(k, v, *cache, start=start, n_new=n_new, acc=acc, pos=pos)
    for b in range(B):
        for h in range(Hkv):
            for t in range(int(n_new[b, h])):
                r = int(start[b, h]) + t
                if 0 <= r < C:
                    assert torch.equal(cache[0][b, h, r], whole[0][b, h, t]) and pos[b, h, r] == t and acc[b, h, r] == 0
    assert int((pos >= 0).sum()) == 40 + 26 + 7 + 0
    ko = torch.empty((B, Hkv, 6, d), dtype=torch.bfloat16, device=DEV)
    vo = torch.empty_like(ko)
    fa.fa_kv4_read(*whole, ko, vo, slots=rows)
    full, fullv = torch.empty((B, Hkv, 128, d), dtype=torch.bfloat16, device=DEV), torch.empty((B, Hkv, 128, d), dtype=torch.bfloat16, device=DEV)
    fa.fa_kv4_read(*whole, full, fullv)
    for t, r in enumerate([5, None, 39, 40, 0, 5]):
        if r is None:
            assert (ko[:, :, t] == 0).all() and (vo[:, :, t] == 0).all()
        elif r < N:
            assert torch.equal(ko[:, :, t], full[:, :, r]) and torch.equal(vo[:, :, t], fullv[:, :, r])


@pytest.mark.parametrize("rot", [False, True])
def test_append_values_that_break_a_scale(rot):
    """Zeros, numbers near the ends of bf16's range, an infinity, a NaN."""
    from exact_io_aware_85_b200 import fa
    d = 128
    k = torch.zeros((1, 1, 7, d), dtype=torch.bfloat16, device=DEV)
    k[0, 0, 1] = 1e-40
    k[0, 0, 2, 5] = 3e38
    k[0, 0, 3, 7] = float("inf")
    k[0, 0, 4, 9] = float("nan")
    k[0, 0, 5, 11] = -float("inf")
    k[0, 0, 6] = 1.0
    signs = _signs(d, 3) if rot else None
    cache = _cache(1, 1, 128, d)
    fa.fa_kv4_append(k, k, *cache, signs=signs)
    scales = cache[3][0, 0, :7].float()
    assert scales[0] == 0 and (cache[2][0, 0, 0] == 0x88).all()
    assert torch.isnan(scales[3:6]).all() and torch.isfinite(scales[[0, 1, 2, 6]]).all()
    assert torch.isnan(cache[1][0, 0, 3:6].float()).all()
    assert ((cache[2][0, 0, :7] & 15) > 0).all() and ((cache[2][0, 0, :7] >> 4) > 0).all()
    out, outv = (torch.empty((1, 1, 7, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    fa.fa_kv4_read(*cache, out, outv, signs=signs)
    assert torch.isnan(out[0, 0, 3:6].float()).all() and torch.isnan(outv[0, 0, 3:6].float()).all()
    assert (out[0, 0, 0] == 0).all() and torch.isfinite(outv[0, 0, 2].float()).all()
    assert abs(float(outv[0, 0, 2, 5]) / 3e38 - 1) < 2.0 ** -6


def _bounds(d, N, terms, lse, pv, o):
    es = (2.0 ** -17 + d * 2.0 ** -24) * terms
    x = (lse.abs() + terms) / math.log(2) * 2.0 ** -22
    chain = (N / 128 + 64) * 2.0 ** -24
    t_lse = es + x + chain + 2.0 ** -21
    t_o = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -16) * pv + (2 * (es + x)[..., None]) * pv
    return t_o, t_lse, 2 * t_lse


CASES = [
    # B, H, Hkv, C, d, rotated, weights, lens (one per sequence; heads of one differ by one row)
    (1, 1, 1, 128, 64, False, True, [1]),
    (1, 4, 4, 128, 128, True, True, [0]),
    (2, 8, 2, 256, 128, False, True, [256, 17]),
    (2, 8, 2, 640, 128, True, True, [129, 640]),
    (3, 12, 4, 384, 64, True, True, [15, 16, 384]),
    (1, 16, 1, 1024, 64, False, True, [1000]),
    (1, 24, 2, 512, 128, True, True, [511]),
    (2, 16, 1, 768, 256, True, True, [640, 3]),
    (1, 6, 6, 2048, 256, False, False, [2047]),
    (2, 10, 2, 4224, 128, False, False, [4200, 0]),
    (1, 8, 1, 9088, 256, False, True, [9000]),
    (1, 3, 1, 70016, 128, True, True, [70001]),
    (40, 8, 8, 256, 64, False, True, [(i * 37) % 257 for i in range(40)]),
]


@pytest.mark.parametrize("B,H,Hkv,C,d,rot,weights,lens", CASES)
def test_decode_matches_reference(B, H, Hkv, C, d, rot, weights, lens):
    from exact_io_aware_85_b200 import fa
    seed = C + d + H
    lens = torch.tensor([[max(0, n - (h % 2)) for h in range(Hkv)] for n in lens], dtype=torch.int32)
    k, v = _randn(seed, B, Hkv, C, d), _randn(seed + 1, B, Hkv, C, d)
    q = _randn(seed + 2, B, H, d)
    signs = _signs(d, seed) if rot else None
    cache = _cache(B, Hkv, C, d)
    fa.fa_kv4_append(k, v, *cache, signs=signs, n_new=lens.to(DEV))
    acc0 = torch.rand((B, Hkv, C), device=DEV)
    acc = acc0.clone() if weights else None
    o = torch.full((B, H, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B, H), float("nan"), device=DEV)
    ws = torch.full((fa.fa_decode_kv4_workspace_bytes(B, H, Hkv, C, d, weights),), 255, dtype=torch.uint8, device=DEV)
    scale = 1 / math.sqrt(d)
    fa.fa_decode_kv4(q, *cache, lens.to(DEV), o, lse, scale, ws, signs=signs, acc=acc)
    torch.cuda.synchronize()
    assert fa.fa_check_status() == fa.FA_OK
    kr = R.values(cache[0].cpu(), cache[1].cpu().float().nan_to_num(0), None if signs is None else signs.cpu())
    vr = R.values(cache[2].cpu(), cache[3].cpu().float().nan_to_num(0))
    # the terms of a score are those of the basis in which the cache holds the keys
    ro, rl, rw, pv, terms = R.decode(q.cpu().double(), kr, vr, lens, scale)
    if signs is not None:
        qh = R.rotate(q.cpu().double(), signs.cpu()) / d
        kh = R.values(cache[0].cpu(), cache[1].cpu().float().nan_to_num(0))
        terms = R.decode(qh, kh, vr, lens, scale)[4]
    live = torch.isfinite(rl)
    t_o, t_lse, t_w = _bounds(d, C, terms, torch.where(live, rl, torch.zeros_like(rl)), pv, ro)
    assert ((o.cpu().double() - ro).abs() <= t_o).all()
    assert (lse.cpu()[~live] == -math.inf).all() and (o.cpu()[~live] == 0).all()
    assert ((lse.cpu().double() - rl).abs() <= t_lse)[live].all()
    if weights:
        got = acc.cpu().double() - acc0.cpu().double()
        t = t_w.view(B, Hkv, -1).amax(-1)[..., None] * rw + 2.0 ** -22 * (1 + rw)
        assert ((got - rw).abs() <= t).all()
        for b in range(B):
            for h in range(Hkv):
                n = int(lens[b, h])
                assert torch.equal(acc[b, h, n:], acc0[b, h, n:])


def test_decode_peaked_and_growing_scores():
    """Scores that grow along the cache (the running maximum moves all the time) and one key that takes all."""
    from exact_io_aware_85_b200 import fa
    B, H, Hkv, C, d = 1, 4, 1, 2048, 128
    k = torch.randn((B, Hkv, C, d)) * 0.05
    q = torch.ones((B, H, d))
    q[:, 1] = -1
    q[:, 2] = 4
    k += torch.linspace(-3, 3, C)[None, None, :, None]
    v = torch.randn((B, Hkv, C, d))
    q, k, v = (t.to(torch.bfloat16).to(DEV) for t in (q, k, v))
    cache = _cache(B, Hkv, C, d)
    fa.fa_kv4_append(k, v, *cache)
    lens = torch.full((B, Hkv), C, dtype=torch.int32, device=DEV)
    o, lse, acc = torch.empty((B, H, d), dtype=torch.bfloat16, device=DEV), torch.empty((B, H), device=DEV), torch.zeros((B, Hkv, C), device=DEV)
    ws = torch.empty(fa.fa_decode_kv4_workspace_bytes(B, H, Hkv, C, d, True), dtype=torch.uint8, device=DEV)
    fa.fa_decode_kv4(q, *cache, lens, o, lse, 0.25, ws, acc=acc)
    kr, vr = (R.values(cache[a].cpu(), cache[a + 1].cpu().float()) for a in (0, 2))
    ro, rl, rw, pv, terms = R.decode(q.cpu().double(), kr, vr, lens.cpu(), 0.25)
    t_o, t_lse, t_w = _bounds(d, C, terms, rl, pv, ro)
    assert ((o.cpu().double() - ro).abs() <= t_o).all()
    assert ((lse.cpu().double() - rl).abs() <= t_lse).all()
    assert ((acc.cpu().double() - rw).abs() <= t_w.amax() * rw + 2.0 ** -22 * (1 + rw)).all()


def test_decode_value_scales_of_any_size():
    """Rows of V whose scales differ by many orders of magnitude, and rows of zeros: what a light key with large
    values gives has to survive beside a heavy key with small ones."""
    from exact_io_aware_85_b200 import fa
    B, H, Hkv, C, d = 1, 8, 2, 512, 64
    g = torch.Generator().manual_seed(9)
    k = torch.randn((B, Hkv, C, d), generator=g)
    v = torch.randn((B, Hkv, C, d), generator=g) * 10.0 ** (torch.randint(-12, 13, (B, Hkv, C, 1), generator=g).float())
    v[:, 1] *= 1e-20
    v[:, :, ::5] = 0
    q = torch.randn((B, H, d), generator=g)
    q, k, v = (t.to(torch.bfloat16).to(DEV) for t in (q, k, v))
    cache = _cache(B, Hkv, C, d)
    fa.fa_kv4_append(k, v, *cache)
    lens = torch.full((B, Hkv), C, dtype=torch.int32, device=DEV)
    o, lse = torch.empty((B, H, d), dtype=torch.bfloat16, device=DEV), torch.empty((B, H), device=DEV)
    ws = torch.empty(fa.fa_decode_kv4_workspace_bytes(B, H, Hkv, C, d, False), dtype=torch.uint8, device=DEV)
    fa.fa_decode_kv4(q, *cache, lens, o, lse, 0.5, ws)
    kr, vr = (R.values(cache[a].cpu(), cache[a + 1].cpu().float()) for a in (0, 2))
    ro, rl, _, pv, terms = R.decode(q.cpu().double(), kr, vr, lens.cpu(), 0.5)
    t_o, t_lse, _ = _bounds(d, C, terms, rl, pv, ro)
    assert ((o.cpu().double() - ro).abs() <= t_o).all()
    assert ((lse.cpu().double() - rl).abs() <= t_lse).all()


def test_decode_nan_stays_in_its_head():
    """A row that was not finite makes its head's outputs NaN, and no other head's."""
    from exact_io_aware_85_b200 import fa
    B, H, Hkv, C, d = 1, 4, 2, 256, 128
    k, v = _randn(1, B, Hkv, C, d), _randn(2, B, Hkv, C, d)
    k[0, 1, 40, 3] = float("inf")
    q = _randn(3, B, H, d)
    cache = _cache(B, Hkv, C, d)
    fa.fa_kv4_append(k, v, *cache)
    lens = torch.full((B, Hkv), 200, dtype=torch.int32, device=DEV)
    o, lse = torch.empty((B, H, d), dtype=torch.bfloat16, device=DEV), torch.empty((B, H), device=DEV)
    ws = torch.empty(fa.fa_decode_kv4_workspace_bytes(B, H, Hkv, C, d, False), dtype=torch.uint8, device=DEV)
    fa.fa_decode_kv4(q, *cache, lens, o, lse, 0.1, ws)
    assert torch.isfinite(o[0, :2].float()).all() and torch.isfinite(lse[0, :2]).all()
    assert torch.isnan(o[0, 2:].float()).all() and torch.isnan(lse[0, 2:]).all()
    lens[0, 1] = 40  # behind the last row it does not matter
    fa.fa_decode_kv4(q, *cache, lens, o, lse, 0.1, ws)
    assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()


def test_lengths_outside_the_cache_are_clamped():
    from exact_io_aware_85_b200 import fa
    B, H, Hkv, C, d = 2, 2, 1, 256, 64
    k, v, q = _randn(1, B, Hkv, C, d), _randn(2, B, Hkv, C, d), _randn(3, B, H, d)
    cache = _cache(B, Hkv, C, d)
    fa.fa_kv4_append(k, v, *cache)
    ws = torch.empty(fa.fa_decode_kv4_workspace_bytes(B, H, Hkv, C, d, True), dtype=torch.uint8, device=DEV)
    out = []
    for lens in ([[C + 5], [-4]], [[C], [0]]):
        o, lse = torch.empty((B, H, d), dtype=torch.bfloat16, device=DEV), torch.empty((B, H), device=DEV)
        acc = torch.zeros((B, Hkv, C), device=DEV)
        fa.fa_decode_kv4(q, *cache, torch.tensor(lens, dtype=torch.int32, device=DEV), o, lse, 0.125, ws, acc=acc)
        out.append((o, lse, acc))
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_decode_is_repeatable_on_streams_and_in_graphs():
    """The same bits every time: again, on another stream, from a graph that follows the lengths, and from two
    graphs that share a workspace and run one after the other."""
    from exact_io_aware_85_b200 import fa
    B, H, Hkv, C, d = 2, 8, 2, 1024, 128
    k, v, q = _randn(1, B, Hkv, C, d), _randn(2, B, Hkv, C, d), _randn(3, B, H, d)
    signs = _signs(d, 1)
    cache = _cache(B, Hkv, C, d)
    fa.fa_kv4_append(k, v, *cache, signs=signs)
    ws = torch.empty(fa.fa_decode_kv4_workspace_bytes(B, H, Hkv, C, d, True), dtype=torch.uint8, device=DEV)
    lens = torch.full((B, Hkv), 700, dtype=torch.int32, device=DEV)

    def buffers():
        return (torch.zeros((B, H, d), dtype=torch.bfloat16, device=DEV), torch.zeros((B, H), device=DEV),
                torch.zeros((B, Hkv, C), device=DEV))

    def step(b, stream=None):
        fa.fa_decode_kv4(q, *cache, lens, b[0], b[1], 0.08, ws, signs=signs, acc=b[2], stream=stream)

    first, again, other, g1, g2 = (buffers() for _ in range(5))
    step(first)
    step(again)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(other, side)
    torch.cuda.synchronize()
    graphs = []
    for b in (g1, g2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(b)
        graphs.append(graph)
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for b in (again, other, g1, g2):
        assert all(torch.equal(x, y) for x, y in zip(first, b))
    lens.fill_(123)
    for b in (first, g1):
        b[2].zero_()
    step(first)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, g1))
    assert fa.fa_check_status() == fa.FA_OK


def test_binding_refusals_on_a_gpu():
    from exact_io_aware_85_b200 import fa
    B, H, Hkv, C, d = 1, 2, 1, 128, 64
    cache = _cache(B, Hkv, C, d)
    q = torch.zeros((B, H, d), dtype=torch.bfloat16, device=DEV)
    o, lse = torch.empty_like(q), torch.empty((B, H), device=DEV)
    lens = torch.zeros((B, Hkv), dtype=torch.int32, device=DEV)
    ws = torch.empty(fa.fa_decode_kv4_workspace_bytes(B, H, Hkv, C, d, False), dtype=torch.uint8, device=DEV)
    good = dict(q=q, kc=cache[0], ks=cache[1], vc=cache[2], vs=cache[3], lens=lens, o=o, lse=lse, scale=0.1, workspace=ws)
    fa.fa_decode_kv4(**good)
    for name, bad in (("q", q.float()), ("q", q[:, :1]), ("ks", cache[1].float()), ("vc", cache[2].cpu()),
                      ("lens", lens.long()), ("lens", lens[0]), ("o", None), ("workspace", ws[:256]),
                      ("vs", cache[3].transpose(0, 2)), ("lse", lse.expand(B, H).double())):
        with pytest.raises(fa.FAError):
            fa.fa_decode_kv4(**dict(good, **{name: bad}))
    with pytest.raises(fa.FAError):
        fa.fa_decode_kv4(**dict(good, acc=torch.zeros((B, Hkv, C), device=DEV)))  # the workspace is too small with acc


@pytest.mark.parametrize("power", [-100, -60, 60, 100])
def test_decode_queries_of_any_size(power):
    """Queries far from one, with a softmax scale that brings the scores back."""
    from exact_io_aware_85_b200 import fa
    B, H, Hkv, C, d = 1, 4, 2, 256, 64
    q = (_randn(1, B, H, d).float() * 2.0 ** power).to(torch.bfloat16)
    k, v = _randn(2, B, Hkv, C, d), _randn(3, B, Hkv, C, d)
    for signs in (None, _signs(d, 4)):
        cache = _cache(B, Hkv, C, d)
        fa.fa_kv4_append(k, v, *cache, signs=signs)
        lens = torch.full((B, Hkv), C, dtype=torch.int32, device=DEV)
        o, lse = torch.empty((B, H, d), dtype=torch.bfloat16, device=DEV), torch.empty((B, H), device=DEV)
        ws = torch.empty(fa.fa_decode_kv4_workspace_bytes(B, H, Hkv, C, d, False), dtype=torch.uint8, device=DEV)
        scale = 2.0 ** -power / 8
        fa.fa_decode_kv4(q, *cache, lens, o, lse, scale, ws, signs=signs)
        cs = None if signs is None else signs.cpu()
        kr, vr = R.values(cache[0].cpu(), cache[1].cpu().float(), cs), R.values(cache[2].cpu(), cache[3].cpu().float())
        ro, rl, _, pv, terms = R.decode(q.cpu().double(), kr, vr, lens.cpu(), scale)
        # in the rotated basis the terms of a score can be larger: a row's terms there are at most |q| |k| in norm
        norms = scale * q.cpu().double().norm(dim=-1) * kr.norm(dim=-1).amax(-1).repeat_interleave(H // Hkv, 1)
        t_o, t_lse, _ = _bounds(d, C, torch.maximum(terms, norms), rl, pv, ro)
        assert ((o.cpu().double() - ro).abs() <= t_o).all()
        assert ((lse.cpu().double() - rl).abs() <= t_lse).all()


def test_a_cache_past_four_gigabytes():
    """Row offsets past 2^32 bytes, and scores past 2^31 bytes: the second head's last rows carry everything."""
    from exact_io_aware_85_b200 import fa
    B, H, Hkv, C, d = 1, 8, 2, 1 << 25, 128
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    kc, vc = (torch.full((B, Hkv, C, d // 2), 0x88, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros((B, Hkv, C), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    cache = (kc, ks, vc, vs)
    n = 5
    k, v, q = _randn(1, B, Hkv, n, d), _randn(2, B, Hkv, n, d), _randn(3, B, H, d)
    k = (k.float() * 20).to(torch.bfloat16)
    start = torch.tensor([[0, C - n]], dtype=torch.int32, device=DEV)
    acc, pos = torch.zeros((B, Hkv, C), device=DEV), torch.zeros((B, Hkv, C), dtype=torch.int32, device=DEV)
    fa.fa_kv4_append(k, v, *cache, start=start, acc=acc, pos=pos)
    assert pos[0, 1, C - n:].tolist() == list(range(n)) and pos[0, 0, :n].tolist() == list(range(n))
    lens = torch.tensor([[n, C]], dtype=torch.int32, device=DEV)
    o, lse = torch.empty((B, H, d), dtype=torch.bfloat16, device=DEV), torch.empty((B, H), device=DEV)
    ws = torch.empty(fa.fa_decode_kv4_workspace_bytes(B, H, Hkv, C, d, True), dtype=torch.uint8, device=DEV)
    scale = 1 / math.sqrt(d)
    fa.fa_decode_kv4(q, *cache, lens, o, lse, scale, ws, acc=acc)
    torch.cuda.synchronize()
    assert fa.fa_check_status() == fa.FA_OK
    for hk, lo in ((0, 0), (1, C - n)):
        kr, vr = (R.values(cache[a][:, hk:hk + 1, lo:lo + n].cpu(), cache[a + 1][:, hk:hk + 1, lo:lo + n].cpu().float())
                  for a in (0, 2))
        qh = q.cpu().double()[:, 4 * hk:4 * hk + 4]
        s = scale * qh[0] @ kr[0, 0].T                      # the other C - n rows score zero, with values of zero
        zeros = C - n if hk else 0
        l = torch.exp(s).sum(-1) + zeros
        p = torch.exp(s) / l[:, None]
        want = p @ vr[0, 0]
        # V's codes c enter the products as c + 8 and the eights leave by a subtraction: sum u (c + 8) and 8 sum u,
        # u = p vs, are sums of numbers of at most 15 u, each addition rounded to 2^-24 of the sum so far, 15 sum u.
        # A warp adds a block of 32 of every 480 keys of its CTA's part in two additions, and 20 more join the parts:
        # adds * 2^-24 * (15 + 8) sum u, which counts where the weighty rows' codes are zero (want is near zero there)
        adds = 2 * (C // (148 * 480) + 1) + 20
        eights = adds * 2.0 ** -24 * 23 * (p @ cache[3][0, hk, lo:lo + n].cpu().double())[:, None]
        assert ((o[0, 4 * hk:4 * hk + 4].cpu().double() - want).abs()
                <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -10) * (p @ vr[0, 0].abs()) + eights).all()
        # sums of 2^25 equal terms in chains of 2^25 / (148 * 480): 2^9 roundings of 2^-24
        assert ((lse[0, 4 * hk:4 * hk + 4].cpu().double() - torch.log(l)).abs() <= 2.0 ** -12).all()
        got = acc[0, hk, lo:lo + n].cpu().double()
        assert ((got - p.sum(0)).abs() <= 2.0 ** -11 * p.sum(0) + 1e-7).all()
    slots = torch.empty((B, Hkv, 3), dtype=torch.int32, device=DEV)
    seen = torch.full((B,), C, dtype=torch.int32, device=DEV)
    acc.fill_(1.0)
    acc[0, 1, C - 2] = 0.5
    acc[0, 1, C - 9] = 0.25
    pos.fill_(7)
    fa.fa_evict_slots(acc, pos, lens, seen, slots, C, 1, 1)
    assert slots[0, 1].tolist() == [C - 9, C - 2, C - 1] and slots[0, 0].tolist() == [n, n + 1, n + 2]
    ko, vo = torch.empty((B, Hkv, 3, d), dtype=torch.bfloat16, device=DEV), torch.empty((B, Hkv, 3, d), dtype=torch.bfloat16, device=DEV)
    fa.fa_kv4_read(*cache, ko, vo, slots=slots)
    want = R.values(cache[2][0, 1, C - 2:].cpu(), cache[3][0, 1, C - 2:].cpu().float())
    assert torch.equal(vo[0, 1, 1:].cpu(), want.to(torch.bfloat16))


def test_decode_rows_without_values_keep_their_weight():
    """Rows whose V is zero, or tiny, beside rows whose V is not: they take their share of the softmax all the same,
    in every order (the sum is held relative to a reference that follows score and value scale)."""
    from exact_io_aware_85_b200 import fa
    B, H, Hkv, C, d = 1, 4, 1, 2048, 64
    g = torch.Generator().manual_seed(11)
    q, k = torch.randn((B, H, d), generator=g), torch.randn((B, Hkv, C, d), generator=g)
    base = torch.randn((B, Hkv, C, d), generator=g)
    rows = torch.arange(C)[:, None]
    for which, small in (("early", rows < C - 3), ("late", rows >= 3), ("most", rows % 700 != 5), ("all", rows >= 0)):
        for factor in (0.0, 1e-24, 1e-12):
            v = torch.where(small, base * factor, base)
            qq, kk, vv = (t.to(torch.bfloat16).to(DEV) for t in (q * 2, k, v))
            cache = _cache(B, Hkv, C, d)
            fa.fa_kv4_append(kk, vv, *cache)
            lens = torch.full((B, Hkv), C, dtype=torch.int32, device=DEV)
            o, lse, acc = torch.empty((B, H, d), dtype=torch.bfloat16, device=DEV), torch.empty((B, H), device=DEV), torch.zeros((B, Hkv, C), device=DEV)
            ws = torch.empty(fa.fa_decode_kv4_workspace_bytes(B, H, Hkv, C, d, True), dtype=torch.uint8, device=DEV)
            fa.fa_decode_kv4(qq, *cache, lens, o, lse, 0.5, ws, acc=acc)
            kr, vr = (R.values(cache[a].cpu(), cache[a + 1].cpu().float()) for a in (0, 2))
            ro, rl, rw, pv, terms = R.decode(qq.cpu().double(), kr, vr, lens.cpu(), 0.5)
            _, t_lse, t_w = _bounds(d, C, terms, rl, pv, ro)
            assert ((lse.cpu().double() - rl).abs() <= t_lse).all(), (which, factor)
            assert ((acc.cpu().double() - rw).abs() <= t_w.amax() * rw + 2.0 ** -22 * (1 + rw)).all(), (which, factor)
            # O's own rounding to bf16 is 2^-8 of it; P's to fp16 (2^-11, or 2^-25 2^8 absolute beside the largest u)
            # and the offset's cancellation (2^-20 sum p vs, at most 8 times the largest |o|) stay below another 2^-8
            top = ro.abs().amax(-1, keepdim=True) + pv.amax(-1, keepdim=True)
            assert ((o.cpu().double() - ro).abs() <= 2.0 ** -7 * top).all(), (which, factor)
