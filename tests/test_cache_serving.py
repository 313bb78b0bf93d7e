"""The cache operators together, as a serving loop uses them: a prompt's forward, the weight its keys received,
eviction to a budget, the surviving rows into the 4-bit cache; then decoding steps, each of which takes a row
(evicting the lightest one), writes its token there and attends.  Every step is checked against 64-bit references
on the state that the step found, eagerly and replayed from one captured graph."""
import math

import pytest
import torch

import cache_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("B,H,Hkv,N,budget,d,rot,graph", [(2, 8, 2, 300, 96, 128, True, False),
                                                          (1, 4, 4, 150, 120, 64, False, True),
                                                          (2, 6, 1, 200, 64, 256, True, True)])
def test_prompt_then_tokens(B, H, Hkv, N, budget, d, rot, graph):
    from exact_io_aware_85_b200 import fa
    g = torch.Generator().manual_seed(N)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    q, k, v = rnd(B, H, N, d), rnd(B, Hkv, N, d), rnd(B, Hkv, N, d)
    signs = (torch.randint(0, 2, (d,), generator=g) * 2 - 1).float().to(DEV) if rot else None
    cs = None if signs is None else signs.cpu()
    scale, C, recent, sink = 1 / math.sqrt(d), 128, 16, 4
    i32 = dict(dtype=torch.int32, device=DEV)
    # the prompt
    o, lse, w = torch.empty_like(q), torch.empty((B, H, N), device=DEV), torch.empty((B, Hkv, N), device=DEV)
    fa.fa_fwd_gqa(q, k, v, o, lse, True, scale)
    ws = torch.empty(fa.fa_key_weights_workspace_bytes(B, H, Hkv, N, d, N), dtype=torch.uint8, device=DEV)
    fa.fa_key_weights(q, k, lse, w, True, scale, ws)
    idx, lens = torch.empty((B, Hkv, budget), **i32), torch.empty((B, Hkv), **i32)
    fa.fa_evict_keep(w, idx, lens, recent, sink)
    cache = [torch.zeros((B, Hkv, C, d // 2), dtype=torch.uint8, device=DEV), torch.zeros((B, Hkv, C), dtype=torch.bfloat16, device=DEV)]
    cache = cache + [t.clone() for t in cache]
    acc, pos = torch.zeros((B, Hkv, C), device=DEV), torch.zeros((B, Hkv, C), **i32)
    fa.fa_kv4_append(k, v, *cache, signs=signs, rows=idx, w=w, acc=acc, pos=pos)
    for b in range(B):
        for h in range(Hkv):
            want = R.evict_keep(w[b, h].tolist(), budget, recent, sink, N)
            assert idx[b, h].tolist() == want == pos[b, h, :budget].tolist()
            assert torch.equal(acc[b, h, :budget], w[b, h, idx[b, h].long()])
    # tokens
    seen = torch.full((B,), N, **i32)
    slots = torch.empty((B, Hkv, 1), **i32)
    qt, kt, vt = torch.empty((B, H, d), dtype=torch.bfloat16, device=DEV), *(
        torch.empty((B, Hkv, 1, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ot, lt = torch.empty_like(qt), torch.empty((B, H), device=DEV)
    wsd = torch.empty(fa.fa_decode_kv4_workspace_bytes(B, H, Hkv, C, d, True), dtype=torch.uint8, device=DEV)

    def step():
        fa.fa_evict_slots(acc, pos, lens, seen, slots, budget + 3, recent, sink)
        fa.fa_kv4_append(kt, vt, *cache, signs=signs, slots=slots, acc=acc, pos=pos, base=seen)
        fa.fa_decode_kv4(qt, *cache, lens, ot, lt, scale, wsd, signs=signs, acc=acc)
        seen.add_(1)

    if graph:
        run = torch.cuda.CUDAGraph()
        with torch.cuda.graph(run):
            step()
    for t in range(6):
        for x in (qt, kt, vt):
            x.copy_(rnd(*x.shape))
        acc0, pos0, lens0, seen0 = (x.cpu() for x in (acc, pos, lens, seen))
        run.replay() if graph else step()
        torch.cuda.synchronize()
        assert fa.fa_check_status() == fa.FA_OK
        kr, vr = R.values(cache[0].cpu(), cache[1].cpu().float(), cs), R.values(cache[2].cpu(), cache[3].cpu().float())
        ro, rl, rw, pv, _ = R.decode(qt.cpu().double(), kr, vr, lens.cpu(), scale)
        for b in range(B):
            for h in range(Hkv):
                want, n = R.evict_slots(acc0[b, h].tolist(), pos0[b, h].tolist(), int(lens0[b, h]), int(seen0[b]),
                                        budget + 3, 1, recent, sink)
                r = want[0]
                assert slots[b, h].tolist() == want and int(lens[b, h]) == n and int(pos[b, h, r]) == N + t
                # the new row holds the token: within half a step of 1/7 of its largest rotated value
                y = R.rotate(kt[b, h, 0].cpu().double(), cs)
                got = (R.unpack(cache[0][b, h, r].cpu()) - 8).double() * float(cache[1][b, h, r])
                assert ((got - y).abs() <= 0.51 * float(cache[1][b, h, r])).all()
                acc0[b, h, r] = 0
        # 2^-8 of O and of each weight; scores of at most 2^4 here: 2^-12 covers what their arithmetic adds
        assert ((ot.cpu().double() - ro).abs() <= 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2.0 ** -12) * pv).all()
        assert ((lt.cpu().double() - rl).abs() <= 2.0 ** -12).all()
        assert ((acc.cpu().double() - acc0.double() - rw).abs() <= 2.0 ** -11 * rw + 2.0 ** -22 * (acc0 + 1)).all()
