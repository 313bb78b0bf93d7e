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


@pytest.mark.parametrize("how", ["queued", "graph"])
def test_calls_wait_for_one_another(how):
    """The kernels come onto the GPU while those before them still run: a layer-like chain of calls whose inputs
    are written just before by slow kernels gives the bits of the same calls with a synchronisation after each."""
    from exact_io_aware_85_b200 import fa
    B, H, Hkv, N, C, d, T = 2, 8, 2, 640, 384, 128, 12
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    q, k, v, qt = rnd(B, H, N, d), rnd(B, Hkv, N, d), rnd(B, Hkv, N, d), rnd(B, H, d)
    signs = (torch.randint(0, 2, (d,), generator=g) * 2 - 1).float().to(DEV)
    big = rnd(4096, 4096)
    i32 = dict(dtype=torch.int32, device=DEV)
    scale = 1 / math.sqrt(d)
    wsk = torch.empty(fa.fa_key_weights_workspace_bytes(B, H, Hkv, N, d, 100), dtype=torch.uint8, device=DEV)
    wsd = torch.empty(fa.fa_decode_kv4_workspace_bytes(B, H, Hkv, C, d, True), dtype=torch.uint8, device=DEV)

    def state():
        z = lambda *s, t=torch.float32: torch.zeros(s, dtype=t, device=DEV)  # noqa: E731
        bf = torch.bfloat16
        return dict(q=z(B, H, N, d, t=bf), k=z(B, Hkv, N, d, t=bf), v=z(B, Hkv, N, d, t=bf), o=z(B, H, N, d, t=bf), lse=z(B, H, N),
                    w=z(B, Hkv, N), idx=z(B, Hkv, 300, t=torch.int32), lens=z(B, Hkv, t=torch.int32), acc=z(B, Hkv, C),
                    pos=z(B, Hkv, C, t=torch.int32), seen=torch.full((B,), N, **i32), slots=z(B, Hkv, 2, t=torch.int32),
                    cache=[z(B, Hkv, C, d // 2, t=torch.uint8), z(B, Hkv, C, t=bf), z(B, Hkv, C, d // 2, t=torch.uint8), z(B, Hkv, C, t=bf)],
                    qt=z(B, H, d, t=bf), kt=z(B, Hkv, 2, d, t=bf), vt=z(B, Hkv, 2, d, t=bf), ot=z(B, H, d, t=bf), lt=z(B, H),
                    kr=z(B, Hkv, C, d, t=bf), vr=z(B, Hkv, C, d, t=bf), tmp=torch.empty_like(big))

    def chain(s, wait):
        torch.mm(big, big, out=s["tmp"])  # what follows queues behind it
        for x, y in (("q", q), ("k", k), ("v", v), ("qt", qt)):
            s[x].copy_(y)
        wait()
        fa.fa_fwd_gqa(s["q"], s["k"], s["v"], s["o"], s["lse"], True, scale)
        wait()
        fa.fa_key_weights(s["q"], s["k"], s["lse"], s["w"], True, scale, wsk, window=100)
        wait()
        fa.fa_evict_keep(s["w"], s["idx"], s["lens"], 16, 4)
        wait()
        fa.fa_kv4_append(s["k"], s["v"], *s["cache"], signs=signs, rows=s["idx"], w=s["w"], acc=s["acc"], pos=s["pos"])
        wait()
        for t in range(T):
            s["kt"].copy_(k[:, :, 2 * t:2 * t + 2])
            s["vt"].copy_(v[:, :, 2 * t:2 * t + 2])
            wait()
            fa.fa_evict_slots(s["acc"], s["pos"], s["lens"], s["seen"], s["slots"], 310, 16, 4)
            wait()
            fa.fa_kv4_append(s["kt"], s["vt"], *s["cache"], signs=signs, slots=s["slots"], acc=s["acc"], pos=s["pos"], base=s["seen"])
            wait()
            fa.fa_decode_kv4(s["qt"], *s["cache"], s["lens"], s["ot"], s["lt"], scale, wsd, signs=signs, acc=s["acc"])
            wait()
            s["qt"].copy_(s["ot"])
            s["seen"].add_(2)
            wait()
        fa.fa_kv4_read(*s["cache"], s["kr"], s["vr"], signs=signs, lens=s["lens"])
        wait()

    want = state()
    chain(want, torch.cuda.synchronize)
    got = state()
    if how == "graph":
        run = torch.cuda.CUDAGraph()
        with torch.cuda.graph(run):
            chain(got, lambda: None)
        run.replay()
    else:
        chain(got, lambda: None)
    torch.cuda.synchronize()
    assert fa.fa_check_status() == fa.FA_OK
    for name, x in want.items():
        if name != "tmp":
            for a, b in zip(x if isinstance(x, list) else [x], got[name] if isinstance(x, list) else [got[name]]):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
    assert bool((want["lens"] == 310).all()) and bool(want["ot"].float().abs().sum() > 0)


@pytest.mark.parametrize("how", ["queued", "graph"])
def test_calls_wait_for_other_streams(how):
    """A call behind one of its own kind and behind an event of another stream, on which its inputs are written late."""
    from exact_io_aware_85_b200 import fa
    B, H, Hkv, C, d = 2, 8, 2, 256, 128
    g = torch.Generator().manual_seed(4)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    k, v, q, big = rnd(B, Hkv, C, d), rnd(B, Hkv, C, d), rnd(B, H, d), rnd(4096, 4096)
    ws = torch.empty(fa.fa_decode_kv4_workspace_bytes(B, H, Hkv, C, d, False), dtype=torch.uint8, device=DEV)
    lens = torch.full((B, Hkv), C, dtype=torch.int32, device=DEV)

    def state():
        cache = [torch.zeros((B, Hkv, C, d // 2), dtype=torch.uint8, device=DEV), torch.zeros((B, Hkv, C), dtype=torch.bfloat16, device=DEV)]
        return dict(k=torch.zeros_like(k), v=torch.zeros_like(v), q=torch.zeros_like(q), o=torch.zeros_like(q),
                    lse=torch.zeros((B, H), device=DEV), cache=cache + [t.clone() for t in cache], tmp=torch.empty_like(big))

    def chain(s, side):
        main = torch.cuda.current_stream()
        fa.fa_kv4_append(s["k"], s["v"], *s["cache"])  # zeros
        side.wait_stream(main)
        with torch.cuda.stream(side):
            torch.mm(big, big, out=s["tmp"])
            s["k"].copy_(k)
            s["v"].copy_(v)
        fa.fa_decode_kv4(s["q"], *s["cache"], lens, s["o"], s["lse"], 0.1, ws)
        main.wait_stream(side)
        fa.fa_kv4_append(s["k"], s["v"], *s["cache"])
        side.wait_stream(main)
        with torch.cuda.stream(side):
            torch.mm(big, big, out=s["tmp"])
            s["q"].copy_(q)
        fa.fa_kv4_append(s["k"], s["v"], *s["cache"])
        main.wait_stream(side)
        fa.fa_decode_kv4(s["q"], *s["cache"], lens, s["o"], s["lse"], 0.1, ws)

    want = state()
    want["k"].copy_(k), want["v"].copy_(v), want["q"].copy_(q)
    fa.fa_kv4_append(want["k"], want["v"], *want["cache"])
    torch.cuda.synchronize()
    fa.fa_decode_kv4(want["q"], *want["cache"], lens, want["o"], want["lse"], 0.1, ws)
    torch.cuda.synchronize()
    for _ in range(3):
        got, side = state(), torch.cuda.Stream()
        torch.cuda.synchronize()
        if how == "graph":
            run = torch.cuda.CUDAGraph()
            with torch.cuda.graph(run):
                chain(got, side)
            run.replay()
        else:
            chain(got, side)
        torch.cuda.synchronize()
        for a, b in zip([want["o"], want["lse"], *want["cache"]], [got["o"], got["lse"], *got["cache"]]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
