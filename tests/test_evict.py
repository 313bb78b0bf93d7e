"""Eviction by accumulated weight against a sort: the answers are whole numbers and have to be equal."""
import pytest
import torch

import cache_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _weights(seed, *shape, kind="heavy"):
    g = torch.Generator().manual_seed(seed)
    if kind == "ties":  # few different values: the order among equals decides
        return torch.randint(0, 4, shape, generator=g).float()
    if kind == "odd":   # signs, infinities, NaN, both zeros
        w = torch.randn(shape, generator=g)
        pick = torch.randint(0, 10, shape, generator=g)
        for n, x in enumerate((float("inf"), -float("inf"), float("nan"), 0.0, -0.0)):
            w[pick == n] = x
        return w
    if kind == "near":  # differences in the last bits
        return (1.0 + torch.randint(0, 64, shape, generator=g).float() * 2.0 ** -23)
    return torch.exp(2 * torch.randn(shape, generator=g))


@pytest.mark.parametrize("B,Hkv,C,keep,recent,sink,kind", [
    (1, 1, 1, 1, 0, 0, "heavy"), (1, 2, 100, 30, 5, 4, "heavy"), (2, 3, 1000, 999, 0, 0, "ties"),
    (2, 2, 1025, 64, 32, 4, "ties"), (1, 2, 5000, 4097, 100, 0, "odd"), (1, 1, 70001, 20000, 50, 4, "heavy"),
    (1, 2, 3001, 1500, 0, 0, "near"), (1, 1, 300, 400, 10, 4, "heavy"), (1, 1, 40000, 1, 0, 0, "near"),
    (2, 80, 257, 100, 3, 3, "odd"),
    # many heads: one CTA each, whose rows do not fit its registers
    (2, 80, 20001, 5000, 50, 4, "heavy"), (1, 150, 33000, 17000, 0, 0, "ties"),
    # a cluster whose rows do not, and a list of equals that overflows
    (1, 1, 140000, 60000, 10, 4, "heavy"), (1, 2, 60000, 30001, 10, 4, "near")])
def test_keep(B, Hkv, C, keep, recent, sink, kind):
    from exact_io_aware_85_b200 import fa
    w = _weights(C + keep, B, Hkv, C, kind=kind)
    g = torch.Generator().manual_seed(1)
    for lens in (None, torch.randint(0, C + 1, (B, Hkv), generator=g, dtype=torch.int32)):
        idx = torch.full((B, Hkv, keep), -7, dtype=torch.int32, device=DEV)
        count = torch.full((B, Hkv), -7, dtype=torch.int32, device=DEV)
        fa.fa_evict_keep(w.to(DEV), idx, count, recent, sink, lens=None if lens is None else lens.to(DEV))
        for b in range(B):
            for h in range(0, Hkv, max(1, Hkv // 4)):
                n = C if lens is None else int(lens[b, h])
                want = R.evict_keep(w[b, h, :n].tolist(), keep, recent, sink, n)
                assert int(count[b, h]) == len(want) == min(n, keep)
                assert idx[b, h].tolist() == want + [-1] * (keep - len(want))


@pytest.mark.parametrize("B,Hkv,C,budget,T,recent,sink,kind", [
    (1, 1, 1, 1, 1, 0, 0, "heavy"), (2, 2, 128, 100, 1, 10, 4, "heavy"), (1, 3, 1000, 1000, 17, 200, 4, "ties"),
    (2, 1, 4096, 4095, 1, 256, 4, "ties"), (1, 1, 70000, 66001, 500, 1000, 4, "heavy"), (1, 2, 500, 500, 500, 10, 2, "odd"),
    (1, 2, 2048, 2000, 64, 1999, 4, "near"), (3, 50, 300, 256, 2, 8, 2, "odd"),
    (1, 150, 20100, 20001, 300, 100, 4, "heavy"), (1, 150, 33000, 33000, 1, 100, 4, "ties"),
    (1, 1, 150000, 140000, 1000, 100, 4, "near"), (1, 2, 140000, 140000, 1, 100, 4, "heavy")])
def test_slots(B, Hkv, C, budget, T, recent, sink, kind):
    from exact_io_aware_85_b200 import fa
    acc = _weights(C + T, B, Hkv, C, kind=kind)
    g = torch.Generator().manual_seed(2)
    pos = torch.argsort(torch.rand((B, Hkv, C), generator=g), -1).to(torch.int32)
    seen = torch.randint(C, C + 5, (B,), generator=g, dtype=torch.int32)
    full = torch.full((B, Hkv), budget, dtype=torch.int32)
    part = torch.randint(max(0, budget - T - 2), budget + 1, (B, Hkv), generator=g, dtype=torch.int32)
    for lens in (full, part, torch.zeros_like(full), full + 100):
        slots = torch.full((B, Hkv, T), -7, dtype=torch.int32, device=DEV)
        got = lens.to(DEV)
        fa.fa_evict_slots(acc.to(DEV), pos.to(DEV), got, seen.to(DEV), slots, budget, recent, sink)
        for b in range(B):
            for h in range(0, Hkv, max(1, Hkv // 4)):
                want, n = R.evict_slots(acc[b, h].tolist(), pos[b, h].tolist(), int(lens[b, h]), int(seen[b]), budget, T,
                                        recent, sink)
                assert int(got[b, h]) == n and slots[b, h].tolist() == want


def test_slots_in_a_graph_walk_through_the_cache():
    """A captured step, replayed: the lengths it left are the ones that it reads next."""
    from exact_io_aware_85_b200 import fa
    C, budget = 128, 6
    acc = torch.arange(C, 0, -1, dtype=torch.float32, device=DEV).view(1, 1, C)
    pos = torch.arange(C, dtype=torch.int32, device=DEV).view(1, 1, C)
    lens, seen = torch.full((1, 1), 4, dtype=torch.int32, device=DEV), torch.full((1,), 4, dtype=torch.int32, device=DEV)
    slots = torch.empty((1, 1, 1), dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_evict_slots(acc, pos, lens, seen, slots, budget, 0, 0)
    got = []
    for _ in range(3):
        graph.replay()
        got.append((int(slots), int(lens)))
    # the third step finds the cache full; rows 4 and 5 hold positions >= seen = 4 and go last, so row 3 is the lightest
    assert got == [(4, 5), (5, 6), (3, 6)]
