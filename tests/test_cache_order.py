"""Kernels that come onto the GPU while those before them run touch memory only behind their wait.

On the CPU: inline assembly that reads or writes memory tells the compiler so; without it the compiler takes a load
for a function of its address and may move it, above the wait too.  On the GPU: rows read out of a cache and appended
right behind, so that the append's inputs are what the kernel before it is still writing."""
import glob
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda"


def _statements(src):
    """(line, volatile, text) of every asm statement of a source."""
    for m in re.finditer(r"\basm(\s+volatile)?\s*\(", src):
        depth, i, quoted = 1, m.end(), False
        while depth:
            c = src[i]
            if c == '"' and src[i - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            i += 1
        yield src.count("\n", 0, m.start()) + 1, bool(m.group(1)), src[m.end():i - 1]


def test_assembly_that_touches_memory_says_so():
    loads = 0
    for path in sorted(glob.glob(os.path.join(ROOT, "exact_io_aware_85_b200", "csrc", "*.cu*"))):
        for line, volatile, text in _statements(open(path).read()):
            ops = " ".join(re.findall(r'"((?:[^"\\]|\\.)*)"', text.split('"memory"')[0]))
            if re.search(r"\b(ld|st|red|atom|cp|multimem)\.|\[%", ops):
                assert volatile, f"{os.path.basename(path)}:{line}: touches memory, is not volatile"
            if re.search(r"\bld\.global|griddepcontrol\.wait", ops):
                loads += 1
                assert '"memory"' in text, f'{os.path.basename(path)}:{line}: no "memory" clobber'
    assert loads >= 2


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["queued", "graph"])
@pytest.mark.parametrize("d,rot", [(64, False), (128, True), (256, True)])
def test_rows_read_and_appended_right_behind(how, d, rot):
    """A cache compacted through buffers that each pass writes anew: reads and contiguous appends in a row give the
    bits that they give with a synchronisation after each call."""
    from exact_io_aware_85_b200 import fa
    B, Hkv, T, C, passes = 2, 4, 2000, 2048, 6
    g = torch.Generator().manual_seed(d)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    signs = (torch.randint(0, 2, (d,), generator=g) * 2 - 1).float().to(DEV) if rot else None
    k, v = rnd(B, Hkv, C, d), rnd(B, Hkv, C, d)
    # every pass takes other rows, in another order
    picks = [torch.stack([torch.randperm(T if t else C, generator=g)[:T] for _ in range(B * Hkv)])
             .view(B, Hkv, T).to(torch.int32).to(DEV) for t in range(passes)]

    def cache():
        c = [torch.zeros((B, Hkv, C, d // 2), dtype=torch.uint8, device=DEV), torch.zeros((B, Hkv, C), dtype=torch.bfloat16, device=DEV)]
        return c + [t.clone() for t in c]

    def state():
        return cache(), cache(), torch.zeros((B, Hkv, T, d), dtype=torch.bfloat16, device=DEV), \
            torch.zeros((B, Hkv, T, d), dtype=torch.bfloat16, device=DEV)

    def chain(s, wait):
        a, b, kr, vr = s
        fa.fa_kv4_append(k, v, *a, signs=signs)
        wait()
        for pick in picks:
            fa.fa_kv4_read(*a, kr, vr, signs=signs, slots=pick)
            wait()
            fa.fa_kv4_append(kr, vr, *b, signs=signs)
            wait()
            a, b = b, a

    want, got = state(), state()
    chain(want, torch.cuda.synchronize)
    if how == "graph":
        run = torch.cuda.CUDAGraph()
        with torch.cuda.graph(run):
            chain(got, lambda: None)
        run.replay()
    else:
        chain(got, lambda: None)
    torch.cuda.synchronize()
    assert fa.fa_check_status() == fa.FA_OK
    for x, y in zip([*want[0], *want[1], *want[2:]], [*got[0], *got[1], *got[2:]]):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert bool(want[3].float().abs().sum() > 0)


@pytest.mark.gpu
def test_calls_at_the_same_time():
    """Decoding steps and key weights on two streams, a workspace each, over the same cache and prompt: the bits of
    the calls alone."""
    from exact_io_aware_85_b200 import fa
    B, H, Hkv, N, C, d = 2, 8, 2, 900, 4096, 128
    g = torch.Generator().manual_seed(8)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    q, k, v, ck, cv = rnd(B, H, N, d), rnd(B, Hkv, N, d), rnd(B, Hkv, N, d), rnd(B, Hkv, C, d), rnd(B, Hkv, C, d)
    o, lse = torch.empty_like(q), torch.empty((B, H, N), device=DEV)
    fa.fa_fwd_gqa(q, k, v, o, lse, True, d ** -0.5)
    cache = [torch.zeros((B, Hkv, C, d // 2), dtype=torch.uint8, device=DEV), torch.zeros((B, Hkv, C), dtype=torch.bfloat16, device=DEV)]
    cache += [t.clone() for t in cache]
    fa.fa_kv4_append(ck, cv, *cache)
    lens = torch.tensor([[C, 5], [77, 3000]], dtype=torch.int32, device=DEV)
    qs = [rnd(B, H, d) for _ in range(2)]

    def buffers():
        return dict(o=torch.zeros_like(qs[0]), lse=torch.zeros((B, H), device=DEV), acc=torch.zeros((B, Hkv, C), device=DEV),
                    w=torch.zeros((B, Hkv, N), device=DEV),
                    ws=torch.empty(fa.fa_decode_kv4_workspace_bytes(B, H, Hkv, C, d, True), dtype=torch.uint8, device=DEV),
                    wk=torch.empty(fa.fa_key_weights_workspace_bytes(B, H, Hkv, N, d, 300), dtype=torch.uint8, device=DEV))

    def calls(b, i, stream):
        for _ in range(6):
            fa.fa_decode_kv4(qs[i], *cache, lens, b["o"], b["lse"], 0.1, b["ws"], acc=b["acc"], stream=stream)
            fa.fa_key_weights(q, k, lse, b["w"], True, d ** -0.5, b["wk"], window=300, stream=stream)

    want = [buffers(), buffers()]
    for i in (0, 1):
        calls(want[i], i, None)
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [buffers(), buffers()]
        torch.cuda.synchronize()
        for i in (0, 1):
            calls(got[i], i, streams[i])
        torch.cuda.synchronize()
        assert fa.fa_check_status() == fa.FA_OK
        for x, y in zip(want, got):
            assert all(torch.equal(x[n], y[n]) for n in ("o", "lse", "acc", "w"))
