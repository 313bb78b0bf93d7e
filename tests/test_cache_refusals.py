"""The cache operators refuse bad arguments before any launch (no GPU needed), and their workspaces
are functions of the sizes alone."""
import ctypes

import pytest
import torch

vp, ci, cf, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
GOOD, ODD4, ODD8, ODD2 = vp(1 << 20), vp((1 << 20) + 4), vp((1 << 20) + 8), vp((1 << 20) + 2)
ODD16 = vp((1 << 20) + 16)
INVALID, UNSUPPORTED, ALIGNMENT = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from exact_io_aware_85_b200 import build
    build.build_library()
    from exact_io_aware_85_b200 import fa
    return fa.lib


def _call(f, order, given, **over):
    a = dict(given, **over)
    return f(*[a[n] for n in order.split()])


def test_append(lib):
    order = "k v signs w rows slots start n_new base kc ks vc vs acc pos B Hkv N T C ldw d stream"
    base = dict({n: GOOD for n in "k v kc ks vc vs acc pos".split()},
                **{n: None for n in "signs w rows slots start n_new base stream".split()},
                B=1, Hkv=2, N=5, T=5, C=128, ldw=0, d=128)
    go = lambda **o: _call(lib.fa_kv4_append, order, base, **o)  # noqa: E731
    for n in "k v kc ks vc vs".split():
        assert go(**{n: None}) == INVALID, n
        assert go(**{n: ODD8}) == ALIGNMENT, n
    for n in "k v".split():
        assert go(**{n: ODD16}) == ALIGNMENT, n     # read 32 bytes at a time
    for n in "acc pos".split():
        assert go(**{n: ODD4}) == ALIGNMENT, n
    for n in "signs w rows slots start n_new base".split():
        assert go(**dict({n: ODD2}, ldw=5)) == ALIGNMENT, n
    for n in "B Hkv N T C".split():
        assert go(**{n: 0}) == INVALID, n
    assert go(T=6) == INVALID                       # more rows than the source has
    assert go(slots=GOOD, start=GOOD) == INVALID    # two destinations
    assert go(w=GOOD, ldw=4) == INVALID             # w shorter than the source
    assert go(C=100) == INVALID                     # capacity not a multiple of 128
    assert go(d=96) == UNSUPPORTED
    assert go(C=(1 << 30) + 128) == UNSUPPORTED
    assert go(B=1 << 16, Hkv=1 << 15) == UNSUPPORTED


def test_read(lib):
    order = "kc ks vc vs signs slots lens k v B Hkv T C first d stream"
    base = dict({n: GOOD for n in "kc ks vc vs k v".split()}, signs=None, slots=None, lens=None, stream=None, B=1, Hkv=2,
                T=5, C=128, first=0, d=64)
    go = lambda **o: _call(lib.fa_kv4_read, order, base, **o)  # noqa: E731
    for n in "kc ks vc vs k v".split():
        assert go(**{n: None}) == INVALID, n
        assert go(**{n: ODD8}) == ALIGNMENT, n
    for n in "k v".split():
        assert go(**{n: ODD16}) == ALIGNMENT, n
    for n in "signs slots lens".split():
        assert go(**{n: ODD2}) == ALIGNMENT, n
    assert go(T=0) == INVALID and go(first=-1) == INVALID and go(C=64) == INVALID
    assert go(slots=GOOD, first=3) == INVALID       # two sources
    assert go(d=32) == UNSUPPORTED


def test_decode(lib):
    order = "q kc ks vc vs signs lens o lse acc B H Hkv C d scale ws nws stream"
    base = dict({n: GOOD for n in "q kc ks vc vs lens o lse ws".split()}, signs=None, acc=None, stream=None, B=1, H=8,
                Hkv=2, C=256, d=128, scale=0.1, nws=1 << 40)
    go = lambda **o: _call(lib.fa_decode_kv4, order, base, **o)  # noqa: E731
    for n in "q kc ks vc vs lens o lse ws".split():
        assert go(**{n: None}) == INVALID, n
    for n in "q kc ks vc vs o acc ws".split():
        assert go(**{n: ODD8}) == ALIGNMENT, n
    for n in "lens lse signs".split():
        assert go(**{n: ODD2}) == ALIGNMENT, n
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert go(scale=s) == INVALID
    assert go(H=7) == INVALID and go(H=0) == INVALID and go(Hkv=0) == INVALID and go(B=0) == INVALID
    assert go(C=0) == INVALID and go(C=200) == INVALID
    assert go(d=96) == UNSUPPORTED and go(H=34) == UNSUPPORTED     # 17 query heads share a key/value head
    assert go(B=65536, H=2, Hkv=1) == UNSUPPORTED
    need = lib.fa_decode_kv4_workspace_bytes(1, 8, 2, 256, 128, 1)
    assert need > lib.fa_decode_kv4_workspace_bytes(1, 8, 2, 256, 128, 0) > 0
    assert go(nws=need - 1, acc=GOOD) == INVALID
    for a in ((1, 7, 2, 256, 128, 0), (1, 8, 2, 200, 128, 0), (1, 8, 2, 256, 96, 0), (1, 34, 2, 256, 64, 0)):
        assert lib.fa_decode_kv4_workspace_bytes(*a) == 0


def test_evict(lib):
    order = "w lens idx count B Hkv C keep recent sink stream"
    base = dict(w=GOOD, lens=None, idx=GOOD, count=GOOD, B=1, Hkv=1, C=10, keep=5, recent=2, sink=2, stream=None)
    go = lambda **o: _call(lib.fa_evict_keep, order, base, **o)  # noqa: E731
    for n in "w idx count".split():
        assert go(**{n: None}) == INVALID and go(**{n: ODD2}) == ALIGNMENT
    assert go(lens=ODD2) == ALIGNMENT
    for n in "B Hkv C keep".split():
        assert go(**{n: 0}) == INVALID
    assert go(recent=-1) == INVALID and go(sink=-1) == INVALID
    assert go(recent=4) == INVALID                  # more rows protected than kept
    assert go(C=(1 << 30) + 1) == UNSUPPORTED
    order2 = "acc pos lens seen slots B Hkv C budget T recent sink stream"
    base2 = dict({n: GOOD for n in "acc pos lens seen slots".split()}, B=1, Hkv=1, C=10, budget=8, T=3, recent=0, sink=0,
                 stream=None)
    go = lambda **o: _call(lib.fa_evict_slots, order2, base2, **o)  # noqa: E731
    for n in "acc pos lens seen slots".split():
        assert go(**{n: None}) == INVALID and go(**{n: ODD2}) == ALIGNMENT
    for n in "B Hkv C budget T".split():
        assert go(**{n: 0}) == INVALID
    assert go(budget=11) == INVALID and go(T=9) == INVALID and go(recent=-1) == INVALID and go(sink=-1) == INVALID


def test_key_weights(lib):
    order = "q k lse w n_rows B H Hkv N ldw d causal window scale ws nws stream"
    base = dict({n: GOOD for n in "q k lse w ws".split()}, n_rows=None, stream=None, B=1, H=4, Hkv=2, N=50, ldw=50, d=64,
                causal=1, window=8, scale=0.1, nws=1 << 40)
    go = lambda **o: _call(lib.fa_key_weights, order, base, **o)  # noqa: E731
    for n in "q k lse w ws".split():
        assert go(**{n: None}) == INVALID, n
    for n in "q k ws".split():
        assert go(**{n: ODD8}) == ALIGNMENT, n
    for n in "lse w n_rows".split():
        assert go(**{n: ODD2}) == ALIGNMENT, n
    for n in "B H Hkv N window".split():
        assert go(**{n: 0}) == INVALID, n
    assert go(H=3) == INVALID and go(ldw=49) == INVALID and go(scale=0.0) == INVALID
    assert go(d=96) == UNSUPPORTED and go(scale=1e-30) == UNSUPPORTED
    assert lib.fa_key_weights_workspace_bytes(1, 4, 2, 50, 64, 8) > 0
    assert go(nws=0) == INVALID
    assert lib.fa_key_weights_workspace_bytes(1, 3, 2, 50, 64, 8) == 0


def test_binding_refuses_what_is_not_a_cuda_tensor(lib):
    """The Python entry points name the argument; CPU tensors are refused before the library is called."""
    from exact_io_aware_85_b200 import fa
    if not torch.cuda.is_available():
        with pytest.raises(fa.FAError):
            fa.fa_evict_keep(None, None, None, 0, 0)
        with pytest.raises(fa.FAError):
            fa.fa_kv4_append(None, None, None, None, None, None)
        with pytest.raises(fa.FAError):
            fa.fa_decode_kv4(None, torch.zeros(1, 1, 128, 32, dtype=torch.uint8), None, None, None, None, None, None, 1.0,
                             None)
