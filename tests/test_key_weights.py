"""The attention weight that each key of a prompt received, against 64-bit column sums of the softmax matrix.

Tolerance: a weight is exp(x) with x = scale q.k - lse formed in fp32: the products are exact, d additions
(d 2^-24 of the terms' magnitudes), the roundings of scale q.k and lse in log2 units (2^-23 of each) and the
exponential itself (2^-21): relative errors of the terms, hence of the sum, whose additions run in chains of at
most n / 64 + 64 terms."""
import math

import pytest
import torch

import cache_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _inputs(B, H, Hkv, N, d, seed, causal, n_rows=None):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((B, H, N, d), generator=g).to(torch.bfloat16)
    k = torch.randn((B, Hkv, N, d), generator=g).to(torch.bfloat16)
    scale = 1 / math.sqrt(d)
    s = scale * q.double().view(B, Hkv, H // Hkv, N, d) @ k.double()[:, :, None].transpose(-1, -2)
    dead = torch.ones(N, N).triu(1).bool() if causal else torch.zeros(N, N).bool()
    s = s.view(B, H, N, N).masked_fill(dead, -math.inf)
    if n_rows is not None:
        for b in range(B):
            s[b, :, :, int(n_rows[b]):] = -math.inf
    lse = torch.logsumexp(s, -1).float().nan_to_num(0.0, posinf=0.0, neginf=0.0)
    terms = scale * float((q.double().abs().amax((0, 1, 2)) * k.double().abs().amax((0, 1, 2))).sum())
    return q, k, lse, scale, terms


def _tol(d, n, terms, lse):
    top = float(lse.abs().max())
    return d * 2.0 ** -24 * terms + (terms + top) * 1.45 * 2.0 ** -23 + 2.0 ** -21 + (n / 64 + 64) * 2.0 ** -24


@pytest.mark.parametrize("B,H,Hkv,N,d,causal,window,ragged", [
    (1, 1, 1, 1, 64, True, 1, False), (1, 4, 2, 100, 64, True, 100, False), (2, 4, 1, 333, 128, True, 333, True),
    (1, 8, 2, 640, 128, True, 64, False), (1, 6, 3, 257, 256, True, 300, False), (2, 3, 3, 300, 64, False, 17, True),
    (1, 2, 2, 1500, 128, False, 1500, False), (1, 16, 1, 513, 64, True, 200, True), (1, 32, 8, 1024, 128, True, 1, False),
    (3, 2, 1, 129, 256, False, 128, True), (1, 4, 4, 2049, 64, True, 2049, False), (2, 2, 2, 700, 256, True, 100, True)])
def test_against_column_sums(B, H, Hkv, N, d, causal, window, ragged):
    from exact_io_aware_85_b200 import fa
    g = torch.Generator().manual_seed(N)
    n_rows = torch.randint(0, N + 1, (B,), generator=g, dtype=torch.int32) if ragged else None
    q, k, lse, scale, terms = _inputs(B, H, Hkv, N, d, N + d, causal, n_rows)
    w = torch.full((B, Hkv, N + 5), -3.0, device=DEV)
    ws = torch.full((fa.fa_key_weights_workspace_bytes(B, H, Hkv, N, d, window),), 255, dtype=torch.uint8, device=DEV)
    fa.fa_key_weights(q.to(DEV), k.to(DEV), lse.to(DEV), w, causal, scale, ws, window=window,
                      n_rows=None if n_rows is None else n_rows.to(DEV))
    torch.cuda.synchronize()
    assert fa.fa_check_status() == fa.FA_OK
    want = R.key_weights(q.double(), k.double(), lse.double(), causal, scale, window, n_rows)
    assert (w[:, :, N:] == -3).all()  # columns behind N stay as they were
    got = w[:, :, :N].cpu().double()
    assert ((got - want).abs() <= _tol(d, N * (H // Hkv), terms, lse) * want).all()
    if ragged:
        for b in range(B):
            assert (got[b, :, int(n_rows[b]):] == 0).all()


def test_with_the_forwards_logsumexp_the_weights_add_up():
    """q, k and fa_fwd_gqa's own lse: every query row gives its keys a total of one."""
    from exact_io_aware_85_b200 import fa
    B, H, Hkv, N, d = 1, 8, 2, 777, 128
    g = torch.Generator().manual_seed(4)
    q = torch.randn((B, H, N, d), generator=g).to(torch.bfloat16).to(DEV)
    k, v = (torch.randn((B, Hkv, N, d), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    o, lse = torch.empty_like(q), torch.empty((B, H, N), device=DEV)
    fa.fa_fwd_gqa(q, k, v, o, lse, True, 1 / math.sqrt(d))
    w = torch.empty((B, Hkv, N), device=DEV)
    ws = torch.empty(fa.fa_key_weights_workspace_bytes(B, H, Hkv, N, d, N), dtype=torch.uint8, device=DEV)
    fa.fa_key_weights(q, k, lse, w, True, 1 / math.sqrt(d), ws)
    # the forward's lse is good to 1e-3 absolute by its own contract
    assert abs(float(w.double().sum()) / (H * N) - 1) <= 1e-3


def test_rows_that_hold_anything_outside_the_window():
    """lse, q and k behind the sequences, and lse and q before the window, are not looked at."""
    from exact_io_aware_85_b200 import fa
    B, H, Hkv, N, d, window = 2, 4, 2, 300, 64, 40
    n_rows = torch.tensor([300, 170], dtype=torch.int32)
    q, k, lse, scale, _ = _inputs(B, H, Hkv, N, d, 3, True, n_rows)
    ws = torch.empty(fa.fa_key_weights_workspace_bytes(B, H, Hkv, N, d, window), dtype=torch.uint8, device=DEV)
    out = []
    for dirty in (False, True):
        a, b, c = q.clone(), k.clone(), lse.clone()
        if dirty:
            for i in range(B):
                n = int(n_rows[i])
                a[i, :, n:], b[i, :, n:], c[i, :, n:] = float("nan"), float("inf"), float("nan")
                a[i, :, :n - window], c[i, :, :n - window] = float("nan"), float("-inf")
        w = torch.empty((B, Hkv, N), device=DEV)
        fa.fa_key_weights(a.to(DEV), b.to(DEV), c.to(DEV), w, True, scale, ws, window=window, n_rows=n_rows.to(DEV))
        out.append(w)
    assert torch.equal(*out)


def test_the_same_bits_again_and_from_a_graph():
    from exact_io_aware_85_b200 import fa
    B, H, Hkv, N, d = 2, 8, 2, 1111, 128
    n_rows = torch.tensor([1111, 640], dtype=torch.int32, device=DEV)
    q, k, lse, scale, _ = _inputs(B, H, Hkv, N, d, 5, True, n_rows.cpu())
    q, k, lse = q.to(DEV), k.to(DEV), lse.to(DEV)
    ws = torch.empty(fa.fa_key_weights_workspace_bytes(B, H, Hkv, N, d, 500), dtype=torch.uint8, device=DEV)
    w = [torch.empty((B, Hkv, N), device=DEV) for _ in range(4)]
    fa.fa_key_weights(q, k, lse, w[0], True, scale, ws, window=500, n_rows=n_rows)
    ws.fill_(255)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fa.fa_key_weights(q, k, lse, w[1], True, scale, ws, window=500, n_rows=n_rows, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_key_weights(q, k, lse, w[2], True, scale, ws, window=500, n_rows=n_rows)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w[0], w[1]) and torch.equal(w[0], w[2])
    n_rows.fill_(300)  # the graph follows the lengths
    graph.replay()
    fa.fa_key_weights(q, k, lse, w[3], True, scale, ws, window=500, n_rows=n_rows)
    torch.cuda.synchronize()
    assert torch.equal(w[2], w[3]) and (w[3][:, :, 300:] == 0).all()
    assert fa.fa_check_status() == fa.FA_OK


def test_log_sum_exps_that_are_not_finite():
    """A row with lse = +infinity gives nothing; one with NaN makes the weight of every key it sees NaN."""
    from exact_io_aware_85_b200 import fa
    B, H, Hkv, N, d = 1, 2, 2, 300, 64
    q, k, lse, scale, _ = _inputs(B, H, Hkv, N, d, 6, True)
    lse[0, 0, 200] = float("inf")
    lse[0, 1, 200] = float("nan")
    ws = torch.empty(fa.fa_key_weights_workspace_bytes(B, H, Hkv, N, d, N), dtype=torch.uint8, device=DEV)
    w = torch.empty((B, Hkv, N), device=DEV)
    fa.fa_key_weights(q.to(DEV), k.to(DEV), lse.to(DEV), w, True, scale, ws)
    want = R.key_weights(q.double(), k.double(), lse.double(), True, scale, N)
    assert torch.isnan(w[0, 1, :201]).all() and torch.isfinite(w[0, 1, 201:]).all()
    # relative 2^-16 covers what the finite rows' arithmetic may be off (see the tolerance above)
    assert ((w[0, 0].cpu().double() - want[0, 0]).abs() <= 2.0 ** -16 * want[0, 0]).all()
