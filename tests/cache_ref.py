"""64-bit references of the 4-bit cache operators (torch on the CPU), from their definitions in include/fa.h."""
from __future__ import annotations

import math

import torch


def walsh(d):
    h = torch.ones((1, 1), dtype=torch.float64)
    while h.shape[0] < d:
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
    return h


def rotate(x, signs):
    return x if signs is None else (x * signs.double()) @ walsh(x.shape[-1])


def quantise(x, signs=None):
    """codes (int, 1..15), scale (bf16 values in float64) and y of rows x (float64)."""
    y = rotate(x, signs)
    amax = y.abs().amax(-1)
    s = (amax / 7).to(torch.float32).to(torch.bfloat16).double()
    c = torch.where(s[..., None] > 0, torch.round(y / s[..., None]).clamp(-7, 7), torch.zeros_like(y))
    return (c + 8).to(torch.int64), s, y


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).to(torch.uint8)


def unpack(packed):
    p = packed.to(torch.int64)
    return torch.stack((p & 15, p >> 4), -1).reshape(*p.shape[:-1], -1)


def values(packed, scale, signs=None):
    """The values that rows stand for, in the original basis."""
    d = 2 * packed.shape[-1]
    y = (unpack(packed) - 8).double() * scale.double()[..., None]
    return y if signs is None else (y @ walsh(d)) * signs.double() / d


def decode(q, k, v, lens, scale):
    """q [B,H,d], k, v [B,Hkv,C,d] (float64, original basis), lens [B,Hkv] -> o, lse, weights [B,Hkv,C],
    and per (b, h): sum_j p_j |v_j| (the size of what rounding P and O can move) and
    max_j scale sum_i |q_i k_ji| (the size of the terms of a score)."""
    B, H, d = q.shape
    Hkv, C = k.shape[1], k.shape[2]
    g = H // Hkv
    o = torch.zeros((B, H, d), dtype=torch.float64)
    lse = torch.full((B, H), -math.inf, dtype=torch.float64)
    w = torch.zeros((B, Hkv, C), dtype=torch.float64)
    pv, terms = torch.zeros_like(o), torch.zeros((B, H), dtype=torch.float64)
    for b in range(B):
        for hk in range(Hkv):
            n = max(0, min(int(lens[b, hk]), C))
            if not n:
                continue
            at = slice(hk * g, (hk + 1) * g)
            s = scale * q[b, at] @ k[b, hk, :n].T
            p = torch.softmax(s, -1)
            lse[b, at] = torch.logsumexp(s, -1)
            o[b, at] = p @ v[b, hk, :n]
            w[b, hk, :n] = p.sum(0)
            pv[b, at] = p @ v[b, hk, :n].abs()
            terms[b, at] = (scale * q[b, at].abs() @ k[b, hk, :n].abs().T).amax(-1)
    return o, lse, w, pv, terms


def key_weights(q, k, lse, causal, scale, window, n_rows=None):
    B, H, N, d = q.shape
    Hkv = k.shape[1]
    w = torch.zeros((B, Hkv, N), dtype=torch.float64)
    for b in range(B):
        n = N if n_rows is None else max(0, min(int(n_rows[b]), N))
        lo = max(0, n - window)
        for h in range(H):
            p = torch.exp(scale * q[b, h, lo:n] @ k[b, h // (H // Hkv), :n].T - lse[b, h, lo:n, None])
            w[b, h // (H // Hkv), :n] += (torch.tril(p, diagonal=lo) if causal else p).sum(0)
    return w


def _order(w):
    """Weights as numbers that sort: NaN above infinity, -0 with 0."""
    return [(1, 0.0) if math.isnan(x) else (0, x + 0.0) for x in w]


def evict_keep(w, keep, n_recent, n_sink, length):
    """One head: the ascending list of the rows that stay."""
    key = _order(w)
    held = lambda j: j < n_sink or j >= length - n_recent  # noqa: E731
    rows = sorted(range(length), key=lambda j: ((0, 0, 0) if held(j) else (1, -key[j][0], -key[j][1]), j))
    return sorted(rows[:keep])


def evict_slots(acc, pos, length, seen, budget, T, n_recent, n_sink):
    """One head: the rows that T new tokens take, and the new length."""
    length = max(0, min(length, budget))
    free = list(range(length, min(budget, length + T)))
    key = _order(acc)
    held = lambda j: pos[j] < n_sink or pos[j] >= seen - n_recent  # noqa: E731
    rows = sorted(range(length), key=lambda j: ((2, 0.0) if held(j) else key[j], -j))
    return free + sorted(rows[:T - len(free)]), min(budget, length + T)
