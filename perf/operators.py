"""The serving operators around the 4-bit key/value cache: cases, inputs, plain forms and definitions.

Four operators: the attention weight that each key of a prompt received (``weights``), eviction by that
weight (``keep``: which rows of a prompt stay; ``slots``: which rows of a full cache new tokens replace),
writing and reading rows of the cache held in 4 bits (``append``), and one decoding step over it (``decode``).
"""
import math

import torch

own = False

GROUP = 128  # cache capacities are multiples of this many rows


def listed():
    return [
        # a SnapKV-like observation window: the last 64 queries of 8 prompts of 32768 tokens, 8 key/value heads
        _weights("weights window 64 of 32768", 8, 32, 8, 32768, 128, True, 64, False),
        # every query of one prompt of the prefill length
        _weights("weights prompt 8192", 1, 32, 8, 8192, 128, True, 8192, False),
        # the smallest call: one short ragged batch, where latency counts
        _weights("weights short 333", 2, 4, 2, 333, 64, True, 333, True),
        # a prompt's end: 32768 rows down to 4096 in each of 64 heads
        _keep("keep 4096 of 32768", 8, 8, 32768, 4096, 64, 4, False),
        # every decoding step of a full cache: one row makes room
        _slots("slots 1 of 4096", 8, 8, 4096, 4096, 1, 256, 4, False),
        # a chunk of 512 tokens into one very long cache
        _slots("slots 512 of 131000", 1, 8, 131072, 131000, 512, 1024, 4, False),
        # a prompt batch of the prefill size into the cache, and its history read back for the next chunk
        _append("append prompt 8192", 4, 8, 8192, 8192, 8192, 128, True, "front"),
        # a token of 8 sequences into replaced rows of a 32768-row cache
        _append("append token", 8, 8, 1, 1, 32768, 128, True, "slots"),
        # the surviving rows of one long prompt, head dim 256
        _append("append kept 4000 of 20001", 1, 8, 20001, 4000, 4096, 256, False, "rows"),
        # the decoding workload: 8 sequences, 32768 rows, 8 key/value heads shared by 4 query heads each
        _decode("decode 8 x 32768", 8, 32, 8, 32768, 32768, 128, True, True, False),
        # a short single sequence without grouping: latency
        _decode("decode 1 x 1000", 1, 8, 8, 1024, 1000, 64, False, False, False),
        # a ragged batch, 8 query heads per key/value head, head dim 256
        _decode("decode ragged 16 x 16384", 16, 32, 4, 16384, 16384, 256, False, True, True),
    ]


def _weights(name, B, H, Hkv, N, d, causal, window, ragged):
    return {"name": name, "op": "weights", "B": B, "H": H, "Hkv": Hkv, "N": N, "d": d, "causal": causal,
            "window": window, "ragged": ragged}


def _keep(name, B, Hkv, N, keep, recent, sink, ragged):
    return {"name": name, "op": "keep", "B": B, "Hkv": Hkv, "N": N, "keep": keep, "recent": recent, "sink": sink,
            "ragged": ragged}


def _slots(name, B, Hkv, C, budget, T, recent, sink, ragged):
    return {"name": name, "op": "slots", "B": B, "Hkv": Hkv, "C": C, "budget": budget, "T": T, "recent": recent,
            "sink": sink, "ragged": ragged}


def _append(name, B, Hkv, N, T, C, d, rotate, how):
    return {"name": name, "op": "append", "B": B, "Hkv": Hkv, "N": N, "T": T, "C": C, "d": d, "rotate": rotate,
            "how": how}


def _decode(name, B, H, Hkv, C, rows, d, rotate, weights, ragged):
    return {"name": name, "op": "decode", "B": B, "H": H, "Hkv": Hkv, "C": C, "rows": rows, "d": d, "rotate": rotate,
            "weights": weights, "ragged": ragged}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _up(n):
    return -(-n // GROUP) * GROUP


def draw(rng):
    op = rng.choice(["weights", "keep", "slots", "append", "append", "decode", "decode", "decode"])
    d = rng.choice([64, 128, 256])
    Hkv, g, B = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8, 12, 16]), _log(rng, 1, 16)
    ragged = rng.random() < 0.5
    if op == "weights":
        g = min(g, 32 // Hkv)
        N = _log(rng, 1, 9000)
        B = max(1, min(B, int(32 * 8192 * 8192 / (Hkv * g * N * N * max(1, d // 128)))))
        window = N if rng.random() < 0.5 else _log(rng, 1, N)
        c = _weights("", B, Hkv * g, Hkv, N, d, rng.random() < 0.8, window, ragged)
    elif op == "keep":
        N = _log(rng, 2, 100000)
        B = max(1, min(B, 8 * 8 * 32768 // (N * Hkv)))
        keep = _log(rng, 1, N)
        recent = rng.randint(0, keep // 2)
        c = _keep("", B, Hkv, N, keep, recent, min(4, keep - recent), ragged)
    elif op == "slots":
        budget = _log(rng, 40, 131072)
        B = max(1, min(B, 8 * 131072 // (budget * Hkv)))
        T = 1 if rng.random() < 0.5 else _log(rng, 1, max(1, budget // 8))
        c = _slots("", B, Hkv, _up(budget), budget, T, rng.randint(0, budget // 4), 4, ragged)
    elif op == "append":
        how = rng.choice(["front", "slots", "rows"])
        N = _log(rng, 1, 20000)
        T = max(1, N // rng.randint(2, 6)) if how == "rows" else N
        B = max(1, min(B, 4 * 8 * 8192 * 128 // (N * Hkv * d)))
        c = _append("", B, Hkv, N, T, _up(T + rng.randint(0, 2 * T)), d, rng.random() < 0.5, how)
    else:
        rows = _log(rng, 1, 60000)
        B = max(1, min(B, 8 * 8 * 32768 * 128 // (_up(rows) * Hkv * d)))
        c = _decode("", B, Hkv * g, Hkv, _up(rows), rows, d, rng.random() < 0.5, rng.random() < 0.5, ragged)
    del c["name"]
    return c


# ---- inputs --------------------------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def _ints(gen, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=gen, device="cuda", dtype=torch.int32)


def _signs(gen, d):
    return (torch.randint(0, 2, (d,), generator=gen, device="cuda") * 2 - 1).float()


def _heavy(gen, *shape):
    """Accumulated weights as they come about: many light keys, a few heavy ones."""
    return torch.exp(2.5 * torch.randn(shape, generator=gen, device="cuda"))


def _random_cache(gen, B, Hkv, C, d):
    """A filled cache: normal rows, quantised (the codes of a rotated and of a plain cache look alike)."""
    codes, scales = [], []
    for sd in (1.0, 0.7):
        c = torch.empty((B, Hkv, C, d // 2), dtype=torch.uint8, device="cuda")
        s = torch.empty((B, Hkv, C), dtype=torch.bfloat16, device="cuda")
        for b in range(B):
            x = torch.randn((Hkv, C, d), generator=gen, device="cuda") * sd
            s[b] = (x.abs().amax(-1) / 7).to(torch.bfloat16)
            n = torch.clamp(torch.round(x / s[b].float()[..., None]), -7, 7).to(torch.uint8) + 8 & 15
            c[b] = n[..., 0::2] | (n[..., 1::2] << 4)
        codes.append(c)
        scales.append(s)
    return codes[0], scales[0], codes[1], scales[1]


def _lse_rows(q, k, scale, causal, lo):
    """Row log-sum-exp of rows lo.. for one head, 32 bits."""
    s = q[lo:].float() @ k.float().T * scale
    if causal:
        i = torch.arange(lo, q.shape[0], device="cuda")
        s.masked_fill_(torch.arange(k.shape[0], device="cuda")[None, :] > i[:, None], float("-inf"))
    return torch.logsumexp(s, -1)


def prepare(case, seed):
    c, gen = case, _gen(seed)
    op, B, Hkv = c["op"], c["B"], c["Hkv"]
    s = {"case": c, "op": op}
    if op == "weights":
        H, N, d = c["H"], c["N"], c["d"]
        s["q"], s["k"] = _normal(gen, B, H, N, d), _normal(gen, B, Hkv, N, d)
        s["scale"] = 1 / math.sqrt(d)
        s["n_rows"] = _ints(gen, max(1, N // 3), N + 1, B) if c["ragged"] else None
        # rows that no window reaches hold an ordinary value
        s["lse"] = (torch.log(torch.arange(1, N + 1, device="cuda").float()) + 0.5).expand(B, H, N).contiguous()
        lens = s["n_rows"].tolist() if c["ragged"] else [N] * B
        for b in range(B):
            for h in range(H):
                n = lens[b]
                lo = max(0, n - c["window"])
                s["lse"][b, h, lo:n] = _lse_rows(s["q"][b, h, :n], s["k"][b, h // (H // Hkv), :n], s["scale"],
                                                 c["causal"], lo)
        s["w"] = torch.zeros((B, Hkv, N), device="cuda")
    elif op == "keep":
        s["w"] = _heavy(gen, B, Hkv, c["N"])
        s["lens"] = _ints(gen, 1, c["N"] + 1, B, Hkv) if c["ragged"] else None
        s["idx"] = torch.empty((B, Hkv, c["keep"]), dtype=torch.int32, device="cuda")
        s["count"] = torch.empty((B, Hkv), dtype=torch.int32, device="cuda")
    elif op == "slots":
        C, budget = c["C"], c["budget"]
        s["acc"] = _heavy(gen, B, Hkv, C)
        # positions of the rows: the cache has been through many replacements
        s["pos"] = torch.argsort(torch.rand((B, Hkv, C), generator=gen, device="cuda"), -1).to(torch.int32)
        s["seen"] = torch.full((B,), C, dtype=torch.int32, device="cuda")
        s["lens"] = (_ints(gen, budget // 2, budget + 1, B, Hkv) if c["ragged"] else
                     torch.full((B, Hkv), budget, dtype=torch.int32, device="cuda"))
        s["slots"] = torch.empty((B, Hkv, c["T"]), dtype=torch.int32, device="cuda")
    elif op == "append":
        N, T, C, d = c["N"], c["T"], c["C"], c["d"]
        s["k"], s["v"] = _normal(gen, B, Hkv, N, d), _normal(gen, B, Hkv, N, d)
        s["signs"] = _signs(gen, d) if c["rotate"] else None
        s["w"] = _heavy(gen, B, Hkv, N)
        s["cache"] = (torch.zeros((B, Hkv, C, d // 2), dtype=torch.uint8, device="cuda"),
                      torch.zeros((B, Hkv, C), dtype=torch.bfloat16, device="cuda"),
                      torch.zeros((B, Hkv, C, d // 2), dtype=torch.uint8, device="cuda"),
                      torch.zeros((B, Hkv, C), dtype=torch.bfloat16, device="cuda"))
        s["acc"] = torch.zeros((B, Hkv, C), device="cuda")
        s["pos"] = torch.zeros((B, Hkv, C), dtype=torch.int32, device="cuda")
        s["base"] = _ints(gen, 0, 1000, B)
        pick = lambda n: torch.argsort(torch.rand((B, Hkv, n), generator=gen, device="cuda"), -1)[..., :T]  # noqa: E731
        s["slots"] = pick(C).to(torch.int32).contiguous() if c["how"] == "slots" else None
        s["rows"] = pick(N).sort(-1).values.to(torch.int32).contiguous() if c["how"] == "rows" else None
        s["k_out"] = torch.empty((B, Hkv, T, d), dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.empty_like(s["k_out"])
    else:
        H, C, d = c["H"], c["C"], c["d"]
        s["q"] = _normal(gen, B, H, d)
        s["cache"] = _random_cache(gen, B, Hkv, C, d)
        s["signs"] = _signs(gen, d) if c["rotate"] else None
        # a rotated row is sqrt(d) times as long as the row it came from
        if c["rotate"]:
            s["cache"] = (s["cache"][0], s["cache"][1] * math.sqrt(d), s["cache"][2], s["cache"][3])
        s["lens"] = (_ints(gen, 0, c["rows"] + 1, B, Hkv) if c["ragged"] else
                     torch.full((B, Hkv), c["rows"], dtype=torch.int32, device="cuda"))
        s["acc"] = _heavy(gen, B, Hkv, C) if c["weights"] else None
        s["scale"] = 1 / math.sqrt(d)
        s["o"] = torch.empty((B, H, d), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((B, H), device="cuda")
    return s


# ---- one pass --------------------------------------------------------------------------------------------------


def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _hadamard(d, dtype):
    """The Sylvester Walsh-Hadamard matrix: entry (i, j) is -1 to the number of ones of i & j."""
    i = torch.arange(d, device="cuda")
    x = i[:, None] & i[None, :]
    x = x ^ (x >> 4)
    x = x ^ (x >> 2)
    x = x ^ (x >> 1)
    return (1 - 2 * (x & 1)).to(dtype)


def _plain_weights(s):
    c = s["case"]
    B, H, Hkv, N, W = c["B"], c["H"], c["Hkv"], c["N"], min(c["window"], c["N"])
    n = s["n_rows"].long() if s["n_rows"] is not None else torch.full((B,), N, device="cuda")
    i = n[:, None] - W + torch.arange(W, device="cuda")  # the query rows of each sequence's window
    at = i.clamp(min=0)[:, None, :].expand(B, H, W)
    q = torch.gather(s["q"], 2, at[..., None].expand(B, H, W, c["d"])).float().view(B, Hkv, H // Hkv, W, c["d"])
    lse = torch.gather(s["lse"], 2, at).view(B, Hkv, H // Hkv, W)
    p = torch.matmul(q, s["k"].float()[:, :, None].transpose(-1, -2))
    p = p.mul_(s["scale"]).sub_(lse[..., None]).exp_()
    j = torch.arange(N, device="cuda")
    dead = (i[:, :, None] < 0) | (j >= n[:, None, None])
    if c["causal"]:
        dead = dead | (j > i[:, :, None])
    p.masked_fill_(dead[:, None, None], 0.0)
    s["w"].copy_(p.sum(3).sum(2))
    return s["w"]


def _plain_keep(s):
    c = s["case"]
    N, keep = c["N"], c["keep"]
    n = s["lens"].long() if s["lens"] is not None else torch.full((c["B"], c["Hkv"]), N, device="cuda")
    j = torch.arange(N, device="cuda")
    w = s["w"].masked_fill((j < c["sink"]) | (j >= n[..., None] - c["recent"]), float("inf"))
    w = w.masked_fill(j >= n[..., None], float("-inf"))
    first = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    first = first.masked_fill(first >= n[..., None], N).sort(-1).values
    s["idx"].copy_(first.masked_fill(first == N, -1))
    s["count"].copy_(n.clamp(max=keep))
    return s["idx"], s["count"]


def _plain_slots(s):
    c = s["case"]
    C, budget, T = c["C"], c["budget"], c["T"]
    n = s["lens"].long()
    j = torch.arange(C, device="cuda")
    held = (s["pos"] < c["sink"]) | (s["pos"] >= s["seen"][:, None, None] - c["recent"])
    w = s["acc"].masked_fill(held, torch.finfo(torch.float32).max)
    # the order in which rows are taken: free rows from the front, then the lightest, the last row first among equals
    free = (budget - n).clamp(min=0, max=T)
    taken = torch.where(j < n[..., None], w, float("inf"))[..., :budget].flip(-1)
    light = budget - 1 - torch.sort(taken, dim=-1, stable=True).indices[..., :T]
    t = torch.arange(T, device="cuda")
    light = light.masked_fill(t >= (T - free)[..., None], C).sort(-1).values  # the rows replaced, ascending
    back = torch.gather(light, -1, (t - free[..., None]).clamp(min=0))
    s["slots"].copy_(torch.where(t < free[..., None], n[..., None] + t, back))
    s["lens"].copy_((n + T).clamp(max=budget))
    return s["slots"], s["lens"]


def _plain_append(s):
    c = s["case"]
    B, Hkv, T = c["B"], c["Hkv"], c["T"]
    t = torch.arange(T, device="cuda").expand(B, Hkv, T)
    src = s["rows"].long() if s["rows"] is not None else t
    dst = s["slots"].long() if s["slots"] is not None else t
    _plain_write(s["k"], s["signs"], src, dst, s["cache"][0], s["cache"][1])
    _plain_write(s["v"], None, src, dst, s["cache"][2], s["cache"][3])
    s["acc"].scatter_(2, dst, torch.gather(s["w"], 2, src))
    s["pos"].scatter_(2, dst, (src + s["base"][:, None, None]).to(torch.int32))
    # and the rows as the cache holds them, in the order in which they were written
    _plain_read(s["cache"][0], s["cache"][1], s["signs"], dst, s["k_out"])
    _plain_read(s["cache"][2], s["cache"][3], None, dst, s["v_out"])
    return s["k_out"], s["v_out"], s["acc"], s["pos"]


def _plain_write(x, signs, src, dst, codes, scales):
    d = x.shape[-1]
    y = torch.gather(x, 2, src[..., None].expand(*src.shape, d))
    # a rotated value can lie next to the border of two codes: 64 bits
    y = y.float() if signs is None else (y.double() * signs.double()) @ _hadamard(d, torch.float64)
    scale = (y.abs().amax(-1).float() / 7).to(torch.bfloat16)
    n = torch.round(y / scale[..., None].to(y.dtype)).clamp(-7, 7)
    n = torch.where(scale[..., None] == 0, torch.zeros_like(n), n).to(torch.int16) + 8
    n = (n[..., 0::2] | (n[..., 1::2] << 4)).to(torch.uint8)
    codes.scatter_(2, dst[..., None].expand(*dst.shape, d // 2), n)
    scales.scatter_(2, dst, scale)


def _plain_read(codes, scales, signs, dst, to):
    d = to.shape[-1]
    x = _unpack(torch.gather(codes, 2, dst[..., None].expand(*dst.shape, d // 2)), torch.gather(scales, 2, dst))
    to.copy_(x if signs is None else (x @ _hadamard(d, torch.float32)) * signs / d)


def _unpack(codes, scale):
    x = torch.stack((codes & 15, codes >> 4), -1).view(*codes.shape[:-1], -1).float().sub_(8)
    return x.mul_(scale.float()[..., None])


def _plain_decode(s):
    c = s["case"]
    B, H, Hkv, C, d = c["B"], c["H"], c["Hkv"], c["C"], c["d"]
    kc, ks, vc, vs = s["cache"]
    q = s["q"].double()
    if s["signs"] is not None:
        q = (q * s["signs"].double()) @ _hadamard(d, torch.float64) / d
    q = q.float().view(B, Hkv, H // Hkv, d)
    x = torch.matmul(q, _unpack(kc, ks).transpose(-1, -2)).mul_(s["scale"])
    live = torch.arange(C, device="cuda") < s["lens"][..., None]
    x = x.masked_fill(~live[:, :, None], float("-inf"))
    some = (s["lens"] > 0)[:, :, None]
    m = torch.where(some, x.amax(-1), torch.zeros((), device="cuda"))
    p = torch.exp(x - m[..., None])
    l = p.sum(-1)
    p = p / torch.where(some, l, torch.ones((), device="cuda"))[..., None]
    s["o"].copy_(torch.matmul(p, _unpack(vc, vs)).view(B, H, d))
    s["lse"].copy_((m + torch.log(l)).view(B, H))
    if s["acc"] is None:
        return s["o"], s["lse"]
    s["acc"].add_(p.sum(2))
    return s["o"], s["lse"], s["acc"]


_plain = {"weights": _plain_weights, "keep": _plain_keep, "slots": _plain_slots, "append": _plain_append,
          "decode": _plain_decode}


def _workspace(s, nbytes):
    """A program's workspace: made once, kept."""
    if "ws" not in s:
        s["ws"] = torch.empty(nbytes(), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _own_weights(s):
    from exact_io_aware_85_b200 import fa
    c = s["case"]
    ws = _workspace(s, lambda: fa.fa_key_weights_workspace_bytes(c["B"], c["H"], c["Hkv"], c["N"], c["d"], c["window"]))
    fa.fa_key_weights(s["q"], s["k"], s["lse"], s["w"], c["causal"], s["scale"], ws, window=c["window"],
                      n_rows=s["n_rows"])
    return s["w"]


def _own_keep(s):
    from exact_io_aware_85_b200 import fa
    c = s["case"]
    fa.fa_evict_keep(s["w"], s["idx"], s["count"], c["recent"], c["sink"], lens=s["lens"])
    return s["idx"], s["count"]


def _own_slots(s):
    from exact_io_aware_85_b200 import fa
    c = s["case"]
    fa.fa_evict_slots(s["acc"], s["pos"], s["lens"], s["seen"], s["slots"], c["budget"], c["recent"], c["sink"])
    return s["slots"], s["lens"]


def _own_append(s):
    from exact_io_aware_85_b200 import fa
    fa.fa_kv4_append(s["k"], s["v"], *s["cache"], signs=s["signs"], rows=s["rows"], slots=s["slots"], w=s["w"],
                     acc=s["acc"], pos=s["pos"], base=s["base"])
    fa.fa_kv4_read(*s["cache"], s["k_out"], s["v_out"], signs=s["signs"], slots=s["slots"])
    return s["k_out"], s["v_out"], s["acc"], s["pos"]


def _own_decode(s):
    from exact_io_aware_85_b200 import fa
    c = s["case"]
    ws = _workspace(s, lambda: fa.fa_decode_kv4_workspace_bytes(c["B"], c["H"], c["Hkv"], c["C"], c["d"], c["weights"]))
    fa.fa_decode_kv4(s["q"], *s["cache"], s["lens"], s["o"], s["lse"], s["scale"], ws, signs=s["signs"], acc=s["acc"])
    return (s["o"], s["lse"]) if s["acc"] is None else (s["o"], s["lse"], s["acc"])


_own = {"weights": _own_weights, "keep": _own_keep, "slots": _own_slots, "append": _own_append,
        "decode": _own_decode}


# ---- what a pass cannot do without -------------------------------------------------------------------------------


def work(case):
    c = case
    B, Hkv = c["B"], c["Hkv"]
    if c["op"] == "weights":
        H, N, W, d = c["H"], c["N"], min(c["window"], c["N"]), c["d"]
        pairs = W * N - (W * (W - 1) // 2 if c["causal"] else 0)  # (query, key) pairs of one head
        if c["ragged"]:  # lengths between a third of N and N: the expected share
            pairs = pairs * 0.5
        return {"bytes": 2 * B * d * (Hkv * N + H * W) + 4 * B * (H * W + Hkv * N), "flops": 2.0 * B * H * pairs * d}
    if c["op"] == "keep":
        n = c["N"] * (0.5 if c["ragged"] else 1)
        return {"bytes": 4 * B * Hkv * (n + c["keep"] + 1), "flops": B * Hkv * n}
    if c["op"] == "slots":
        n = c["budget"] * (0.75 if c["ragged"] else 1)
        return {"bytes": 4 * B * Hkv * (2 * n + c["T"] + 2), "flops": B * Hkv * n}
    if c["op"] == "append":
        d, rows = c["d"], B * Hkv * c["T"]
        row = d // 2 + 2  # a row of the cache
        return {"bytes": 2 * rows * (2 * (2 * d + row)) + 12 * rows,
                "flops": rows * d * (8 + (2 * math.log2(d) if c["rotate"] else 0))}
    H, d = c["H"], c["d"]
    n = B * Hkv * c["rows"] * (0.5 if c["ragged"] else 1)
    return {"bytes": n * (d + 4 + (8 if c["weights"] else 0)) + B * H * (4 * d + 4), "flops": 4.0 * n * (H // Hkv) * d}


# ---- the definitions, in 64 bits ---------------------------------------------------------------------------------


def _walsh(d):
    """The Walsh-Hadamard matrix by its doubling: H_2n = [[H, H], [H, -H]]."""
    h = torch.ones((1, 1), dtype=torch.float64, device="cuda")
    while h.shape[0] < d:
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
    return h


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "weights":
        return _exact_weights(c, s)
    if c["op"] == "append":
        return _exact_append(c, s)
    if c["op"] == "decode":
        return _exact_decode(c, s)
    return None  # eviction answers in row numbers


def _exact_weights(c, s):
    g, w = c["H"] // c["Hkv"], torch.zeros((c["B"], c["Hkv"], c["N"]), dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        n = int(s["n_rows"][b]) if s["n_rows"] is not None else c["N"]
        lo = max(0, n - c["window"])
        for h in range(c["H"]):
            x = s["scale"] * (s["q"][b, h, lo:n].double() @ s["k"][b, h // g, :n].double().T)
            p = torch.exp(x - s["lse"][b, h, lo:n, None].double())
            w[b, h // g, :n] += (torch.tril(p, diagonal=lo) if c["causal"] else p).sum(0)
    return w


def _exact_append(c, s):
    B, Hkv, N, T, d = c["B"], c["Hkv"], c["N"], c["T"], c["d"]
    h, outs = _walsh(d), []
    acc = s["acc"].double()
    for x, signs in ((s["k"], s["signs"]), (s["v"], None)):
        to = torch.empty((B, Hkv, T, d), dtype=torch.float64, device="cuda")
        for b in range(B):
            for k in range(Hkv):
                y = x[b, k].double() if s["rows"] is None else x[b, k, s["rows"][b, k].long()].double()
                if signs is not None:
                    y = torch.einsum("td,d,de->te", y, signs.double(), h)
                # the scale is a number of the format: bf16, as the cache stores it
                f = (y.abs().max(-1, keepdim=True).values / 7).to(torch.bfloat16).double()
                y = f * torch.round(y / f).clip(-7, 7)
                to[b, k] = y if signs is None else torch.einsum("te,ed,d->td", y, h, signs.double()) / d
        outs.append(to)
    for b in range(B):
        for k in range(Hkv):
            src = slice(0, T) if s["rows"] is None else s["rows"][b, k].long()
            dst = slice(0, T) if s["slots"] is None else s["slots"][b, k].long()
            acc[b, k, dst] = s["w"][b, k, src].double()
    return outs[0], outs[1], acc, None


def _exact_decode(c, s):
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    g, (kc, ks, vc, vs) = H // Hkv, s["cache"]
    o = torch.zeros((B, H, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device="cuda")
    acc = s["acc"].double() if s["acc"] is not None else None

    def rows(codes, scale, n):
        x = torch.empty((n, d), dtype=torch.float64, device="cuda")
        x[:, 0::2], x[:, 1::2] = (codes[:n] % 16).double(), (codes[:n] // 16).double()
        return (x - 8) * scale[:n].double()[:, None]

    for b in range(B):
        for k in range(Hkv):
            n = int(s["lens"][b, k])
            if n == 0:
                continue
            at = slice(k * g, (k + 1) * g)
            q = s["q"][b, at].double()
            if s["signs"] is not None:
                q = torch.einsum("gd,d,de->ge", q, s["signs"].double(), _walsh(d)) / d
            x = s["scale"] * (q @ rows(kc[b, k], ks[b, k], n).T)
            lse[b, at] = torch.logsumexp(x, -1)
            p = torch.softmax(x, -1)
            o[b, at] = p @ rows(vc[b, k], vs[b, k], n)
            if acc is not None:
                acc[b, k, :n] += p.sum(0)
    return (o, lse) if acc is None else (o, lse, acc)
