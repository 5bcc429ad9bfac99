"""The paged 4-bit cache and the operators around it, as cases that can be timed and checked.

Four operators, in the order in which a serving step uses them:

  plan    block tables, slot maps and positions from the requests' lengths
  rope    RMS norm of every query and key head with the position rotation
  append  INT4 quantisation of new keys and values into the pages of a slot map
  attend  attention of a ragged batch of query rows over the pages

`run` computes them in plain torch where `own` is false and through
bit_kv_cache_qwm_gb300.paged where it is true.

Cache bytes: pool [pages][kv heads][block]; a block of p token slots holds
  K codes [p][d/2]     channel c in byte c/2, bits 4 (c mod 2)
  K params [p][d/32]   float16 (zero, scale) per group of 32 channels
  V codes, V params    the same for the value
A page that no request holds keeps whatever its last owner left there, here
bytes that read as NaN.
"""
import math
import random

import torch

own = False

GROUP = 32
CLAMP = 60000.0


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one token for each of 48 requests in flight: the plan of a decode step
        {"name": "plan-decode", "op": "plan", "requests": 48, "new_lo": 1, "new_hi": 1, "cached_lo": 200,
         "cached_hi": 32760, "page": 16, "rows": 64, "lens": 1},
        # a batch of prompts at once, pages of 64 tokens
        {"name": "plan-prompts", "op": "plan", "requests": 240, "new_lo": 1, "new_hi": 800, "cached_lo": 0,
         "cached_hi": 4680, "page": 64, "rows": 98280, "lens": 2},
        # the queries and keys of a small decode batch, grouped heads
        {"name": "rope-decode", "op": "rope", "dtype": "bf16", "rows": 16, "heads": 40, "kv_heads": 8, "d": 128,
         "rot": 128, "axes": 1, "interleaved": False, "fused": True},
        # one chunk of a video model: frame, row and column positions on three sections of the channels
        {"name": "rope-chunk", "op": "rope", "dtype": "bf16", "rows": 4680, "heads": 24, "kv_heads": 24, "d": 128,
         "rot": 128, "axes": 3, "interleaved": False, "fused": True},
        # float32, half the channels rotated, adjacent pairs
        {"name": "rope-f32", "op": "rope", "dtype": "f32", "rows": 32760, "heads": 12, "kv_heads": 4, "d": 64,
         "rot": 32, "axes": 1, "interleaved": True, "fused": False},
        # one token for each of 48 requests into the cache
        {"name": "append-decode", "op": "append", "dtype": "bf16", "rows": 48, "kv_heads": 8, "d": 128, "page": 16,
         "pad": 16},
        # one chunk of a video model into the cache
        {"name": "append-chunk", "op": "append", "dtype": "bf16", "rows": 4680, "kv_heads": 24, "d": 128, "page": 128,
         "pad": 0},
        # one request far into its stream, one query token
        {"name": "attend-one", "op": "attend", "dtype": "bf16", "requests": 1, "new_lo": 1, "new_hi": 1,
         "cached_lo": 98279, "cached_hi": 98279, "heads": 40, "kv_heads": 8, "d": 128, "page": 64, "causal": True,
         "window": 0, "lens": 3},
        # a decode batch of ragged requests
        {"name": "attend-batch", "op": "attend", "dtype": "bf16", "requests": 48, "new_lo": 1, "new_hi": 1,
         "cached_lo": 200, "cached_hi": 16380, "heads": 32, "kv_heads": 8, "d": 128, "page": 16, "causal": True,
         "window": 0, "lens": 4},
        # a video chunk over its stream, every cached token visible
        {"name": "attend-chunk", "op": "attend", "dtype": "bf16", "requests": 1, "new_lo": 4680, "new_hi": 4680,
         "cached_lo": 28080, "cached_hi": 28080, "heads": 24, "kv_heads": 24, "d": 128, "page": 128, "causal": False,
         "window": 0, "lens": 5},
        # prompts with cached prefixes, causal, grouped heads
        {"name": "attend-prompts", "op": "attend", "dtype": "bf16", "requests": 4, "new_lo": 900, "new_hi": 4096,
         "cached_lo": 0, "cached_hi": 4000, "heads": 32, "kv_heads": 8, "d": 128, "page": 64, "causal": True,
         "window": 0, "lens": 6},
        # float32, a sliding window, odd lengths
        {"name": "attend-f32", "op": "attend", "dtype": "f32", "requests": 3, "new_lo": 30, "new_hi": 260,
         "cached_lo": 100, "cached_hi": 4680, "heads": 8, "kv_heads": 4, "d": 64, "page": 16, "causal": True,
         "window": 1001, "lens": 7},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "append", "attend", "attend", "attend"])
    if op == "plan":
        return {"op": op, "requests": _log(rng, 1, 240), "new_lo": 0, "new_hi": _log(rng, 1, 400),
                "cached_lo": 0, "cached_hi": _log(rng, 16, 32760), "page": rng.choice([16, 32, 64, 128]),
                "rows": 98280 if rng.random() < 0.5 else 240 * 400 + rng.randrange(100), "lens": rng.randrange(1 << 30)}
    if op == "rope":
        d = rng.choice([64, 128])
        hk = rng.choice([1, 2, 4, 8])
        return {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "rows": _log(rng, 1, 9001),
                "heads": hk * rng.choice([1, 2, 3, 4, 5, 6]), "kv_heads": hk, "d": d,
                "rot": rng.choice([d, d // 2]), "axes": rng.choice([1, 3]), "interleaved": rng.random() < 0.5,
                "fused": rng.random() < 0.5}
    if op == "append":
        return {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "rows": _log(rng, 1, 9001),
                "kv_heads": rng.choice([1, 2, 4, 8]), "d": rng.choice([64, 128]), "page": rng.choice([16, 32, 64, 128]),
                "pad": rng.choice([0, 3, 40])}
    c = {"op": op, "dtype": "bf16", "d": rng.choice([64, 128, 128]), "page": rng.choice([16, 32, 64, 128]),
         "kv_heads": rng.choice([1, 2, 4, 8]), "causal": True, "window": 0, "lens": rng.randrange(1 << 30)}
    c["heads"] = c["kv_heads"] * rng.choice([1, 2, 3, 4, 5, 8])
    kind = rng.choice(["decode", "decode", "prompts", "chunk", "f32"])
    if kind == "decode":  # one token, or a few drafted ones
        c |= {"requests": _log(rng, 1, 64), "new_lo": 1, "new_hi": rng.choice([1, 1, 4]), "cached_lo": 0,
              "cached_hi": _log(rng, 100, 16000), "window": rng.choice([0, 0, 513])}
    elif kind == "prompts":
        c |= {"requests": rng.choice([1, 2, 3, 5]), "new_lo": 1, "new_hi": _log(rng, 50, 2000), "cached_lo": 0,
              "cached_hi": _log(rng, 50, 4000), "window": rng.choice([0, 0, 700])}
    elif kind == "chunk":
        n = _log(rng, 200, 4680)
        c |= {"requests": 1, "new_lo": n, "new_hi": n, "cached_lo": 0, "cached_hi": _log(rng, 1000, 28080),
              "causal": False, "heads": 8, "kv_heads": 8}
    else:
        c |= {"dtype": "f32", "requests": rng.choice([1, 2, 5]), "new_lo": 1, "new_hi": _log(rng, 1, 200),
              "cached_lo": 0, "cached_hi": _log(rng, 50, 4680), "window": rng.choice([0, 300])}
    return c


def _lengths(case):
    """(cached, new) tokens of each request, from the case alone."""
    r = random.Random(case["lens"])
    n = range(case["requests"])
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in n]
    cached = [r.randint(case["cached_lo"], case["cached_hi"]) for _ in n]
    return cached, new


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _size(case):
    return 2 if case["dtype"] == "bf16" else 4


def _block_bytes(d, page):
    return page * (d + d // 4)


def _pairs(cached, new, causal, window):
    """(visible pairs, tokens that some row sees) of one request."""
    n = cached + new
    if not causal:
        return new * n, n if new else 0
    seen = lambda m: m * (m + 1) // 2  # noqa: E731  the first m positions, each seeing all before it
    pairs = seen(n) - seen(cached)
    if window:
        late = lambda m: max(0, m - window) * (max(0, m - window) + 1) // 2  # noqa: E731
        pairs -= late(n) - late(cached)
    return pairs, (min(n, new + window - 1) if window else n) if new else 0


def work(case):
    op = case["op"]
    if op == "plan":
        cached, new = _lengths(case)
        p = case["page"]
        need = sum((c + n + p - 1) // p - (c + p - 1) // p for c, n in zip(cached, new))
        # lengths in and out, offsets, the new pages' ids in and out, the open page of each request, slots and positions
        return {"bytes": 20 * case["requests"] + 8 * need + 12 * case["rows"], "flops": 0}
    if op == "rope":
        n = case["rows"] * (case["heads"] + case["kv_heads"]) * case["d"]
        return {"bytes": 2 * n * _size(case) + case["rows"] * (case["rot"] * 4 + 4 * case["axes"]), "flops": 8 * n}
    if op == "append":
        n = 2 * case["rows"] * case["kv_heads"] * case["d"]
        # in, the packed bytes out, and the values they stand for out
        return {"bytes": 2 * n * _size(case) + n * 5 // 8 + 8 * (case["rows"] + case["pad"]), "flops": 8 * n}
    cached, new = _lengths(case)
    both = [_pairs(c, n, case["causal"], case["window"]) for c, n in zip(cached, new)]
    d, rows = case["d"], sum(new)
    return {"bytes": sum(t for _, t in both) * case["kv_heads"] * (d + d // 4) + 2 * rows * case["heads"] * d * _size(case),
            "flops": 4 * d * case["heads"] * sum(p for p, _ in both)}


# ---------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _int(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _pages(g, cached, new, page, spare):
    """A block table over a shuffled pool: each request's pages, -1 behind them, and the pool's other pages."""
    held = [(c + page - 1) // page for c in cached]
    total = [(c + n + page - 1) // page for c, n in zip(cached, new)]
    n_pages = sum(total) + spare
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    width = max(1, max(total))
    first = torch.cumsum(_int([0] + held[:-1]), 0)
    j = torch.arange(width, device="cuda")[None, :]
    own_ = j < _int(held)[:, None]
    at = torch.where(own_, first[:, None] + j, 0)
    return n_pages, torch.where(own_, order[at], -1).to(torch.int32), order[sum(held):].contiguous()


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    if op == "plan":
        cached, new = _lengths(case)
        n_pages, table, free = _pages(g, cached, new, case["page"], 37)
        free_pages = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
        free_pages[: free.numel()] = free
        return {"op": op, "kv_len": _int(cached), "new_len": _int(new), "table": table, "free_pages": free_pages,
                "free_count": _int([free.numel()]), "page": case["page"], "rows": case["rows"]}
    if op == "rope":
        T, hq, hk, d, rot, axes = (case[x] for x in ("rows", "heads", "kv_heads", "d", "rot", "axes"))
        dt = _dtype(case)
        if case["fused"]:  # views of one projection's output, values behind them
            x = (_normal(g, T, hq + 2 * hk, d) * 1.7).to(dt)
            q, k = x[:, :hq], x[:, hq:hq + hk]
        else:
            q, k = (_normal(g, T, hq, d) * 1.7).to(dt), (_normal(g, T, hk, d) * 1.7).to(dt)
        n_pos = 40000
        inv = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        angle = torch.arange(n_pos, device="cuda", dtype=torch.float64)[:, None] * inv[None, :]
        cos_sin = torch.cat([torch.cos(angle), torch.sin(angle)], 1).float()
        pos = torch.randint(0, n_pos, (T, axes), generator=g, device="cuda", dtype=torch.int32)
        half = rot // 2
        sections = [half] if axes == 1 else [half - 2 * (half * 3 // 8), half * 3 // 8, half * 3 // 8]
        return {"op": op, "q": q, "k": k, "wq": (1 + 0.2 * _normal(g, d)).to(dt), "wk": (1 + 0.2 * _normal(g, d)).to(dt),
                "cos_sin": cos_sin, "positions": pos, "interleaved": case["interleaved"], "sections": sections,
                "axis": _int(sum(([a] * n for a, n in enumerate(sections)), []), torch.int64), "eps": 1e-6}
    d, hk, page = case["d"], case["kv_heads"], case["page"]
    dt = _dtype(case)
    if op == "append":
        T = case["rows"] + case["pad"]
        n_pages = (T + page - 1) // page + 5
        slots = torch.randperm(n_pages * page, generator=g, device="cuda")[:T]
        slots[case["rows"]:] = -1
        sigma = torch.exp(_normal(g, hk, d))
        return {"op": op, "k": (_normal(g, T, hk, d) * sigma).to(dt), "v": _normal(g, T, hk, d).to(dt),
                "slots": slots, "pool": torch.full((n_pages, hk, _block_bytes(d, page)), 255, dtype=torch.uint8, device="cuda")}
    cached, new = _lengths(case)
    after = [c + n for c, n in zip(cached, new)]
    n_pages, table, _ = _pages(g, after, [0] * len(after), page, 3)
    n, groups = n_pages, d // GROUP
    codes = torch.randint(0, 256, (2, n, hk, page * d // 2), generator=g, device="cuda", dtype=torch.uint8)
    scale = 0.15 + 0.2 * torch.rand((2, n, hk, page, groups), generator=g, device="cuda")
    zero = scale * (-7.5 + 1.5 * torch.randn((2, n, hk, page, groups), generator=g, device="cuda"))
    params = torch.stack([zero, scale], -1).half().view(torch.uint8).reshape(2, n, hk, page * groups * 4)
    pool = torch.cat([codes[0], params[0], codes[1], params[1]], -1).contiguous()
    pool[:, :, :][_unheld(table, n)] = 255
    rows = sum(new)
    return {"op": op, "q": _normal(g, rows, case["heads"], d).to(dt), "pool": pool, "table": table,
            "kv_len": _int(after), "cu_rows": torch.cumsum(_int([0] + new), 0).to(torch.int32), "max_new": max(new),
            "causal": case["causal"], "window": case["window"], "page": page}


def _unheld(table, n_pages):
    held = torch.zeros(n_pages + 1, dtype=torch.bool, device="cuda")
    held[table.reshape(-1).long()] = True  # -1 marks the extra last entry
    return ~held[:n_pages]


# ---------------------------------------------------------------- the plain forms
def _plan(s):
    """Pages from the top of the free stack in the requests' order, a slot and a position for every new row."""
    p, rows = s["page"], s["rows"]
    old, new, table = s["kv_len"].long(), s["new_len"].long(), s["table"]
    after = old + new
    held, total = (old + p - 1) // p, (after + p - 1) // p
    need = total - held
    first = torch.cumsum(need, 0) - need
    cu = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)])
    count = s["free_count"].long()
    ok = (need.sum() <= count) & (total.max() <= table.shape[1]) & (cu[-1] <= rows) & (new.min() >= 0) & (old.min() >= 0)
    j = torch.arange(table.shape[1], device=table.device)[None, :]
    fresh = (j >= held[:, None]) & (j < total[:, None]) & ok
    at = (count - 1 - first[:, None] - (j - held[:, None])).clamp(0, s["free_pages"].numel() - 1)
    table.copy_(torch.where(fresh, s["free_pages"][at], table))
    t = torch.arange(rows, device=table.device)
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=new.numel() - 1)
    real = (t < cu[-1]) & ok
    pos = torch.where(real, old[b] + t - cu[b], 0)
    slot = table[b, pos // p].long() * p + pos % p
    return {"kv_len": torch.where(ok, after, old).int(), "free_count": (count - torch.where(ok, need.sum(), 0)).int(),
            "cu_rows": torch.where(ok, cu, 0).int(), "slots": torch.where(real, slot, -1),
            "positions": torch.where(real, pos, -1).int(), "table": table}


def _rotate(s, x, w):
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
    rot = s["cos_sin"].shape[1]
    half = rot // 2
    pair = torch.arange(half, device=x.device)
    at = s["positions"].long()[:, s["axis"]]
    cos, sin = s["cos_sin"][at, pair][:, None], s["cos_sin"][at, half + pair][:, None]
    one, two = (x[..., 0:rot:2], x[..., 1:rot:2]) if s["interleaved"] else (x[..., :half], x[..., half:rot])
    a, b = one * cos - two * sin, two * cos + one * sin
    turned = torch.stack([a, b], -1).flatten(-2) if s["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _quantise(x):
    """(codes, zero, scale) of the last dimension's groups of 32, in float32."""
    x = torch.where(torch.isnan(x), 0.0, x.float()).clamp(-CLAMP, CLAMP).unflatten(-1, (-1, GROUP))
    low, high = x.amin(-1), x.amax(-1)
    zero, scale = low.half(), ((high - low) / torch.full_like(high, 15.0)).half()
    z, r = zero.float()[..., None], scale.float()[..., None]
    codes = torch.where(r > 0, torch.round((x - z) / r), 0.0).clamp(0, 15)
    return codes.flatten(-2), zero, scale


def _append(s):
    """The packed bytes of every row that has a slot, at that slot; returns the values they stand for and the pool."""
    pool, real = s["pool"], s["slots"] >= 0
    hk, block = pool.shape[1:]
    d = s["k"].shape[-1]
    page = block * 4 // (5 * d)
    at = s["slots"][real][:, None, None]
    head = torch.arange(hk, device=pool.device)[None, :, None]
    byte = torch.arange(d // 2, device=pool.device)

    def put(x, base):
        codes, zero, scale = _quantise(x)
        c = codes[real].to(torch.uint8)
        pool[at // page, head, base + at % page * (d // 2) + byte] = c[..., 0::2] | (c[..., 1::2] << 4)
        params = torch.stack([zero, scale], -1).view(torch.uint8).flatten(-2)
        pool[at // page, head, base + page * d // 2 + at % page * (d // 8) + byte[:d // 8]] = params[real]
        value = codes.unflatten(-1, (-1, GROUP)) * scale.float()[..., None] + zero.float()[..., None]
        return torch.where(real[:, None, None], value.flatten(-2), 0.0).to(x.dtype)

    return [put(s["k"], 0), put(s["v"], block // 2), pool]


def _dequantise(blocks, base, d, page):
    """Values [..., page, d] of one half (keys or values) of the blocks [..., bytes], float32."""
    codes = blocks[..., base:base + page * d // 2].unflatten(-1, (page, d // 2))
    params = blocks[..., base + page * d // 2:base + page * d * 5 // 8].contiguous().view(torch.float16)
    params = params.unflatten(-1, (page, d // GROUP, 2)).float()
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    return (c * params[..., 1:] + params[..., :1]).flatten(-2)


def _attend(s):
    q, pool, table = s["q"], s["pool"], s["table"]
    T, hq, d = q.shape
    hk, block, page = pool.shape[1], pool.shape[2], s["page"]
    B, m = table.shape[0], s["max_new"]
    blocks = pool[table.long().clamp(min=0)].transpose(1, 2)               # [B, hk, pages, block]
    k, v = (_dequantise(blocks, h * block // 2, d, page).flatten(2, 3) for h in (0, 1))
    n = torch.arange(k.shape[2], device=q.device)
    live = (n < s["kv_len"][:, None])[:, None, :, None]
    k, v = torch.where(live, k, 0.0), torch.where(live, v, 0.0)
    cu = s["cu_rows"].long()
    rows = cu[1:] - cu[:-1]
    i = torch.arange(m, device=q.device)
    at = torch.where(i < rows[:, None], cu[:-1, None] + i, 0)               # [B, m]
    x = q.float()[at].unflatten(2, (hk, hq // hk)).permute(0, 2, 3, 1, 4)   # [B, hk, group, m, d]
    score = torch.matmul(x.flatten(2, 3), k.transpose(-1, -2)).unflatten(2, (hq // hk, m)) / math.sqrt(d)
    where = (s["kv_len"] - rows)[:, None] + i                               # [B, m] position of each row
    sees = n < s["kv_len"][:, None, None]
    if s["causal"]:
        sees = sees & (n <= where[..., None])
    if s["window"]:
        sees = sees & (n > where[..., None] - s["window"])
    score = torch.where(sees[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isfinite(top), top, 0.0))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (hq // hk, m)) / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)                              # [B, m, hq, d]
    t = torch.arange(T, device=q.device)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return o[b, t - cu[b]].to(q.dtype)


def run(s):
    op = s["op"]
    if own:
        from bit_kv_cache_qwm_gb300 import paged
        if op == "plan":
            r = paged.qwm_paged_plan(s["kv_len"], s["new_len"], s["table"], s["free_pages"], s["free_count"], s["page"], s["rows"])
            return {"kv_len": r.kv_len, "free_count": r.free_count, "cu_rows": r.cu_rows, "slots": r.slots,
                    "positions": r.positions, "table": s["table"]}
        if op == "rope":
            return list(paged.qwm_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cos_sin"], s["positions"], eps=s["eps"],
                                               interleaved=s["interleaved"], sections=s["sections"]))
        if op == "append":
            k_hat, v_hat = torch.empty_like(s["k"]), torch.empty_like(s["v"])
            paged.qwm_paged_append(s["k"], s["v"], s["pool"], s["slots"], k_hat=k_hat, v_hat=v_hat)
            return [k_hat, v_hat, s["pool"]]
        return paged.qwm_paged_attend(s["q"], s["pool"], s["table"], s["kv_len"], s["cu_rows"], max_new=s["max_new"],
                                      causal=s["causal"], window=s["window"])
    if op == "plan":
        return _plan(s)
    if op == "rope":
        return [_rotate(s, s["q"], s["wq"]).to(s["q"].dtype), _rotate(s, s["k"], s["wk"]).to(s["k"].dtype)]
    return _append(s) if op == "append" else _attend(s)


# ---------------------------------------------------------------- in 64 bits, from the definitions
def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None
    s = prepare(case, seed)
    if op == "rope":
        out = []
        for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
            x, w = x.double(), w.double()
            y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * w
            z = y.clone()
            rot = case["rot"]
            for j in range(rot // 2):
                a, b = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + rot // 2)
                row = s["cos_sin"][s["positions"][:, int(s["axis"][j])].long()].double()
                c, n = row[:, j, None], row[:, rot // 2 + j, None]
                z[..., a] = y[..., a] * c - y[..., b] * n
                z[..., b] = y[..., a] * n + y[..., b] * c
            out.append(z)
        return out
    if op == "append":
        out = []
        for x in (s["k"], s["v"]):
            y = x.double()
            z = torch.empty_like(y)
            for g in range(y.shape[-1] // GROUP):
                part = y[..., g * GROUP:(g + 1) * GROUP]
                low, high = part.min(-1, keepdim=True).values, part.max(-1, keepdim=True).values
                zero, scale = low.half().double(), ((high - low) / 15).half().double()
                code = ((part - zero) / torch.where(scale == 0, 1.0, scale)).round().clamp(0, 15)
                z[..., g * GROUP:(g + 1) * GROUP] = zero + torch.where(scale == 0, 0.0, code) * scale
            z[s["slots"] < 0] = 0
            out.append(z)
        return out + [None]  # the pool's bytes have no value in 64 bits
    q, d, page = s["q"].double(), case["d"], case["page"]
    out = torch.zeros_like(q)
    cu, lens, group = s["cu_rows"].tolist(), s["kv_len"].tolist(), case["heads"] // case["kv_heads"]
    section = page * d // 2, page * d // 8
    for b, n in enumerate(lens):
        held = s["pool"][s["table"][b, :(n + page - 1) // page].long()]
        here = torch.arange(n, device=q.device)
        at = n - (cu[b + 1] - cu[b]) + torch.arange(cu[b + 1] - cu[b], device=q.device)[:, None]
        hidden = torch.zeros((at.shape[0], n), dtype=torch.bool, device=q.device)
        if case["causal"]:
            hidden |= here > at
        if case["window"]:
            hidden |= here <= at - case["window"]
        if n == 0 or at.shape[0] == 0:
            continue
        for h in range(case["kv_heads"]):
            kv = []
            for base in (0, sum(section)):
                codes = held[:, h, base:base + section[0]].reshape(-1, d // 2)[:n]
                par = held[:, h, base + section[0]:base + sum(section)].contiguous().view(torch.float16).reshape(-1, d // GROUP, 2)[:n].double()
                full = torch.empty((n, d), dtype=torch.float64, device=q.device)
                full[:, 0::2], full[:, 1::2] = (codes % 16).double(), (codes // 16).double()
                kv.append(full * par[..., 1].repeat_interleave(GROUP, 1) + par[..., 0].repeat_interleave(GROUP, 1))
            for j in range(h * group, (h + 1) * group):
                logits = (q[cu[b]:cu[b + 1], j] @ kv[0].T / math.sqrt(d)).masked_fill(hidden, -math.inf)
                out[cu[b]:cu[b + 1], j] = torch.nan_to_num(torch.softmax(logits, -1), nan=0.0) @ kv[1]
    return out
