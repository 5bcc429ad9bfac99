"""The paged 8-bit cache and attention over selected pages, as cases that can be timed and checked.

Four operators, in the order in which a serving step uses them:

  append  new keys and values into the pages of their requests, in 8 bits with a scale for each
          block of 16 tokens and head
  read    the tokens of requests back out of the pages
  attend  attention of a ragged batch of query rows over the pages
  sparse  the bounds of the pages that the step wrote, the pages that a cheap score selects for each
          request and key/value head, and the attention over these alone

`run` computes them in plain torch where `own` is false and through
bit_kv_cache_qwm_gb300.paged where it is true.

Cache bytes: pool [pages][kv heads][block]; a block of p token slots holds
  K codes [p][d], V codes [p][d]  e4m3
  scales [p / 16][2]              float16, a power of two each: K's and V's of 16 slots
  and zeros or anything up to a multiple of 16 bytes.
Scales are powers of two from 2^-15 to 2^7, the least that brings the block's largest magnitude to
448, so that one that grows with a later token leaves the codes before it what they were, but for
those that fall below the normal numbers.  Slots that hold no token, and pages that no request
holds, keep whatever was there, here bytes that read as NaN.

Bounds: [pages][kv heads][2 d + 16] bytes: the largest, then the smallest value of each channel over
the page's tokens as int8, and their scale as float32.  The score of a page for a query row is the
largest product that a key within the bounds could have with it, with the row in int8 as well; all
of it is exact in whole numbers but for two products in float32.
"""
import math
import random

import torch

own = False

BLOCK = 16                     # tokens that share a scale
LOW, HIGH = -15, 7             # exponents of the scales
CLAMP = 448.0 * 2.0 ** HIGH


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one token for each of 48 requests into the cache
        {"name": "append-decode", "op": "append", "dtype": "bf16", "requests": 48, "new_lo": 1, "new_hi": 1,
         "cached_lo": 200, "cached_hi": 900, "kv_heads": 8, "d": 128, "page": 16, "lens": 1},
        # one chunk of a video model into its stream, which ends inside a block
        {"name": "append-chunk", "op": "append", "dtype": "bf16", "requests": 1, "new_lo": 4680, "new_hi": 4680,
         "cached_lo": 4677, "cached_hi": 4677, "kv_heads": 24, "d": 128, "page": 128, "lens": 2},
        # what a few short requests hold, in float32, for a look at what the encoding costs
        {"name": "read-f32", "op": "read", "dtype": "f32", "requests": 5, "new_lo": 20, "new_hi": 300,
         "cached_lo": 0, "cached_hi": 100, "kv_heads": 4, "d": 64, "page": 32, "lens": 3},
        # a long request handed on to another cache
        {"name": "read-long", "op": "read", "dtype": "bf16", "requests": 1, "new_lo": 98280, "new_hi": 98280,
         "cached_lo": 0, "cached_hi": 0, "kv_heads": 8, "d": 128, "page": 64, "lens": 4},
        # one request far into its stream, one query token
        {"name": "attend-one", "op": "attend", "dtype": "bf16", "requests": 1, "new_lo": 1, "new_hi": 1,
         "cached_lo": 98279, "cached_hi": 98279, "heads": 40, "kv_heads": 8, "d": 128, "page": 64, "causal": True,
         "window": 0, "lens": 5},
        # a decode batch of ragged requests
        {"name": "attend-batch", "op": "attend", "dtype": "bf16", "requests": 48, "new_lo": 1, "new_hi": 1,
         "cached_lo": 200, "cached_hi": 16380, "heads": 32, "kv_heads": 8, "d": 128, "page": 16, "causal": True,
         "window": 0, "lens": 6},
        # a video chunk over its stream, every cached token visible
        {"name": "attend-chunk", "op": "attend", "dtype": "bf16", "requests": 1, "new_lo": 4680, "new_hi": 4680,
         "cached_lo": 28080, "cached_hi": 28080, "heads": 24, "kv_heads": 24, "d": 128, "page": 128, "causal": False,
         "window": 0, "lens": 7},
        # prompts with cached prefixes, causal, grouped heads
        {"name": "attend-prompts", "op": "attend", "dtype": "bf16", "requests": 4, "new_lo": 900, "new_hi": 4096,
         "cached_lo": 0, "cached_hi": 4000, "heads": 32, "kv_heads": 8, "d": 128, "page": 64, "causal": True,
         "window": 0, "lens": 8},
        # float32, a sliding window, odd lengths
        {"name": "attend-f32", "op": "attend", "dtype": "f32", "requests": 3, "new_lo": 30, "new_hi": 260,
         "cached_lo": 100, "cached_hi": 4680, "heads": 8, "kv_heads": 4, "d": 64, "page": 16, "causal": True,
         "window": 1001, "lens": 9},
        # one token of a request at the end of a long stream: 16,384 of its 374,400 tokens
        {"name": "sparse-one", "op": "sparse", "dtype": "bf16", "requests": 1, "new_lo": 1, "new_hi": 1,
         "cached_lo": 374399, "cached_hi": 374399, "heads": 40, "kv_heads": 8, "d": 128, "page": 64, "causal": True,
         "width": 256, "sink": 1, "lens": 10},
        # a decode batch, 2,048 tokens of each request
        {"name": "sparse-batch", "op": "sparse", "dtype": "bf16", "requests": 48, "new_lo": 1, "new_hi": 1,
         "cached_lo": 200, "cached_hi": 32760, "heads": 32, "kv_heads": 8, "d": 128, "page": 32, "causal": True,
         "width": 64, "sink": 1, "lens": 11},
        # a video chunk over the pages of a long stream that suit it best, and its own
        {"name": "sparse-chunk", "op": "sparse", "dtype": "bf16", "requests": 1, "new_lo": 4680, "new_hi": 4680,
         "cached_lo": 98280, "cached_hi": 98280, "heads": 24, "kv_heads": 24, "d": 128, "page": 128, "causal": False,
         "width": 166, "sink": 0, "lens": 12},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "read", "attend", "attend", "attend", "sparse", "sparse"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "kv_heads": rng.choice([1, 2, 4, 8]),
         "d": rng.choice([64, 128, 128]), "page": rng.choice([16, 32, 64, 128, 256]), "lens": rng.randrange(1 << 30)}
    if op in ("append", "read"):
        n = rng.choice([1, 1, 3, 17, 60])
        return c | {"requests": n, "new_lo": 0 if n > 1 else 1, "new_hi": _log(rng, 1, 9001 // n), "cached_lo": 0,
                    "cached_hi": _log(rng, 1, 2000)}
    c |= {"dtype": "bf16", "causal": True, "heads": c["kv_heads"] * rng.choice([1, 2, 3, 4, 5, 8])}
    if op == "sparse":
        kind = rng.choice(["decode", "decode", "drafts", "chunk", "f32"])
        if kind == "chunk":
            n = _log(rng, 100, 4680)
            c |= {"requests": 1, "new_lo": n, "new_hi": n, "cached_lo": 4000, "cached_hi": _log(rng, 4000, 60000),
                  "causal": rng.random() < 0.5, "heads": 8, "kv_heads": 8}
        else:
            n = {"decode": 1, "drafts": 5, "f32": 3}[kind]
            c |= {"requests": _log(rng, 1, 64), "new_lo": 1, "new_hi": n, "cached_lo": 0,
                  "cached_hi": _log(rng, 1000, 20000), "dtype": "f32" if kind == "f32" else "bf16"}
        tail = (c["new_hi"] + c["page"] - 2) // c["page"] + 1
        return c | {"width": tail + _log(rng, 1, 1 + 4000 // c["page"]), "sink": rng.choice([0, 1, 2])}
    c["window"] = 0
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
    if sum(new) == 0:
        new[0] = 1
    return cached, new


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _size(case):
    return 2 if case["dtype"] == "bf16" else 4


def _block_bytes(d, page):
    return 2 * page * d + (page // BLOCK * 4 + 15) // 16 * 16


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
    op, hk, d, page = case["op"], case["kv_heads"], case["d"], case["page"]
    cached, new = _lengths(case)
    rows = sum(new)
    if op in ("append", "read"):
        n = 2 * rows * hk * d
        # append: in, the packed bytes out, and the values they stand for out; read: bytes in, values out
        return {"bytes": (2 if op == "append" else 1) * n * _size(case) + n + n // (8 * d), "flops": 4 * n if op == "append" else n}
    token = hk * (2 * d + 4 / BLOCK)
    q_out = 2 * rows * case["heads"] * d * _size(case)
    if op == "attend":
        both = [_pairs(c, n, case["causal"], case["window"]) for c, n in zip(cached, new)]
        return {"bytes": int(sum(t for _, t in both) * token) + q_out, "flops": 4 * d * case["heads"] * sum(p for p, _ in both)}
    pages = [(c + n + page - 1) // page for c, n in zip(cached, new)]
    kept = [c - (p - min(p, case["width"])) * page for c, p in zip(cached, pages)]
    both = [_pairs(c, n, case["causal"], 0) for c, n in zip(kept, new)]
    touched = sum((c + n + page - 1) // page - c // page for c, n in zip(cached, new))
    # bounds of all pages in, those of the pages written out and these pages' keys in; the scores' products
    # (a bound for either sign of a channel), the selected pages; outputs
    return {"bytes": int(sum(t for _, t in both) * token) + q_out + hk * (2 * d + 16) * (sum(pages) + touched) +
            hk * touched * page * d + 4 * hk * sum(min(p, case["width"]) for p in pages),
            "flops": case["heads"] * d * (4 * sum(p for p, _ in both) + 4 * sum(n * p for n, p in zip(new, pages)))}


# ---------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _int(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _table(g, lens, page, spare):
    """A block table over a shuffled pool: each request's pages, -1 behind them."""
    held = [(n + page - 1) // page for n in lens]
    n_pages = sum(held) + spare
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    first = torch.cumsum(_int([0] + held[:-1]), 0)
    j = torch.arange(max(1, max(held)), device="cuda")[None, :]
    mine = j < _int(held)[:, None]
    return n_pages, torch.where(mine, order[torch.where(mine, first[:, None] + j, 0)], -1).to(torch.int32)


def _fill(g, pool, table, lens, d, page, topics):
    """Keys and values of `lens` tokens of each request into the pool, a few requests' pages at a time; the
    slots behind them stay as they are.  topics > 0: the keys of a page have that much in common."""
    hk = pool.shape[1]
    sigma = torch.exp(0.5 * _normal(g, hk, d))
    for b, n in enumerate(lens):
        for j0 in range(0, (n + page - 1) // page, 1 + 65536 // page):
            j1 = min((n + page - 1) // page, j0 + 1 + 65536 // page)
            ids = table[b, j0:j1].long()
            k = _normal(g, j1 - j0, hk, page, d) * (1 - topics) + _normal(g, j1 - j0, hk, 1, d) * topics
            live = (torch.arange(j0 * page, j1 * page, device="cuda") < n).view(j1 - j0, 1, page, 1)
            for half, x in ((0, k * sigma[:, None]), (1, _normal(g, j1 - j0, hk, page, d))):
                code, scale = _encode(torch.where(live, x.bfloat16().float(), 0.0).unflatten(2, (-1, BLOCK)))
                code = torch.where(live, code.flatten(2, 3), 255).flatten(2)
                pool[ids, :, half * page * d:(half + 1) * page * d] = code
                at = _scales(pool, d, page)
                at[ids, :, :, half] = torch.where(live.view(j1 - j0, 1, -1, BLOCK)[..., 0], scale.half(), at[ids, :, :, half])


def prepare(case, seed):
    g = _generator(seed)
    op, hk, d, page = case["op"], case["kv_heads"], case["d"], case["page"]
    dt = _dtype(case)
    cached, new = _lengths(case)
    after = [c + n for c, n in zip(cached, new)]
    rows = sum(new)
    n_pages, table = _table(g, after, page, 3)
    pool = torch.full((n_pages, hk, _block_bytes(d, page)), 255, dtype=torch.uint8, device="cuda")
    _fill(g, pool, table, cached if op == "append" else after, d, page, 0.5 if op == "sparse" else 0.0)
    s = {"op": op, "d": d, "page": page, "pool": pool, "table": table, "kv_len": _int(after), "max_new": max(new),
         "cu_rows": torch.cumsum(_int([0] + new), 0).to(torch.int32), "rows": rows, "dtype": dt}
    if op == "append":  # a token in a hundred is larger than those before it
        grow = torch.where(torch.rand((rows, hk, 1), generator=g, device="cuda") < 0.01, 20.0, 1.0)
        s |= {"k": (_normal(g, rows, hk, d) * torch.exp(_normal(g, hk, d)) * grow).to(dt), "v": (_normal(g, rows, hk, d) * grow).to(dt)}
    elif op == "attend":
        s |= {"q": _normal(g, rows, case["heads"], d).to(dt), "causal": case["causal"], "window": case["window"]}
    elif op == "sparse":
        bounds = torch.full((n_pages, hk, 2 * d + 16), 255, dtype=torch.uint8, device="cuda")
        for b, (c, n) in enumerate(zip(cached, after)):
            for j0 in range(0, c // page, 1 + 65536 // page):  # the full pages that earlier steps left
                ids = table[b, j0:min(c // page, j0 + 1 + 65536 // page)].long()
                _put_bounds(bounds, ids, _bounds_of(pool, ids, torch.full_like(ids, page), d, page))
        s |= {"q": _normal(g, rows, case["heads"], d).to(dt), "bounds": bounds, "width": case["width"], "sink": case["sink"],
              "causal": case["causal"], "window": 0}
    return s


# ---------------------------------------------------------------- the plain forms
def _power(e):
    """2^e for whole e from -126 to 127, float32."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _scale_for(amax):
    """The least power of two whose 448-fold is no less than amax, within the range of the scales."""
    m, x = torch.frexp(amax)
    return _power(torch.where(amax > 0, x.int() - 9 + (m > 0.875).int(), LOW).clamp(LOW, HIGH))


def _clean(x):
    return torch.where(torch.isnan(x), 0.0, x.float()).clamp(-CLAMP, CLAMP)


def _to_codes(x):
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _value(code):
    return code.contiguous().view(torch.float8_e4m3fn).float()


def _encode(x):
    """Codes and scales of blocks [..., 16, d] that hold nothing else."""
    scale = _scale_for(x.abs().amax((-1, -2)))
    return _to_codes(x / scale[..., None, None]), scale


def _codes(pool, half, d, page):
    return pool[..., half * page * d:(half + 1) * page * d].unflatten(-1, (page, d))


def _scales(pool, d, page):
    """[pages, heads, page / 16, 2], a view of the pool."""
    return pool[..., 2 * page * d:2 * page * d + page // BLOCK * 4].view(torch.float16).unflatten(-1, (page // BLOCK, 2))


def _blocks(s):
    """The blocks of 16 slots that the step writes, [requests, most]: whether there is one, its number in its
    request, the page's id and the block's place in the page; [.., 16]: the rows of its slots, whether a slot
    gets one, and whether one holds a token from before."""
    cu, page = s["cu_rows"].long(), s["page"]
    rows = (cu[1:] - cu[:-1])[:, None]
    end = s["kv_len"].long()[:, None]
    start = end - rows
    j = start // BLOCK + torch.arange((s["max_new"] + BLOCK - 2) // BLOCK + 1, device=cu.device)
    there = (j * BLOCK < end) & (rows > 0)
    at = torch.where(there, j * BLOCK // page, 0)
    pg = torch.gather(s["table"].long(), 1, at)
    n = j[..., None] * BLOCK + torch.arange(BLOCK, device=cu.device)
    fresh = (n >= start[..., None]) & (n < end[..., None])
    row = torch.where(fresh, cu[:-1, None, None] + n - start[..., None], 0)
    return there, pg, j * BLOCK % page // BLOCK, row, fresh, n < start[..., None]


def _append(s):
    there, *rest = _blocks(s)
    pg, sub, row, fresh, before = (x[there] for x in rest)
    d, page, pool = s["d"], s["page"], s["pool"]
    fresh, before = fresh[:, None, :, None], before[:, None, :, None]                 # [blocks, 1, 16, 1]
    out = []
    for half, x in ((0, s["k"]), (1, s["v"])):
        new = torch.where(fresh, _clean(x)[row].transpose(1, 2), 0.0)                  # [blocks, heads, 16, d]
        scale = _scale_for(new.abs().amax((-1, -2)))
        codes = _codes(pool, half, d, page).unflatten(2, (-1, BLOCK))
        old, had = codes[pg, :, sub], _scales(pool, d, page)[pg, :, sub, half].float()
        scale = torch.where(before.any(2)[..., 0], torch.maximum(had, scale), scale)
        moved = _to_codes(_value(old) * (had / scale)[..., None, None])
        code = _to_codes(new / scale[..., None, None])
        code = torch.where(fresh, code, torch.where(before, moved, old))
        _scales(pool, d, page)[pg, :, sub, half] = scale.half()
        codes[pg, :, sub] = code
        hat = torch.empty_like(x)
        hat[row[fresh[:, 0, :, 0]]] = (_value(code) * scale[..., None, None]).transpose(1, 2)[fresh[:, 0, :, 0]].to(x.dtype)
        out.append(hat)
    return out + [pool]


def _places(s):
    """Page and slot of every row."""
    t = torch.arange(s["rows"], device=s["table"].device)
    cu = s["cu_rows"].long()
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    n = s["kv_len"].long()[b] - cu[b + 1] + t
    return s["table"][b, n // s["page"]].long(), n % s["page"]


def _read(s):
    pg, at = _places(s)
    d, page, pool = s["d"], s["page"], s["pool"]
    scale = _scales(pool, d, page)[pg, :, at // BLOCK].float()
    return [(_value(_codes(pool, h, d, page)[pg, :, at]) * scale[..., h, None]).to(s["dtype"]) for h in (0, 1)]


def _values(blocks, half, d, page):
    """Values [..., page, d] of one half of the blocks [..., bytes], float32."""
    scale = _scales(blocks, d, page)[..., half].float()
    return (_value(_codes(blocks, half, d, page)).unflatten(-2, (-1, BLOCK)) * scale[..., None, None]).flatten(-3, -2)


def _bounds_of(pool, ids, count, d, page):
    """(largest, smallest int8 [n, heads, d], scale [n, heads]) of the first `count` keys of pages."""
    k = _values(pool[ids], 0, d, page)
    live = (torch.arange(page, device=k.device) < count[:, None])[:, None, :, None]
    high = torch.where(live, k, -math.inf).amax(2)
    low = torch.where(live, k, math.inf).amin(2)
    scale = torch.maximum(high.abs(), low.abs()).amax(-1) / torch.full_like(high[..., 0], 127.0)
    by = torch.where(scale > 0, scale, 1.0)[..., None]
    return torch.round(high / by).to(torch.int8), torch.round(low / by).to(torch.int8), scale


def _put_bounds(bounds, ids, b):
    high, low, scale = b
    d = high.shape[-1]
    bounds[ids, :, :d], bounds[ids, :, d:2 * d] = high.view(torch.uint8), low.view(torch.uint8)
    bounds[ids, :, 2 * d:] = torch.cat([scale[..., None], torch.zeros_like(scale)[..., None].expand(-1, -1, 3)], -1).view(torch.uint8)


def _bounds(s):
    """The bounds of the pages that hold rows of the step."""
    page = s["page"]
    rows = (s["cu_rows"][1:] - s["cu_rows"][:-1]).long()[:, None]
    end = s["kv_len"].long()[:, None]
    j = (end - rows) // page + torch.arange((s["max_new"] + page - 2) // page + 1, device=end.device)
    there = (j * page < end) & (rows > 0)
    ids = torch.gather(s["table"].long(), 1, torch.where(there, j, 0))[there]
    count = (end - j * page).clamp(max=page)[there]
    for i in range(0, ids.numel(), 1024):
        _put_bounds(s["bounds"], ids[i:i + 1024], _bounds_of(s["pool"], ids[i:i + 1024], count[i:i + 1024], s["d"], page))


def _select(s):
    """The step's pages, the first `sink`, and those with the highest scores, `width` in all, in their order."""
    q, table, page, width, bounds, d = s["q"], s["table"].long(), s["page"], s["width"], s["bounds"], s["d"]
    hk, group = bounds.shape[1], q.shape[1] // bounds.shape[1]
    x = torch.where(torch.isnan(q), 0.0, q.float()).clamp(-3.4028234663852886e38, 3.4028234663852886e38)
    top = x.abs().amax(-1, keepdim=True)
    unit = torch.where(top >= 2.0 ** -100, top / torch.full_like(top, 127.0), 0.0)
    whole = torch.where(unit > 0, torch.round(x / torch.where(unit > 0, unit, 1.0)), 0.0).clamp(-127, 127)
    cu = s["cu_rows"].long()
    rows, end = cu[1:] - cu[:-1], s["kv_len"].long()
    i = torch.arange(s["max_new"], device=q.device)
    real = i < rows[:, None]                                                            # [B, m]
    at = torch.where(real, cu[:-1, None] + i, 0)
    whole = whole[at].unflatten(2, (hk, group)).transpose(1, 2).flatten(2, 3)           # [B, hk, m group, d]
    unit = unit[at][..., 0].unflatten(2, (hk, group)).transpose(1, 2).flatten(2, 3)
    real = real[:, None, :, None].expand(-1, hk, -1, group).flatten(2, 3)
    known = bounds[table.clamp(min=0)].transpose(1, 2)                                   # [B, hk, pages, bytes]
    high = known[..., :d].contiguous().view(torch.int8).float()
    low = known[..., d:2 * d].contiguous().view(torch.int8).float()
    scale = known[..., 2 * d:2 * d + 4].contiguous().view(torch.float32)[..., 0]
    # whole numbers below 2^24: exact in float32 in any order
    dots = torch.matmul(whole.clamp(min=0), high.transpose(-1, -2)) + torch.matmul(whole.clamp(max=0), low.transpose(-1, -2))
    score = dots * scale[:, :, None, :] * unit[..., None]
    score = torch.where(real[..., None], score, -math.inf).amax(2)                       # [B, hk, pages]
    j = torch.arange(table.shape[1], device=q.device)
    count = (end + page - 1) // page
    kind = (j < s["sink"]).int() + 2 * (j >= ((end - rows) // page)[:, None]).int()
    kind = torch.where(j < count[:, None], kind.clamp(max=2), -1)[:, None].expand(-1, hk, -1)
    score = torch.where(kind == 1, math.inf, score)                                      # the first ones in their order
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices              # then the kind goes first
    order = torch.gather(order, 2, torch.sort(torch.gather(kind, 2, order), dim=-1, descending=True, stable=True).indices)
    kept = torch.minimum(count, torch.full_like(count, width))
    if order.shape[2] < width:
        order = torch.cat([order, order.new_zeros(*order.shape[:2], width - order.shape[2])], 2)
    w = torch.arange(width, device=q.device)
    order = torch.where(w < kept[:, None, None], order[..., :width], table.shape[1])
    order = torch.sort(order, dim=-1).values
    out = torch.gather(table[:, None].expand(-1, hk, -1), 2, order.clamp(max=table.shape[1] - 1))
    out = torch.where((w < kept[:, None, None]) & (rows > 0)[:, None, None], out, -1).int()
    return out, torch.where(rows > 0, end - page * (count - kept), 0).int()


def _attend(s, table, kv_len):
    """table: [requests, pages], or [requests, heads, pages]."""
    q, pool = s["q"], s["pool"]
    T, hq, d = q.shape
    hk, page = pool.shape[1], s["page"]
    m = s["max_new"]
    head = torch.arange(hk, device=q.device)[:, None]
    blocks = pool[(table[:, None] if table.dim() == 2 else table).long().clamp(min=0), head]   # [B, hk, pages, bytes]
    k, v = (_values(blocks, h, d, page).flatten(2, 3) for h in (0, 1))
    n = torch.arange(k.shape[2], device=q.device)
    live = (n < kv_len[:, None])[:, None, :, None]
    k, v = torch.where(live, k, 0.0), torch.where(live, v, 0.0)
    cu = s["cu_rows"].long()
    rows = cu[1:] - cu[:-1]
    i = torch.arange(m, device=q.device)
    at = torch.where(i < rows[:, None], cu[:-1, None] + i, 0)               # [B, m]
    x = q.float()[at].unflatten(2, (hk, hq // hk)).permute(0, 2, 3, 1, 4)   # [B, hk, group, m, d]
    score = torch.matmul(x.flatten(2, 3), k.transpose(-1, -2)).unflatten(2, (hq // hk, m)) / math.sqrt(d)
    where = (kv_len - rows)[:, None] + i                                    # [B, m] position of each row
    sees = n < kv_len[:, None, None]
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
        step = (s["table"], s["kv_len"], s["cu_rows"])
        if op == "append":
            k_hat, v_hat = torch.empty_like(s["k"]), torch.empty_like(s["v"])
            paged.qwm_paged8_append(s["k"], s["v"], s["pool"], *step, k_hat=k_hat, v_hat=v_hat)
            return [k_hat, v_hat, s["pool"]]
        if op == "read":
            return list(paged.qwm_paged8_read(s["pool"], *step, s["rows"], s["d"], dtype=s["dtype"]))
        if op == "attend":
            return paged.qwm_paged8_attend(s["q"], s["pool"], *step, max_new=s["max_new"], causal=s["causal"], window=s["window"])
        paged.qwm_paged8_bounds(s["pool"], s["bounds"], *step, max_new=s["max_new"])
        pages, lens = paged.qwm_paged8_select(s["q"], s["bounds"], *step, s["page"], s["width"], sink=s["sink"])
        o = paged.qwm_paged8_attend(s["q"], s["pool"], pages, lens, s["cu_rows"], max_new=s["max_new"], causal=s["causal"])
        return [s["bounds"], pages, lens, o]
    if op == "append":
        return _append(s)
    if op == "read":
        return _read(s)
    if op == "attend":
        return _attend(s, s["table"], s["kv_len"])
    _bounds(s)
    pages, lens = _select(s)
    return [s["bounds"], pages, lens, _attend(s, pages, lens)]


# ---------------------------------------------------------------- in 64 bits, from the definitions
def _two_to(e):
    """2^e, float64."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(code):
    """The value of each e4m3 byte, float64."""
    c = code.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    x = torch.where(e > 0, (8 + m) * _two_to(e - 10), m * 2.0 ** -9)
    return torch.where(c > 127, -x, x)


def _nearest(x):
    """Multiples of 2^-9 and four bits nearest to x (|x| <= 448), ties to even: what e4m3 holds."""
    step = _two_to(torch.frexp(x.abs().clamp(min=2.0 ** -6)).exponent - 4)
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    op, d, page = case["op"], case["d"], case["page"]
    cu, lens = s["cu_rows"].tolist(), s["kv_len"].tolist()
    hk = case["kv_heads"]

    def held(b, h, half, lo, hi, ids=None):
        """Values of tokens lo to hi of a request (of a list of pages)."""
        ids = s["table"][b] if ids is None else ids
        got = s["pool"][ids[lo // page:(hi + page - 1) // page].long(), h]
        c = got[:, half * page * d:(half + 1) * page * d].reshape(-1, d)
        f = got[:, 2 * page * d:2 * page * d + page // 4].contiguous().view(torch.float16).reshape(-1, 2)[:, half]
        full = _e4m3(c) * f.double().repeat_interleave(BLOCK)[:, None]
        return full[lo % page:lo % page + hi - lo]

    if op == "append":
        out = []
        for half, x in ((0, s["k"]), (1, s["v"])):
            y = x.double()
            z = torch.empty_like(y)
            for b, n in enumerate(lens):
                start = n - cu[b + 1] + cu[b]
                for t in range(start // BLOCK * BLOCK, n, BLOCK):
                    lo, hi = cu[b] + max(t, start) - start, cu[b] + min(t + BLOCK, n) - start
                    if lo >= hi:
                        continue
                    top = y[lo:hi].abs().amax((0, 2))
                    size = torch.full_like(top, 2.0 ** LOW)
                    for e in range(LOW, HIGH):
                        size = torch.where(top > 448 * 2.0 ** e, 2.0 ** (e + 1), size)
                    if t < start:
                        had = s["pool"][int(s["table"][b, t // page]), :, 2 * page * d:2 * page * d + page // 4]
                        had = had.contiguous().view(torch.float16).reshape(hk, -1, 2)[:, t % page // BLOCK, half]
                        size = torch.maximum(size, had.double())
                    z[lo:hi] = _nearest(y[lo:hi] / size[:, None]) * size[:, None]
            out.append(z)
        return out + [None]  # the pool's bytes have no value in 64 bits
    if op == "read":
        out = []
        for half in (0, 1):
            z = torch.empty((s["rows"], hk, d), dtype=torch.float64, device="cuda")
            for b, n in enumerate(lens):
                for h in range(hk):
                    if cu[b] < cu[b + 1]:
                        z[cu[b]:cu[b + 1], h] = held(b, h, half, n - cu[b + 1] + cu[b], n)
            out.append(z)
        return out
    pages = None
    if op == "sparse":
        _bounds(s)
        pages, short = _select(s)  # whole numbers, by definition in float32
        lens = short.tolist()
    q = s["q"].double()
    out = torch.zeros_like(q)
    group = case["heads"] // hk
    for b, n in enumerate(lens):
        rows = cu[b + 1] - cu[b]
        here = torch.arange(n, device=q.device)
        at = n - rows + torch.arange(rows, device=q.device)[:, None]
        hidden = torch.zeros((rows, n), dtype=torch.bool, device=q.device)
        if case["causal"]:
            hidden |= here > at
        if s["window"]:
            hidden |= here <= at - s["window"]
        if n == 0 or rows == 0:
            continue
        for h in range(hk):
            k, v = (held(b, h, half, 0, n, None if pages is None else pages[b, h]) for half in (0, 1))
            for j in range(h * group, (h + 1) * group):
                logits = (q[cu[b]:cu[b + 1], j] @ k.T / math.sqrt(d)).masked_fill(hidden, -math.inf)
                out[cu[b]:cu[b + 1], j] = torch.nan_to_num(torch.softmax(logits, -1), nan=0.0) @ v
    return out if pages is None else [None, pages, short, out]
