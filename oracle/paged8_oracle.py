"""Plain CPU oracle of the paged 8-bit cache and of the selection of pages.

TEST INFRASTRUCTURE ONLY, like paged_oracle.py: NumPy, each function the formula
written out, no code shared with the CUDA library.  Values and attention are
float64; what is by definition decided in float32 (the bounds' units and codes,
the scores) is done there, one IEEE operation at a time.
"""
from __future__ import annotations

import numpy as np

SLOTS = 16                     # slots that share a scale
LOW, HIGH = -15, 7
CLAMP = 448.0 * 2.0 ** HIGH
f32 = np.float32


# ------------------------------------------------------------------ e4m3
def _table():
    x = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x[c] = (8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9
        if c & 127 == 127:
            x[c] = np.nan
        if c > 127:
            x[c] = -x[c]
    return x


E4M3 = _table()


def encode(x):
    """The e4m3 codes nearest to x (float64, |x| <= 448), ties to the even code."""
    x = np.asarray(x, np.float64)
    grid = E4M3[:127]                                    # ascending, codes 0 .. 126
    i = np.searchsorted(grid, np.abs(x), side="right") - 1
    j = np.minimum(i + 1, 126)
    low, high = np.abs(x) - grid[i], grid[j] - np.abs(x)
    up = (high < low) | ((high == low) & (i % 2 == 1) & (j > i))
    return (np.where(up, j, i) | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def scale_for(amax: float) -> float:
    for e in range(LOW, HIGH):
        if 448.0 * 2.0 ** e >= amax:
            return 2.0 ** e
    return 2.0 ** HIGH


# ------------------------------------------------------------------ blocks
def block_bytes(d: int, page: int) -> int:
    return 2 * page * d + max(16, page // 4)


def codes_of(blk, half: int, d: int, page: int):
    return blk[half * page * d: (half + 1) * page * d].reshape(page, d)


def scales_of(blk, d: int, page: int):
    """[page / 16, 2] float16, a view."""
    return blk[2 * page * d: 2 * page * d + page // 4].view(np.float16).reshape(-1, 2)


def read_block(blk, d: int, page: int):
    """(k_hat, v_hat) float64 [page, d]."""
    s = np.repeat(scales_of(blk, d, page).astype(np.float64), SLOTS, 0)
    with np.errstate(invalid="ignore"):
        return [E4M3[codes_of(blk, h, d, page)] * s[:, h: h + 1] for h in (0, 1)]


def append(pool, k, v, table, kv_len, cu, page: int):
    """The pool after the step, and (k_hat, v_hat) float64 (NaN in rows that get none)."""
    pool = pool.copy()
    d, hk = k.shape[2], k.shape[1]
    hats = [np.full(k.shape, np.nan), np.full(k.shape, np.nan)]
    for b, n in enumerate(kv_len):
        first = int(n) - int(cu[b + 1] - cu[b])
        for t in range(max(first, 0) // SLOTS * SLOTS, int(n), SLOTS):
            lo, hi = max(t, first), min(t + SLOTS, int(n))
            pg = int(table[b, t // page])
            if lo >= hi or not 0 <= pg < pool.shape[0]:
                continue
            at = t % page
            rows = slice(int(cu[b]) + lo - first, int(cu[b]) + hi - first)
            for h in range(hk):
                for half, x in ((0, k), (1, v)):
                    y = np.asarray(x[rows, h], np.float64)
                    y = np.clip(np.where(np.isnan(y), 0.0, y), -CLAMP, CLAMP)
                    codes, scales = codes_of(pool[pg, h], half, d, page), scales_of(pool[pg, h], d, page)
                    s = scale_for(np.abs(y).max())
                    if first > t:
                        had = float(scales[at // SLOTS, half])
                        if had >= s:
                            s = had
                        else:
                            codes[at: at + first - t] = encode(E4M3[codes[at: at + first - t]] * (had / s))
                    codes[at + lo - t: at + hi - t] = encode(y / s)
                    scales[at // SLOTS, half] = s
                    hats[half][rows, h] = E4M3[codes[at + lo - t: at + hi - t]] * s
    return pool, hats[0], hats[1]


def gather(pool, ids, n: int, head: int, d: int, page: int):
    """(k_hat, v_hat, known) [n, d] of the first n tokens of a list of pages."""
    k, v, known = np.zeros((n, d)), np.zeros((n, d)), np.zeros(n, bool)
    for j in range(-(-n // page)):
        pg = int(ids[j])
        if 0 <= pg < pool.shape[0]:
            kb, vb = read_block(pool[pg, head], d, page)
            m = min(page, n - j * page)
            k[j * page: j * page + m], v[j * page: j * page + m] = kb[:m], vb[:m]
            known[j * page: j * page + m] = True
    return k, v, known


def attend(q, pool, table, kv_len, cu, page: int, causal: bool, window: int, sigma: float):
    """(O, lse, spread, vmax) like paged_oracle.attend; table [requests, pages] or [requests, kv_heads, pages]."""
    rows, hq, d = q.shape
    hk = pool.shape[1]
    group = hq // hk
    O, lse = np.zeros((rows, hq, d)), np.full((rows, hq), -np.inf)
    spread, vmax = np.zeros((rows, hq)), np.zeros((rows, hq))
    for b in range(len(kv_len)):
        n, lo, hi = int(kv_len[b]), int(cu[b]), int(cu[b + 1])
        if hi == lo:
            continue
        for h in range(hk):
            k, v, known = gather(pool, table[b] if table.ndim == 2 else table[b, h], n, h, d, page)
            tok = np.arange(n)
            for i in range(hi - lo):
                at = n - (hi - lo) + i
                sees = known.copy()
                if causal:
                    sees &= tok <= at
                if window:
                    sees &= tok > at - window
                if not sees.any():
                    continue
                x = q[lo + i, h * group: (h + 1) * group]                          # [group, d]
                s = sigma * (x @ k[sees].T)
                m = s.max(1, keepdims=True)
                p = np.exp(s - m)
                z = slice(h * group, (h + 1) * group)
                O[lo + i, z] = p @ v[sees] / p.sum(1, keepdims=True)
                lse[lo + i, z] = m[:, 0] + np.log(p.sum(1))
                spread[lo + i, z] = (np.abs(x) @ np.abs(k[sees]).T).max(1) * abs(sigma)
                vmax[lo + i, z] = np.abs(v[sees]).max()
    return O, lse, spread, vmax


# ------------------------------------------------------------------ selection
def bounds(pool, old, table, kv_len, cu, page: int, d: int):
    """The bounds' bytes after the step, from those before."""
    out = old.copy()
    for b, n in enumerate(kv_len):
        first = int(n) - int(cu[b + 1] - cu[b])
        if first >= n:
            continue
        for j in range(max(first, 0) // page, -(-int(n) // page)):
            pg = int(table[b, j])
            if not 0 <= pg < pool.shape[0]:
                continue
            for h in range(pool.shape[1]):
                k = read_block(pool[pg, h], d, page)[0][: min(page, int(n) - j * page)].astype(f32)
                high, low = k.max(0), k.min(0)
                unit = f32(max(np.abs(high).max(), np.abs(low).max())) / f32(127)
                by = unit if unit > 0 else f32(1)
                out[pg, h, :d] = np.rint(high / by).astype(np.int8).view(np.uint8)
                out[pg, h, d: 2 * d] = np.rint(low / by).astype(np.int8).view(np.uint8)
                out[pg, h, 2 * d:] = np.array([unit, 0, 0, 0], f32).view(np.uint8)
    return out


def scores(q, bnd, ids, d: int):
    """[pages] float32: the scores of pages `ids` of one head (bnd [pages, bytes]) for query rows q [m, d]; NaN
    where the id is out of range or the bounds are NaN."""
    q = np.asarray(q, f32)
    q = np.clip(np.where(np.isnan(q), f32(0), q), -np.finfo(f32).max, np.finfo(f32).max)
    top = np.abs(q).max(1, keepdims=True)
    unit = np.where(top >= f32(2.0 ** -100), top / f32(127), f32(0)).astype(f32)
    x = np.where(unit > 0, np.clip(np.rint(q / np.where(unit > 0, unit, f32(1))), -127, 127), 0).astype(np.int64)
    out = np.full(len(ids), np.nan, f32)
    ids = np.asarray(ids)
    known = (ids >= 0) & (ids < bnd.shape[0])
    b = bnd[ids[known]]
    high, low = (np.ascontiguousarray(b[:, z * d: (z + 1) * d]).view(np.int8).astype(np.float64) for z in (0, 1))
    S = np.maximum(x, 0) @ high.T + np.minimum(x, 0) @ low.T       # whole numbers below 2^24: exact
    with np.errstate(over="ignore"):
        out[known] = ((S.astype(f32) * np.ascontiguousarray(b[:, 2 * d: 2 * d + 4]).view(f32)[:, 0]) * unit).max(0)
    return out


def select(q, bnd, table, kv_len, cu, page: int, width: int, sink: int, d: int):
    """(pages [requests, kv_heads, width], lens [requests])."""
    B, hk = len(kv_len), bnd.shape[1]
    group = q.shape[1] // hk
    pages, lens = np.full((B, hk, width), -1, np.int32), np.zeros(B, np.int32)
    for b, n in enumerate(kv_len):
        n, lo, hi = int(n), int(cu[b]), int(cu[b + 1])
        count, tail = -(-n // page), max(n - (hi - lo), 0) // page
        kept = min(count, width)
        if hi == lo or count - tail > kept:
            continue
        lens[b] = n - page * (count - kept)
        for h in range(hk):
            s = scores(q[lo:hi, h * group: (h + 1) * group].reshape(-1, d), bnd[:, h], table[b, :count], d)
            own = list(range(tail, count))
            first = list(range(min(sink, tail, kept - len(own))))
            rest = [j for j in range(len(first), tail)]
            rest.sort(key=lambda j: (bool(np.isnan(s[j])), 0 if np.isnan(s[j]) else -s[j], j))
            take = sorted(own + first + rest[: kept - len(own) - len(first)])
            pages[b, h, :kept] = table[b, take]
    return pages, lens
