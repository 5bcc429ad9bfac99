"""Plain CPU oracle of the paged 4-bit cache and the norm and rotation step.

TEST INFRASTRUCTURE ONLY, like qwm_oracle.py: float64 NumPy, each function the
formula written out, no code shared with the CUDA library.  The one decision
taken in float32, one IEEE operation at a time, is the 4-bit code (that is its
definition); float16 parameters are rounded to nearest even.
"""
from __future__ import annotations

import numpy as np

GROUP = 32
CLAMP = 60000.0
f32 = np.float32


# ------------------------------------------------------------------ quantiser
def quantize_int4(x):
    """(codes uint8, zero f16, scale f16) of groups along the last axis of x
    [..., d] (values of the input dtype, exactly in float32)."""
    x = np.asarray(x, dtype=f32)
    x = np.where(np.isnan(x), f32(0), x)
    x = np.clip(x, f32(-CLAMP), f32(CLAMP)).reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    mn, mx = x.min(-1), x.max(-1)
    zero = mn.astype(np.float16)
    scale = ((mx - mn) / f32(15)).astype(np.float16)
    z, s = zero.astype(f32)[..., None], scale.astype(f32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        q = (x - z) / s
    codes = np.where(s > 0, np.clip(np.rint(np.where(s > 0, q, 0)), 0, 15), 0).astype(np.uint8)
    return codes.reshape(*codes.shape[:-2], codes.shape[-2] * GROUP), zero, scale


def dequantize_int4(codes, zero, scale):
    """zero + code scale in float64."""
    c = codes.astype(np.float64).reshape(*codes.shape[:-1], codes.shape[-1] // GROUP, GROUP)
    return (zero.astype(np.float64)[..., None] + c * scale.astype(np.float64)[..., None]).reshape(codes.shape)


def block_offsets(d: int, page: int) -> dict:
    """Byte offsets of a block's sections and its size."""
    k = page * d // 2
    kp = k + page * (d // GROUP) * 4
    return {"kcode": 0, "kqp": k, "vcode": kp, "vqp": kp + k, "bytes": 2 * kp}


def write_slot(pool, slot: int, head: int, k, v, d: int, page: int):
    """Store one token of one head (k, v: [d]) into pool [pages, heads, bytes] uint8."""
    off = block_offsets(d, page)
    blk = pool[slot // page, head]
    at = slot % page
    for x, oc, op in ((k, off["kcode"], off["kqp"]), (v, off["vcode"], off["vqp"])):
        codes, zero, scale = quantize_int4(x)
        blk[oc + at * d // 2: oc + (at + 1) * d // 2] = codes[0::2] | (codes[1::2] << 4)
        par = np.stack([zero, scale], -1).astype(np.float16).view(np.uint8).reshape(-1)
        n = par.size
        blk[op + at * n: op + (at + 1) * n] = par


def read_block(blk, d: int, page: int):
    """(k_hat, v_hat) float64 [page, d] of one block's bytes."""
    off = block_offsets(d, page)
    out = []
    for oc, op in ((off["kcode"], off["kqp"]), (off["vcode"], off["vqp"])):
        raw = blk[oc: oc + page * d // 2].reshape(page, d // 2)
        codes = np.empty((page, d), np.uint8)
        codes[:, 0::2], codes[:, 1::2] = raw & 15, raw >> 4
        par = np.ascontiguousarray(blk[op: op + page * (d // GROUP) * 4]).view(np.float16).reshape(page, d // GROUP, 2)
        out.append(dequantize_int4(codes, par[..., 0], par[..., 1]))
    return out


# ------------------------------------------------------------------ bookkeeping
def plan(kv_len, new_len, table, free_pages, free_count: int, page: int, rows: int):
    """The plan's outputs (kv_len, free_count, cu_rows, slots, positions, table), or None when it does not fit."""
    B = len(kv_len)
    table = np.array(table)
    held = [-(-int(n) // page) for n in kv_len]
    total = [-(-(int(n) + int(m)) // page) for n, m in zip(kv_len, new_len)]
    if min(kv_len) < 0 or min(new_len) < 0 or sum(new_len) > rows or max(total) > table.shape[1] \
            or sum(total) - sum(held) > free_count:
        return None
    cu, slots, positions = [0], np.full(rows, -1, np.int64), np.full(rows, -1, np.int32)
    for b in range(B):
        for j in range(held[b], total[b]):
            free_count -= 1
            table[b, j] = free_pages[free_count]
        for i in range(int(new_len[b])):
            pos = int(kv_len[b]) + i
            positions[cu[-1] + i] = pos
            slots[cu[-1] + i] = int(table[b, pos // page]) * page + pos % page
        cu.append(cu[-1] + int(new_len[b]))
    return np.asarray(kv_len) + np.asarray(new_len), free_count, np.array(cu, np.int32), slots, positions, table


def release(keep_len, kv_len, table, free_pages, free_count: int, page: int):
    """The release's state after the call: (kv_len, table, free_pages, free_count)."""
    kv_len, table, free_pages = np.array(kv_len), np.array(table), np.array(free_pages)
    for b in range(len(kv_len)):
        for j in range(-(-int(keep_len[b]) // page), -(-int(kv_len[b]) // page)):
            free_pages[free_count] = table[b, j]
            free_count += 1
            table[b, j] = -1
        kv_len[b] = keep_len[b]
    return kv_len, table, free_pages, free_count


# ------------------------------------------------------------------ norm and rotation
def norm_rope(x, w, cos_sin, positions, axis, eps: float, interleaved: bool):
    """x [rows, heads, d]; w [d] or None; cos_sin [n, rot]; positions [rows, axes]; axis [rot/2]."""
    x = np.asarray(x, np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if w is not None:
        y = y * np.asarray(w, np.float64)
    rot = cos_sin.shape[1]
    out = y.copy()
    for j in range(rot // 2):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
        c = cos_sin[positions[:, axis[j]], j].astype(np.float64)[:, None]
        s = cos_sin[positions[:, axis[j]], rot // 2 + j].astype(np.float64)[:, None]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
    return out


# ------------------------------------------------------------------ attention
def gather(pool, table_row, n: int, head: int, d: int, page: int):
    """(k_hat, v_hat, known) [n, d] of the first n tokens of a request: tokens of a page id out of range are unknown."""
    k, v, known = np.zeros((n, d)), np.zeros((n, d)), np.zeros(n, bool)
    for j in range(-(-n // page)):
        pg = int(table_row[j])
        if 0 <= pg < pool.shape[0]:
            kb, vb = read_block(pool[pg, head], d, page)
            m = min(page, n - j * page)
            k[j * page: j * page + m], v[j * page: j * page + m] = kb[:m], vb[:m]
            known[j * page: j * page + m] = True
    return k, v, known


def attend(q, pool, table, kv_len, cu_rows, page: int, causal: bool, window: int, sigma: float):
    """(O, lse, spread): q [rows, heads, d] float64.  spread [rows, heads] =
    max over visible tokens of sigma sum_c |q_c k_c| (what the rounding of a
    product sum scales with) and, last, max |v_hat| of the request."""
    rows, hq, d = q.shape
    hk = pool.shape[1]
    group = hq // hk
    O, lse = np.zeros((rows, hq, d)), np.full((rows, hq), -np.inf)
    spread, vmax = np.zeros((rows, hq)), np.zeros((rows, hq))
    for b in range(len(kv_len)):
        n, lo, hi = int(kv_len[b]), int(cu_rows[b]), int(cu_rows[b + 1])
        for h in range(hk):
            k, v, known = gather(pool, table[b], n, h, d, page)
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
                for g in range(group):
                    x = q[lo + i, h * group + g]
                    s = sigma * (k[sees] @ x)
                    m = s.max()
                    p = np.exp(s - m)
                    O[lo + i, h * group + g] = p @ v[sees] / p.sum()
                    lse[lo + i, h * group + g] = m + np.log(p.sum())
                    spread[lo + i, h * group + g] = (np.abs(k[sees]) @ np.abs(x)).max() * abs(sigma)
                    vmax[lo + i, h * group + g] = np.abs(v[sees]).max()
    return O, lse, spread, vmax
