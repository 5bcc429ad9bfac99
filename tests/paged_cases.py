"""Shared set-up of the paged cache's tests: seeded batches and tolerances.

Only tests import this file.
"""
from __future__ import annotations

import numpy as np

from oracle import paged_oracle as P

EPS2 = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}   # half a step, relative


def bf16(x):
    """float32 values rounded to bfloat16 (nearest even)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32)


def rounded(x, dtype: str):
    return bf16(x) if dtype == "bf16" else np.asarray(x, np.float32)


class Batch:
    """Requests with cached tokens in a shuffled pool.  Slots that hold no
    token, and pages that no request holds, are 0xFF bytes (NaN parameters)."""

    def __init__(self, seed, cached, new, heads, kv_heads, d, page, dtype="bf16", q_sigma=1.0, spare=3):
        r = np.random.default_rng(seed)
        self.cached, self.new = list(cached), list(new)
        self.d, self.page, self.heads, self.kv_heads, self.dtype = d, page, heads, kv_heads, dtype
        self.kv_len = np.array([c + n for c, n in zip(cached, new)], np.int32)
        held = [-(-int(n) // page) for n in self.kv_len]
        n_pages = sum(held) + spare
        order = r.permutation(n_pages).astype(np.int32)
        self.table = np.full((len(held), max(1, max(held))), -1, np.int32)
        self.pool = np.full((n_pages, kv_heads, P.block_offsets(d, page)["bytes"]), 255, np.uint8)
        at = 0
        for b, m in enumerate(held):
            self.table[b, :m] = order[at: at + m]
            at += m
        self.free = order[at:]
        off = P.block_offsets(d, page)
        sigma = np.exp(0.5 * r.standard_normal((kv_heads, d)))
        for b, n in enumerate(self.kv_len):
            k = rounded(r.standard_normal((n, kv_heads, d)) * sigma, dtype)
            v = rounded(r.standard_normal((n, kv_heads, d)), dtype)
            for x, oc, op in ((k, off["kcode"], off["kqp"]), (v, off["vcode"], off["vqp"])):
                codes, zero, scale = P.quantize_int4(x)
                packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
                par = np.stack([zero, scale], -1).view(np.uint8).reshape(n, kv_heads, d // 8)
                w = par.shape[-1]
                for i in range(n):
                    pg, s = self.table[b, i // page], i % page
                    self.pool[pg, :, oc + s * d // 2: oc + (s + 1) * d // 2] = packed[i]
                    self.pool[pg, :, op + s * w: op + (s + 1) * w] = par[i]
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.rows = int(self.cu[-1])
        self.q = rounded(r.standard_normal((self.rows, heads, d)) * q_sigma, dtype)


def attend_tolerance(O, spread, vmax, n: int, dtype: str, tensor: bool):
    """Bound of |O_gpu - O| per element.

    Float32 kernel: a logit of d products is off by at most (d + 3) 2^-24
    sigma sum |q k| (d <= 128; the sum, the scale and the exponent's argument)
    and exp2 by 2^-22, so p is off by 2 delta relative to the normalised sum;
    the sums of p and of p v add at most (n / 16 + 100) roundings each.
    Tensor kernels: k_hat is rounded once to float16 (2^-11 |k| a term, and
    the same once more for the code's subtraction-free sum), Q is exact,
    products accumulate in float32; P and V_hat are rounded to float16 (2^-11
    each), a P below float16's normal range by 2^-25 absolute.  Then one
    rounding to the output's dtype."""
    d32 = 131 * EPS2["f32"]
    if tensor:
        delta = spread * (EPS2["f16"] * 1.01 + d32) + 2.0 ** -21
        rel = np.expm1(2 * delta) + 2.02 * EPS2["f16"] + n * 2.0 ** -25 + (n + 200) * EPS2["f32"]
    else:
        delta = spread * d32 + 2.0 ** -22
        rel = np.expm1(2 * delta) + 2 * (n / 16 + 100) * EPS2["f32"]
    return (rel * vmax)[..., None] * (1 + EPS2[dtype]) + EPS2[dtype] * np.abs(O) + 1e-30
