"""Shared set-up of the 8-bit cache's tests: seeded batches and tolerances.

Only tests import this file.
"""
from __future__ import annotations

import numpy as np

from oracle import paged8_oracle as P8
from paged_cases import EPS2, rounded


class Batch8:
    """Requests with cached tokens in a shuffled 8-bit pool.  Slots that hold no
    token, and pages that no request holds, are 0xFF bytes (NaN codes and scales)."""

    def __init__(self, seed, cached, new, heads, kv_heads, d, page, dtype="bf16", q_sigma=1.0, spare=3, width=None):
        r = np.random.default_rng(seed)
        self.cached, self.new = list(cached), list(new)
        self.d, self.page, self.heads, self.kv_heads, self.dtype = d, page, heads, kv_heads, dtype
        self.kv_len = np.array([c + n for c, n in zip(cached, new)], np.int32)
        held = [-(-int(n) // page) for n in self.kv_len]
        n_pages = sum(held) + spare
        order = r.permutation(n_pages).astype(np.int32)
        self.table = np.full((len(held), width or max(1, max(held))), -1, np.int32)
        at = 0
        for b, m in enumerate(held):
            self.table[b, :m] = order[at: at + m]
            at += m
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.rows = int(self.cu[-1])
        sigma = np.exp(0.5 * r.standard_normal((kv_heads, d)))
        total = int(self.kv_len.sum())
        self.k = rounded(r.standard_normal((total, kv_heads, d)) * sigma, dtype)     # every token, cached and new
        self.v = rounded(r.standard_normal((total, kv_heads, d)), dtype)
        self.empty = np.full((n_pages, kv_heads, P8.block_bytes(d, page)), 255, np.uint8)
        all_cu = np.concatenate([[0], np.cumsum(self.kv_len)])
        self.pool = P8.append(self.empty, self.k, self.v, self.table, self.kv_len, all_cu, page)[0]
        self.q = rounded(r.standard_normal((self.rows, heads, d)) * q_sigma, dtype)

    def rows_of(self, x, first, count):
        """Rows of `count[b]` tokens of each request from its token `first[b]` on, of a tensor of all tokens."""
        base = np.concatenate([[0], np.cumsum(self.kv_len)])
        return np.concatenate([x[base[b] + f: base[b] + f + c] for b, (f, c) in enumerate(zip(first, count))])


def attend8_tolerance(O, spread, vmax, n: int, dtype: str, tensor: bool):
    """Bound of |O_gpu - O| per element.

    k_hat and v_hat are exact in float16 and in float32, and so is q scaled by a
    power of two.  A logit of d products is off by at most (d + 3) 2^-24 sigma sum
    |q k| (d <= 128; the sum, the scale and the exponent's argument), exp2 by
    2^-22, so p is off by 2 delta relative to the normalised sum; the sums of p and
    of p v add at most (n / 16 + 100) roundings each in the float32 kernel and
    n + 200 in the tensor kernels, which round P to float16 besides (2^-11, and
    below float16's normal range 2^-25 absolute) and whose exp2 and rescaling are
    off by 2^-21.  Kernel 2 in float32 takes q and P as two float16 terms, off by 2^-22
    of each (4 2^-24 more in delta, 2^-22 in P), sums a step's 16 tokens in two MMAs
    that cut off below 2^-23 each, and adds the steps up like the float32 kernel.
    Then one rounding to the output's dtype."""
    d32 = 131 * EPS2["f32"]
    if tensor and dtype == "f32":
        delta = spread * (d32 + 4 * EPS2["f32"]) + 2.0 ** -21
        rel = np.expm1(2 * delta) + 2 * 2.0 ** -22 + 2 * (n / 16 + 100) * EPS2["f32"]
    elif tensor:
        delta = spread * d32 + 2.0 ** -21
        rel = np.expm1(2 * delta) + 1.01 * EPS2["f16"] + n * 2.0 ** -25 + (n + 200) * EPS2["f32"]
    else:
        delta = spread * d32 + 2.0 ** -22
        rel = np.expm1(2 * delta) + 2 * (n / 16 + 100) * EPS2["f32"]
    return (rel * vmax)[..., None] * (1 + EPS2[dtype]) + EPS2[dtype] * np.abs(O) + 1e-30
