"""The 8-bit cache's calls as their documentation allows them and no other test makes
them."""
import numpy as np
import pytest
import torch

from oracle import paged8_oracle as P8
from paged8_cases import Batch8
from test_gpu_paged8_cache import BOUNDS, all_bounds, before, dev, host, paged  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ a step in slices
@pytest.mark.parametrize("cached,new,cuts", [([100, 3, 40], [30, 40, 1], (0, 1, 2, 3)), ([3, 70], [33, 50], (0, 1, 2)),
                                             ([0, 0, 5, 16], [100, 20, 17, 60], (0, 1, 3, 4)), ([20] * 6, [1, 1, 1, 1, 60, 2], (0, 4, 6))])
@pytest.mark.parametrize("freed", [False, True])
def test_append_and_read_of_a_step_in_slices(paged, cached, new, cuts, freed):  # noqa: F811
    """cu_rows[a: b + 1] of a step begin behind the first row: the rows ahead belong
    to no request of the call.  Nothing is reported, no byte but the step's blocks
    changes, and pages ahead of those may have been given up (-1 in the tables)."""
    B = Batch8(21, cached, new, 2, 2, 64, 16, "f32")
    k, v = (B.rows_of(x, cached, new) for x in (B.k, B.v))
    pool0 = before(B)
    want, kh, vh = P8.append(pool0, k, v, B.table, B.kv_len, B.cu, 16)
    table = B.table.copy()
    if freed:
        for b, c in enumerate(cached):
            table[b, :c // 16] = -1
    pool, lens, cu, t = dev(pool0), dev(B.kv_len), dev(B.cu), dev(table)
    status = i32([0])
    hats = [torch.full((B.rows, 2, 64), 9.0, device="cuda") for _ in range(4)]
    for a, b in zip(cuts[:-1], cuts[1:]):
        step = t[a:b].contiguous(), lens[a:b], cu[a:b + 1]
        paged.qwm_paged8_append(dev(k), dev(v), pool, *step, k_hat=hats[0], v_hat=hats[1], status=status)
        assert int(status.item()) == 0, (a, b)
        paged.qwm_paged8_read(pool, *step, B.rows, 64, dtype=torch.float32, k_out=hats[2], v_out=hats[3], status=status)
        assert int(status.item()) == 0, (a, b)
        assert bool((hats[2][int(B.cu[b]):] == 9.0).all())
    assert np.array_equal(host(pool), want)
    for got, x in zip(hats, (kh, vh, kh, vh)):
        assert np.array_equal(host(got), x)


# ------------------------------------------------------------------ scores without a finite value
@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_pages_without_bounds_come_behind_scores_of_minus_infinity(paged, rows, d):  # noqa: F811
    """Infinite queries against keys of the other sign score -inf on every page; pages
    out of range and bounds that are NaN still come last, in few rows and in many."""
    page, count, hk = 16, 300, 2
    bnd = np.zeros((count, hk, 2 * d + 16), np.uint8)
    bnd[..., :d], bnd[..., d:2 * d] = 120, 90
    bnd[..., 2 * d:2 * d + 4] = np.array([0.5], np.float32).view(np.uint8)
    table = np.random.default_rng(3).permutation(count).astype(np.int32)[None]
    none = [2, 5, 140, 141]
    bnd[table[0, none[0]], :, 2 * d:2 * d + 4] = np.array([np.nan], np.float32).view(np.uint8)
    table[0, none[1]], table[0, none[2]] = -1, count
    bnd[table[0, none[3]], :, 2 * d:2 * d + 4] = np.array([np.nan], np.float32).view(np.uint8)
    q = np.full((rows, 2 * hk, d), -np.inf, np.float32)
    lens, cu = np.array([count * page], np.int32), np.array([0, rows], np.int32)
    own = count - (count * page - rows) // page
    rest = [j for j in range(count - own) if j not in none]
    status = i32([0])
    for width in (own + 1, own + 7, own + len(rest), own + len(rest) + 2):
        got, _ = paged.qwm_paged8_select(dev(q), dev(bnd), dev(table), dev(lens), dev(cu), page, width, status=status)
        take = sorted((rest + none)[:width - own]) + list(range(count - own, count))
        assert np.array_equal(host(got)[0], np.tile(table[0, take], (hk, 1))), width
        assert np.array_equal(host(got), P8.select(q, bnd, table, lens, cu, page, width, 0, d)[0])
    assert int(status.item()) == BOUNDS


# ------------------------------------------------------------------ outputs in other tensors' memory
def test_a_selection_into_its_queries_bounds_or_status(paged):  # noqa: F811
    """pages and lens in the memory of q, of the bounds or of the status word are
    refused; neighbours of them in one allocation are not."""
    B = Batch8(3, [200], [2], 2, 1, 64, 16, "f32")
    step = dev(B.table), dev(B.kv_len), dev(B.cu)
    bnd = all_bounds(B)
    n_q, n_b = B.q.size, bnd.size // 4
    mem = torch.zeros(n_q + n_b + 4 + 8, dtype=torch.int32, device="cuda")
    q, status = mem[:n_q].view(torch.float32).view(B.q.shape), mem[n_q + n_b: n_q + n_b + 1]
    bounds = mem[n_q: n_q + n_b].view(torch.uint8).view(bnd.shape)
    q.copy_(dev(B.q)), bounds.copy_(dev(bnd))
    want, want_len = paged.qwm_paged8_select(q, bounds, *step, 16, 4, status=status)
    saved = mem.clone()
    at = lambda i, m: mem[i: i + m]  # noqa: E731
    for kw in (dict(pages=at(0, 4).view(1, 1, 4)), dict(pages=at(n_q - 1, 4).view(1, 1, 4)), dict(pages=at(n_q + n_b - 1, 4).view(1, 1, 4)),
               dict(pages=at(n_q + n_b - 3, 4).view(1, 1, 4)), dict(pages=at(n_q + n_b, 4).view(1, 1, 4)), dict(lens=at(n_q - 1, 1)),
               dict(lens=at(n_q, 1)), dict(lens=at(n_q + n_b, 1))):
        with pytest.raises(ValueError, match="memory of its own"):
            paged.qwm_paged8_select(q, bounds, *step, 16, 4, status=status, **kw)
    assert torch.equal(mem, saved)
    got, got_len = paged.qwm_paged8_select(q, bounds, *step, 16, 4, status=status, pages=at(n_q + n_b + 4, 4).view(1, 1, 4),
                                           lens=at(n_q + n_b + 1, 1))
    assert torch.equal(got, want) and torch.equal(got_len, want_len) and torch.equal(mem[:n_q + n_b + 1], saved[:n_q + n_b + 1])


def test_two_outputs_in_one_tensor(paged):  # noqa: F811
    """Values into the keys' tensor, or the stored values of one into the other's
    input, are refused; two slices of one tensor are not."""
    B = Batch8(4, [20], [30], 2, 2, 64, 16, "f32")
    step, pool = (dev(B.table), dev(B.kv_len), dev(B.cu)), dev(B.pool)
    k, v = dev(B.rows_of(B.k, [20], [30])), dev(B.rows_of(B.v, [20], [30]))
    both = torch.zeros((30, 4, 64), device="cuda")
    saved = pool.clone()
    for call in (lambda: paged.qwm_paged8_read(pool, *step, 30, 64, dtype=torch.float32, k_out=both[:, :2], v_out=both[:, :2]),
                 lambda: paged.qwm_paged8_append(k, v, pool, *step, k_hat=both[:, :2], v_hat=both[:, :2]),
                 lambda: paged.qwm_paged8_append(k, v, pool, *step, k_hat=v), lambda: paged.qwm_paged8_append(k, v, pool, *step, v_hat=k)):
        with pytest.raises(ValueError, match="apart"):
            call()
    assert torch.equal(pool, saved) and bool((both == 0).all())
    paged.qwm_paged8_read(pool, *step, 30, 64, dtype=torch.float32, k_out=both[:, :2], v_out=both[:, 2:])
    rk, rv = paged.qwm_paged8_read(pool, *step, 30, 64, dtype=torch.float32)
    assert torch.equal(both, torch.cat([rk, rv], 1))
    for none in (torch.empty((0, 2, 64), device="cuda"), both[:0, :2]):
        paged.qwm_paged8_read(pool, step[0], step[1], i32([0, 0]), 0, 64, dtype=torch.float32, k_out=none, v_out=none)
        paged.qwm_paged8_append(k[:0], v[:0], pool, step[0], step[1], i32([0, 0]), k_hat=none, v_hat=none)


def test_diagnostics_of_more_rows_than_requests_of_a_call(paged):  # noqa: F811
    """Every query is a request of its own there, and a call takes 8,192."""
    from bit_kv_cache_qwm_gb300 import diagnostics
    r = np.random.default_rng(11)
    K, V = (dev(r.standard_normal((1, 200, 64)).astype(np.float32)) for _ in range(2))
    q = dev(r.standard_normal((1, 8200, 64)).astype(np.float32))
    args = dict(page_tokens=16, widths=(3,))
    key = "weight_in_3_pages"
    got = diagnostics.measure_paged8(K, V, q, 0.125, **args)
    parts = [diagnostics.measure_paged8(K, V, q[:, a:b].contiguous(), 0.125, **args)[key] for a, b in ((0, 4100), (4100, 8200))]
    # float32 means of 4,100 and 8,200 values in (0, 1)
    assert got[key] == pytest.approx(sum(parts) / 2, rel=1e-5)


@pytest.mark.parametrize("max_new", [0, 2 ** 31, 2 ** 62, 2 ** 63 - 1])
def test_bounds_with_any_hint(paged, max_new):  # noqa: F811
    B = Batch8(5, [100, 3], [300, 20], 2, 2, 64, 16, "f32")
    old = np.zeros((B.empty.shape[0], 2, 144), np.uint8)
    got = dev(old)
    paged.qwm_paged8_bounds(dev(B.pool), got, dev(B.table), dev(B.kv_len), dev(B.cu), max_new=max_new)
    assert np.array_equal(host(got), P8.bounds(B.pool, old, B.table, B.kv_len, B.cu, 16, 64))


# ------------------------------------------------------------------ many rows over many pages
def walk(pages, rows, group, requests, kv_heads, page_slots):
    """(row tiles, page tiles) that a CTA of the scores of many rows goes through for
    requests of `pages` earlier pages and `rows` rows: tiles of 128 of either,
    page tiles dealt to as many CTAs as there are SMs for each request and head."""
    want = -(-torch.cuda.get_device_properties(0).multi_processor_count // (requests * kv_heads))
    parts = min(want, -(-page_slots // 128))
    assert parts == want     # so the rows of a request are not split
    return [(-(-r * group // 128), -(-(-(-p // 128)) // parts)) for p, r in zip(pages, rows)]


def long_tables(seed, count, new, heads, kv_heads, d, page, odd=False):
    """A step over `count` pages of each request with random bounds, no pool behind
    them; `odd`: with the queries, bounds and ids that a score has rules for."""
    r = np.random.default_rng(seed)
    n_pages = sum(count)
    bnd = np.zeros((n_pages, kv_heads, 2 * d + 16), np.uint8)
    x = np.sort(r.integers(-127, 128, (n_pages, kv_heads, 2, d)), axis=2)[:, :, ::-1]
    bnd[..., :2 * d] = x.reshape(n_pages, kv_heads, 2 * d).astype(np.int8).view(np.uint8)
    bnd[..., 2 * d:2 * d + 4] = np.exp(r.standard_normal((n_pages, kv_heads, 1))).astype(np.float32).view(np.uint8)
    order = r.permutation(n_pages).astype(np.int32)
    table = np.full((len(count), max(count)), -1, np.int32)
    at = 0
    for b, m in enumerate(count):
        table[b, :m] = order[at:at + m]
        at += m
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    lens = np.array([m * page - int(r.integers(0, page)) for m in count], np.int32)
    q = r.standard_normal((int(cu[-1]), heads, d)).astype(np.float32)
    if odd:
        for b, m in enumerate(count):
            for j in r.choice(m, m // 6, replace=False):        # in every tile of pages
                table[b, j] = r.choice([-1, n_pages, 2 ** 31 - 1, -5])
            for j in r.choice(m, m // 6, replace=False):
                if 0 <= table[b, j] < n_pages:
                    bnd[table[b, j], :, 2 * d:2 * d + 4] = np.array([r.choice([np.nan, 0.0, 1e-30])], np.float32).view(np.uint8)
            same = [j for j in r.choice(m, m // 3, replace=False) if 0 <= table[b, j] < n_pages]
            bnd[table[b, same]] = bnd[table[b, same[0]]]        # equal scores
        for i in range(q.shape[0]):
            h, kind = int(r.integers(heads)), i % 7
            if kind == 0:
                q[i, h, :4] = np.nan, 3.0, -np.inf, np.inf
            elif kind == 1:
                q[i] = np.nan
            elif kind == 2:
                q[i, h] = 0.0
            elif kind == 3:
                q[i] *= np.float32(1e-38)
            elif kind == 4:
                q[i, h] = np.float32(2.0 ** -101)
            elif kind == 5:
                q[i] = np.float32(2.0 ** -100) * np.sign(q[i])
    return bnd, table, lens, cu, q


STEP = [800, 1700, 790, 1000, 129, 385, 1650, 641], [60, 40, 110, 330, 70, 0, 135, 5]     # pages, rows of eight requests


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("odd", [False, True])
def test_scores_of_many_rows_over_several_tiles_of_pages(paged, d, odd):  # noqa: F811
    """A CTA goes on to another tile of pages, behind one, two and more tiles of
    rows; its steps, and its tiles of pages, come round the four places that it
    keeps for each."""
    count, new = STEP
    heads, kv_heads, page, group = 16, 8, 16, 2
    bnd, table, lens, cu, q = long_tables(30 + d, count, new, heads, kv_heads, d, page, odd)
    walks = walk([(n - m) // page for n, m in zip(lens, new)], new, group, len(count), kv_heads, table.shape[1])
    assert {nr for nr, pages in walks if pages > 1} >= {1, 2, 3, 6} and {nr for nr, pages in walks if pages > 4} >= {1, 3}
    assert sum(new) * group > 8 * len(count)       # not the scores of few rows
    status = i32([0])
    for width, sink in ((40, 1), (300, 0)):
        with np.errstate(invalid="ignore", over="ignore"):
            want, wl = P8.select(q, bnd, table, lens, cu, page, width, sink, d)
        for _ in range(10):
            got, gl = paged.qwm_paged8_select(dev(q), dev(bnd), dev(table), dev(lens), dev(cu), page, width, sink=sink, status=status)
            assert np.array_equal(host(gl), wl) and np.array_equal(host(got), want)
    assert int(status.item()) == (BOUNDS if odd else 0)


@pytest.mark.parametrize("limit", [0, 300, 3000, 30000])
def test_a_wait_that_runs_out_over_several_tiles_of_pages(paged, monkeypatch, limit):  # noqa: F811
    """As in the test of waits for one tile: the call ends, names pages of the
    request, reports what ran out, and the next one is whole again."""
    count, new = STEP
    bnd, table, lens, cu, q = long_tables(40, count, new, 16, 8, 64, 16)
    args = dev(q), dev(bnd), dev(table), dev(lens), dev(cu), 16, 40
    status = i32([0])
    want, wl = paged.qwm_paged8_select(*args, status=status)
    assert int(status.item()) == 0
    monkeypatch.setenv("QWM_FAULT_INJECT", f"wait={limit}")
    got, gl = paged.qwm_paged8_select(*args, status=status)
    torch.cuda.synchronize()
    monkeypatch.delenv("QWM_FAULT_INJECT")
    bits = int(status.item())
    assert bits in (0, 4) and torch.equal(gl, wl)
    for b in range(len(count)):
        for h in range(8):
            ids = [x for x in host(got)[b, h].tolist() if x >= 0]
            assert len(ids) == len(set(ids)) == (40 if new[b] else 0) and set(ids) <= set(table[b].tolist())
    if bits == 0:
        assert torch.equal(got, want)
    status.zero_()
    assert torch.equal(paged.qwm_paged8_select(*args, status=status)[0], want) and int(status.item()) == 0


def test_a_prompt_among_single_tokens(paged):  # noqa: F811
    """63 single tokens and a prompt that together count as few rows."""
    count, new = [20 + 3 * b for b in range(63)] + [400], [1] * 63 + [449]
    bnd, table, lens, cu, q = long_tables(50, count, new, 1, 1, 64, 16)
    assert sum(new) <= 8 * len(new)
    want, wl = P8.select(q, bnd, table, lens, cu, 16, 31, 1, 64)
    got, gl = paged.qwm_paged8_select(dev(q), dev(bnd), dev(table), dev(lens), dev(cu), 16, 31, sink=1)
    assert np.array_equal(host(gl), wl) and np.array_equal(host(got), want)
