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
    none = torch.empty((0, 2, 64), device="cuda")
    paged.qwm_paged8_read(pool, step[0], step[1], i32([0, 0]), 0, 64, dtype=torch.float32, k_out=none, v_out=none)


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
