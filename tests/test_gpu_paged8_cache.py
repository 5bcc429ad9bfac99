"""qwm_paged8_append, qwm_paged8_read, qwm_paged8_bounds and qwm_paged8_select on
the GPU against the oracle: every byte, index and length is equal."""
import numpy as np
import pytest
import torch

from oracle import paged8_oracle as P8
from paged8_cases import Batch8
from paged_cases import rounded

pytestmark = pytest.mark.gpu

SATURATED, BOUNDS, NAN, CAPACITY = 0x2, 0x8, 0x10, 0x20


@pytest.fixture(scope="module")
def paged():
    from bit_kv_cache_qwm_gb300 import build
    build.build()
    from bit_kv_cache_qwm_gb300 import paged as p
    return p


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def host(t):
    return t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()


def before(B):
    """The pool before the step of a batch: its cached tokens alone."""
    cu = np.concatenate([[0], np.cumsum(B.cached)])
    zero = [0] * len(B.cached)
    return P8.append(B.empty, B.rows_of(B.k, zero, B.cached), B.rows_of(B.v, zero, B.cached), B.table, B.cached, cu, B.page)[0]


STEPS = [([0], [1]), ([5], [1]), ([15, 16, 17, 0], [1, 1, 1, 1]), ([0, 3, 100], [0, 45, 7]), ([31], [66]), ([0] * 5, [1, 2, 16, 17, 33]),
         ([7, 40, 9], [9, 0, 24]), ([0, 0, 5, 0], [0, 3, 0, 0]), (list(range(40)), [1] * 40), ([1] * 70, [3, 0] * 35)]


@pytest.mark.parametrize("d,page,dtype", [(128, 16, "bf16"), (64, 32, "f32"), (128, 64, "f32"), (64, 256, "bf16"), (128, 128, "bf16")])
@pytest.mark.parametrize("cached,new", STEPS)
def test_append_and_read_match_the_oracle(paged, cached, new, d, page, dtype):
    B = Batch8(1, cached, new, 2, 2, d, page, dtype)
    r = np.random.default_rng(2)
    scale = np.exp(2.0 * r.standard_normal((B.rows, 2, 1)))      # scales grow, or do not
    k, v = (rounded(x * scale, dtype) for x in (B.rows_of(B.k, cached, new), B.rows_of(B.v, cached, new)))
    pool0 = before(B)
    want, kh, vh = P8.append(pool0, k, v, B.table, B.kv_len, B.cu, page)
    pool, table, lens, cu = dev(pool0), dev(B.table), dev(B.kv_len), dev(B.cu)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    # rows behind the last request stay as they are
    kd, vd = (torch.cat([dev(x, dtype), torch.full((3, 2, d), 7.0, device="cuda").to(dev(x, dtype).dtype)]) for x in (k, v))
    gk, gv = torch.full_like(kd, 3.0), torch.full_like(vd, 3.0)
    paged.qwm_paged8_append(kd, vd, pool, table, lens, cu, k_hat=gk, v_hat=gv, status=status)
    assert int(status.item()) == 0
    assert np.array_equal(host(pool), want)
    for got, hat in ((gk, kh), (gv, vh)):
        assert np.array_equal(host(got)[: B.rows], hat) and (host(got)[B.rows:] == 3.0).all()
    # the step's tokens again, and every token of every request
    rk, rv = paged.qwm_paged8_read(pool, table, lens, cu, B.rows, d, dtype=kd.dtype, status=status)
    assert np.array_equal(host(rk), kh) and np.array_equal(host(rv), vh)
    all_cu = np.concatenate([[0], np.cumsum(B.kv_len)]).astype(np.int32)
    total = int(all_cu[-1])
    ok, ov = (torch.full((total + 2, 2, d), 5.0, dtype=kd.dtype, device="cuda") for _ in range(2))
    paged.qwm_paged8_read(pool, table, lens, dev(all_cu), total + 2, d, dtype=kd.dtype, k_out=ok, v_out=ov, status=status)
    for b, n in enumerate(B.kv_len):
        for h in range(2):
            a, c, _ = P8.gather(want, B.table[b], int(n), h, d, page)
            assert np.array_equal(host(ok)[all_cu[b]: all_cu[b + 1], h], a)
            assert np.array_equal(host(ov)[all_cu[b]: all_cu[b + 1], h], c)
    assert (host(ok)[total:] == 5.0).all() and int(status.item()) == 0


def test_append_token_by_token_and_views(paged):
    """A fused projection's views in, a [heads, rows, d] tensor out, a token at a
    time; the sizes grow, so that scales do."""
    d, page, hk, n = 128, 32, 3, 50
    r = np.random.default_rng(3)
    grow = 2.0 ** (np.arange(n) / 4.0)[:, None, None]
    k, v = (rounded(r.standard_normal((n, hk, d)) * 1e-3 * grow, "bf16") for _ in range(2))
    table = np.array([[2, 0]], np.int32)
    want = np.full((3, hk, P8.block_bytes(d, page)), 255, np.uint8)
    pool = dev(want)
    x = dev(np.concatenate([np.zeros_like(k), k, v], 1), "bf16")
    for i in range(n):
        want, kh, vh = P8.append(want, k[i: i + 1], v[i: i + 1], table, [i + 1], [0, 1], page)
        hat = torch.empty((2, hk, 1, d), dtype=torch.bfloat16, device="cuda")
        y = x[i: i + 1]
        paged.qwm_paged8_append(y[:, hk: 2 * hk], y[:, 2 * hk:], pool, dev(table), dev(np.array([i + 1], np.int32)),
                                dev(np.array([0, 1], np.int32)), k_hat=hat[0].transpose(0, 1), v_hat=hat[1].transpose(0, 1))
        assert np.array_equal(host(hat[0].transpose(0, 1)), kh) and np.array_equal(host(hat[1].transpose(0, 1)), vh), i
    assert np.array_equal(host(pool), want)
    ok, ov = (torch.empty((hk, n, d), device="cuda").transpose(0, 1) for _ in range(2))
    paged.qwm_paged8_read(pool, dev(table), dev(np.array([n], np.int32)), dev(np.array([0, n], np.int32)), n, d, dtype=torch.float32,
                          k_out=ok, v_out=ov)
    for h in range(hk):
        a, c, _ = P8.gather(want, table[0], n, h, d, page)
        assert np.array_equal(host(ok)[:, h], a) and np.array_equal(host(ov)[:, h], c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_of_nan_infinite_and_extreme_values(paged, dtype):
    d, page = 64, 16
    x = np.zeros((6, 1, d), np.float32)
    x[0, 0, :4] = np.nan, 1.0, -2.0, 3e-6
    x[1, 0, :3] = np.inf, -np.inf, 5.0
    x[2, 0, :3] = 57344.0, 60000.0, -1e30
    x[3, 0, :4] = 1e-40, -1e-40, 2.0 ** -24, -0.0
    x[4, 0] = 448.0 * 2.0 ** -15
    x[5, 0] = 449.0 * 2.0 ** -15
    x = rounded(x, dtype)
    table = np.arange(6, dtype=np.int32)[:, None]                # a request a row: scales do not mix
    lens, cu = np.ones(6, np.int32), np.arange(7, dtype=np.int32)
    empty = np.full((6, 1, P8.block_bytes(d, page)), 255, np.uint8)
    want, kh, _ = P8.append(empty, x, -x, table, lens, cu, page)
    pool, hat, status = dev(empty), torch.empty((6, 1, d), device="cuda", dtype=dev(x, dtype).dtype), torch.zeros(1, dtype=torch.int32, device="cuda")
    paged.qwm_paged8_append(dev(x, dtype), dev(-x, dtype), pool, dev(table), dev(lens), dev(cu), k_hat=hat, status=status)
    assert np.array_equal(host(pool), want) and np.array_equal(host(hat), kh)
    assert int(status.item()) == NAN | SATURATED


def test_bad_pages_lengths_and_offsets_are_passed_over(paged):
    B = Batch8(5, [20, 30, 3], [5, 40, 6], 2, 1, 64, 16, "f32")
    k, v = (B.rows_of(x, B.cached, B.new) for x in (B.k, B.v))
    n_pages = B.empty.shape[0]
    pool0 = before(B)
    for page_id in (-1, n_pages, 2 ** 31 - 1, -2 ** 31):
        table = B.table.copy()
        table[1, 3] = page_id                                    # tokens 48 to 63 of request 1
        want, kh, vh = P8.append(pool0, k, v, table, B.kv_len, B.cu, 16)
        pool, status = dev(pool0), torch.zeros(1, dtype=torch.int32, device="cuda")
        gk = torch.full((B.rows, 1, 64), 9.0, device="cuda")
        paged.qwm_paged8_append(dev(k), dev(v), pool, dev(table), dev(B.kv_len), dev(B.cu), k_hat=gk, status=status)
        assert np.array_equal(host(pool), want) and int(status.item()) == BOUNDS
        assert np.array_equal(np.where(np.isnan(kh), 9.0, kh), host(gk))
        status.zero_()
        rk, _ = paged.qwm_paged8_read(pool, dev(table), dev(B.kv_len), dev(B.cu), B.rows, 64, dtype=torch.float32, status=status)
        assert np.array_equal(np.where(np.isnan(kh), 0.0, kh), host(rk)) and int(status.item()) == BOUNDS
    # lengths and offsets out of range: reported, nothing outside the request's own pages is written
    for lens, cu in (([25, 2 ** 31 - 1, 9], B.cu), ([25, -7, 9], B.cu), ([25, 10, 9], B.cu), (B.kv_len, [0, 5, 2, 51]),
                     (B.kv_len, [-5, 5, 45, 51]), (B.kv_len, [0, 5, 45, 2 ** 31 - 1]), (B.kv_len, [0, 2 ** 31 - 1, -2 ** 31, 51])):
        pool, status = dev(pool0), torch.zeros(1, dtype=torch.int32, device="cuda")
        lens, cu = dev(np.array(lens, np.int32)), dev(np.array(cu, np.int32))
        paged.qwm_paged8_append(dev(k), dev(v), pool, dev(B.table), lens, cu, status=status)
        assert int(status.item()) == BOUNDS
        spare = sorted(set(range(n_pages)) - set(B.table.ravel().tolist()))
        assert (host(pool)[spare] == 255).all()
        status.zero_()
        paged.qwm_paged8_read(pool, dev(B.table), lens, cu, B.rows, 64, dtype=torch.float32, status=status)
        assert int(status.item()) == BOUNDS
        bnd = paged.paged8_page_bounds(n_pages, 1, 64)
        status.zero_()
        paged.qwm_paged8_bounds(pool, bnd, dev(B.table), lens, cu, max_new=40, status=status)
        assert int(status.item()) & BOUNDS
        status.zero_()
        paged.qwm_paged8_select(dev(B.q), bnd, dev(B.table), lens, cu, 16, 2, status=status)
        assert int(status.item()) & BOUNDS


@pytest.mark.parametrize("d,page,dtype", [(128, 16, "bf16"), (64, 64, "f32"), (128, 256, "bf16"), (64, 128, "bf16"), (128, 64, "bf16"),
                                          (64, 32, "bf16")])
@pytest.mark.parametrize("max_new", [None, 1, 0, 10 ** 6])
def test_bounds_match_the_oracle(paged, d, page, dtype, max_new):
    B = Batch8(6, [0, 70, 15, 300, 64], [0, 1, 2, 300, 90], 2, 2, d, page, dtype)
    old = np.random.default_rng(0).integers(0, 256, (B.empty.shape[0], 2, 2 * d + 16)).astype(np.uint8)
    want = P8.bounds(B.pool, old, B.table, B.kv_len, B.cu, page, d)
    got, status = dev(old), torch.zeros(1, dtype=torch.int32, device="cuda")
    paged.qwm_paged8_bounds(dev(B.pool), got, dev(B.table), dev(B.kv_len), dev(B.cu), max_new=300 if max_new is None else max_new,
                            status=status)
    assert np.array_equal(host(got), want) and int(status.item()) == 0
    # a page of zeros
    zero = P8.append(B.empty, 0 * B.k, 0 * B.v, B.table, B.kv_len, np.concatenate([[0], np.cumsum(B.kv_len)]), page)[0]
    paged.qwm_paged8_bounds(dev(zero), got, dev(B.table), dev(B.kv_len), dev(B.cu), max_new=1)
    assert np.array_equal(host(got), P8.bounds(zero, want, B.table, B.kv_len, B.cu, page, d))


def all_bounds(B):
    full = np.full((B.empty.shape[0], B.kv_heads, 2 * B.d + 16), 255, np.uint8)
    return P8.bounds(B.pool, full, B.table, B.kv_len, np.concatenate([[0], np.cumsum(B.kv_len)]), B.page, B.d)


@pytest.mark.parametrize("heads,kv_heads,d,page,dtype", [(6, 2, 128, 16, "bf16"), (3, 3, 64, 32, "f32"), (16, 1, 128, 16, "f32"),
                                                         (8, 4, 64, 16, "bf16")])
@pytest.mark.parametrize("cached,new", [([900, 0, 50, 333], [1, 1, 0, 1]), ([2100], [5]), ([700, 10, 400], [70, 3, 100]),
                                        ([255, 256, 257], [1, 1, 1])])
@pytest.mark.parametrize("width,sink", [(8, 0), (12, 2), (1, 0), (40, 1), (200, 3)])
def test_select_matches_the_oracle(paged, cached, new, heads, kv_heads, d, page, dtype, width, sink):
    B = Batch8(7, cached, new, heads, kv_heads, d, page, dtype)
    bnd = all_bounds(B)
    want, lens = P8.select(B.q, bnd, B.table, B.kv_len, B.cu, page, width, sink, d)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, gl = paged.qwm_paged8_select(dev(B.q, dtype), dev(bnd), dev(B.table), dev(B.kv_len), dev(B.cu), page, width, sink=sink,
                                      status=status)
    assert np.array_equal(host(gl), lens) and np.array_equal(host(got), want)
    over = any(n and -(-(c + n) // page) - c // page > width for c, n in zip(cached, new))
    assert int(status.item()) == (CAPACITY if over else 0)


def test_select_ties_signs_and_odd_queries(paged):
    """Equal scores go to the lower page, zeros of either sign are equal, queries
    of NaN and infinities count as the definition says; pages out of range and
    bounds that are NaN come last."""
    d, page, n = 64, 16, 16 * 60 + 1
    B = Batch8(8, [n - 1] * 4, [1] * 4, 4, 2, d, page, "f32")
    bnd = all_bounds(B)
    bnd[B.table[0]] = bnd[B.table[0, 0]]                          # every page of request 0 the same
    bnd[B.table[1, 7], :, 2 * d: 2 * d + 4] = np.array([np.nan], np.float32).view(np.uint8)
    bnd[B.table[1, 9:50], :, 2 * d: 2 * d + 4] = np.array([0.0], np.float32).view(np.uint8)
    q = B.q.copy()
    q[1, 0] = 0.0
    q[2, 0, :4] = np.nan, np.inf, -np.inf, 1e30
    q[2, 2] = np.nan
    q[3, 0] *= 1e-38
    q[3, 1] = 0.0
    q[3, 2:] = 2.0 ** -101
    for width, sink in ((20, 0), (59, 1), (60, 0), (2, 5)):
        with np.errstate(invalid="ignore"):
            want, lens = P8.select(q, bnd, B.table, B.kv_len, B.cu, page, width, sink, d)
        got, gl = paged.qwm_paged8_select(dev(q), dev(bnd), dev(B.table), dev(B.kv_len), dev(B.cu), page, width, sink=sink)
        for b in (0, 2, 3):
            assert np.array_equal(host(got)[b], want[b]), (width, sink, b)
        assert np.array_equal(host(gl), lens)
        if width < 60:
            assert B.table[1, 7] not in host(got)[1]
    table = B.table.copy()
    table[0, 3], table[0, 4] = -1, B.empty.shape[0]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, _ = paged.qwm_paged8_select(dev(q), dev(bnd), dev(table), dev(B.kv_len), dev(B.cu), page, 59, status=status)
    assert int(status.item()) == BOUNDS
    assert (host(got)[0] == np.concatenate([table[0, :3], table[0, 5:]])).all()


def test_select_over_a_long_table(paged):
    """More pages than the keys kept on chip (16,384), with scores spread wide."""
    d, hk, page, n_pages = 64, 1, 16, 20000
    r = np.random.default_rng(9)
    bnd = np.zeros((n_pages, hk, 2 * d + 16), np.uint8)
    bnd[..., : 2 * d] = r.integers(-127, 128, (n_pages, hk, 2 * d)).astype(np.int8).view(np.uint8)
    bnd[..., 2 * d: 2 * d + 4] = np.exp(3 * r.standard_normal((n_pages, hk, 1))).astype(np.float32).view(np.uint8)
    table = r.permutation(n_pages).astype(np.int32)[None]
    q = r.standard_normal((2, 2, d)).astype(np.float32)
    lens, cu = np.array([n_pages * page - 3], np.int32), np.array([0, 2], np.int32)
    for width in (1, 300, 19999):
        want, wl = P8.select(q, bnd, table, lens, cu, page, width, 1, d)
        got, gl = paged.qwm_paged8_select(dev(q), dev(bnd), dev(table), dev(lens), dev(cu), page, width, sink=1)
        assert np.array_equal(host(gl), wl) and np.array_equal(host(got), want)


def test_many_requests(paged):
    """8,192 requests, some without rows."""
    r = np.random.default_rng(10)
    n = 8192
    cached, new = r.integers(0, 40, n), r.integers(0, 3, n)
    new[:2] = 0, 1
    held = -(-(cached + new) // 16)
    table = np.full((n, 3), -1, np.int32)
    order = r.permutation(int(held.sum())).astype(np.int32)
    at = 0
    for b in range(n):
        table[b, : held[b]] = order[at: at + held[b]]
        at += held[b]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    rows = int(cu[-1])
    k, v = r.standard_normal((2, rows, 1, 64)).astype(np.float32)
    pool0 = np.zeros((order.size, 1, P8.block_bytes(64, 16)), np.uint8)
    pool0[:, :, -16:] = np.tile(np.array([2.0 ** -15], np.float16).view(np.uint8), 8)
    lens = (cached + new).astype(np.int32)
    want = P8.append(pool0, k, v, table, lens, cu, 16)
    pool, status = dev(pool0), torch.zeros(1, dtype=torch.int32, device="cuda")
    step = dev(table), dev(lens), dev(cu)
    paged.qwm_paged8_append(dev(k), dev(v), pool, *step, status=status)
    assert np.array_equal(host(pool), want[0])
    rk, rv = paged.qwm_paged8_read(pool, *step, rows, 64, dtype=torch.float32, status=status)
    assert np.array_equal(host(rk), want[1]) and np.array_equal(host(rv), want[2])
    old = np.zeros((order.size, 1, 144), np.uint8)
    bnd = dev(old)
    paged.qwm_paged8_bounds(pool, bnd, *step, max_new=2, status=status)
    assert np.array_equal(host(bnd), P8.bounds(want[0], old, table, lens, cu, 16, 64))
    q = r.standard_normal((rows, 2, 64)).astype(np.float32)
    pages, ls = paged.qwm_paged8_select(dev(q), bnd, *step, 16, 2, status=status)
    wp, wl = P8.select(q, host(bnd), table, lens, cu, 16, 2, 0, 64)
    assert np.array_equal(host(pages), wp) and np.array_equal(host(ls), wl) and int(status.item()) == 0
