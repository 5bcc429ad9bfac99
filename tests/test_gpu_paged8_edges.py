"""The 8-bit cache's calls at the edge of what they promise."""
import numpy as np
import pytest
import torch

from oracle import paged8_oracle as P8
from paged8_cases import Batch8, attend8_tolerance
from test_gpu_paged8_cache import all_bounds, dev, host, paged  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ waits that run out
@pytest.mark.parametrize("limit", [0, 300, 3000, 30000])
@pytest.mark.parametrize("cached,new,d", [([3000, 500], [300, 100], 128), ([9000], [130], 64)])
def test_a_wait_that_runs_out(paged, monkeypatch, limit, cached, new, d):  # noqa: F811
    """The bounded waits of the tcgen05 kernels limited to so few cycles that some
    may run out: the calls end, the attention's rows are what they were or NaN, the
    selection still names pages of the request, the status bit says whether any
    wait ran out, and the next calls are whole again."""
    B = Batch8(1, cached, new, 8, 4, d, 16, "bf16")
    q, pool, bnd = dev(B.q, "bf16"), dev(B.pool), dev(all_bounds(B))
    step = dev(B.table), dev(B.kv_len), dev(B.cu)
    status = i32([0])

    def select():
        return paged.qwm_paged8_select(q, bnd, *step, 16, 30, status=status)

    def attend():
        lse = torch.empty(B.rows, 8, device="cuda")
        o = paged.qwm_paged8_attend(q, pool, *step, max_new=max(new), lse=lse, status=status, kernel=paged.PAGED_TC)
        torch.cuda.synchronize()
        return o, lse

    want, (ref, ref_lse) = select(), attend()
    assert int(status.item()) == 0
    monkeypatch.setenv("QWM_FAULT_INJECT", f"wait={limit}")
    pages, lens = select()
    bits = int(status.item())
    assert bits in (0, 4)       # a wait that has ended at its first look does not run out
    status.zero_()
    out, lse = attend()
    monkeypatch.delenv("QWM_FAULT_INJECT")
    lost = torch.isnan(lse)
    assert torch.isnan(out[lost].float()).all() and torch.equal(out[~lost], ref[~lost])
    assert int(status.item()) in ((4,) if lost.any() else (0, 4))
    assert torch.equal(lens, want[1])
    got = host(pages)
    for b in range(len(cached)):
        held = -(-(cached[b] + new[b]) // 16)
        for h in range(4):
            mine = got[b, h][got[b, h] >= 0].tolist()
            assert len(mine) == min(30, held) and set(mine) <= set(B.table[b, :held].tolist())
    if bits == 0:
        assert torch.equal(pages, want[0])
    status.zero_()
    again, (out, lse) = select(), attend()
    assert torch.equal(again[0], want[0]) and torch.equal(out, ref) and torch.equal(lse, ref_lse) and int(status.item()) == 0


# ------------------------------------------------------------------ offsets beyond 32 bits
@pytest.mark.parametrize("page", [16, 256])
def test_pool_beyond_4_gib(paged, page):  # noqa: F811
    """Pages at the far end of a pool of more than 2^32 bytes."""
    d, hk = 128, 8
    block = P8.block_bytes(d, page)
    n_pages = (1 << 32) // (block * hk) + 40
    B = Batch8(2, [300, 40], [20, 1], 16, hk, d, page, "bf16")
    used = B.empty.shape[0]
    far = n_pages - used                                          # page p of the batch is page far + p
    assert far * hk * block > 1 << 32
    pool = torch.empty((n_pages, hk, block), dtype=torch.uint8, device="cuda")
    pool[:40].fill_(255)
    before = P8.append(B.empty, B.rows_of(B.k, [0, 0], B.cached), B.rows_of(B.v, [0, 0], B.cached), B.table, B.cached,
                       np.concatenate([[0], np.cumsum(B.cached)]), page)[0]
    pool[far:] = dev(before)
    table = np.where(B.table >= 0, B.table + far, -1).astype(np.int32)
    step = dev(table), dev(B.kv_len), dev(B.cu)
    k, v = (B.rows_of(x, B.cached, B.new) for x in (B.k, B.v))
    status = i32([0])
    paged.qwm_paged8_append(dev(k, "bf16"), dev(v, "bf16"), pool, *step, status=status)
    want, kh, vh = P8.append(before, k, v, B.table, B.kv_len, B.cu, page)
    assert np.array_equal(host(pool[far:]), want) and bool((pool[:40] == 255).all())
    rk, rv = paged.qwm_paged8_read(pool, *step, B.rows, d, status=status)
    assert np.array_equal(host(rk), kh) and np.array_equal(host(rv), vh)
    bnd = paged.paged8_page_bounds(n_pages, hk, d)
    bnd[far:] = dev(P8.bounds(before, np.zeros((used, hk, 2 * d + 16), np.uint8), B.table, np.array(B.cached),
                              np.concatenate([[0], np.cumsum(B.cached)]), page, d))
    paged.qwm_paged8_bounds(pool, bnd, *step, max_new=20, status=status)
    pages, lens = paged.qwm_paged8_select(dev(B.q, "bf16"), bnd, *step, page, 4, sink=1, status=status)
    wp, wl = P8.select(B.q, host(bnd[far:]), B.table, B.kv_len, B.cu, page, 4, 1, d)
    assert np.array_equal(host(lens), wl) and np.array_equal(host(pages), np.where(wp >= 0, wp + far, -1))
    O, _, spread, vmax = P8.attend(B.q.astype(np.float64), want, B.table, B.kv_len, B.cu, page, True, 0, d ** -0.5)
    for kernel in (1, 2, 3):
        o = paged.qwm_paged8_attend(dev(B.q, "bf16"), pool, *step, max_new=20, status=status, kernel=kernel)
        assert (np.abs(host(o) - O) <= attend8_tolerance(O, spread, vmax, 320, "bf16", kernel != 1)).all()
    assert int(status.item()) == 0


# ------------------------------------------------------------------ shapes of calls
def test_no_rows(paged):  # noqa: F811
    """Tensors without rows, and steps that bring none."""
    B = Batch8(3, [40, 9], [0, 0], 4, 2, 64, 16, "bf16")
    step, pool, bnd = (dev(B.table), dev(B.kv_len), dev(B.cu)), dev(B.pool), dev(all_bounds(B))
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    status = i32([0])
    for rows in (0, 3):
        kv = torch.zeros((rows, 2, 64), dtype=torch.bfloat16, device="cuda")
        qq = torch.ones((rows, 4, 64), dtype=torch.bfloat16, device="cuda")
        hat = torch.full_like(kv, 5.0)
        paged.qwm_paged8_append(kv, kv, pool, *step, k_hat=hat, status=status)
        assert np.array_equal(host(pool), B.pool) and bool((hat == 5.0).all())
        rk, _ = paged.qwm_paged8_read(pool, *step, rows, 64, k_out=hat, status=status)
        assert rk is hat and bool((hat == 5.0).all())
        paged.qwm_paged8_bounds(pool, bnd, *step, status=status)
        assert np.array_equal(host(bnd), all_bounds(B))
        pages, lens = paged.qwm_paged8_select(qq, bnd, *step, 16, 2, status=status)
        assert bool((pages == -1).all()) and bool((lens == 0).all())
        out = torch.full_like(qq, 7.0)
        paged.qwm_paged8_attend(qq, pool, pages, lens, step[2], max_new=1, out=out, status=status)
        assert bool((out == 7.0).all())
    assert paged.qwm_paged8_attend(q, pool, *step).shape == (0, 4, 64) and none.shape[0] == 0
    assert int(status.item()) == 0


def test_a_row_of_length_one_and_queries_before_the_first_token(paged):  # noqa: F811
    """A request that brings more rows than it has tokens: the rows ahead of its
    first token see nothing, and are reported by the calls that write or read them."""
    B = Batch8(4, [0], [1], 4, 2, 128, 16, "bf16")
    cu = i32([0, 4])
    q = torch.randn((4, 4, 128), device="cuda").bfloat16()
    status = i32([0])
    for kernel in (1, 2, 3):
        lse = torch.zeros((4, 4), device="cuda")
        o = paged.qwm_paged8_attend(q, dev(B.pool), dev(B.table), dev(B.kv_len), cu, max_new=4, lse=lse, kernel=kernel)
        assert bool((o[:3] == 0).all()) and bool((lse[:3] == -np.inf).all()) and bool(torch.isfinite(lse[3]).all())
        _, v, _ = P8.gather(B.pool, B.table[0], 1, 0, 128, 16)
        assert np.array_equal(host(o[3, 0]), v[0])
    rk, _ = paged.qwm_paged8_read(dev(B.pool), dev(B.table), dev(B.kv_len), cu, 4, 128, status=status)
    assert int(status.item()) == 8 and bool((rk[:3] == 0).all())
    assert np.array_equal(host(rk[3, 1]), P8.gather(B.pool, B.table[0], 1, 1, 128, 16)[0][0])


def test_more_rows_than_tokens_among_single_tokens(paged):  # noqa: F811
    """The same where the calls go row by row."""
    B = Batch8(14, [0, 5, 40, 31], [1, 1, 2, 1], 4, 2, 64, 16, "f32")
    cu = np.array([0, 3, 4, 6, 7], np.int32)                      # request 0 has one token and three rows
    table, lens = B.table, B.kv_len
    r = np.random.default_rng(1)
    k, v = r.standard_normal((2, 7, 2, 64)).astype(np.float32)
    want, kh, vh = P8.append(B.pool, k, v, table, lens, cu, 16)
    pool, status = dev(B.pool), i32([0])
    hat = torch.full((7, 2, 64), 9.0, device="cuda")
    paged.qwm_paged8_append(dev(k), dev(v), pool, dev(table), dev(lens), dev(cu), k_hat=hat, status=status)
    assert np.array_equal(host(pool), want) and int(status.item()) == 8
    assert np.array_equal(host(hat), np.where(np.isnan(kh), 9.0, kh))
    _, rv = paged.qwm_paged8_read(pool, dev(table), dev(lens), dev(cu), 7, 64, dtype=torch.float32)
    assert np.array_equal(host(rv), np.where(np.isnan(vh), 0.0, vh))


@pytest.mark.parametrize("kernel", [1, 2, 3])
def test_all_pages_selected_is_the_whole_attention(paged, kernel):  # noqa: F811
    B = Batch8(5, [500, 33, 1200], [3, 40, 1], 8, 2, 128, 32, "bf16")
    step, pool = (dev(B.table), dev(B.kv_len), dev(B.cu)), dev(B.pool)
    q = dev(B.q, "bf16")
    width = B.table.shape[1] + 3
    pages, lens = paged.qwm_paged8_select(q, dev(all_bounds(B)), *step, 32, width)
    assert torch.equal(lens, step[1])
    a = paged.qwm_paged8_attend(q, pool, *step, max_new=40, kernel=kernel)
    b = paged.qwm_paged8_attend(q, pool, pages, lens, step[2], max_new=40, kernel=kernel)
    assert torch.equal(a, b)


def test_a_shared_prefix_and_a_step_in_two_calls(paged):  # noqa: F811
    """Two requests that begin with the same pages read them like any other; a step
    of single tokens and a prompt in a call each gives what one call gives."""
    B = Batch8(6, [128, 128, 700], [1, 1, 90], 6, 2, 128, 64, "bf16")
    table = B.table.copy()
    table[1, :2] = table[0, :2]
    q, pool, bnd = dev(B.q, "bf16"), dev(B.pool), dev(all_bounds(B))
    lens, cu = dev(B.kv_len), dev(B.cu)
    O, _, spread, vmax = P8.attend(B.q.astype(np.float64), B.pool, table, B.kv_len, B.cu, 64, True, 0, 128 ** -0.5)
    out = torch.empty_like(q)
    for a, b, most in ((0, 2, 1), (2, 3, 90)):
        paged.qwm_paged8_attend(q, pool, dev(table[a:b]), lens[a:b], cu[a:b + 1], max_new=most, out=out)
    assert (np.abs(host(out) - O) <= attend8_tolerance(O, spread, vmax, 790, "bf16", True)).all()
    rk, _ = paged.qwm_paged8_read(pool, dev(table[:2]), lens[:2], i32([0, 129, 258]), 258, 128)
    assert torch.equal(rk[:128], rk[129:257])
    whole = paged.qwm_paged8_select(q, bnd, dev(table), lens, cu, 64, 4)
    for a, b in ((0, 2), (2, 3)):
        part = paged.qwm_paged8_select(q, bnd, dev(table[a:b]), lens[a:b], cu[a:b + 1], 64, 4)
        assert torch.equal(part[0], whole[0][a:b]) and torch.equal(part[1], whole[1][a:b])


def test_a_request_cut_back_inside_a_block(paged):  # noqa: F811
    """Tokens appended behind a cut keep to the block's scale where earlier tokens
    are left in it, and start anew where none are; the bounds forget what was cut."""
    d, page = 64, 16
    r = np.random.default_rng(7)
    table = np.array([[1, 0, 2]], np.int32)
    pool0 = np.full((3, 1, P8.block_bytes(d, page)), 255, np.uint8)
    big = (100 * r.standard_normal((40, 1, d))).astype(np.float32)
    small = (0.01 * r.standard_normal((10, 1, d))).astype(np.float32)
    first = P8.append(pool0, big, big, table, [40], [0, 40], page)[0]
    for keep in (32, 35, 16, 0):
        n = keep + 10
        want, kh, _ = P8.append(first, small, small, table, [n], [0, 10], page)
        pool, hat = dev(first), torch.empty((10, 1, d), device="cuda")
        step = dev(table), i32([n]), i32([0, 10])
        paged.qwm_paged8_append(dev(small), dev(small), pool, *step, k_hat=hat)
        assert np.array_equal(host(pool), want) and np.array_equal(host(hat), kh)
        bnd = torch.zeros((3, 1, 2 * d + 16), dtype=torch.uint8, device="cuda")
        paged.qwm_paged8_bounds(pool, bnd, *step, max_new=10)
        assert np.array_equal(host(bnd), P8.bounds(want, np.zeros((3, 1, 2 * d + 16), np.uint8), table, [n], [0, 10], page, d))


def test_calls_on_a_side_stream(paged):  # noqa: F811
    B = Batch8(8, [400], [30], 8, 2, 128, 64, "bf16")
    q, pool, bnd = dev(B.q, "bf16"), dev(B.pool), dev(all_bounds(B))
    step = dev(B.table), dev(B.kv_len), dev(B.cu)

    def work():
        p, n = paged.qwm_paged8_select(q, bnd, *step, 64, 4)
        return p, n, paged.qwm_paged8_attend(q, pool, p, n, step[2], max_new=30), paged.qwm_paged8_read(pool, *step, B.rows, 128)[0]

    want = work()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = work()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_selection_into_its_own_inputs(paged):  # noqa: F811
    """pages and lens in the memory of the table, the lengths, the first rows or one
    another are refused; neighbours of them in one allocation are not."""
    B = Batch8(3, [200], [1], 2, 1, 64, 16, "bf16")
    q, bnd = dev(B.q, "bf16"), dev(all_bounds(B))
    n = B.table.shape[1]
    mem = torch.zeros(2 * n + 8, dtype=torch.int32, device="cuda")
    table, lens, cu = mem[:n].view(1, n), mem[n:n + 1], mem[n + 1:n + 3]
    table.copy_(dev(B.table)), lens.copy_(dev(B.kv_len)), cu.copy_(dev(B.cu))
    want, want_len = paged.qwm_paged8_select(q, bnd, table, lens, cu, 16, 4)
    before = mem.clone()
    free = mem[n + 3:]
    for kw in (dict(pages=mem[:4].view(1, 1, 4)), dict(pages=mem[n - 1:n + 3].view(1, 1, 4)),
               dict(pages=mem[n + 2:n + 6].view(1, 1, 4)), dict(lens=lens), dict(lens=mem[3:4]), dict(lens=cu[1:]),
               dict(pages=free[:4].view(1, 1, 4), lens=free[3:4])):
        with pytest.raises(ValueError, match="memory of its own"):
            paged.qwm_paged8_select(q, bnd, table, lens, cu, 16, 4, **kw)
    assert torch.equal(mem, before)
    got, got_len = paged.qwm_paged8_select(q, bnd, table, lens, cu, 16, 4, pages=free[:4].view(1, 1, 4), lens=free[4:5])
    assert torch.equal(got, want) and torch.equal(got_len, want_len) and torch.equal(mem[:n + 3], before[:n + 3])


@pytest.mark.parametrize("dtype,kernel", [("bf16", 1), ("bf16", 2), ("bf16", 3), ("f32", 1), ("f32", 2)])
def test_results_do_not_depend_on_the_run(paged, dtype, kernel):  # noqa: F811
    B = Batch8(9, [5000, 10, 300], [9, 2, 40], 8, 2, 64, 32, dtype)
    args = dev(B.q, dtype), dev(B.pool), dev(B.table), dev(B.kv_len), dev(B.cu)
    ref = paged.qwm_paged8_attend(*args, max_new=40, kernel=kernel)
    for _ in range(5):
        assert torch.equal(paged.qwm_paged8_attend(*args, max_new=40, kernel=kernel), ref)


@pytest.mark.parametrize("cached,new,d", [([9000], [130], 64), ([12000, 300, 5000], [300, 20, 90], 128)])
def test_selections_do_not_depend_on_the_run(paged, cached, new, d):  # noqa: F811
    """Several tiles of pages and of rows, often, alone and beside another stream's
    work that moves the warps' timing."""
    B = Batch8(10, cached, new, 8, 4, d, 16, "bf16")
    q, bnd = dev(B.q, "bf16"), dev(all_bounds(B))
    step = dev(B.table), dev(B.kv_len), dev(B.cu)
    want, _ = P8.select(B.q, host(bnd), B.table, B.kv_len, B.cu, 16, 30, 1, d)
    noise, side = torch.randn(2048, 2048, device="cuda"), torch.cuda.Stream()
    for i in range(60):
        if i % 2:
            with torch.cuda.stream(side):
                noise = torch.tanh(noise @ noise)
        got, _ = paged.qwm_paged8_select(q, bnd, *step, 16, 30, sink=1)
        assert np.array_equal(host(got), want), i


def test_diagnostics_of_the_8_bit_cache(paged):  # noqa: F811
    """Errors of the read-back values against the oracle's encoding, and the weight
    in the selected pages: all of it in all pages, a share of it in fewer."""
    from bit_kv_cache_qwm_gb300 import diagnostics
    r = np.random.default_rng(11)
    H, N, d, page = 2, 333, 64, 32
    K, V = (r.standard_normal((H, N, d)).astype(np.float32) for _ in range(2))
    q = r.standard_normal((H, 5, d)).astype(np.float32)
    got = diagnostics.measure_paged8(dev(K), dev(V), dev(q), d ** -0.5, page_tokens=page, widths=(3, 11))
    _, kh, vh = P8.append(np.full((11, H, P8.block_bytes(d, page)), 255, np.uint8), K.transpose(1, 0, 2), V.transpose(1, 0, 2),
                          np.arange(11)[None], [N], [0, N], page)
    for key, a, b in (("key_rel_error", kh, K), ("value_rel_error", vh, V)):
        b = b.transpose(1, 0, 2)
        assert got[key] == pytest.approx(np.linalg.norm(a - b) / np.linalg.norm(b), rel=1e-4)
    # three pages (the last holds 13 tokens) are 77 of 333 tokens: no even share is known beforehand
    assert got["weight_in_11_pages"] == pytest.approx(1.0, abs=1e-5) and 0 < got["weight_in_3_pages"] < 1
