"""qwm_paged8_attend on the GPU against the oracle, in all its kernels, over
tables of requests and of heads; and the 8-bit cache's calls together as a
serving loop, eager and captured."""
import numpy as np
import pytest
import torch

from oracle import paged8_oracle as P8
from paged8_cases import Batch8, attend8_tolerance
from test_gpu_paged8_cache import BOUNDS, all_bounds, dev, host, paged  # noqa: F401

pytestmark = pytest.mark.gpu

KERNELS = [1, 2, 3]


def run(paged, B, kernel, causal=True, window=0, pool=None, table=None, lens=None, scale=0.0, q=None, max_new=None, status=None):
    lse = torch.full((B.rows, B.heads), 99.0, device="cuda")
    o = paged.qwm_paged8_attend(dev(B.q if q is None else q, B.dtype), dev(B.pool if pool is None else pool),
                                dev(B.table if table is None else table), dev(B.kv_len if lens is None else lens), dev(B.cu),
                                max_new=max(B.new) if max_new is None else max_new, causal=causal, window=window, scale=scale, lse=lse,
                                kernel=kernel, status=status)
    return host(o), host(lse)


def check(paged, B, kernel, causal=True, window=0, table=None, lens=None, scale=0.0):
    sigma = scale or B.d ** -0.5
    table = B.table if table is None else table
    lens = B.kv_len if lens is None else lens
    O, lse, spread, vmax = P8.attend(B.q.astype(np.float64), B.pool, table, lens, B.cu, B.page, causal, window, sigma)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, gl = run(paged, B, kernel, causal, window, table=table, lens=lens, scale=scale, status=status)
    assert int(status.item()) == 0
    n = int(max(lens))
    tol = attend8_tolerance(O, spread, vmax, n, B.dtype, kernel != 1)
    assert (np.abs(got - O) <= tol).all(), np.max(np.abs(got - O) / tol)
    seen = np.isfinite(lse)
    assert np.array_equal(seen, np.isfinite(gl)) and (gl[~seen] == -np.inf).all()
    # log2 and the sum's roundings beside the logits'
    slack = 2 * spread * 131 * 2.0 ** -24 + (n + 300) * 2.0 ** -23 + 2.0 ** -20 + np.abs(np.where(seen, lse, 0)) * 2.0 ** -22
    assert (np.abs(np.where(seen, gl - lse, 0)) <= slack).all()


SHAPES = [([0], [1]), ([63], [1]), ([500, 0, 33, 128], [1, 1, 1, 0]), ([1000], [2]), ([0, 70, 1], [4, 3, 1]), ([5, 900], [30, 7]),
          ([0, 200], [129, 40]), ([300], [257]), ([0, 0, 9], [0, 1, 0])]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("heads,kv_heads,d,page", [(4, 2, 128, 16), (5, 1, 64, 32), (3, 3, 128, 128), (8, 1, 128, 64), (6, 2, 64, 256)])
@pytest.mark.parametrize("cached,new", SHAPES)
@pytest.mark.parametrize("mask", ["causal", "full", "window"])
def test_attend_matches_the_oracle(paged, kernel, heads, kv_heads, d, page, cached, new, mask):  # noqa: F811
    B = Batch8(1, cached, new, heads, kv_heads, d, page, "bf16")
    check(paged, B, kernel, causal=mask != "full", window=40 if mask == "window" else 0)


@pytest.mark.parametrize("kernel", [1, 2])
@pytest.mark.parametrize("heads,kv_heads,d,page", [(4, 2, 128, 16), (5, 1, 64, 32)])
@pytest.mark.parametrize("cached,new", SHAPES)
@pytest.mark.parametrize("mask", ["causal", "full", "window"])
def test_attend_in_float32(paged, kernel, heads, kv_heads, d, page, cached, new, mask):  # noqa: F811
    B = Batch8(2, cached, new, heads, kv_heads, d, page, "f32")
    check(paged, B, kernel, causal=mask != "full", window=17 if mask == "window" else 0, scale=0.2)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("cached,new,page", [([700, 300], [1, 1], 16), ([900], [5], 32), ([2000, 40], [150, 30], 64)])
def test_attend_over_a_table_of_each_head(paged, kernel, cached, new, page):  # noqa: F811
    B = Batch8(3, cached, new, 6, 3, 128, page, "bf16")
    width = 9
    table, lens = P8.select(B.q, all_bounds(B), B.table, B.kv_len, B.cu, page, width, 1, 128)
    assert (table[:, 0] != table[:, 1]).any()
    for causal in (True, False):
        check(paged, B, kernel, causal=causal, table=table, lens=lens)


@pytest.mark.parametrize("kernel", KERNELS)
def test_bytes_that_no_append_wrote_reach_no_row(paged, kernel):  # noqa: F811
    """Slots behind a request, and tokens hidden from a row, may hold anything:
    NaN codes, scales of NaN or infinity."""
    B = Batch8(4, [37, 100], [40, 60], 4, 2, 128, 32, "bf16")
    want, lse = run(paged, B, kernel)
    r = np.random.default_rng(0)
    pool = B.pool.copy()
    for b, n in enumerate(B.kv_len):                              # behind the last token: other garbage
        last = B.table[b, (n - 1) // 32]
        if n % 32:
            for half in (0, 1):
                for h in range(2):
                    P8.codes_of(pool[last, h], half, 128, 32)[n % 32:] = r.integers(0, 256, (32 - n % 32, 128))
    got, gl = run(paged, B, kernel, pool=pool)
    assert np.array_equal(got, want) and np.array_equal(gl, lse)
    # the last 16 tokens of request 1 are hidden from all rows but its last 16
    n = int(B.kv_len[1])
    for code, scale in ((0x7f, 1.0), (0xff, np.nan), (0x7e, np.inf), (0x55, -np.inf), (0x7e, 65504.0)):
        pool = B.pool.copy()
        for t in range(n - n % 16, n):
            pg = B.table[1, t // 32]
            for half in (0, 1):
                P8.codes_of(pool[pg, 0], half, 128, 32)[t % 32] = code
            P8.scales_of(pool[pg, 0], 128, 32)[t % 32 // 16] = scale
        got, gl = run(paged, B, kernel, pool=pool)
        rows = slice(0, B.rows - n % 16 if n % 16 else B.rows)
        assert np.array_equal(got[rows], want[rows]) and np.array_equal(gl[rows], lse[rows]), (code, scale)


@pytest.mark.parametrize("kernel", KERNELS)
def test_scales_at_both_ends_and_mixed(paged, kernel):  # noqa: F811
    """Blocks at 2^-15, at 2^7 and far apart from each other."""
    for ks, vs in ((2.0 ** -15, 2.0 ** -15), (1.0, 2.0 ** 7), (None, None)):
        B = Batch8(5, [200, 77], [1, 20], 4, 2, 128, 16, "bf16")
        r = np.random.default_rng(1)
        s = P8.scales_of
        for pg in range(B.pool.shape[0]):
            for h in range(2):
                if np.isfinite(s(B.pool[pg, h], 128, 16)[0, 0].astype(np.float64)):
                    s(B.pool[pg, h], 128, 16)[0] = (ks or 2.0 ** int(r.integers(-9, -5)), vs or 2.0 ** int(r.integers(-15, 8)))
        check(paged, B, kernel)


@pytest.mark.parametrize("kernel", KERNELS)
def test_rows_of_nan_and_pages_out_of_range(paged, kernel):  # noqa: F811
    B = Batch8(6, [100, 260], [3, 9], 4, 2, 128, 16, "bf16")
    clean, lse = run(paged, B, kernel)
    q = B.q.copy()
    q[4, 1, 7] = np.nan
    got, gl = run(paged, B, kernel, q=q)
    assert np.isnan(got[4, 1]).all() and np.isnan(gl[4, 1])
    keep = np.ones((B.rows, 4), bool)
    keep[4, 1] = False
    assert np.array_equal(got[keep], clean[keep]) and np.array_equal(gl[keep], lse[keep])
    for bad in (-1, B.pool.shape[0], 2 ** 31 - 1):
        table = B.table.copy()
        table[1, 5] = bad
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        O, wl, spread, vmax = P8.attend(B.q.astype(np.float64), B.pool, table, B.kv_len, B.cu, 16, True, 0, 128 ** -0.5)
        got, gl = run(paged, B, kernel, table=table, status=status)
        assert int(status.item()) == BOUNDS
        assert (np.abs(got - O) <= attend8_tolerance(O, spread, vmax, 300, "bf16", kernel != 1)).all()


@pytest.mark.parametrize("heads,kv_heads,d,page,cached,new", [(3, 1, 128, 64, [9000], [7]), (8, 2, 64, 16, [5000, 700], [40, 300]),
                                                              (1, 1, 128, 256, [0, 3000], [500, 1])])
def test_float32_of_any_size(paged, heads, kv_heads, d, page, cached, new):  # noqa: F811
    """Large, small and subnormal queries, rows of zeros: float32 on the tensor
    cores scales each row by a power of two."""
    B = Batch8(9, cached, new, heads, kv_heads, d, page, "f32")
    r = np.random.default_rng(3)
    B.q *= (2.0 ** r.integers(-8, 3, (B.rows, heads, 1))).astype(np.float32)
    B.q[0, 0] = 0.0
    B.q[B.rows - 1, 0] *= np.float32(1e-39)
    B.q[B.rows // 2, 0, 1:] *= np.float32(1e-6)                  # one channel far above the others
    check(paged, B, 2)


@pytest.mark.parametrize("cached,new,heads,kv_heads", [([9000], [1], 5, 1), ([20000], [3], 4, 2), ([6000, 10, 3000], [1, 1, 1], 8, 2),
                                                       ([5000], [300], 2, 1)])
def test_long_requests_are_split(paged, cached, new, heads, kv_heads):  # noqa: F811
    B = Batch8(7, cached, new, heads, kv_heads, 128, 64, "bf16")
    for kernel in KERNELS:
        check(paged, B, kernel)


def test_strided_and_in_place(paged):  # noqa: F811
    B = Batch8(8, [300, 64], [1, 4], 4, 2, 128, 32, "bf16")
    args = dev(B.pool), dev(B.table), dev(B.kv_len), dev(B.cu)
    want = paged.qwm_paged8_attend(dev(B.q, "bf16"), *args, max_new=4)
    wide = torch.full((B.rows + 2, 7, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[: B.rows, 1:5] = dev(B.q, "bf16")
    q = wide[:, 1:5]
    out = torch.full((4, B.rows + 2, 128), 5.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    paged.qwm_paged8_attend(q, *args, max_new=4, out=out)
    assert torch.equal(out[: B.rows], want) and bool((out[B.rows:] == 5.0).all())
    paged.qwm_paged8_attend(q, *args, max_new=4, out=q)
    assert torch.equal(wide[: B.rows, 1:5], want) and bool((wide[B.rows:] == 3.0).all()) and bool((wide[:, 0] == 3.0).all())


def loop(paged, sparse, dtype, capture):  # noqa: F811
    """Prompts, then single tokens and drafts, with a request cut back between; every
    output against the oracle."""
    r = np.random.default_rng(12)
    B, hq, hk, d, page, n_pages, width_t = 3, 4, 2, 64, 16, 60, 20
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pool = paged.paged8_pool(n_pages, hk, d, page)
    pool.fill_(255)
    bounds = paged.paged8_page_bounds(n_pages, hk, d)
    bounds.fill_(255)
    table = torch.full((B, width_t), -1, dtype=torch.int32, device="cuda")
    free, count, lens = torch.randperm(n_pages, device="cuda").int(), i32([n_pages]), i32([0] * B)
    ref, ref_b = host(pool), host(bounds)
    status = i32([0])
    steps = [[70, 33, 1], [1, 1, 1], [1, 5, 1], [1, 1, 0], [40, 1, 90], [1, 1, 1], [1, 1, 1]]
    rows = max(sum(s) for s in steps)
    new_t = i32([0] * B)
    x = torch.zeros((rows, hq + 2 * hk, d), dtype=tdt, device="cuda")
    got = {}
    width = 8

    def step():
        plan = paged.qwm_paged_plan(lens, new_t, table, free, count, page, rows, status=status)
        kh = torch.zeros((rows, hk, d), dtype=tdt, device="cuda")
        paged.qwm_paged8_append(x[:, hq:hq + hk], x[:, hq + hk:], pool, table, plan.kv_len, plan.cu_rows, k_hat=kh, status=status)
        t, n = table, plan.kv_len
        if sparse:
            paged.qwm_paged8_bounds(pool, bounds, table, plan.kv_len, plan.cu_rows, max_new=90, status=status)
            t, n = paged.qwm_paged8_select(x[:, :hq], bounds, table, plan.kv_len, plan.cu_rows, page, width, sink=1, status=status)
        o = torch.zeros((rows, hq, d), dtype=tdt, device="cuda")
        paged.qwm_paged8_attend(x[:, :hq], pool, t, n, plan.cu_rows, max_new=90, out=o, status=status)
        got.update(plan=plan, kh=kh, t=t, n=n, o=o)

    graph = None
    if capture:
        step()                                                    # nothing new: a warm-up that changes nothing
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    for i, new in enumerate(steps):
        new_t.copy_(i32(new))
        x.copy_(torch.from_numpy(r.standard_normal(x.shape).astype(np.float32)).to(tdt))
        graph.replay() if capture else step()
        torch.cuda.synchronize()
        plan, T = got["plan"], sum(new)
        tb, n, cu = host(table), host(plan.kv_len), host(plan.cu_rows)
        y = host(x).astype(np.float64)
        ref, kh, _ = P8.append(ref, y[:T, hq:hq + hk], y[:T, hq + hk:], tb, n, cu, page)
        assert np.array_equal(host(pool), ref) and np.array_equal(host(got["kh"])[:T], kh), i
        if sparse:
            ref_b = P8.bounds(ref, ref_b, tb, n, cu, page, d)
            assert np.array_equal(host(bounds), ref_b), i
            wt, wn = P8.select(y[:T, :hq], ref_b, tb, n, cu, page, width, 1, d)
            assert np.array_equal(host(got["t"]), wt) and np.array_equal(host(got["n"]), wn), i
            tb, n = wt, wn
        O, _, spread, vmax = P8.attend(y[:T, :hq], ref, tb, n, cu, page, True, 0, d ** -0.5)
        tol = attend8_tolerance(O, spread, vmax, int(max(n)), dtype, True)
        assert (np.abs(host(got["o"])[:T] - O) <= tol).all(), i
        assert (host(got["o"])[T:] == 0).all()
        lens.copy_(plan.kv_len), count.copy_(plan.free_count)
        if i == 3:                                                # request 0 gives up 30 tokens, request 2 ends
            keep = host(lens) - np.array([30, 0, host(lens)[2]])
            paged.qwm_paged_release(i32(keep.tolist()), lens, table, free, count, page, status=status)
    assert int(status.item()) == 0


@pytest.mark.parametrize("capture", [False, True])
@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_serving_loop(paged, sparse, dtype, capture):  # noqa: F811
    loop(paged, sparse, dtype, capture)


def test_two_streams_and_two_graphs(paged):  # noqa: F811
    """Steps of two pools at once on two streams, and replayed from two graphs,
    give what each gives alone."""
    cases = [Batch8(20, [3000, 50], [1, 1], 8, 2, 128, 64, "bf16"), Batch8(21, [2500, 700], [1, 1], 8, 2, 128, 64, "bf16")]
    state = []
    for B in cases:
        s = dict(q=dev(B.q, "bf16"), pool=dev(B.pool), table=dev(B.table), lens=dev(B.kv_len), cu=dev(B.cu), bounds=dev(all_bounds(B)))
        state.append(s)

    def step(s):
        paged.qwm_paged8_bounds(s["pool"], s["bounds"], s["table"], s["lens"], s["cu"])
        t, n = paged.qwm_paged8_select(s["q"], s["bounds"], s["table"], s["lens"], s["cu"], 64, 10)
        return paged.qwm_paged8_attend(s["q"], s["pool"], t, n, s["cu"], max_new=1), \
            paged.qwm_paged8_attend(s["q"], s["pool"], s["table"], s["lens"], s["cu"], max_new=1)

    want = [step(s) for s in state]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in state]
    graphs = []
    for s in state:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = step(s)
        graphs.append((g, o))
    for _ in range(5):
        got = []
        for s, st in zip(state, streams):
            with torch.cuda.stream(st):
                got.append(step(s))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        for (g, o), st in zip(graphs, streams):
            for x in o:
                x.zero_()
        torch.cuda.synchronize()
        for (g, o), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for (g, o), b in zip(graphs, want):
            assert torch.equal(o[0], b[0]) and torch.equal(o[1], b[1])
