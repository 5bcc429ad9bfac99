"""qwm_paged_plan, qwm_paged_release, qwm_paged_append and qwm_qk_norm_rope on
the GPU against the oracle, and the four calls together as a serving loop."""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from paged_cases import EPS2, Batch, attend_tolerance, bf16, rounded

pytestmark = pytest.mark.gpu


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
    return t.cpu().numpy()


def layout(seed, cached, page, width, spare):
    r = np.random.default_rng(seed)
    held = [-(-int(c) // page) for c in cached]
    order = r.permutation(sum(held) + spare).astype(np.int32)
    table = np.full((len(held), width), -1, np.int32)
    at = 0
    for b, m in enumerate(held):
        table[b, :m] = order[at: at + m]
        at += m
    free = np.full(order.size, -1, np.int32)
    free[:spare] = order[at:]
    return table, free


@pytest.mark.parametrize("requests,page,most,pad", [(1, 16, 1, 0), (1, 64, 700, 3), (48, 16, 1, 16), (48, 128, 300, 0),
                                                    (240, 32, 60, 100), (1025, 16, 9, 7), (3000, 256, 4, 1),
                                                    (8192, 16, 3, 5)])
def test_plan_matches_the_oracle(paged, requests, page, most, pad):
    r = np.random.default_rng(requests)
    cached, new = r.integers(0, 500, requests), r.integers(0, most + 1, requests)
    width = -(-(500 + most) // page) + 2
    need = sum(-(-(int(c) + int(m)) // page) - -(-int(c) // page) for c, m in zip(cached, new))
    table, free = layout(3, cached, page, width, need + 5)
    rows = int(new.sum()) + pad
    want = P.plan(cached, new, table, free, need + 5, page, rows)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = dev(table)
    fp, fc, kl = dev(free), dev(np.array([need + 5], np.int32)), dev(cached.astype(np.int32))
    got = paged.qwm_paged_plan(kl, dev(new.astype(np.int32)), t, fp, fc, page, rows, status=status)
    assert int(status.item()) == 0
    assert np.array_equal(host(got.kv_len), want[0]) and int(got.free_count.item()) == want[1]
    for a, b in zip((got.cu_rows, got.slots, got.positions, t), want[2:]):
        assert np.array_equal(host(a), b)
    assert np.array_equal(host(fp), free) and int(fc.item()) == need + 5 and np.array_equal(host(kl), cached)
    # in place, as a serving loop runs it
    t2 = dev(table)
    out = paged.PagedPlan(kl, fc, got.cu_rows, got.slots, got.positions)
    paged.qwm_paged_plan(kl, dev(new.astype(np.int32)), t2, fp, fc, page, rows, out=out)
    assert np.array_equal(host(kl), want[0]) and int(fc.item()) == want[1] and torch.equal(t, t2)
    assert np.array_equal(host(out.slots), want[3])


@pytest.mark.parametrize("why,status_bit", [("pages", 0x20), ("rows", 0x20), ("width", 0x20), ("negative", 0x8), ("count", 0x8)])
def test_plan_that_does_not_fit_changes_nothing(paged, why, status_bit):
    cached, new, page = np.array([20, 0, 64], np.int32), np.array([30, 9, 1], np.int32), 16
    table, free = layout(1, cached, page, 6, 8)
    rows, count = 60, 8
    if why == "pages":
        count = 3           # 2 + 1 + 1 are needed
    if why == "rows":
        rows = 39
    if why == "width":
        table = table[:, :4].copy()
    if why == "negative":
        new[1] = -1
    if why == "count":
        count = free.size + 1
    t, fc, kl = dev(table), dev(np.array([count], np.int32)), dev(cached)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = paged.qwm_paged_plan(kl, dev(new), t, dev(free), fc, page, rows, status=status)
    assert int(status.item()) == status_bit
    assert np.array_equal(host(t), table) and np.array_equal(host(got.kv_len), cached)
    assert int(got.free_count.item()) == count
    assert (got.slots == -1).all() and (got.positions == -1).all() and (got.cu_rows == 0).all()


def test_plan_with_a_bad_page_gives_its_rows_no_slot(paged):
    cached, new, page = np.array([20, 3], np.int32), np.array([20, 2], np.int32), 16
    table, free = layout(1, cached, page, 6, 4)
    free[3] = 999                       # the first page handed out
    table[1, 0] = -7
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = dev(table)
    got = paged.qwm_paged_plan(dev(cached), dev(new), t, dev(free), dev(np.array([4], np.int32)), page, 22, status=status)
    assert int(status.item()) == 8 and int(t[0, 2].item()) == -1
    slots = host(got.slots)
    assert (slots[:12] >= 0).all() and (slots[12:] == -1).all()
    assert np.array_equal(host(got.positions), [*range(20, 40), 3, 4])


@pytest.mark.parametrize("requests,page", [(1, 16), (7, 64), (1300, 16), (8192, 32)])
def test_release_and_plan_again(paged, requests, page):
    r = np.random.default_rng(requests)
    cached = r.integers(0, 300, requests).astype(np.int32)
    keep = np.where(r.random(requests) < 0.5, 0, (cached * r.random(requests)).astype(np.int32)).astype(np.int32)
    keep[-1] = cached[-1]
    table, free = layout(2, cached, page, -(-300 // page), 3)
    want = P.release(keep, cached, table, free, 3, page)
    kl, t, fp, fc = dev(cached), dev(table), dev(free), dev(np.array([3], np.int32))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(2):                  # the second call has nothing left to do
        paged.qwm_paged_release(dev(keep), kl, t, fp, fc, page, status=status)
        assert int(status.item()) == 0
        assert np.array_equal(host(kl), want[0]) and np.array_equal(host(t), want[1])
        assert int(fc.item()) == want[3] and np.array_equal(host(fp)[: want[3]], want[2][: want[3]])
    new = np.full(requests, 2, np.int32)
    p = P.plan(want[0], new, want[1], want[2], want[3], page, 2 * requests)
    got = paged.qwm_paged_plan(kl, dev(new), t, fp, fc, page, 2 * requests)
    assert (p is None) == bool((got.slots == -1).all())
    if p is not None:
        assert np.array_equal(host(got.slots), p[3])


def test_release_refuses_what_is_out_of_range(paged):
    cached, page = np.array([40, 20, 10], np.int32), 16
    table, free = layout(2, cached, page, 4, 1)
    kl, t, fp, fc = dev(cached), dev(table), dev(free), dev(np.array([1], np.int32))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    paged.qwm_paged_release(dev(np.array([41, -1, 10], np.int32)), kl, t, fp, fc, page, status=status)
    assert int(status.item()) == 8
    assert np.array_equal(host(kl), cached) and np.array_equal(host(t), table) and int(fc.item()) == 1
    # more pages than the pool has: nothing changes
    status.zero_()
    fc.fill_(free.size)
    paged.qwm_paged_release(dev(np.zeros(3, np.int32)), kl, t, fp, fc, page, status=status)
    assert int(status.item()) == 0x20 and np.array_equal(host(kl), cached) and np.array_equal(host(t), table)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,page,rows", [(1, 16, 1), (3, 16, 50), (8, 64, 33), (2, 256, 300)])
def test_append_is_bit_exact(paged, dtype, d, heads, page, rows):
    """Bytes of the pool against the oracle's, rows without a slot and slots
    without a row left as they were, and x_hat."""
    r = np.random.default_rng(rows + heads)
    k = rounded(r.standard_normal((rows, heads, d)) * np.exp(r.standard_normal((heads, d))), dtype)
    v = rounded(r.standard_normal((rows, heads, d)), dtype)
    k[0, 0, :32] = 1.5                          # a constant group: scale 0
    v[0, 0, :32] = np.arange(32) % 2 * 15       # codes exactly 0 and 15
    v[-1, -1, -32:] = rounded(r.standard_normal(32) * 1e-7, dtype)   # subnormal parameters
    k[-1, -1, -32:] = np.arange(32) - 7.5 if dtype == "f32" else (np.arange(32) - 8)   # ties among the codes
    n_pages = -(-rows // page) + 2
    slots = r.permutation(n_pages * page)[:rows].astype(np.int64)
    if rows > 4:
        slots[2] = -1
        slots[rows // 2] = -(1 << 40)
    pool = r.integers(0, 256, (n_pages, heads, P.block_offsets(d, page)["bytes"])).astype(np.uint8)
    want = pool.copy()
    for i in range(rows):
        if slots[i] >= 0:
            for h in range(heads):
                P.write_slot(want, int(slots[i]), h, k[i, h], v[i, h], d, page)
    got = dev(pool)
    kh, vh = (torch.full((rows, heads, d), 9.0, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda") for _ in "kv")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    paged.qwm_paged_append(dev(k, dtype), dev(v, dtype), got, dev(slots), k_hat=kh, v_hat=vh, status=status)
    assert int(status.item()) == 0
    assert np.array_equal(host(got), want)
    for x, hat in ((k, kh), (v, vh)):
        c, z, s = P.quantize_int4(x)
        xh = P.dequantize_int4(c, z, s)
        xh[slots < 0] = 0
        # one rounding to float32 (the sum), one to the dtype
        assert (np.abs(host(hat.float()) - xh) <= (EPS2["f32"] + (EPS2[dtype] if dtype == "bf16" else 0)) * 1.01 * np.abs(xh)).all()
    again = dev(pool)
    paged.qwm_paged_append(dev(k, dtype), dev(v, dtype), again, dev(slots))     # without x_hat
    assert torch.equal(again, got)


def test_append_of_what_float16_cannot_hold(paged):
    """NaN becomes 0, infinities and large values +-60000, with status bits;
    the stored values are finite in float16."""
    r = np.random.default_rng(5)
    base = r.standard_normal((4, 2, 128)).astype(np.float32)
    k, v = base.copy(), base[::-1].copy()
    k[0, 0, 3], k[1, 1, 40] = np.nan, np.inf
    v[2, 0, 5], v[2, 0, 6], v[3, 1, 100] = -np.inf, np.inf, 3e38
    k[3, 0, :32] = 60000.0
    k[3, 0, 1] = -60000.0
    slots = np.arange(4, dtype=np.int64) + 7
    pool = np.zeros((1, 2, P.block_offsets(128, 16)["bytes"]), np.uint8)
    for what, expect in ((k, 0x12), (v, 0x2), (base, 0)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = dev(pool)
        paged.qwm_paged_append(dev(what), dev(base), got, dev(slots), status=status)
        assert int(status.item()) == expect
        want = pool.copy()
        for i in range(4):
            for h in range(2):
                P.write_slot(want, int(slots[i]), h, what[i, h], base[i, h], 128, 16)
        assert np.array_equal(host(got), want)
        for h in range(2):
            assert all(np.abs(x).max() <= 65504 for x in P.read_block(host(got)[0, h], 128, 16))


def test_append_strides_and_slots_out_of_range(paged):
    """Views of one fused tensor, head-major x_hat; a slot behind the pool
    stores nothing and is reported."""
    r = np.random.default_rng(6)
    fused = dev(r.standard_normal((9, 8, 128)).astype(np.float32), "bf16")
    k, v = fused[:, 2:4], fused[:, 6:8]
    slots = np.array([0, 5, 31, 32, 16, 2, 3, 1 << 40, -1], np.int64)
    pool = torch.zeros((2, 2, P.block_offsets(128, 16)["bytes"]), dtype=torch.uint8, device="cuda")
    hm = torch.zeros((2, 9, 128), dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    paged.qwm_paged_append(k, v, pool, dev(slots), k_hat=hm.transpose(0, 1), status=status)
    assert int(status.item()) == 8
    ref = torch.zeros_like(pool)
    keep = slots.copy()
    keep[(slots >= 32)] = -1
    kh = torch.empty((9, 2, 128), dtype=torch.bfloat16, device="cuda")
    paged.qwm_paged_append(k.contiguous(), v.contiguous(), ref, dev(keep), k_hat=kh)
    assert torch.equal(ref, pool) and torch.equal(hm.transpose(0, 1), kh)
    assert (kh[3] == 0).all() and (kh[7:] == 0).all()


# ------------------------------------------------------------------ norm and rotation
def rope_table(n, rot, base=10000.0):
    inv = base ** (-np.arange(0, rot, 2) / rot)
    ang = np.arange(n)[:, None] * inv[None]
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def rope_tolerance(y, dtype):
    """|out - exact|: the norm's factor is off by (d + 6) 2^-24 at most (d
    squares, the mean, the root, the reciprocal), x' by two more roundings, a
    rotation by three roundings of terms not larger than |x'_a| + |x'_b|; then
    one rounding to the dtype."""
    big = np.abs(y).max(-1, keepdims=True)
    return 2 * 140 * EPS2["f32"] * big + EPS2[dtype] * np.abs(y) + (1e-30 if dtype == "f32" else 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot,axes,interleaved", [(128, 128, 1, False), (128, 64, 1, False), (128, 128, 3, False),
                                                    (64, 64, 1, True), (64, 16, 1, True), (128, 32, 2, False),
                                                    (128, 128, 4, True), (64, 48, 3, False)])
@pytest.mark.parametrize("rows,heads,kv_heads", [(1, 1, 1), (13, 24, 8), (40, 5, 1)])
def test_norm_and_rotation(paged, dtype, d, rot, axes, interleaved, rows, heads, kv_heads):
    r = np.random.default_rng(rows * d + rot)
    q, k = (rounded(r.standard_normal((rows, h, d)) * 1.7, dtype) for h in (heads, kv_heads))
    wq, wk = (rounded(1 + 0.2 * r.standard_normal(d), dtype) for _ in "qk")
    table = rope_table(5000, rot)
    pos = r.integers(0, 5000, (rows, axes)).astype(np.int32)
    cut = np.sort(r.integers(0, rot // 2 + 1, axes - 1))
    sections = np.diff(np.concatenate([[0], cut, [rot // 2]])).astype(int)
    axis = np.repeat(np.arange(axes), sections)
    a, b = paged.qwm_qk_norm_rope(dev(q, dtype), dev(k, dtype), dev(wq, dtype), dev(wk, dtype), dev(table), dev(pos),
                                  eps=1e-5, interleaved=interleaved, sections=list(sections))
    for got, x, w in ((a, q, wq), (b, k, wk)):
        want = P.norm_rope(x, w, table, pos, axis, 1e-5, interleaved)
        assert (np.abs(host(got.float()) - want) <= rope_tolerance(want, dtype)).all()


def test_norm_and_rotation_without_weights_keys_or_copies(paged):
    """No weight, no keys, [rows] positions, views, in place, padding rows."""
    r = np.random.default_rng(3)
    x = rounded(r.standard_normal((11, 9, 128)), "bf16")
    table = rope_table(100, 128)
    pos = r.integers(0, 100, 11).astype(np.int32)
    pos[4], pos[9] = -1, 100
    fused = dev(x, "bf16")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k = fused[:, :6], fused[:, 6:8]
    paged.qwm_qk_norm_rope(q, k, None, None, dev(table), dev(pos), q_out=q, k_out=k, status=status)
    assert int(status.item()) == 8
    want = P.norm_rope(x[:, :8], None, table, np.clip(pos, 0, 99)[:, None], np.zeros(64, int), 1e-6, False)
    got = host(fused.float())
    real = (pos >= 0) & (pos < 100)
    assert (np.abs(got[real][:, :8] - want[real]) <= rope_tolerance(want, "bf16")[real]).all()
    assert np.array_equal(got[~real], x[~real]) and np.array_equal(got[:, 8], x[:, 8])
    one, none = paged.qwm_qk_norm_rope(dev(x, "bf16"), None, None, None, dev(table), dev(np.clip(pos, 0, 99)))
    assert none is None and torch.equal(one[real][:, :8], fused[torch.from_numpy(real).cuda()][:, :8])


def test_norm_of_extreme_rows(paged):
    """A zero row stays zero; one of large values does not overflow what
    float32 holds (squares of 1e15)."""
    x = np.zeros((2, 1, 128), np.float32)
    x[1] = 1e15
    table = rope_table(4, 128)
    got, _ = paged.qwm_qk_norm_rope(dev(x), None, None, None, dev(table), dev(np.zeros(2, np.int32)))
    assert (host(got)[0] == 0).all()
    assert np.abs(host(got)[1] - 1.0).max() <= 2 * 140 * EPS2["f32"]


# ------------------------------------------------------------------ the four together
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [0, 24])
def test_serving_loop(paged, dtype, window):
    """Prompts, single tokens, a request that ends and one that takes its
    place, padded rows in every step: each step's attention against the oracle
    over the pages as they are, and the pages against the oracle's bytes."""
    r = np.random.default_rng(17)
    B, hq, hk, d, page, rows, width = 3, 6, 2, 128, 16, 64, 8
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    n_pages = 14
    pool = torch.full((n_pages, hk, paged.qwm_paged_block_bytes(d, page)), 255, dtype=torch.uint8, device="cuda")
    ref_pool = host(pool)
    table = np.full((B, width), -1, np.int32)
    free, count, lens = r.permutation(n_pages).astype(np.int32), n_pages, np.zeros(B, np.int64)
    t, fp, fc, kl = dev(table), dev(free), dev(np.array([count], np.int32)), dev(lens.astype(np.int32))
    cs = rope_table(300, d)
    wq, wk = (rounded(1 + 0.1 * r.standard_normal(d), dtype) for _ in "qk")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for new, keep in (([30, 17, 0], None), ([1, 1, 12], None), ([1, 1, 1], None), ([2, 0, 1], [0, 19, 9]), ([20, 1, 40], None)):
        if keep is not None:
            lens, table, free, count = P.release(keep, lens, table, free, count, page)
            paged.qwm_paged_release(dev(np.array(keep, np.int32)), kl, t, fp, fc, page, status=status)
        lens, count, cu, slots, positions, table = P.plan(lens, new, table, free, count, page, rows)
        plan = paged.qwm_paged_plan(kl, dev(np.array(new, np.int32)), t, fp, fc, page, rows, status=status)
        kl, fc = plan.kv_len, plan.free_count
        assert np.array_equal(host(kl), lens) and np.array_equal(host(plan.slots), slots) and np.array_equal(host(t), table)
        x = dev(rounded(r.standard_normal((rows, hq + 2 * hk, d)), dtype), dtype)
        q, k = paged.qwm_qk_norm_rope(x[:, :hq], x[:, hq:hq + hk], dev(wq, dtype), dev(wk, dtype), dev(cs), plan.positions,
                                      q_out=torch.zeros((rows, hq, d), dtype=td, device="cuda"),
                                      k_out=torch.zeros((rows, hk, d), dtype=td, device="cuda"), status=status)
        used = int(cu[-1])
        want_q = P.norm_rope(host(x[:used, :hq].float()), wq, cs, positions[:used, None], np.zeros(d // 2, int), 1e-6, False)
        assert (np.abs(host(q[:used].float()) - want_q) <= rope_tolerance(want_q, dtype)).all() and (q[used:] == 0).all()
        paged.qwm_paged_append(k, x[:, hq + hk:], pool, plan.slots, status=status)
        kn, vn = host(k.float()), host(x[:, hq + hk:].float())
        for i in range(used):
            for h in range(hk):
                P.write_slot(ref_pool, int(slots[i]), h, kn[i, h], vn[i, h], d, page)
        assert np.array_equal(host(pool), ref_pool)
        o = paged.qwm_paged_attend(q, pool, t, plan.kv_len, plan.cu_rows, max_new=max(new), window=window, status=status)
        O, _, spread, vmax = P.attend(host(q[:used].float()).astype(np.float64), ref_pool, table, lens, cu, page, True, window, d ** -0.5)
        tol = attend_tolerance(O, spread, vmax, int(lens.max()), dtype, dtype == "bf16")
        assert (np.abs(host(o[:used].float()) - O) <= tol).all()
    assert int(status.item()) == 0


def test_step_captured_into_a_graph(paged):
    """The four calls captured once and replayed for several decode steps,
    updating lengths and pages in place, give what eager calls give."""
    def state():
        g = torch.Generator(device="cuda").manual_seed(3)
        pool = torch.full((20, 2, paged.qwm_paged_block_bytes(64, 16)), 255, dtype=torch.uint8, device="cuda")
        s = {"pool": pool, "t": torch.full((4, 6), -1, dtype=torch.int32, device="cuda"),
             "fp": torch.randperm(20, generator=g, device="cuda").int(), "fc": torch.tensor([20], dtype=torch.int32, device="cuda"),
             "kl": torch.zeros(4, dtype=torch.int32, device="cuda"), "new": torch.tensor([1, 1, 0, 1], dtype=torch.int32, device="cuda"),
             "x": torch.zeros((6, 8, 64), dtype=torch.bfloat16, device="cuda"),
             "out": torch.zeros((6, 4, 64), dtype=torch.bfloat16, device="cuda"), "cs": dev(rope_table(100, 64))}
        s["plan"] = paged.PagedPlan(s["kl"], s["fc"], *(torch.zeros(n, dtype=dt, device="cuda")
                                                       for n, dt in ((5, torch.int32), (6, torch.int64), (6, torch.int32))))
        return s

    def step(s):
        p = paged.qwm_paged_plan(s["kl"], s["new"], s["t"], s["fp"], s["fc"], 16, 6, out=s["plan"])
        x = s["x"]
        q, k = paged.qwm_qk_norm_rope(x[:, :4], x[:, 4:6], None, None, s["cs"], p.positions, q_out=x[:, :4], k_out=x[:, 4:6])
        paged.qwm_paged_append(k, x[:, 6:], s["pool"], p.slots)
        paged.qwm_paged_attend(q, s["pool"], s["t"], p.kv_len, p.cu_rows, max_new=1, out=s["out"])

    xs = [torch.randn((6, 8, 64), generator=torch.Generator(device="cuda").manual_seed(i), device="cuda").bfloat16() for i in range(40)]
    a, b = state(), state()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step(b)
    for x in xs:
        a["x"].copy_(x)
        step(a)
        b["x"].copy_(x)
        g.replay()
        for key in ("pool", "t", "kl", "fc", "out"):
            assert torch.equal(a[key], b[key]), key
    assert host(a["kl"]).tolist() == [40, 40, 0, 40]


def test_diagnostics_measure_the_paged_encoding(paged):
    """The attention-shift diagnostics' INT4 entry against the oracle's own
    quantiser on the same keys, values and queries."""
    from bit_kv_cache_qwm_gb300 import diagnostics
    r = np.random.default_rng(8)
    K, V = (rounded(r.standard_normal((2, 300, 128)), "bf16") for _ in "kv")
    q = r.standard_normal((2, 20, 128)).astype(np.float32)
    got = diagnostics.measure_paged(dev(K), dev(V), dev(q), 128 ** -0.5)
    k64, v64, q64 = K.astype(np.float64), V.astype(np.float64), q.astype(np.float64)
    kh, vh = (P.dequantize_int4(*P.quantize_int4(x)) for x in (K, V))
    rel = lambda a, b: np.sqrt(((a - b) ** 2).sum() / (b ** 2).sum())  # noqa: E731
    L, Lq = q64 @ k64.swapaxes(1, 2), q64 @ kh.swapaxes(1, 2)
    soft = lambda x: np.exp(x - x.max(-1, keepdims=True)) / np.exp(x - x.max(-1, keepdims=True)).sum(-1, keepdims=True)  # noqa: E731
    O, Oq = soft(L / 128 ** 0.5) @ v64, soft(Lq / 128 ** 0.5) @ vh
    for key, want in (("key_rel_error", rel(kh, k64)), ("value_rel_error", rel(vh, v64)), ("logit_rel_error", rel(Lq, L)),
                      ("output_rel_error", rel(Oq, O))):
        assert got[key] == pytest.approx(want, rel=1e-3), key
    assert abs(got["top1_change"] - (L.argmax(-1) != Lq.argmax(-1)).mean()) <= 1 / 40


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_calls_that_follow_without_a_pause(paged, dtype):
    """The kernels of a step are placed on the GPU while the one ahead runs out:
    prompts and decode steps through four layers give the same bits whether the
    host waits after every call, never, or replays captured steps."""
    B, hq, hk, d, page, layers = 8, 8, 2, 128, 16, 4
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(5)
    xs = {n: torch.randn((layers, n, hq + 2 * hk, d), generator=g, device="cuda").to(td) for n in (B * 150, B)}
    cs = dev(rope_table(300, d))
    i32 = dict(dtype=torch.int32, device="cuda")

    def state():
        return {"pool": [torch.full((120, hk, paged.qwm_paged_block_bytes(d, page)), 255, dtype=torch.uint8, device="cuda")
                         for _ in range(layers)],
                "t": torch.full((B, 16), -1, **i32), "fp": torch.arange(120, **i32), "fc": torch.tensor([120], **i32),
                "kl": torch.zeros(B, **i32), "plan": {n: (torch.zeros(B + 1, **i32), torch.zeros(n, dtype=torch.int64, device="cuda"),
                                                          torch.zeros(n, **i32)) for n in xs}}

    def step(s, n, wait=lambda: None):
        new = torch.full((B,), n // B, **i32)
        p = paged.qwm_paged_plan(s["kl"], new, s["t"], s["fp"], s["fc"], page, n, out=paged.PagedPlan(s["kl"], s["fc"], *s["plan"][n]))
        wait()
        y = 0
        for x, pool in zip(xs[n], s["pool"]):
            x = x + y
            q, k = paged.qwm_qk_norm_rope(x[:, :hq], x[:, hq:hq + hk], None, None, cs, p.positions)
            wait()
            paged.qwm_paged_append(k, x[:, hq + hk:], pool, p.slots)
            wait()
            o = paged.qwm_paged_attend(q, pool, s["t"], p.kv_len, p.cu_rows, max_new=n // B)
            wait()
            y = torch.cat([o, o[:, :2 * hk]], 1)
        return o

    a, b, c = state(), state(), state()
    torch.cuda.synchronize()
    want = [step(a, n, torch.cuda.synchronize).clone() for n in [B * 150] + [B] * 20]
    got = [step(b, n).clone() for n in [B * 150] + [B] * 20]
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    step(c, B * 150)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        out = step(c, B)
    for x in want[1:]:
        graph.replay()
        assert torch.equal(out, x)
    for s in (b, c):
        assert torch.equal(s["kl"], a["kl"]) and all(torch.equal(x, y) for x, y in zip(s["pool"], a["pool"]))


def test_behind_copies_fills_and_other_streams(paged):
    """What stands ahead of a call on its stream may be a copy, a fill, or work
    of another stream that it waits for, captured or not."""
    T, hq, hk, d, page = 300, 4, 2, 64, 32
    r = torch.Generator(device="cuda").manual_seed(9)
    src = [torch.randn((T, hq + 2 * hk, d), generator=r, device="cuda").bfloat16() for _ in range(4)]
    pinned = [x.cpu().pin_memory() for x in src]
    cs = dev(rope_table(T, d))
    i32 = dict(dtype=torch.int32, device="cuda")
    width = -(-T // page)
    x = torch.zeros_like(src[0])
    v = torch.zeros((T, hk, d), dtype=torch.bfloat16, device="cuda")
    pool = paged.paged_pool(width, hk, d, page)
    table, out = torch.arange(width, **i32)[None].contiguous(), torch.zeros((T, hq, d), dtype=torch.bfloat16, device="cuda")
    kl, cu, pos = torch.tensor([T], **i32), torch.tensor([0, T], **i32), torch.arange(T, **i32)
    slots = torch.arange(T, device="cuda")
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def step(copy):
        side.wait_stream(main)
        copy()
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000)
            v.copy_(x[:, hq + hk:])
        q, k = paged.qwm_qk_norm_rope(x[:, :hq], x[:, hq:hq + hk], None, None, cs, pos)
        pool.zero_()
        main.wait_stream(side)
        paged.qwm_paged_append(k, v, pool, slots)
        out.zero_()
        paged.qwm_paged_attend(q, pool, table, kl, cu, max_new=T, out=out)

    want = []
    for y in src:
        q, k = paged.qwm_qk_norm_rope(y[:, :hq], y[:, hq:hq + hk], None, None, cs, pos)
        torch.cuda.synchronize()
        p = torch.zeros_like(pool)
        paged.qwm_paged_append(k, y[:, hq + hk:].contiguous(), p, slots)
        torch.cuda.synchronize()
        want.append(paged.qwm_paged_attend(q, p, table, kl, cu, max_new=T))
    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        for y, w in zip(pinned, want):
            def copy():
                x.copy_(y, non_blocking=True)
                side.wait_stream(main)
            step(copy)
            assert torch.equal(out, w)
    torch.cuda.synchronize()
    feed = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        def copy():
            x.copy_(feed)
            side.wait_stream(main)
        step(copy)
    for y, w in zip(src, want):
        feed.copy_(y)
        graph.replay()
        assert torch.equal(out, w)
