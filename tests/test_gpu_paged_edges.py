"""The paged calls on inputs at the edge of what they promise."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from paged_cases import Batch, attend_tolerance, rounded
from test_gpu_paged_attend import KERNELS, dev, kid
from test_gpu_paged_cache import host, rope_table, rope_tolerance

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def paged():
    from bit_kv_cache_qwm_gb300 import build
    build.build()
    from bit_kv_cache_qwm_gb300 import paged as p
    return p


# ------------------------------------------------------------------ rows that are not finite
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("cached,new", [([70, 300], 1), ([70, 300], 40), ([9000, 40], 2), ([9000, 40], 70)])
def test_lse_of_a_row_of_nan(paged, kernel, cached, new):
    """-inf is the lse of a row that sees nothing; that of a row of NaN is NaN,
    whether its item is cut or not, and its neighbours' are what they were."""
    bt = Batch(33, cached, [new, new], 6, 2, 128, 16)
    args = (dev(bt.pool), dev(bt.table), dev(bt.kv_len), dev(bt.cu))
    q = dev(bt.q, "bf16")
    ref, got = (torch.zeros(bt.rows, 6, device="cuda") for _ in range(2))
    paged.qwm_paged_attend(q, *args, max_new=new, kernel=kid(paged, kernel), lse=ref)
    q[0, 1, 5] = float("nan")
    q[-1, 4, 100] = float("nan")
    out = paged.qwm_paged_attend(q, *args, max_new=new, kernel=kid(paged, kernel), lse=got)
    for row in ((0, 1), (bt.rows - 1, 4)):
        assert torch.isnan(got[row]) and torch.isnan(out[row].float()).all()
        got[row] = ref[row]
    assert torch.equal(got, ref) and torch.isfinite(ref).all()


# ------------------------------------------------------------------ waits that run out
@pytest.mark.parametrize("limit", [0, 300, 3000, 30000, 300000])
@pytest.mark.parametrize("cached,new,heads,kv_heads,d", [([100, 0, 300, 20], [300, 513, 257, 700], 24, 24, 64),
                                                         ([20000], [40], 8, 1, 128), ([0, 50], [900, 1500], 32, 4, 128)])
def test_a_wait_that_runs_out_leaves_rows_of_nan(paged, monkeypatch, limit, cached, new, heads, kv_heads, d):
    """The bounded waits of the tcgen05 kernel limited to so few cycles that
    some may run out: the call ends, a row is what it was or NaN throughout,
    the status bit says whether any is, and the next call is whole again."""
    bt = Batch(37, cached, new, heads, kv_heads, d, 32)
    q, args = dev(bt.q, "bf16"), (dev(bt.pool), dev(bt.table), dev(bt.kv_len), dev(bt.cu))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run():
        lse = torch.empty(bt.rows, heads, device="cuda")
        out = paged.qwm_paged_attend(q, *args, max_new=max(new), lse=lse, status=status, kernel=paged.PAGED_TC)
        torch.cuda.synchronize()
        return out, lse

    ref, ref_lse = run()
    assert int(status.item()) == 0
    monkeypatch.setenv("QWM_FAULT_INJECT", f"wait={limit}")
    out, lse = run()
    monkeypatch.delenv("QWM_FAULT_INJECT")
    lost = torch.isnan(lse)
    if limit == 0:
        assert lost.any()
    assert torch.isnan(out[lost].float()).all()
    assert torch.equal(out[~lost], ref[~lost]) and torch.equal(lse[~lost], ref_lse[~lost])
    assert int(status.item()) in ((4,) if lost.any() else (0, 4))
    status.zero_()
    out, lse = run()
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse) and int(status.item()) == 0


# ------------------------------------------------------------------ size of the queries
def check_size(paged, bt, kernel, scale):
    """O and lse of a batch against the oracle.  O's bound is attend_tolerance.
    A logit is off by delta = spread (131 2^-24 + 1.01 2^-11 for the tensor
    kernels, whose k_hat is float16) as derived there, and so is the log-sum-exp
    of logits; beside it the exponentials and the sum (n + 200 roundings), and
    (m + log2 l) ln 2 with m and log2 l rounded: 4 2^-24 |lse|."""
    q = dev(bt.q, "bf16")
    lse = torch.full((bt.rows, bt.heads), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = paged.qwm_paged_attend(q, dev(bt.pool), dev(bt.table), dev(bt.kv_len), dev(bt.cu), max_new=max(bt.new), scale=scale,
                                 lse=lse, status=status, kernel=kernel)
    O, want, spread, vmax = P.attend(bt.q.astype(np.float64), bt.pool, bt.table, bt.kv_len, bt.cu, bt.page, True, 0, scale)
    n, tensor = int(bt.kv_len.max()), kernel != paged.PAGED_SIMT
    with np.errstate(over="ignore"):
        tol = attend_tolerance(O, spread, vmax, n, "bf16", tensor)
    got, l = host(out.float()).astype(np.float64), host(lse).astype(np.float64)
    assert np.isfinite(got).all() and (np.abs(got - O) <= tol).all()
    delta = spread * (131 * 2.0 ** -24 + (1.01 * 2.0 ** -11 if tensor else 0))
    assert (np.abs(l - want) <= delta + np.abs(want) * 2.0 ** -22 + (n + 200) * 2.0 ** -22).all()
    return int(status.item())


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sigma,scale", [(1e-4, 1e3), (1e-6, 1e5), (1e-8, 1e7), (1e-20, 1e19), (1e-38, 1e37)])
def test_small_queries(paged, kernel, d, sigma, scale):
    """Queries far below float16's range (the last partly below float32's
    normal one) with a scale that brings the logits back."""
    bt = Batch(30, [100, 30, 200], [20, 1, 150], 4, 2, d, 16, q_sigma=sigma)
    assert check_size(paged, bt, kid(paged, kernel), scale=scale) == 0


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("scale", [1e-2])
def test_large_normal_small_and_zero_queries_in_one_batch(paged, kernel, scale):
    """Each row's size is its own: rows of 1e5, 1, 1e-5, 1e-9 and 0 beside one
    another, and one large channel among small ones."""
    bt = Batch(31, [100, 30], [40, 300], 4, 2, 128, 16)
    size = np.array([1e5, 1.0, 1e-5, 1e-9, 0.0])[np.random.default_rng(0).integers(0, 5, (bt.rows, 4, 1))]
    bt.q = rounded(bt.q * size, "bf16")
    bt.q[::7, :, 5] = 100.0
    assert check_size(paged, bt, kid(paged, kernel), scale=scale) == 0


@pytest.mark.parametrize("kernel", KERNELS)
def test_zero_queries_and_a_small_scale(paged, kernel):
    """A row of zeros weighs what it sees evenly, whatever the scale."""
    bt = Batch(32, [70, 20], [5, 200], 4, 2, 64, 16)
    bt.q[:] = 0
    for scale in (1e-30, 1.0, 1e30):
        assert check_size(paged, bt, kid(paged, kernel), scale=scale) == 0


# ------------------------------------------------------------------ request counts
def test_plan_at_every_size_of_its_shared_memory():
    """A plan's prefix sums take 12 bytes a request beside the kernel's own
    shared memory: counts around 48 KB, smaller ones first, in a process of its
    own (a larger call before would have raised the limit)."""
    code = """
import numpy as np, torch
from bit_kv_cache_qwm_gb300 import build, paged
from oracle import paged_oracle as P
build.build()
i32 = dict(dtype=torch.int32, device="cuda")
for n in (4052, 4053, 4095, 4096, 4097, 8192):
    for in_place in (False, True):
        r = np.random.default_rng(n)
        new = r.integers(0, 3, n).astype(np.int32)
        free = r.permutation(n).astype(np.int32)
        rows = int(new.sum()) + 3
        table = np.full((n, 1), -1, np.int32)
        want = P.plan(np.zeros(n, np.int64), new, table, free, n, 16, rows)
        t, kl, fc = torch.from_numpy(table).cuda(), torch.zeros(n, **i32), torch.tensor([n], **i32)
        out = paged.PagedPlan(kl, fc, torch.empty(n + 1, **i32), torch.empty(rows, dtype=torch.int64, device="cuda"),
                              torch.empty(rows, **i32)) if in_place else None
        got = paged.qwm_paged_plan(kl, torch.from_numpy(new).cuda(), t, torch.from_numpy(free).cuda(), fc, 16, rows, out=out)
        for a, b in zip((got.kv_len, got.free_count, got.cu_rows, got.slots, got.positions, t), want):
            assert np.array_equal(a.cpu().numpy().ravel(), np.ravel(b)), n
print("done")
"""
    res = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert res.returncode == 0 and res.stdout.strip() == "done", res.stderr[-2000:]


# ------------------------------------------------------------------ tokens that a row does not see
# (zero, scale) in float16 that no append writes: NaN, infinite, and finite ones
# whose values leave float16
BAD_PARAMS = [(np.nan, np.nan), (np.inf, 1.0), (-np.inf, 0.0), (0.0, np.inf), (1.0, np.nan), (60000.0, 60000.0)]


def spoil(bt, b, token, pair):
    """Every parameter of one token of a request becomes `pair`; its codes stay."""
    off, w = P.block_offsets(bt.d, bt.page), bt.d // 32
    pg, s = bt.table[b, token // bt.page], token % bt.page
    raw = np.tile(np.array(pair, np.float16), w).view(np.uint8)
    for o in (off["kqp"], off["vqp"]):
        bt.pool[pg, :, o + s * 4 * w: o + (s + 1) * 4 * w] = raw


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("pair", BAD_PARAMS)
def test_hidden_tokens_have_no_effect(paged, kernel, d, pair):
    """Bytes that no append writes, in tokens that one row sees and another does
    not (behind a causal row, left of a window): the rows that do not see them
    keep their bits."""
    k = kid(paged, kernel)
    for new, window, token, hidden in ((33, 0, 110, range(10)), (300, 0, 390, range(290)), (5, 0, 103, range(3)),
                                       (33, 20, 95, range(15, 33)), (300, 130, 101, range(131, 300)),
                                       (4, 90, 11, range(1, 4))):
        bt = Batch(34, [100, 40], [new, 3], 4, 2, d, 16)
        q, args = dev(bt.q, "bf16"), (dev(bt.table), dev(bt.kv_len), dev(bt.cu))
        f = lambda: paged.qwm_paged_attend(q, dev(bt.pool), *args, max_new=new, window=window, kernel=k)  # noqa: E731
        ref = f()
        spoil(bt, 0, token, pair)
        got = f()
        same = list(hidden) + list(range(new, bt.rows))
        assert torch.equal(got[same], ref[same]), (new, window)


@pytest.mark.parametrize("pair", BAD_PARAMS)
def test_hidden_tokens_have_no_effect_in_float32(paged, pair):
    for new, window, token, hidden in ((33, 0, 110, range(10)), (70, 20, 95, range(15, 70))):
        bt = Batch(35, [100, 40], [new, 3], 4, 2, 64, 16, dtype="f32")
        q, args = dev(bt.q, "f32"), (dev(bt.table), dev(bt.kv_len), dev(bt.cu))
        f = lambda: paged.qwm_paged_attend(q, dev(bt.pool), *args, max_new=new, window=window)  # noqa: E731
        ref = f()
        spoil(bt, 0, token, pair)
        got = f()
        same = list(hidden) + list(range(new, bt.rows))
        assert torch.equal(got[same], ref[same])


@pytest.mark.parametrize("kernel", KERNELS)
def test_a_long_decode_step_with_a_spoilt_token_of_another_row(paged, kernel):
    """Drafts over a long request: the last draft token's bytes reach no row
    before it, in cut items too."""
    bt = Batch(36, [9000], [4], 8, 2, 128, 64)
    q, args = dev(bt.q, "bf16"), (dev(bt.table), dev(bt.kv_len), dev(bt.cu))
    f = lambda: paged.qwm_paged_attend(q, dev(bt.pool), *args, max_new=4, kernel=kid(paged, kernel))  # noqa: E731
    ref = f()
    spoil(bt, 0, 9003, (np.nan, np.nan))
    assert torch.equal(f()[:3], ref[:3])


# ------------------------------------------------------------------ norm and rotation of what is not finite
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot,interleaved", [(128, 64, False), (128, 32, True), (64, 16, False), (64, 48, True), (128, 128, False)])
@pytest.mark.parametrize("what", [np.inf, -np.inf, np.nan])
def test_norm_and_rotation_of_what_is_not_finite(paged, dtype, d, rot, interleaved, what):
    """An infinite channel makes itself NaN (inf times the norm's 0) and, where
    it is rotated, its partner; an infinite or NaN weight reaches its own
    channel and that partner: no other channel and no other head."""
    r = np.random.default_rng(d + rot)
    table, pos = rope_table(50, rot), np.array([3, 17, 40], np.int32)
    axis = np.zeros(rot // 2, int)
    for c in {0, 5, rot // 2, rot - 1, rot % d, (rot + 3) % d, d - 1}:
        x = rounded(r.standard_normal((3, 5, d)), dtype)
        w = rounded(1 + 0.2 * r.standard_normal(d), dtype)
        bad = x.copy()
        bad[1, 2, c] = what
        wbad = w.copy()
        wbad[c] = what
        for xx, ww in ((bad, w), (x, wbad)):
            got, _ = paged.qwm_qk_norm_rope(dev(xx, dtype), None, dev(ww, dtype), None, dev(table), dev(pos), interleaved=interleaved)
            with np.errstate(all="ignore"):
                want = P.norm_rope(xx, ww, table, pos[:, None], axis, 1e-6, interleaved)
            g = host(got.float()).astype(np.float64)
            assert np.array_equal(np.isnan(g), np.isnan(want)), c
            finite = np.isfinite(want)
            assert np.array_equal(g[~finite & ~np.isnan(want)], want[~finite & ~np.isnan(want)])
            tol = rope_tolerance(np.where(finite, want, 0), dtype)
            assert (np.abs(g[finite] - want[finite]) <= tol[finite]).all()


# ------------------------------------------------------------------ logits that float32 cannot tell apart
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("size", [1e3, 1e5, 1e6, 1e7, 1e8, 1e10, 1e15])
@pytest.mark.parametrize("cached,new", [([100, 30], [40, 300]), ([9000], [3])])
def test_large_logits_are_right_or_nan(paged, kernel, size, cached, new):
    """Rows of growing logits.  Kernel 1 takes them all.  A row of the others is
    right, within the bound of its logits' rounding, or NaN in O and lse; it may
    be NaN only where some logit is beyond 2^22."""
    bt = Batch(38, cached, new, 4, 2, 128, 16)
    bt.q = rounded(bt.q * size, "bf16")
    k = kid(paged, kernel)
    lse = torch.empty(bt.rows, bt.heads, device="cuda")
    out = paged.qwm_paged_attend(dev(bt.q, "bf16"), dev(bt.pool), dev(bt.table), dev(bt.kv_len), dev(bt.cu), max_new=max(new),
                                 lse=lse, kernel=k)
    O, want, spread, vmax = P.attend(bt.q.astype(np.float64), bt.pool, bt.table, bt.kv_len, bt.cu, bt.page, True, 0, 128 ** -0.5)
    n, tensor = int(bt.kv_len.max()), k != paged.PAGED_SIMT
    with np.errstate(over="ignore"):
        tol = attend_tolerance(O, spread, vmax, n, "bf16", tensor)
    got, l = host(out.float()).astype(np.float64), host(lse).astype(np.float64)
    lost = np.isnan(l)
    assert tensor or not lost.any()
    assert np.isnan(got[lost]).all() and not np.isnan(got[~lost]).any()
    assert (np.abs(got - O)[~lost] <= tol[~lost]).all()
    delta = spread * (131 * 2.0 ** -24 + (1.01 * 2.0 ** -11 if tensor else 0))
    assert (np.abs(l - want) <= delta + np.abs(want) * 2.0 ** -22 + (n + 200) * 2.0 ** -22)[~lost].all()
    # spread bounds every logit of the row from above
    assert not (lost & (spread <= 2.0 ** 22)).any()
