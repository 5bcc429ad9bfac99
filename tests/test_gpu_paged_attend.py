"""qwm_paged_attend on the GPU against the float64 oracle: every kernel, head
layout, page size and mask, with garbage (NaN bytes) in every slot that holds
no token."""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from paged_cases import Batch, attend_tolerance, rounded

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


def check(paged, bt, kernel, causal=True, window=0, scale=0.0, max_new=None, tail=2, **kw):
    """Run one batch and compare O and lse with the oracle; the `tail` rows
    behind the last request must stay as they were."""
    T = bt.rows + tail
    q = torch.zeros((T, bt.heads, bt.d), dtype=torch.bfloat16 if bt.dtype == "bf16" else torch.float32, device="cuda")
    q[: bt.rows] = dev(bt.q, bt.dtype)
    q[bt.rows:] = float("nan")
    out = torch.full_like(q, 7.0)
    lse = torch.full((T, bt.heads), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    paged.qwm_paged_attend(q, dev(bt.pool), dev(bt.table), dev(bt.kv_len), dev(bt.cu),
                           max_new=max(bt.new) if max_new is None else max_new, causal=causal, window=window, scale=scale,
                           out=out, lse=lse, status=status, kernel=kernel, **kw)
    torch.cuda.synchronize()
    sigma = scale if scale > 0 else 1 / np.sqrt(bt.d)
    O, want_lse, spread, vmax = P.attend(bt.q.astype(np.float64), bt.pool, bt.table, bt.kv_len, bt.cu, bt.page, causal, window, sigma)
    got = out[: bt.rows].float().cpu().numpy().astype(np.float64)
    n = int(bt.kv_len.max())
    tensor = bt.dtype == "bf16" and kernel != paged.PAGED_SIMT
    tol = attend_tolerance(O, spread, vmax, n, bt.dtype, tensor)
    assert np.isfinite(got).all()
    bad = np.abs(got - O) > tol
    assert not bad.any(), (np.argwhere(bad)[:3], np.abs(got - O).max(), (np.abs(got - O) / tol).max())
    gl = lse[: bt.rows].cpu().numpy().astype(np.float64)
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(gl), empty)
    ltol = spread * (2.0 ** -11 * 1.01 if tensor else 0) + (spread + np.abs(np.where(empty, 0, want_lse)) + n + 200) * 2.0 ** -22
    assert (np.abs(gl[~empty] - want_lse[~empty]) <= ltol[~empty]).all()
    assert (got[empty] == 0).all()
    assert (out[bt.rows:] == 7).all() and (lse[bt.rows:] == 7).all()
    return int(status.item())


KERNELS = ["simt", "mma", "tc", "auto"]


def kid(paged, name):
    return {"auto": paged.PAGED_AUTO, "simt": paged.PAGED_SIMT, "mma": paged.PAGED_MMA, "tc": paged.PAGED_TC}[name]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (8, 8), (8, 1), (6, 2), (15, 3)])
def test_single_tokens(paged, kernel, d, heads, kv_heads):
    """One new token for requests of 1 to a few hundred tokens."""
    bt = Batch(1, [0, 1, 15, 16, 17, 63, 64, 65, 127, 200, 333], [1] * 11, heads, kv_heads, d, 16)
    assert check(paged, bt, kid(paged, kernel)) == 0


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 33), (True, 100)])
def test_masks_and_pages(paged, kernel, page, causal, window):
    """Ragged prompts, requests without new tokens among them, odd sizes."""
    bt = Batch(2, [0, 5, 100, 260, 31, 0], [7, 0, 33, 3, 1, 129], 4, 2, 128, page)
    assert check(paged, bt, kid(paged, kernel), causal=causal, window=window) == 0


@pytest.mark.parametrize("kernel", KERNELS)
def test_rows_that_see_nothing(paged, kernel):
    """More query rows than cached tokens: the first rows stand before the
    cache and see nothing (O = 0, lse = -inf), also where a request has no
    token at all."""
    bt = Batch(3, [0, 0, 40], [5, 0, 20], 4, 2, 128, 16)
    bt.kv_len = np.array([2, 0, 60], np.int32)
    assert check(paged, bt, kid(paged, kernel)) == 0
    bt.kv_len = np.array([0, 0, 60], np.int32)
    assert check(paged, bt, kid(paged, kernel)) == 0
    assert check(paged, bt, kid(paged, kernel), causal=False) == 0


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("d", [64, 128])
def test_long_requests_are_split(paged, kernel, d):
    """One request long enough for every CTA to get a part of it, next to
    short ones; the result is the same bit for bit on a second run."""
    bt = Batch(4, [9000, 0, 40], [2, 1, 3], 4, 1, d, 64)
    k = kid(paged, kernel)
    assert check(paged, bt, k) == 0
    a = [paged.qwm_paged_attend(dev(bt.q, "bf16"), dev(bt.pool), dev(bt.table), dev(bt.kv_len), dev(bt.cu), max_new=3, kernel=k)
         for _ in range(2)]
    assert torch.equal(a[0], a[1])


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("hint", [0, 1, 2, 5000])
def test_max_new_is_a_hint(paged, kernel, hint):
    bt = Batch(5, [50, 3, 700], [3, 40, 1], 4, 2, 128, 32)
    assert check(paged, bt, kid(paged, kernel), max_new=hint) == 0


@pytest.mark.parametrize("kernel", KERNELS)
def test_scale_and_large_queries(paged, kernel):
    """Queries beyond float16 with a scale that brings the logits back, and a
    scale that makes the softmax nearly one-hot."""
    bt = Batch(6, [100, 30], [20, 1], 4, 2, 128, 16, q_sigma=3e5)
    assert check(paged, bt, kid(paged, kernel), scale=1e-7) == 0
    bt = Batch(7, [100, 30], [20, 1], 4, 2, 128, 16)
    assert check(paged, bt, kid(paged, kernel), scale=0.5) == 0


@pytest.mark.parametrize("kernel", KERNELS)
def test_strided_rows_in_place_and_head_major(paged, kernel):
    """q as a view of a fused projection, out = q, and [heads][rows] order."""
    bt = Batch(8, [77, 12], [9, 2], 6, 2, 128, 16)
    k = kid(paged, kernel)
    args = (dev(bt.pool), dev(bt.table), dev(bt.kv_len), dev(bt.cu))
    ref = paged.qwm_paged_attend(dev(bt.q, "bf16"), *args, max_new=9, kernel=k)
    fused = torch.zeros((bt.rows, 10, 128), dtype=torch.bfloat16, device="cuda")
    fused[:, 2:8] = dev(bt.q, "bf16")
    view = fused[:, 2:8]
    got = paged.qwm_paged_attend(view, *args, max_new=9, out=view, kernel=k)
    assert got.data_ptr() == view.data_ptr() and torch.equal(view, ref)
    assert (fused[:, :2] == 0).all() and (fused[:, 8:] == 0).all()
    hm = dev(bt.q, "bf16").transpose(0, 1).contiguous()
    o = torch.empty_like(hm)
    paged.qwm_paged_attend(hm.transpose(0, 1), *args, max_new=9, out=o.transpose(0, 1), kernel=k)
    assert torch.equal(o.transpose(0, 1), ref)


@pytest.mark.parametrize("kernel", KERNELS)
def test_bad_tables_and_lengths_are_masked_and_reported(paged, kernel):
    """A page id out of range hides its tokens; a length beyond the table and
    offsets that leave the rows are clamped; each sets the status bit."""
    bt = Batch(9, [100, 90], [3, 2], 4, 2, 128, 16)
    k = kid(paged, kernel)
    for bad in (-1, bt.pool.shape[0], 1 << 30, -(1 << 31)):
        save = bt.table[0, 2]
        bt.table[0, 2] = bad
        assert check(paged, bt, k) == 8
        bt.table[0, 2] = save
    bt.table[1, :] = -1
    assert check(paged, bt, k) == 8          # a request with no valid page at all
    bt = Batch(9, [100, 90], [3, 2], 4, 2, 128, 16)
    full = bt.table.shape[1] * 16
    bt.table[0, : bt.table.shape[1]] = bt.table[0, 0]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (dev(bt.q, "bf16"), dev(bt.pool), dev(bt.table))
    a = paged.qwm_paged_attend(*args, dev(np.array([full + 5000, 92], np.int32)), dev(bt.cu), max_new=3, status=status, kernel=k)
    assert int(status.item()) == 8
    b = paged.qwm_paged_attend(*args, dev(np.array([full, 92], np.int32)), dev(bt.cu), max_new=3, kernel=k)
    assert torch.equal(a, b)
    status.zero_()
    out = torch.full_like(a, 7.0)
    paged.qwm_paged_attend(*args, dev(bt.kv_len), dev(np.array([0, 3, 900], np.int32)), max_new=3, out=out, status=status, kernel=k)
    assert int(status.item()) == 8 and torch.isfinite(out.float()).all()
    status.zero_()
    paged.qwm_paged_attend(*args, dev(np.array([-4, 92], np.int32)), dev(bt.cu), max_new=3, out=out, status=status, kernel=k)
    assert int(status.item()) == 8 and (out[:3] == 0).all()


@pytest.mark.parametrize("kernel", KERNELS)
def test_float32(paged, kernel):
    if kernel not in ("simt", "auto"):
        pytest.skip("bf16 kernel")
    for d in (64, 128):
        bt = Batch(10, [0, 5, 100, 700], [7, 0, 70, 1], 6, 2, d, 16, dtype="f32")
        assert check(paged, bt, kid(paged, kernel)) == 0
        assert check(paged, bt, kid(paged, kernel), window=20) == 0
        bt = Batch(11, [1500, 5], [1, 2], 3, 1, d, 32, dtype="f32")
        assert check(paged, bt, kid(paged, kernel)) == 0


def test_offsets_beyond_32_bits(paged):
    """A pool of more than 2^32 bytes with the request's pages at its end."""
    bt = Batch(12, [300], [2], 8, 8, 128, 256)
    n = (1 << 32) // bt.pool[0].size + 10
    big = torch.zeros((n,) + bt.pool.shape[1:], dtype=torch.uint8, device="cuda")
    shift = n - bt.pool.shape[0]
    big[shift:] = dev(bt.pool)
    args = (dev(bt.kv_len), dev(bt.cu))
    for k in KERNELS:
        a = paged.qwm_paged_attend(dev(bt.q, "bf16"), dev(bt.pool), dev(bt.table), *args, max_new=2, kernel=kid(paged, k))
        b = paged.qwm_paged_attend(dev(bt.q, "bf16"), big, dev(np.where(bt.table >= 0, bt.table + shift, -1).astype(np.int32)),
                                   *args, max_new=2, kernel=kid(paged, k))
        assert torch.equal(a, b)


@pytest.mark.parametrize("kernel", KERNELS)
def test_captured_with_other_lengths_and_on_two_streams(paged, kernel):
    """Two graphs of different batches, replayed at the same time on two
    streams, with lengths changed between capture and replay."""
    k = kid(paged, kernel)
    bts = [Batch(20, [900, 40], [2, 2], 8, 2, 128, 16), Batch(21, [30, 2000, 7], [1, 3, 2], 8, 2, 128, 64)]
    graphs = []
    for bt in bts:
        st = [dev(bt.q, "bf16"), dev(bt.pool), dev(bt.table), dev(np.maximum(bt.kv_len - 5, 0)), dev(bt.cu)]
        out = torch.zeros_like(st[0])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            paged.qwm_paged_attend(*st, max_new=3, out=out, kernel=k)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            paged.qwm_paged_attend(*st, max_new=3, out=out, kernel=k)
        st[3].copy_(dev(bt.kv_len))
        graphs.append((g, s, st, out))
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s, _, _ in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (g, s, st, out), bt in zip(graphs, bts):
        ref = paged.qwm_paged_attend(dev(bt.q, "bf16"), dev(bt.pool), dev(bt.table), dev(bt.kv_len), dev(bt.cu), max_new=3, kernel=k)
        assert torch.equal(out, ref)


@pytest.mark.parametrize("kernel", KERNELS)
def test_many_requests(paged, kernel):
    """More requests than a CTA has threads, most without rows."""
    r = np.random.default_rng(0)
    n = 1300
    cached = r.integers(0, 20, n)
    new = (r.random(n) < 0.2).astype(int)
    bt = Batch(13, cached, new, 2, 2, 64, 16)
    assert check(paged, bt, kid(paged, kernel)) == 0


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("new", [1, 40])
def test_a_row_of_nan_or_infinity_stays_alone(paged, kernel, new):
    """Rows of q that hold NaN or infinity change no other row, of their own
    head group, token or request."""
    bt = Batch(14, [70, 300], [new, new], 6, 2, 128, 16)
    k = kid(paged, kernel)
    args = (dev(bt.pool), dev(bt.table), dev(bt.kv_len), dev(bt.cu))
    q = dev(bt.q, "bf16")
    ref = paged.qwm_paged_attend(q, *args, max_new=new, kernel=k)
    bad = q.clone()
    bad[0, 1, 5] = float("nan")
    bad[-1, 4, 100] = float("inf")
    got = paged.qwm_paged_attend(bad, *args, max_new=new, kernel=k)
    same = torch.ones(got.shape[:2], dtype=torch.bool, device="cuda")
    same[0, 1] = same[-1, 4] = False
    assert torch.equal(got[same], ref[same])
    assert not torch.isfinite(got[0, 1].float()).any()


@pytest.mark.parametrize("kernel", KERNELS)
def test_on_another_stream(paged, kernel):
    """The call runs on the current stream, after what is ahead of it there."""
    bt = Batch(15, [200, 3000], [2, 2], 8, 2, 128, 32)
    k = kid(paged, kernel)
    args = [dev(bt.pool), dev(bt.table), dev(bt.kv_len), dev(bt.cu)]
    ref = paged.qwm_paged_attend(dev(bt.q, "bf16"), *args, max_new=2, kernel=k)
    q = torch.zeros_like(dev(bt.q, "bf16"))
    want = dev(bt.q, "bf16")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        q.copy_(want)
        got = paged.qwm_paged_attend(q, *args, max_new=2, kernel=k)
        after = got.clone()
    s.synchronize()
    assert torch.equal(after, ref)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("d, key", [(64, 2.203125), (128, 1.5625)])
def test_small_weights_beside_a_large_one(paged, kernel, d, key):
    """One token outweighs each of the others by about 2^25.5 and has the value
    0, the others the value 1: O is what the small weights add up to.  All
    codes, logits and values are exact.  P is float16 with the maximum at 2^7
    or more, so a small weight w keeps an error of half its smallest step, 2^-25
    / 2^7, relative to w = 2^-diff; the exponential, the sums of 200 tokens and
    the logit (float32, below 2^5) make less than 2^-16; O is rounded to bf16."""
    page, n = 16, 200
    k = torch.zeros(n, 1, d, dtype=torch.bfloat16, device="cuda")
    v = torch.ones_like(k)
    k[0], v[0] = key, 0
    width = -(-n // page)
    pool = paged.paged_pool(width, 1, d, page)
    table = torch.arange(width, dtype=torch.int32, device="cuda")[None].contiguous()
    paged.qwm_paged_append(k, v, pool, torch.arange(n, device="cuda"))
    q = torch.ones(2, 1, d, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    out = paged.qwm_paged_attend(q, pool, table, torch.tensor([n], **i32), torch.tensor([0, 2], **i32), max_new=2,
                                 causal=False, kernel=kid(paged, kernel))
    diff = np.sqrt(d) * key / np.log(2)
    want = (n - 1) * 2.0 ** -diff / (1 + (n - 1) * 2.0 ** -diff)
    rel = 2.0 ** (diff - 32) + 2.0 ** -16 + 2.0 ** -8
    assert ((out.double().cpu() - want).abs() <= rel * want).all(), out[0, 0, :4]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("new", [1, 300])
def test_in_place(paged, kernel, new):
    """out may be q: every row is read by those who need it before it is
    written, whole items and cut ones alike."""
    bt = Batch(16, [40, 5000, 0, 700], [new] * 4, 8, 2, 64, 16)
    args = (dev(bt.pool), dev(bt.table), dev(bt.kv_len), dev(bt.cu))
    q = dev(bt.q, "bf16")
    ref = paged.qwm_paged_attend(q, *args, max_new=new, kernel=kid(paged, kernel))
    got = paged.qwm_paged_attend(q, *args, max_new=new, kernel=kid(paged, kernel), out=q)
    assert got is q and torch.equal(q, ref)


@pytest.mark.parametrize("kernel", KERNELS)
def test_shared_prefix_and_endless_window(paged, kernel):
    """Two requests whose tables name the same pages read the same tokens (not
    to the same bits: the partition may cut one of them and not the other), and
    a window longer than any cache hides none."""
    bt = Batch(17, [200, 200], [2, 2], 4, 2, 128, 32)
    bt.table[1] = bt.table[0]
    bt.q[2:] = bt.q[:2]
    args = (dev(bt.pool), dev(bt.table), dev(bt.kv_len), dev(bt.cu))
    q = dev(bt.q, "bf16")
    k = kid(paged, kernel)
    got = paged.qwm_paged_attend(q, *args, max_new=2, kernel=k)
    assert check(paged, bt, k) == 0
    assert torch.equal(paged.qwm_paged_attend(q, *args, max_new=2, window=2 ** 40, kernel=k), got)


def test_a_mixed_step_in_two_calls(paged):
    """Single tokens and prompts of one plan, each range of requests in a call
    of its own over the same rows."""
    bt = Batch(18, [300, 5000, 17, 0, 900], [1, 1, 1, 200, 70], 8, 2, 128, 16)
    q, pool, table, lens, cu = dev(bt.q, "bf16"), dev(bt.pool), dev(bt.table), dev(bt.kv_len), dev(bt.cu)
    out = torch.full_like(q, float("nan"))
    for a, b in ((0, 3), (3, 5)):
        paged.qwm_paged_attend(q, pool, table[a:b], lens[a:b], cu[a:b + 1], max_new=max(bt.new[a:b]), out=out)
    O, _, spread, vmax = P.attend(bt.q.astype(np.float64), bt.pool, bt.table, bt.kv_len, bt.cu, bt.page, True, 0, 128 ** -0.5)
    got = out.float().cpu().numpy().astype(np.float64)
    assert (np.abs(got - O) <= attend_tolerance(O, spread, vmax, int(bt.kv_len.max()), "bf16", True)).all()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("heads,kv_heads,new", [(32, 1, 1), (71, 1, 1), (24, 1, 2), (9, 3, 6)])
def test_more_rows_than_a_few_row_item(paged, kernel, heads, kv_heads, new):
    """Wide head groups and drafts: a key/value head's rows fill one to three
    items of 16."""
    bt = Batch(19, [0, 31, 500, 2049], [new, new, 1, new], heads, kv_heads, 64, 16)
    assert check(paged, bt, kid(paged, kernel)) == 0


@pytest.mark.parametrize("kernel", ["tc", "auto"])
def test_items_of_one_cta_differ(paged, kernel):
    """Several items follow one another in a CTA, with queries beyond float16
    in some of them, a page out of range in others, and ragged ends: what an
    item needs must not reach the next."""
    bt = Batch(22, [100, 0, 300, 20], [300, 513, 257, 700], 24, 24, 64, 32)
    large = np.zeros((bt.rows, 1, 1))
    for b in (1, 3):
        large[bt.cu[b]: bt.cu[b + 1]] = 1
    large[bt.cu[0] + 100: bt.cu[0] + 130] = 1     # some rows of an item
    bt.q = rounded(bt.q * np.where(large > 0, 3e5, 1.0), "bf16")
    assert check(paged, bt, kid(paged, kernel), scale=1e-7) == 0
    q, args = dev(bt.q, "bf16"), (dev(bt.pool), dev(bt.kv_len), dev(bt.cu))
    ref = paged.qwm_paged_attend(q, args[0], dev(bt.table), *args[1:], max_new=700, scale=1e-7, kernel=kid(paged, kernel))
    bt.table[2, 3] = bt.pool.shape[0]             # tokens 96 to 127 of request 2
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = paged.qwm_paged_attend(q, args[0], dev(bt.table), *args[1:], max_new=700, scale=1e-7, status=status,
                                 kernel=kid(paged, kernel))
    assert int(status.item()) == 8
    other = np.ones(bt.rows, bool)
    other[bt.cu[2]: bt.cu[3]] = False
    keep = torch.from_numpy(other).cuda()
    assert torch.equal(got[keep], ref[keep]) and not torch.equal(got[~keep], ref[~keep])
