"""The paged calls on inputs at the edge of what they promise."""

import pytest
import torch

from paged_cases import Batch
from test_gpu_paged_attend import KERNELS, dev, kid

pytestmark = pytest.mark.gpu


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
