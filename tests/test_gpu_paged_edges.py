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
