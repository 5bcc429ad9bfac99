"""The paged cache's binding without a GPU: struct layouts against the header
as a C compiler sees it, refusals of the C ABI, refusals of the binding, and
pins of the oracle."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import paged_oracle as P

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def paged():
    from bit_kv_cache_qwm_gb300 import build
    build.build()
    from bit_kv_cache_qwm_gb300 import paged as p
    return p


def test_packed_structs_match_the_header(paged, tmp_path):
    """Size, and offset of the last field, of every argument struct."""
    want = {"qwm_qk_norm_rope_args": (paged._ROPE, "eps", 4), "qwm_paged_plan_args": (paged._PLAN, "page_tokens", 8),
            "qwm_paged_release_args": (paged._RELEASE, "page_tokens", 8),
            "qwm_paged_append_args": (paged._APPEND, "page_tokens", 4), "qwm_paged_attend_args": (paged._ATTEND, "kernel", 8)}
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "qwm.h"\nint main(void){' + "".join(
        f'printf("%zu %zu\\n", sizeof({n}), offsetof({n}, {last}));' for n, (_, last, _) in want.items()) + "return 0;}\n")
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n")
    for line, (n, (st, _, tail)) in zip(lines, want.items()):
        size, off = map(int, line.split())
        assert (st.size, st.size - tail) == (size, off), n


@pytest.mark.parametrize("d,page,want", [(128, 16, 2560), (64, 16, 1280), (128, 256, 40960), (96, 16, 0), (128, 24, 0), (128, 8, 0), (128, 512, 0)])
def test_block_bytes(paged, d, page, want):
    assert paged.lib().qwm_paged_block_bytes(d, page) == want
    if want:
        assert P.block_offsets(d, page)["bytes"] == want == paged.qwm_paged_block_bytes(d, page)
    else:
        with pytest.raises(ValueError):
            paged.qwm_paged_block_bytes(d, page)


FAKE = 0x10000   # never touched: every call below is refused before it launches


def rope_args(paged, **kw):
    a = dict(q=(FAKE, 1280, 128), k=(FAKE, 1280, 128), q_out=(FAKE, 1280, 128), k_out=(FAKE, 1280, 128), wq=FAKE, wk=FAKE,
             table=FAKE, pos=FAKE, status=0, rows=4, n_pos=100, dtype=1, d=128, hq=6, hk=2, rot=128, axes=1,
             sections=(64, 0, 0, 0), inter=0, eps=1e-6)
    a.update(kw)
    return paged._ROPE.pack(*a["q"], *a["k"], *a["q_out"], *a["k_out"], a["wq"], a["wk"], a["table"], a["pos"], a["status"],
                            a["rows"], a["n_pos"], a["dtype"], a["d"], a["hq"], a["hk"], a["rot"], a["axes"], *a["sections"],
                            a["inter"], a["eps"])


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), 0), (dict(rows=-1), 1), (dict(dtype=2), 1), (dict(d=96), 2), (dict(d=64), 1), (dict(rot=0), 1),
    (dict(rot=24), 1), (dict(rot=144), 1), (dict(axes=0), 1), (dict(axes=5), 1), (dict(axes=2, sections=(60, 5, 0, 0)), 1),
    (dict(sections=(-1, 0, 0, 0)), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(n_pos=0), 1), (dict(hq=0), 1),
    (dict(hk=-1), 1), (dict(table=0), 1), (dict(pos=0), 1), (dict(q=(0, 1280, 128)), 1), (dict(q=(FAKE + 8, 1280, 128)), 1),
    (dict(q=(FAKE, 1284, 128)), 1), (dict(q_out=(FAKE, 128, 128)), 1), (dict(q_out=(FAKE, 640, 128)), 1),
    (dict(q_out=(FAKE, 1280, 64)), 1), (dict(q_out=(FAKE, 1280, 0)), 1), (dict(k_out=(FAKE, -1280, 128)), 1),
    (dict(wq=FAKE + 2), 1)])
def test_norm_rope_refusals(paged, kw, status, monkeypatch):
    monkeypatch.setenv("QWM_FAULT_INJECT", "launch")
    assert paged.lib().qwm_qk_norm_rope(rope_args(paged, **kw), None) == status
    # the same call without the mistake gets as far as the launch, where the test hook stops it
    assert paged.lib().qwm_qk_norm_rope(rope_args(paged), None) == 6


def plan_args(paged, **kw):
    a = dict(p=[FAKE] * 11, rows=10, n_pages=5, requests=3, max_blocks=4, page=16)
    a.update({k: v for k, v in kw.items() if k != "null"})
    if "null" in kw:
        a["p"] = [0 if i == kw["null"] else FAKE for i in range(11)]
    return paged._PLAN.pack(*a["p"], a["rows"], a["n_pages"], a["requests"], a["max_blocks"], a["page"])


@pytest.mark.parametrize("kw,status", [(dict(null=i), 1) for i in range(10)] + [
    (dict(null=10), 6), (dict(rows=-1), 1), (dict(rows=1 << 31), 1), (dict(n_pages=0), 1), (dict(n_pages=1 << 31), 1),
    (dict(requests=0), 1), (dict(requests=8193), 2), (dict(requests=8192), 6), (dict(max_blocks=0), 1), (dict(page=20), 1),
    (dict(page=512), 1), (dict(rows=0), 6)])
def test_plan_refusals(paged, kw, status, monkeypatch):
    monkeypatch.setenv("QWM_FAULT_INJECT", "launch")
    assert paged.lib().qwm_paged_plan(plan_args(paged, **kw), None) == status


@pytest.mark.parametrize("null,requests,page,status", [(i, 3, 16, 1) for i in range(5)] + [
    (5, 3, 16, 6), (None, 0, 16, 1), (None, 8193, 16, 2), (None, 3, 17, 1), (None, 3, 16, 6)])
def test_release_refusals(paged, null, requests, page, status, monkeypatch):
    monkeypatch.setenv("QWM_FAULT_INJECT", "launch")
    a = paged._RELEASE.pack(*[0 if i == null else FAKE for i in range(6)], 5, requests, 4, page)
    assert paged.lib().qwm_paged_release(a, None) == status


def append_args(paged, **kw):
    a = dict(k=(FAKE, 256, 128), v=(FAKE, 256, 128), kh=(0, 0, 0), vh=(0, 0, 0), pool=FAKE, slots=FAKE, status=0, rows=4,
             n_pages=3, dtype=1, d=128, hk=2, page=16)
    a.update(kw)
    return paged._APPEND.pack(*a["k"], *a["v"], *a["kh"], *a["vh"], a["pool"], a["slots"], a["status"], a["rows"], a["n_pages"],
                              a["dtype"], a["d"], a["hk"], a["page"])


@pytest.mark.parametrize("kw,status", [
    ({}, 6), (dict(rows=0), 0), (dict(rows=-1), 1), (dict(dtype=7), 1), (dict(d=80), 2), (dict(page=48), 2), (dict(hk=0), 1),
    (dict(n_pages=0), 1), (dict(pool=0), 1), (dict(pool=FAKE + 4), 1), (dict(slots=0), 1), (dict(slots=FAKE + 4), 1),
    (dict(k=(FAKE + 2, 256, 128)), 1), (dict(v=(FAKE, 257, 128)), 1), (dict(k=(FAKE, 0, 0)), 6), (dict(kh=(FAKE, 0, 128)), 1),
    (dict(vh=(FAKE, 128, 128)), 1), (dict(vh=(FAKE, 128, 512)), 6), (dict(vh=(FAKE, 128, 384)), 1)])
def test_append_refusals(paged, kw, status, monkeypatch):
    monkeypatch.setenv("QWM_FAULT_INJECT", "launch")
    assert paged.lib().qwm_paged_append(append_args(paged, **kw), None) == status


def attend_args(paged, **kw):
    a = dict(q=(FAKE, 768, 128), out=(FAKE, 768, 128), lse=0, pool=FAKE, table=FAKE, lens=FAKE, cu=FAKE, status=0, ws=FAKE,
             ws_bytes=1 << 40, rows=10, n_pages=5, max_new=4, dtype=1, d=128, hq=6, hk=2, page=16, requests=3, max_blocks=4,
             causal=1, window=0, scale=0.0, kernel=0)
    a.update(kw)
    return paged._ATTEND.pack(*a["q"], *a["out"], *(a[x] for x in (
        "lse", "pool", "table", "lens", "cu", "status", "ws", "ws_bytes", "rows", "n_pages", "max_new", "dtype", "d", "hq", "hk",
        "page", "requests", "max_blocks", "causal", "window", "scale", "kernel")))


@pytest.mark.parametrize("kw,status", [
    ({}, 6), (dict(rows=0), 0), (dict(requests=0), 0), (dict(rows=-1), 1), (dict(dtype=2), 1), (dict(d=256), 2), (dict(page=8), 2),
    (dict(hq=7), 1), (dict(hk=0), 1), (dict(hk=12), 1), (dict(window=-1), 1), (dict(window=5, causal=0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(kernel=4), 1), (dict(kernel=-1), 1), (dict(max_new=-1), 1), (dict(max_blocks=0), 1),
    (dict(max_blocks=1 << 27), 2), (dict(n_pages=0), 1), (dict(pool=0), 1), (dict(pool=FAKE + 8), 1), (dict(table=0), 1),
    (dict(lens=0), 1), (dict(cu=0), 1), (dict(ws=0), 1), (dict(ws=FAKE + 64), 1), (dict(ws_bytes=100), 1),
    (dict(q=(FAKE + 4, 768, 128)), 1), (dict(out=(FAKE, 768, 64)), 1), (dict(out=(FAKE, 512, 128)), 1),
    (dict(out=(FAKE, 128, 1280)), 6), (dict(rows=1 << 29), 2), (dict(dtype=0, kernel=2), 2), (dict(dtype=0, kernel=3), 2)])
def test_attend_refusals(paged, kw, status, monkeypatch):
    monkeypatch.setenv("QWM_FAULT_INJECT", "launch")
    assert paged.lib().qwm_paged_attend(attend_args(paged, **kw), None) == status


def test_null_arguments(paged):
    L = paged.lib()
    for fn in (L.qwm_qk_norm_rope, L.qwm_paged_plan, L.qwm_paged_release, L.qwm_paged_append, L.qwm_paged_attend):
        assert fn(None, None) == 1
    assert L.qwm_paged_attend_workspace_bytes(96) == 0
    assert L.qwm_paged_attend_kernel_for(0, 8, 2, 1) == 1
    assert [L.qwm_paged_attend_kernel_for(1, 8, 2, n) for n in (0, 1, 8, 9, 4096)] == [2, 2, 2, 3, 3]
    assert L.qwm_paged_attend_kernel_for(1, 8, 3, 1) == -1


def test_the_binding_refuses_host_tensors_and_wrong_shapes(paged):
    """Refused before the library is called, so no host pointer reaches a kernel."""
    x = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    pool = torch.zeros((3, 2, 2560), dtype=torch.uint8)
    for call in (lambda: paged.qwm_paged_append(x, x, pool, i.long()),
                 lambda: paged.qwm_paged_attend(x, pool, i.view(2, 2), i, i),
                 lambda: paged.qwm_qk_norm_rope(x, x, None, None, torch.zeros(4, 128), i),
                 lambda: paged.qwm_paged_plan(i, i, i.view(4, 1), i, i, 16, 4),
                 lambda: paged.qwm_paged_release(i, i, i.view(4, 1), i, i, 16)):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ pins of the oracle
def test_oracle_quantiser_by_hand():
    """A group 0, 1, ..., 15, 0, 1, ..., 15: zero 0, scale 1, codes the values;
    ties to even; a constant group has scale 0."""
    x = np.tile(np.arange(16, dtype=np.float32), 2)
    c, z, s = P.quantize_int4(x)
    assert z[0] == 0 and s[0] == 1 and np.array_equal(c, x) and np.array_equal(P.dequantize_int4(c, z, s), x)
    y = x.copy()
    y[1:4] = 0.5, 1.5, 2.5
    assert P.quantize_int4(y)[0][1:4].tolist() == [0, 2, 2]
    c, z, s = P.quantize_int4(np.full(32, -3.25, np.float32))
    assert s[0] == 0 and not c.any() and (P.dequantize_int4(c, z, s) == -3.25).all()
    c, z, s = P.quantize_int4(np.array([np.nan, np.inf, -np.inf] + [0] * 29, np.float32))
    assert (z[0], s[0]) == (-60000, 8000) and c[:3].tolist() == [8, 15, 0]


@pytest.mark.parametrize("scale", [1e-6, 1.0, 3e4])
def test_oracle_quantiser_error_bound(scale):
    """|x - x_hat| <= scale/2 + the roundings of zero and scale to float16
    (half a step of zero, and 15 times half a step of scale; 2^-25 in the
    subnormal range)."""
    x = (np.random.default_rng(0).standard_normal((50, 128)) * scale).astype(np.float32)
    x = np.clip(x, -60000, 60000)
    c, z, s = P.quantize_int4(x)
    err = np.abs(P.dequantize_int4(c, z, s) - x).reshape(50, 4, 32).max(-1)
    z64, s64 = np.abs(z.astype(np.float64)), s.astype(np.float64)
    slack = np.maximum(z64 * 2.0 ** -11, 2.0 ** -25) + 15 * np.maximum(s64 * 2.0 ** -11, 2.0 ** -25)
    assert (err <= s64 / 2 * (1 + 1e-6) + slack * 1.01).all()


def test_oracle_block_round_trip_and_attention():
    """Bytes written slot by slot read back as the quantised values, and the
    attention over them is torch's softmax attention."""
    r = np.random.default_rng(1)
    d, page, hk = 64, 16, 2
    pool = np.full((3, hk, P.block_offsets(d, page)["bytes"]), 255, np.uint8)
    k, v = r.standard_normal((2, 20, hk, d)).astype(np.float32)
    table = np.array([[2, 0]])
    for i in range(20):
        for h in range(hk):
            P.write_slot(pool, int(table[0, i // page]) * page + i % page, h, k[i, h], v[i, h], d, page)
    kh = P.dequantize_int4(*P.quantize_int4(k))
    vh = P.dequantize_int4(*P.quantize_int4(v))
    for h in range(hk):
        a, b, known = P.gather(pool, table[0], 20, h, d, page)
        assert known.all() and np.array_equal(a, kh[:, h]) and np.array_equal(b, vh[:, h])
    q = r.standard_normal((3, 4, d))
    O, lse, _, _ = P.attend(q, pool, table, [20], [0, 3], page, True, 6, 0.3)
    T = torch.from_numpy
    n = np.arange(20)
    at = 17 + np.arange(3)[:, None]
    mask = T((n <= at) & (n > at - 6))
    want = torch.nn.functional.scaled_dot_product_attention(
        T(q).transpose(0, 1), T(kh).transpose(0, 1).repeat_interleave(2, 0), T(vh).transpose(0, 1).repeat_interleave(2, 0),
        attn_mask=mask, scale=0.3).transpose(0, 1)
    assert np.abs(O - want.numpy()).max() <= 1e-12
    logits = 0.3 * torch.einsum("ihd,nhd->hin", T(q), T(kh).repeat_interleave(2, 1)).masked_fill(~mask, -np.inf)
    assert np.abs(lse - torch.logsumexp(logits, -1).T.numpy()).max() <= 1e-12


def test_oracle_rotation_is_a_rotation():
    """Norms are kept, and the dot product of two rotated rows depends on the
    difference of their positions alone."""
    r = np.random.default_rng(2)
    rot = 64
    inv = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    ang = np.arange(200)[:, None] * inv
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    x = r.standard_normal((2, 1, 64))
    for inter in (False, True):
        f = lambda a, b: P.norm_rope(x, None, table, np.array([[a], [b]]), np.zeros(32, int), 0.0, inter)  # noqa: E731
        y = f(3, 10)
        assert np.allclose((y * y).mean(-1), 1.0)
        assert np.isclose((y[0] * y[1]).sum(), (f(103, 110)[0] * f(103, 110)[1]).sum())


def test_oracle_plan_by_hand():
    """Two requests on pages of 16: the open page is filled first, new pages
    come off the top of the stack in the requests' order."""
    kv, free_count, cu, slots, pos, table = P.plan([14, 16], [3, 2], [[5, -1], [7, -1]], [9, 8, 4], 3, 16, 6)
    assert kv.tolist() == [17, 18] and free_count == 1 and cu.tolist() == [0, 3, 5]
    assert table.tolist() == [[5, 4], [7, 8]]
    assert slots.tolist() == [5 * 16 + 14, 5 * 16 + 15, 4 * 16, 8 * 16, 8 * 16 + 1, -1]
    assert pos.tolist() == [14, 15, 16, 16, 17, -1]
    assert P.plan([14, 16], [3, 2], [[5, -1], [7, -1]], [9, 8, 4], 1, 16, 6) is None
