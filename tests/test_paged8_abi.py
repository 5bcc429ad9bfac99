"""The 8-bit cache's binding without a GPU: struct layouts against the header as
a C compiler sees it, exported symbols, refusals of the C ABI and of the binding
(every call is refused, or stopped by the test hook, before it launches), and
pins of the oracle."""
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from oracle import paged8_oracle as P8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000   # never touched


@pytest.fixture(scope="module")
def paged():
    from bit_kv_cache_qwm_gb300 import build
    build.build()
    from bit_kv_cache_qwm_gb300 import paged as p
    return p


@pytest.fixture(autouse=True)
def stop_at_the_launch(monkeypatch):
    monkeypatch.setenv("QWM_FAULT_INJECT", "launch")


def test_packed_structs_match_the_header(paged, tmp_path):
    want = {"qwm_paged8_append_args": (paged._APPEND8, "max_blocks", 4), "qwm_paged8_read_args": (paged._READ8, "max_blocks", 4),
            "qwm_paged8_attend_args": (paged._ATTEND8, "reserved", 4), "qwm_paged8_bounds_args": (paged._BOUNDS8, "max_blocks", 8),
            "qwm_paged8_select_args": (paged._SELECT8, "sink", 8)}
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "qwm.h"\nint main(void){' + "".join(
        f'printf("%zu %zu\\n", sizeof({n}), offsetof({n}, {last}));' for n, (_, last, _) in want.items()) + "return 0;}\n")
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n")
    for line, (n, (st, _, tail)) in zip(lines, want.items()):
        assert (st.size, st.size - tail) == tuple(map(int, line.split())), n


def test_every_declared_symbol_is_exported(paged):
    from bit_kv_cache_qwm_gb300 import qwm
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "qwm.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(qwm_paged8_[a-z0-9_]+)\s*\(", src))
    assert names == set(qwm.EXPORTS8)
    for n in names:
        assert hasattr(paged.lib(), n), n


@pytest.mark.parametrize("d,page,want", [(128, 16, 4112), (64, 16, 2064), (128, 32, 8208), (64, 64, 8208), (128, 128, 32800),
                                         (128, 256, 65600), (96, 16, 0), (128, 24, 0), (128, 8, 0), (128, 512, 0)])
def test_block_bytes(paged, d, page, want):
    assert paged.lib().qwm_paged8_block_bytes(d, page) == want
    if want:
        assert P8.block_bytes(d, page) == want == paged.qwm_paged8_block_bytes(d, page)
        assert paged._PAGE8[d, want] == page
    else:
        with pytest.raises(ValueError):
            paged.qwm_paged8_block_bytes(d, page)


STEP = [(dict(table=0), 1), (dict(lens=0), 1), (dict(cu=0), 1), (dict(table=FAKE + 2), 1), (dict(lens=FAKE + 1), 1),
        (dict(cu=FAKE + 3), 1), (dict(status=FAKE + 2), 1), (dict(status=FAKE), 6), (dict(pool=0), 1), (dict(pool=FAKE + 4), 1),
        (dict(n_pages=0), 1), (dict(n_pages=1 << 31), 1), (dict(d=80), 2), (dict(page=48), 2), (dict(hk=0), 1),
        (dict(hk=65537), 1), (dict(requests=-1), 1), (dict(requests=8193), 2), (dict(requests=8192), 6), (dict(requests=0), 0),
        (dict(max_blocks=0), 1), (dict(max_blocks=1 << 27), 2)]
ROWS = [({}, 6), (dict(rows=0), 0), (dict(rows=-1), 1), (dict(rows=1 << 31), 1), (dict(dtype=2), 1), (dict(k=(0, 256, 128)), 1),
        (dict(k=(FAKE + 2, 256, 128)), 1), (dict(v=(FAKE, 257, 128)), 1), (dict(v=(FAKE, -256, 128)), 1)]


def append_args(paged, **kw):
    a = dict(k=(FAKE, 256, 128), v=(FAKE, 256, 128), kh=(0, 0, 0), vh=(0, 0, 0), pool=FAKE, table=FAKE, lens=FAKE, cu=FAKE,
             status=0, rows=4, n_pages=3, dtype=1, d=128, hk=2, page=16, requests=3, max_blocks=4)
    a.update(kw)
    return paged._APPEND8.pack(*a["k"], *a["v"], *a["kh"], *a["vh"], *(a[x] for x in (
        "pool", "table", "lens", "cu", "status", "rows", "n_pages", "dtype", "d", "hk", "page", "requests", "max_blocks")))


@pytest.mark.parametrize("kw,status", STEP + ROWS + [
    (dict(k=(FAKE, 0, 0)), 6), (dict(kh=(FAKE, 0, 128)), 1), (dict(vh=(FAKE, 128, 128)), 1), (dict(vh=(FAKE, 128, 512)), 6),
    (dict(vh=(FAKE, 128, 384)), 1), (dict(kh=(FAKE + 8, 256, 128)), 1)])
def test_append_refusals(paged, kw, status):
    assert paged.lib().qwm_paged8_append(append_args(paged, **kw), None) == status


@pytest.mark.parametrize("kw,status", STEP + ROWS + [(dict(k=(FAKE, 0, 0)), 1), (dict(v=(FAKE, 128, 128)), 1),
                                                     (dict(v=(FAKE, 128, 512)), 6)])
def test_read_refusals(paged, kw, status):
    a = dict(k=(FAKE, 256, 128), v=(FAKE, 256, 128), pool=FAKE, table=FAKE, lens=FAKE, cu=FAKE, status=0, rows=4, n_pages=3,
             dtype=1, d=128, hk=2, page=16, requests=3, max_blocks=4)
    a.update(kw)
    args = paged._READ8.pack(*a["k"], *a["v"], *(a[x] for x in (
        "pool", "table", "lens", "cu", "status", "rows", "n_pages", "dtype", "d", "hk", "page", "requests", "max_blocks")))
    assert paged.lib().qwm_paged8_read(args, None) == status


@pytest.mark.parametrize("kw,status", STEP + [({}, 6), (dict(bounds=0), 1), (dict(bounds=FAKE + 8), 1), (dict(max_new=-1), 1),
                                              (dict(max_new=1 << 60), 6), (dict(hk=65536), 2)])
def test_bounds_refusals(paged, kw, status):
    a = dict(pool=FAKE, bounds=FAKE, table=FAKE, lens=FAKE, cu=FAKE, status=0, n_pages=3, max_new=1, d=128, hk=2, page=16,
             requests=3, max_blocks=4)
    a.update(kw)
    assert paged.lib().qwm_paged8_bounds(paged._BOUNDS8.pack(*a.values()), None) == status


@pytest.mark.parametrize("kw,status", [x for x in STEP if "pool" not in x[0]] + [
    ({}, 6), (dict(rows=0), 6), (dict(rows=-1), 1), (dict(rows=1 << 31), 1), (dict(rows=1 << 30, heads=4), 2), (dict(dtype=2), 1),
    (dict(q=(0, 256, 128)), 1), (dict(q=(FAKE + 2, 256, 128)), 1), (dict(q=(FAKE, 257, 128)), 1), (dict(bounds=0), 1),
    (dict(bounds=FAKE + 8), 1), (dict(pages=0), 1), (dict(pages=FAKE + 1), 1), (dict(out=0), 1), (dict(out=FAKE), 1),
    (dict(out=FAKE + 2), 1), (dict(ws=0), 1), (dict(ws=FAKE + 16), 1), (dict(ws_bytes=256 + 256 + 1023), 1), (dict(ws_bytes=256 + 256 + 1024), 6),
    (dict(heads=5), 1), (dict(heads=0), 1), (dict(width=0), 1), (dict(sink=-1), 1), (dict(sink=1 << 30, width=1 << 30), 6)])
def test_select_refusals(paged, kw, status):
    a = dict(q=(FAKE, 256, 128), bounds=FAKE, table=FAKE, lens=FAKE, cu=FAKE, pages=FAKE, out=2 * FAKE, status=0, ws=FAKE,
             ws_bytes=1 << 40, rows=4, n_pages=3, dtype=1, d=128, heads=2, hk=2, page=16, requests=3, max_blocks=4, width=2, sink=0)
    a.update(kw)
    assert paged.lib().qwm_paged8_select(paged._SELECT8.pack(*a["q"], *list(a.values())[1:]), None) == status
    # keys, the rows' units, the rows
    f = paged.lib().qwm_paged8_select_workspace_bytes
    assert f(4, 2, 128, 3, 2, 4) == 256 + 256 + 1024 and f(0, 5, 64, 10, 5, 1000) == 200192
    assert f(-1, 2, 128, 3, 2, 4) == f(4, 0, 128, 3, 2, 4) == f(4, 2, 96, 3, 2, 4) == f(4, 2, 128, 3, 0, 4) == f(4, 2, 128, 3, 2, 0) == 0


@pytest.mark.parametrize("out,lens,cu,status", [(0, 4, 32, 1), (4, 0, 32, 1), (8, 0, 32, 1), (12, 0, 32, 6), (0, 12, 32, 6), (32, 0, 32, 1),
                                                (44, 0, 32, 1), (48, 0, 32, 6), (20, 0, 32, 6), (24, 0, 32, 1)])
def test_select_refuses_lengths_in_its_lengths_or_first_rows(paged, out, lens, cu, status):
    """len_out [3] anywhere in kv_len [3] or cu_rows [4], not beside them."""
    a = [FAKE, 256, 128, FAKE, 3 * FAKE, FAKE + lens, FAKE + cu, 4 * FAKE, FAKE + out, 0, 5 * FAKE, 1 << 40, 4, 3, 1, 128, 2, 2, 16, 3, 4, 2, 0]
    assert paged.lib().qwm_paged8_select(paged._SELECT8.pack(*a), None) == status


def attend_args(paged, **kw):
    a = dict(q=(FAKE, 768, 128), out=(FAKE, 768, 128), lse=0, pool=FAKE, table=FAKE, lens=FAKE, cu=FAKE, status=0, ws=FAKE,
             ws_bytes=1 << 40, rows=10, n_pages=5, max_new=4, dtype=1, d=128, hq=6, hk=2, page=16, requests=3, max_blocks=4,
             causal=1, window=0, scale=0.0, kernel=0, heads=1, reserved=0)
    a.update(kw)
    return paged._ATTEND8.pack(*a["q"], *a["out"], *list(a.values())[2:])


@pytest.mark.parametrize("kw,status", [
    ({}, 6), (dict(heads=2), 6), (dict(heads=3), 1), (dict(heads=0), 1), (dict(reserved=1), 1), (dict(rows=0), 0),
    (dict(requests=0), 0), (dict(rows=-1), 1), (dict(dtype=2), 1), (dict(d=256), 2), (dict(page=8), 2), (dict(hq=7), 1),
    (dict(window=-1), 1), (dict(window=5, causal=0), 1), (dict(scale=float("nan")), 1), (dict(kernel=4), 1), (dict(max_new=-1), 1),
    (dict(max_blocks=1 << 27), 2), (dict(pool=FAKE + 8), 1), (dict(table=FAKE + 1), 1), (dict(lens=FAKE + 2), 1),
    (dict(cu=FAKE + 3), 1), (dict(lse=FAKE + 1), 1), (dict(status=FAKE + 1), 1), (dict(ws=FAKE + 64), 1), (dict(ws_bytes=100), 1),
    (dict(q=(FAKE + 4, 768, 128)), 1), (dict(out=(FAKE, 512, 128)), 1), (dict(rows=1 << 29), 2), (dict(dtype=0, kernel=2), 6),
    (dict(dtype=0, kernel=3), 2), (dict(dtype=0), 6), (dict(hk=1 << 16, hq=1 << 16, page=256, q=(FAKE, 1 << 23, 128), out=(FAKE, 1 << 23, 128)), 2)])
def test_attend_refusals(paged, kw, status):
    assert paged.lib().qwm_paged8_attend(attend_args(paged, **kw), None) == status


def test_null_arguments(paged):
    L = paged.lib()
    for fn in (L.qwm_paged8_append, L.qwm_paged8_read, L.qwm_paged8_attend, L.qwm_paged8_bounds, L.qwm_paged8_select):
        assert fn(None, None) == 1
    assert L.qwm_paged8_attend_workspace_bytes(96) == 0 and L.qwm_paged8_select_workspace_bytes(1, 1, 64, 0, 1, 1) == 256 + 64


def test_the_binding_refuses_host_tensors_and_wrong_shapes(paged):
    """Refused before the library is called, so no host pointer reaches a kernel."""
    x = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    pool = torch.zeros((3, 2, 4112), dtype=torch.uint8)
    bounds = torch.zeros((3, 2, 272), dtype=torch.uint8)
    for call in (lambda: paged.qwm_paged8_append(x, x, pool, i.view(2, 2), i, i),
                 lambda: paged.qwm_paged8_read(pool, i.view(2, 2), i, i, 4, 128),
                 lambda: paged.qwm_paged8_attend(x, pool, i.view(2, 2), i, i),
                 lambda: paged.qwm_paged8_bounds(pool, bounds, i.view(2, 2), i, i),
                 lambda: paged.qwm_paged8_bounds(pool, bounds[..., :100], i.view(2, 2), i, i),
                 lambda: paged.qwm_paged8_select(x, bounds, i.view(2, 2), i, i, 16, 2),
                 lambda: paged.qwm_paged8_block_bytes(128, 48)):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ pins of the oracle
def test_oracle_codes_are_e4m3():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(P8.E4M3, want, equal_nan=True)
    r = np.random.default_rng(0)
    x = np.concatenate([r.standard_normal(20000) * np.exp(3 * r.standard_normal(20000)), P8.E4M3[:127],
                        (P8.E4M3[:126] + P8.E4M3[1:127]) / 2, [0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10, -2.0 ** -11]])
    x = np.clip(x, -448, 448).astype(np.float32)
    got = P8.encode(x.astype(np.float64))
    assert np.array_equal(got, torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_oracle_scales_by_hand():
    assert [P8.scale_for(a) for a in (0.0, 448.0, 448.5, 224.0, 57344.0, 28672.5, 1e-9)] == \
        [2.0 ** -15, 1.0, 2.0, 0.5, 128.0, 128.0, 2.0 ** -15]


def test_oracle_append_in_steps_and_error():
    """A block written token by token holds what one written at once does, but for
    codes that a grown scale moved below the normal numbers; every value is
    within half a step of e4m3 (2^-4 relative, 2^-10 of the scale below its normal
    numbers), and twice that where it was moved."""
    r = np.random.default_rng(1)
    d, page, n = 64, 32, 40
    k, v = ((r.standard_normal((n, 1, d)) * np.exp(2 * r.standard_normal((n, 1, 1)))).astype(np.float32) for _ in range(2))
    table = np.array([[1, 0]], np.int32)
    empty = np.full((2, 1, P8.block_bytes(d, page)), 255, np.uint8)
    at_once = P8.append(empty, k, v, table, [n], [0, n], page)[0]
    pool = empty
    for i in range(n):
        pool, kh, _ = P8.append(pool, k[i: i + 1], v[i: i + 1], table, [i + 1], [0, 1], page)
    a, b = (P8.gather(p, table[0], n, 0, d, page)[0] for p in (at_once, pool))
    s = np.array([float(P8.scales_of(pool[table[0, i // page], 0], d, page)[i % page // 16, 0]) for i in range(n)])[:, None]
    assert np.abs(a - b).max(1).max() <= (2.0 ** -9 * s).max()
    err = np.abs(a - k[:, 0])
    assert (err <= np.maximum(2.0 ** -4 * np.abs(k[:, 0]), 2.0 ** -10 * s) * (1 + 1e-9)).all()
    assert (np.abs(b - k[:, 0]) <= 2 * np.maximum(2.0 ** -4 * np.abs(k[:, 0]), 2.0 ** -10 * s) * (1 + 1e-9)).all()


def test_oracle_scores_bound_the_products():
    """Up to the roundings to int8 (half a unit of either factor), a page's score is
    no less than the product of the row with any key in it, and equals it for a
    page of one key within those roundings."""
    r = np.random.default_rng(2)
    d, page, hk = 64, 16, 2
    n = 50
    k = r.standard_normal((n, hk, d)).astype(np.float32)
    table = np.array([[3, 1, 0, 2]], np.int32)
    pool = P8.append(np.full((4, hk, P8.block_bytes(d, page)), 255, np.uint8), k, k, table, [n], [0, n], page)[0]
    bnd = P8.bounds(pool, np.full((4, hk, 2 * d + 16), 255, np.uint8), table, [n], [0, n], page, d)
    q = r.standard_normal((3, d)).astype(np.float32)
    for h in range(hk):
        kh = P8.gather(pool, table[0], n, h, d, page)[0]
        s = P8.scores(q, bnd[:, h], table[0], d)
        for j in range(4):
            keys = kh[j * page: min(n, (j + 1) * page)]
            unit = bnd[table[0, j], h, 2 * d: 2 * d + 4].view(np.float32)[0]
            qu = np.abs(q).max() / 127
            slack = d * 0.5 * (unit * np.abs(q).max() + qu * np.abs(keys).max() + qu * unit)
            assert s[j] >= (q @ keys.T).max() - slack
    P, lens = P8.select(np.repeat(q[:1, None], 2, 1), bnd, table, [n], [0, 1], page, 2, 0, d)
    assert lens[0] == n - 2 * page and (P[0, :, 1] == table[0, 3]).all()
