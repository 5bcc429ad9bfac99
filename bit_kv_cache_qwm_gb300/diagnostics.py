"""Attention-shift diagnostics on synthetic data.

QuantWM Abstract: 2-bit keys have the smaller reconstruction error but the
larger output error, because small key perturbations change QK^T and shift
the tokens queries select.  roboind article: "The key to a smaller error ..."
(key-only vs value-only quantisation), Figure 2 (the highest-scoring
historical token moves) and Table 1 (the fraction of queries whose
highest-scoring historical token changes against BF16).

The caches are built by the library on the GPU (calibrate, append) for three
encodings of the same keys and values: nearest-centroid assignment without
compensation (the QVG-style baseline the pages compare with), QSAC without
compensation, and QSAC with PSAC (rank r); `qwm_dequantize` gives their
keys, values and coefficients in float32, and the comparisons against the
unquantised keys and values run here in torch (float32).  The paged caches'
quantisers (INT4 `qwm_paged_append` and e4m3 `qwm_paged8_append`, no calibration)
are measured next to them on the same keys, values and queries, and for the
attention over selected pages the share of the softmax weight that they hold.  Measured per encoding:
  top1_change        fraction of (head, query) pairs whose argmax token differs
  logit_rel_error    RMS(q.k - l_quant) / RMS(q.k) over all (query, token) pairs
  key_rel_error      ||K - K_hat|| / ||K||  (Frobenius, all heads)
  value_rel_error    ||V - V_hat|| / ||V||
  output_rel_error_key_only    O with quantised (compensated) keys, exact values
  output_rel_error_value_only  O with exact keys, quantised values
  output_rel_error             both quantised (what qwm_attend computes)

  python -m bit_kv_cache_qwm_gb300.diagnostics --workload bf16-h12-n32760 --heads 0,1,2,3 --rows 256

This module is a measurement tool, not part of the product path: its
comparisons run in eager torch on dequantised copies, and no library call
(calibrate, append, attend) uses it.
"""
import argparse
import json

import numpy as np
import torch

from . import synth

ENCODINGS = (("nearest", False), ("qsac", False), ("qsac", True))


def _rel(a, b):
    return float(torch.linalg.vector_norm(a - b) / torch.linalg.vector_norm(b))


def measure(ctx, K, V, q, sigma: float) -> dict:
    """The diagnostics of one cache (a qwm.Qwm context holding exactly the
    keys K and values V [H, N, d], in cache order) for query rows q [H, M, d]
    (float32 tensors on the context's device)."""
    kh, vh, e, valid = ctx.dequantize()
    kh, vh, e = kh[:, valid], vh[:, valid], e[:, valid]
    Lq = q @ kh.transpose(1, 2)
    if ctx.cfg.rank > 0:
        U = torch.from_numpy(ctx.get_calibration()["U"]).to(q.device).float()   # [H, r, d]
        Lq = Lq + (q @ U.transpose(1, 2)) @ e.transpose(1, 2)
    return compare(K, V, q, sigma, kh, vh, Lq)


def measure_paged(K, V, q, sigma: float, page_tokens: int = 64) -> dict:
    """The same diagnostics of the paged cache's INT4 encoding of K and V
    [H, N, d] (bfloat16 or float32), for query rows q [H, M, d] float32."""
    from . import paged
    H, N, d = K.shape
    pool = paged.paged_pool((N + page_tokens - 1) // page_tokens, H, d, page_tokens, device=K.device)
    kh, vh = torch.empty_like(K, dtype=torch.float32), torch.empty_like(V, dtype=torch.float32)
    paged.qwm_paged_append(K.float().transpose(0, 1), V.float().transpose(0, 1), pool, torch.arange(N, device=K.device),
                           k_hat=kh.transpose(0, 1), v_hat=vh.transpose(0, 1))
    return compare(K.float(), V.float(), q, sigma, kh, vh, q @ kh.transpose(1, 2))


def measure_paged8(K, V, q, sigma: float, page_tokens: int = 64, widths=(16, 64)) -> dict:
    """The same diagnostics of the paged 8-bit cache, read back from its pages, and
    `weight_in_N_pages`: the mean share of a row's softmax weight in the N pages
    that the selection names for that row alone, the last page and the first among
    them."""
    from . import paged
    H, N, d = K.shape
    M = q.shape[1]
    n_pages = (N + page_tokens - 1) // page_tokens
    pool = paged.paged8_pool(n_pages, H, d, page_tokens, device=K.device)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=K.device)  # noqa: E731
    table = torch.arange(n_pages, dtype=torch.int32, device=K.device)[None]
    step = table, i32([N]), i32([0, N])
    paged.qwm_paged8_append(K.float().transpose(0, 1), V.float().transpose(0, 1), pool, *step)
    kh, vh = (x.transpose(0, 1) for x in paged.qwm_paged8_read(pool, *step, N, d, dtype=torch.float32))
    res = compare(K.float(), V.float(), q, sigma, kh, vh, q @ kh.transpose(1, 2))
    bounds = paged.paged8_page_bounds(n_pages, H, d, device=K.device)
    paged.qwm_paged8_bounds(pool, bounds, *step, max_new=N)
    # every query as a request's last token
    rows = q.float().transpose(0, 1).contiguous()
    P = torch.softmax(sigma * (q @ kh.transpose(1, 2)), dim=-1)
    P = torch.nn.functional.pad(P, (0, n_pages * page_tokens - N)).unflatten(-1, (n_pages, page_tokens)).sum(-1)
    most = 8192                                                # requests of a call
    for width in widths:
        parts = []
        for at in range(0, max(M, 1), most):
            m = min(most, M - at)
            parts.append(paged.qwm_paged8_select(rows[at: at + m], bounds, table.expand(m, -1).contiguous(), i32([N] * m),
                                                 torch.arange(m + 1, dtype=torch.int32, device=K.device), page_tokens, width, sink=1)[0])
        pages = torch.cat(parts)
        held = torch.gather(P, 2, pages.transpose(0, 1).long().clamp(min=0)) * (pages.transpose(0, 1) >= 0)
        res[f"weight_in_{width}_pages"] = float(held.sum(-1).mean())
    return res


def compare(K, V, q, sigma: float, kh, vh, Lq) -> dict:
    """The diagnostics of quantised keys kh, values vh and logits Lq against
    the exact ones (all float32)."""
    L = q @ K.transpose(1, 2)                                   # exact logits [H, M, N]
    P = torch.softmax(sigma * L, dim=-1)
    O = P @ V
    Pq = torch.softmax(sigma * Lq, dim=-1)
    return {
        "top1_change": float((Lq.argmax(dim=-1) != L.argmax(dim=-1)).float().mean()),
        "logit_rel_error": float(torch.sqrt(((L - Lq) ** 2).mean() / (L ** 2).mean())),
        "key_rel_error": _rel(kh, K),
        "value_rel_error": _rel(vh, V),
        "output_rel_error_key_only": _rel(Pq @ V, O),
        "output_rel_error_value_only": _rel(P @ vh, O),
        "output_rel_error": _rel(Pq @ vh, O),
    }


def run(workload: str, heads=None, rows: int = 256, n_chunks=None, device=None) -> dict:
    """The three encodings of the workload's keys and values (all appends, or
    the first n_chunks) for `rows` query rows of the given heads."""
    from . import qwm
    wl = synth.workload(workload)
    heads = list(range(wl.heads)) if heads is None else list(heads)
    H, d, C, r = len(heads), wl.head_dim, wl.n_centroids, wl.rank
    n_chunks = wl.n_chunks if n_chunks is None else n_chunks
    dev = torch.device("cuda", 0) if device is None else torch.device(device)
    tdt = torch.bfloat16 if wl.dtype == "bf16" else torch.float32
    T = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dev, tdt)
    ks = [T(synth.keys(wl, ch, heads)) for ch in range(n_chunks)]
    vs = [T(synth.values(wl, ch, heads)) for ch in range(n_chunks)]
    K = torch.cat(ks, dim=1).float()
    V = torch.cat(vs, dim=1).float()
    q = T(synth.queries(wl, 0, heads, m=rows)).float()
    qh = T(synth.hist_queries(wl, 0, heads))
    kf = synth.kmeans_keys(wl, heads)
    init = np.stack([synth.kmeans_init_rows(wl, h, kf.shape[1], C) for h in heads]).astype(np.int32)
    cent = qwm.qwm_kmeans(T(kf), torch.from_numpy(init).to(dev), C, iters=25 if C <= 256 else 5)
    tiles = n_chunks * ((wl.chunk + 127) // 128)
    out = {"workload": wl.name, "heads": heads, "tokens": int(K.shape[1]), "query_rows": rows,
           "rank": r, "n_centroids": C, "encodings": {}}
    for assign, psac in ENCODINGS:
        rank = r if psac else 0
        ctx = qwm.Qwm(H, d, rank, C, dtype=wl.dtype, max_tokens=tiles * 128, max_hist=qh.shape[1], device=dev)
        ctx.set_centroids(cent)
        ctx.set_assignment(assign)
        ctx.calibrate(qh)
        for k, v in zip(ks, vs):
            ctx.append(k, v)
        res = measure(ctx, K, V, q, 1.0 / np.sqrt(d))
        assert ctx.status() == 0
        out["encodings"][f"{assign}{'+psac' if psac else ''}"] = res
        ctx.close()
    out["paged_int4"] = measure_paged(K, V, q, 1.0 / np.sqrt(d))
    out["paged_e4m3"] = measure_paged8(K, V, q, 1.0 / np.sqrt(d))
    return out


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--workload", default="bf16-h12-n32760")
    ap.add_argument("--heads", default="", help="comma-separated head indices (default: all)")
    ap.add_argument("--rows", type=int, default=256)
    ap.add_argument("--chunks", type=int, default=0)
    a = ap.parse_args()
    heads = [int(x) for x in a.heads.split(",")] if a.heads else None
    print(json.dumps(run(a.workload, heads, a.rows, a.chunks or None)))


if __name__ == "__main__":
    main()
