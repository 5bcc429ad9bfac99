"""Thin Python binding of libqwm's paged 4-bit cache (ctypes).

Argument checks and marshalling only; every step runs in the CUDA library, on
the device of its tensors and that device's current stream.  Nothing is kept
between calls: pools, tables and lengths are the caller's tensors, and the
attention's workspace comes from torch's allocator call by call, so calls on
different streams and captured graphs share nothing.

A serving step:

    plan = qwm_paged_plan(kv_len, new_len, table, free_pages, free_count, page_tokens, rows)
    # per layer
    q, k = qwm_qk_norm_rope(q, k, w_q, w_k, cos_sin, plan.positions)
    qwm_paged_append(k, v, pool, plan.slots)
    o = qwm_paged_attend(q, pool, table, plan.kv_len, plan.cu_rows, max_new)
"""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple, Optional, Sequence

import torch

from .qwm import QWM_BF16, QWM_F32, _check, lib

PAGE_TOKENS = (16, 32, 64, 128, 256)
# attention kernels (the `kernel` argument of qwm_paged_attend): automatic
# choice, float32 CUDA cores, bf16 mma.sync for few rows, bf16 tcgen05
PAGED_AUTO, PAGED_SIMT, PAGED_MMA, PAGED_TC = 0, 1, 2, 3

# The argument structs of include/qwm.h, packed in one call each: a pointer or
# 64-bit field is q, a 32-bit one i or f, in the header's order.
_ROPE = struct.Struct("=19q11if")
_PLAN = struct.Struct("=13q3i4x")
_RELEASE = struct.Struct("=7q3i4x")
_APPEND = struct.Struct("=17q4i")
_ATTEND = struct.Struct("=17q9ifi4x")

_Tensor, _BF16, _F32, _I32, _I64 = torch.Tensor, torch.bfloat16, torch.float32, torch.int32, torch.int64
_DTYPES = {torch.bfloat16: QWM_BF16, torch.float32: QWM_F32}
_workspace_bytes: dict = {}
_INT_MAX = 2 ** 31 - 1   # a window beyond it is one as well


class PagedPlan(NamedTuple):
    """What qwm_paged_plan writes (see include/qwm.h)."""
    kv_len: torch.Tensor       # int32 [requests], with the new tokens
    free_count: torch.Tensor   # int32 [1]
    cu_rows: torch.Tensor      # int32 [requests + 1]
    slots: torch.Tensor        # int64 [rows]
    positions: torch.Tensor    # int32 [rows]


# the handle of a device's current stream, without building a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _run(fn, args: bytes, what: str, index: int):
    """fn(args) on device `index` and its current stream."""
    if index == _current_device():
        st = fn(args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(args, _raw_stream(index))
    if st:
        _check(st, what)


# The checks read each attribute of a tensor once, and the number of its device
# (-1: the CPU) for the device itself: a small step costs the host more than
# the GPU.

def _rows(x, what: str, dtype=None, index=None, shape=None):
    """A CUDA tensor [rows, heads, d] in bf16 or float32 with contiguous heads
    of 16-byte aligned vectors (any row and head stride), and where given of
    `dtype` on device `index` and of `shape`; returns (pointer, row stride,
    head stride)."""
    if not isinstance(x, _Tensor) or not x.is_cuda:
        raise ValueError(f"{what}: a CUDA tensor is expected")
    dt, have = x.dtype, x.shape
    if len(have) != 3 or dt not in _DTYPES:
        raise ValueError(f"{what}: a bfloat16 or float32 tensor [rows, heads, d] is expected, got {dt} {tuple(have)}")
    if dtype is not None and (dt is not dtype or x.get_device() != index):
        raise ValueError(f"{what}: expected {dtype} on cuda:{index}, got {dt} on {x.device}")
    if shape is not None and have != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(have)}")
    s0, s1, s2 = x.stride()
    if have[0] <= 1:
        s0 = 0
    if have[1] <= 1:
        s1 = 0
    if s2 != 1 and have[2] != 1:
        raise ValueError(f"{what}: the channels of a head have to be contiguous")
    p = x.data_ptr()
    if (p | (s0 | s1) * (2 if dt is _BF16 else 4)) & 15:
        raise ValueError(f"{what}: pointer and strides have to be multiples of 16 bytes")
    return p, s0, s1


def _like(x):
    """An uninitialised contiguous tensor like x, and its pointer and strides."""
    y = torch.empty_like(x, memory_format=torch.contiguous_format)
    _, h, d = x.shape
    return y, (y.data_ptr(), h * d, d)


def _array(x, what: str, dtype, shape, index: int):
    """The pointer of a contiguous tensor of `dtype` and `shape` (None: any) on device `index`."""
    if not isinstance(x, _Tensor) or x.get_device() != index:
        raise ValueError(f"{what}: a tensor on cuda:{index} is expected")
    have = x.shape
    if x.dtype is not dtype or len(have) != len(shape) or not x.is_contiguous():
        raise ValueError(f"{what}: a contiguous {len(shape)}-d {dtype} tensor is expected, got {x.dtype} {tuple(have)}")
    if have != shape:
        for n, want in zip(have, shape):
            if want is not None and n != want:
                raise ValueError(f"{what}: expected shape {tuple('any' if w is None else w for w in shape)}, got {tuple(have)}")
    return x.data_ptr()


def _status(x, index: int):
    return 0 if x is None else _array(x, "status", _I32, (1,), index)


def _page_tokens(pool, d: int) -> int:
    """Tokens of a page of `pool` [pages, kv_heads, block] for heads of d channels."""
    if not isinstance(pool, _Tensor) or not pool.is_cuda or pool.dtype is not torch.uint8 or pool.dim() != 3 \
            or not pool.is_contiguous():
        raise ValueError("pool: a contiguous CUDA uint8 tensor [pages, kv_heads, block bytes] is expected")
    page, rest = divmod(4 * pool.shape[2], 5 * d)
    if rest or page not in PAGE_TOKENS:
        raise ValueError(f"pool: {pool.shape[2]} bytes are no block of a page of {PAGE_TOKENS} tokens at d = {d}")
    return page


def qwm_paged_block_bytes(head_dim: int, page_tokens: int) -> int:
    """Bytes of one block: page_tokens slots of one key/value head."""
    n = int(lib().qwm_paged_block_bytes(head_dim, page_tokens))
    if n == 0:
        raise ValueError(f"head_dim 64 or 128 and page_tokens of {PAGE_TOKENS} are built, not {head_dim} and {page_tokens}")
    return n


def paged_pool(n_pages: int, kv_heads: int, head_dim: int, page_tokens: int, device=None) -> torch.Tensor:
    """An uninitialised pool [n_pages, kv_heads, block bytes] (one per layer)."""
    return torch.empty((n_pages, kv_heads, qwm_paged_block_bytes(head_dim, page_tokens)), dtype=torch.uint8,
                       device="cuda" if device is None else device)


def qwm_qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], q_weight: Optional[torch.Tensor],
                     k_weight: Optional[torch.Tensor], cos_sin: torch.Tensor, positions: torch.Tensor, eps: float = 1e-6,
                     interleaved: bool = False, sections: Optional[Sequence[int]] = None,
                     q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None):
    """RMS norm of every head of q [rows, heads, d] and k [rows, kv_heads, d]
    (None: queries alone) and the rotation of their first cos_sin.shape[1]
    channels, in one pass.  cos_sin: float32 [n_positions, rot]; positions:
    int32 [rows] or [rows, axes], with `sections` pairs for each axis; a
    negative position leaves the row of an output given by the caller as it
    was.  Returns (q_out, k_out), new tensors where none are given; q_out = q
    works in place."""
    qr = _rows(q, "q")
    T, hq, d = q.shape
    dev, dt = q.get_device(), q.dtype
    if q_out is None:
        q_out, qo = _like(q)
    else:
        qo = _rows(q_out, "q_out", dt, dev, q.shape)
    hk, kr, ko = 0, (0, 0, 0), (0, 0, 0)
    if k is not None:
        kr = _rows(k, "k", dt, dev)
        tk, hk, dk = k.shape
        if tk != T or dk != d:
            raise ValueError(f"k: expected [{T}, kv_heads, {d}], got {tuple(k.shape)}")
        if k_out is None:
            k_out, ko = _like(k)
        else:
            ko = _rows(k_out, "k_out", dt, dev, k.shape)
    elif k_out is not None or k_weight is not None:
        raise ValueError("k_out, k_weight: given without k")
    table = _array(cos_sin, "cos_sin", _F32, (None, None), dev)
    n_pos, rot = cos_sin.shape
    axes = positions.shape[1] if isinstance(positions, _Tensor) and positions.dim() == 2 else 0
    pos = _array(positions, "positions", _I32, (T, axes) if axes else (T,), dev)
    axes = axes or 1
    if axes > 4:
        raise ValueError("positions: 1 to 4 axes")
    if sections is None:
        if axes > 1:
            raise ValueError("sections: needed with several axes")
        s = (rot // 2, 0, 0, 0)
    else:
        s = tuple(sections)
        if len(s) != axes or sum(s) != rot // 2 or min(s) < 0:
            raise ValueError(f"sections: {axes} counts with the sum {rot // 2} are expected, got {s}")
        s += (0,) * (4 - axes)
    wq = 0 if q_weight is None else _array(q_weight, "q_weight", dt, (d,), dev)
    wk = 0 if k_weight is None else _array(k_weight, "k_weight", dt, (d,), dev)
    _run(lib().qwm_qk_norm_rope,
         _ROPE.pack(*qr, *kr, *qo, *ko, wq, wk, table, pos, _status(status, dev), T, n_pos, _DTYPES[dt], d, hq, hk, rot, axes,
                    *s, 1 if interleaved else 0, eps), "qwm_qk_norm_rope", dev)
    return q_out, k_out


def qwm_paged_plan(kv_len: torch.Tensor, new_len: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                   free_count: torch.Tensor, page_tokens: int, rows: int, out: Optional[PagedPlan] = None,
                   status: Optional[torch.Tensor] = None) -> PagedPlan:
    """Pages, slots and positions of a step that adds new_len[b] tokens to each
    request (int32 tensors on the GPU; `rows` rows of storage, at least the
    sum of new_len as the host knows it).  block_table is updated in place;
    the rest is returned, in `out` where given (its kv_len and free_count may
    be the inputs themselves).  Nothing changes when it does not fit: then
    cu_rows is 0 throughout, every slot -1, and `status` has DEV_CAPACITY."""
    if not isinstance(kv_len, _Tensor) or not kv_len.is_cuda:
        raise ValueError("kv_len: a CUDA tensor is expected")
    dev, i32 = kv_len.get_device(), _I32
    a = _array(kv_len, "kv_len", i32, (None,), dev)
    B = kv_len.shape[0]
    b = _array(new_len, "new_len", i32, (B,), dev)
    c = _array(free_pages, "free_pages", i32, (None,), dev)
    d = _array(free_count, "free_count", i32, (1,), dev)
    e = _array(block_table, "block_table", i32, (B, None), dev)
    if out is None:
        # an allocation each: views of a common one cost more
        at, new = kv_len.device, torch.empty
        lens, left, cu = torch.empty_like(kv_len), torch.empty_like(free_count), new(B + 1, dtype=i32, device=at)
        slots, positions = new(rows, dtype=_I64, device=at), new(rows, dtype=i32, device=at)
        out = PagedPlan(lens, left, cu, slots, positions)
        ptr = (lens.data_ptr(), left.data_ptr(), cu.data_ptr(), slots.data_ptr(), positions.data_ptr())
    else:
        ptr = (_array(out.kv_len, "out.kv_len", i32, (B,), dev), _array(out.free_count, "out.free_count", i32, (1,), dev),
               _array(out.cu_rows, "out.cu_rows", i32, (B + 1,), dev), _array(out.slots, "out.slots", _I64, (rows,), dev),
               _array(out.positions, "out.positions", i32, (rows,), dev))
    _run(lib().qwm_paged_plan,
         _PLAN.pack(a, b, c, d, e, *ptr, _status(status, dev), rows, free_pages.shape[0], B, block_table.shape[1],
                    page_tokens), "qwm_paged_plan", dev)
    return out


def qwm_paged_release(keep_len: torch.Tensor, kv_len: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                      free_count: torch.Tensor, page_tokens: int, status: Optional[torch.Tensor] = None):
    """Cut every request back to keep_len[b] tokens (0: it ends) and push the
    pages it gives up on the free stack; kv_len, block_table, free_pages and
    free_count are updated in place."""
    if not isinstance(kv_len, _Tensor) or not kv_len.is_cuda:
        raise ValueError("kv_len: a CUDA tensor is expected")
    dev, i32 = kv_len.get_device(), _I32
    a = _array(kv_len, "kv_len", i32, (None,), dev)
    B = kv_len.shape[0]
    _run(lib().qwm_paged_release,
         _RELEASE.pack(_array(keep_len, "keep_len", i32, (B,), dev), a, _array(block_table, "block_table", i32, (B, None), dev),
                       _array(free_pages, "free_pages", i32, (None,), dev), _array(free_count, "free_count", i32, (1,), dev),
                       _status(status, dev), free_pages.shape[0], B, block_table.shape[1], page_tokens),
         "qwm_paged_release", dev)


def qwm_paged_append(k: torch.Tensor, v: torch.Tensor, pool: torch.Tensor, slots: torch.Tensor,
                     k_hat: Optional[torch.Tensor] = None, v_hat: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None):
    """Quantise keys and values [rows, kv_heads, d] to 4 bits into the slots
    (int64 [rows], -1: no slot) of the pool.  k_hat, v_hat receive the values
    that the stored bytes stand for (0 in rows without a slot)."""
    kr = _rows(k, "k")
    shape, dt, dev = k.shape, k.dtype, k.get_device()
    T, hk, d = shape
    vr = _rows(v, "v", dt, dev, shape)
    page = _page_tokens(pool, d)
    n_pages, hp, _ = pool.shape
    if pool.get_device() != dev or hp != hk:
        raise ValueError(f"pool: expected [pages, {hk}, block] on {k.device}, got {tuple(pool.shape)} on {pool.device}")
    kh = (0, 0, 0) if k_hat is None else _rows(k_hat, "k_hat", dt, dev, shape)
    vh = (0, 0, 0) if v_hat is None else _rows(v_hat, "v_hat", dt, dev, shape)
    _run(lib().qwm_paged_append,
         _APPEND.pack(*kr, *vr, *kh, *vh, pool.data_ptr(), _array(slots, "slots", _I64, (T,), dev), _status(status, dev),
                      T, n_pages, _DTYPES[dt], d, hk, page), "qwm_paged_append", dev)


def _workspace_size(dev: int, d: int) -> int:
    with torch.cuda.device(dev):
        n = int(lib().qwm_paged_attend_workspace_bytes(d))
    if n == 0:
        raise ValueError(f"head_dim 64 or 128 is built, not {d}")
    _workspace_bytes[dev, d] = n
    return n


def qwm_paged_attend(q: torch.Tensor, pool: torch.Tensor, block_table: torch.Tensor, kv_len: torch.Tensor,
                     cu_rows: torch.Tensor, max_new: Optional[int] = None, causal: bool = True, window: int = 0,
                     scale: float = 0.0, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None, kernel: int = PAGED_AUTO) -> torch.Tensor:
    """Attention of the rows of a plan, q [rows, heads, d], over their
    requests' pages (kv_len and cu_rows as qwm_paged_plan returns them).
    max_new: the most rows of one request as the host knows it.  It chooses the
    kernel; absent it is all rows, which runs single tokens of many requests on
    the kernel for prompts, three times slower.  Single tokens and prompts in one step are
    better two calls, on slices block_table[a:b], kv_len[a:b] and
    cu_rows[a:b + 1] with the same q and out.  window > 0: only the last
    `window` tokens up to the row's own.  lse: float32 [rows, heads] to receive
    the log-sum-exp.  Rows behind the last request are left as they were in
    `out`.  status: where a page out of range, or a device wait that ran out
    (its rows are NaN), is reported."""
    qr = _rows(q, "q")
    T, hq, d = q.shape
    dev, dt = q.get_device(), q.dtype
    page = _page_tokens(pool, d)
    n_pages, hk, _ = pool.shape
    if pool.get_device() != dev or hk < 1 or hq % hk:
        raise ValueError(f"pool: kv heads that divide {hq} on {q.device} are expected, got {tuple(pool.shape)} on {pool.device}")
    if out is None:
        out, ot = _like(q)
    else:
        ot = _rows(out, "out", dt, dev, q.shape)
    table = _array(block_table, "block_table", _I32, (None, None), dev)
    B, width = block_table.shape
    lens = _array(kv_len, "kv_len", _I32, (B,), dev)
    cu = _array(cu_rows, "cu_rows", _I32, (B + 1,), dev)
    ls = 0 if lse is None else _array(lse, "lse", _F32, (T, hq), dev)
    n_ws = _workspace_bytes.get((dev, d)) or _workspace_size(dev, d)
    ws = pool.new_empty(n_ws)
    _run(lib().qwm_paged_attend,
         _ATTEND.pack(*qr, *ot, ls, pool.data_ptr(), table, lens, cu, _status(status, dev), ws.data_ptr(), n_ws, T, n_pages,
                      T if max_new is None else max_new, _DTYPES[dt], d, hq, hk, page, B, width, 1 if causal else 0,
                      min(window, _INT_MAX), scale, kernel), "qwm_paged_attend", dev)
    return out


def paged_attend_kernel_for(dtype: torch.dtype, heads: int, kv_heads: int, max_new: int) -> int:
    """The attention kernel (PAGED_SIMT, PAGED_MMA or PAGED_TC) of the automatic choice."""
    return int(lib().qwm_paged_attend_kernel_for(_DTYPES[dtype], heads, kv_heads, max_new))
