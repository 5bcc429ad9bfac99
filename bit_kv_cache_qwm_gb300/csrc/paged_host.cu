// Host side of the paged caches: argument checks, kernel choice and
// launches.  Nothing is kept between calls and nothing is allocated.
#include <math.h>
#include <string.h>

#include "paged_internal.cuh"
#include "paged_launch.cuh"
#include "tcgen05_util.cuh"

using namespace qwm;
using namespace qwm::paged;

namespace {

cudaStream_t S(void* p) { return reinterpret_cast<cudaStream_t>(p); }
qwm_status cuda_status(cudaError_t e) { return e == cudaSuccess ? QWM_OK : QWM_ERR_CUDA; }

// log2 of a page size that is built, else -1
int page_shift(int32_t page) {
  for (int s = 4; s <= 8; ++s)
    if (page == 1 << s) return s;
  return -1;
}

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
// every one a multiple of 4 bytes (NULL is): a kernel that reads an int32 or a
// float elsewhere faults
template <class... P>
bool words(const P*... p) {
  return (aligned(p, 4) && ...);
}

constexpr int64_t kMaxStride = (int64_t)1 << 40;

// A caller's rows: 16-byte aligned vectors everywhere; an output's elements
// must not share an address.
bool rows_ok(const qwm_rows& r, int64_t rows, int64_t heads, int d, int esz, bool output) {
  if (!r.ptr || !aligned(r.ptr, 16)) return false;
  if (r.row_stride < 0 || r.head_stride < 0 || r.row_stride > kMaxStride || r.head_stride > kMaxStride) return false;
  if ((rows > 1 && (r.row_stride * esz) % 16) || (heads > 1 && (r.head_stride * esz) % 16)) return false;
  if (!output) return true;
  const bool row_inner = rows > 1 && (heads <= 1 || r.row_stride < r.head_stride);
  const int64_t si = row_inner ? r.row_stride : r.head_stride, ni = row_inner ? rows : heads;
  const int64_t so = row_inner ? r.head_stride : r.row_stride, no = row_inner ? heads : rows;
  int64_t span = d;
  if (ni > 1) {
    if (si < span) return false;
    if (si > INT64_MAX / 4 / ni) return false;
    span += si * (ni - 1);
  }
  return no <= 1 || so >= span;
}

bool dtype_ok(int32_t t) { return t == QWM_F32 || t == QWM_BF16; }
int esize(int32_t t) { return t == QWM_F32 ? 4 : 2; }
bool dim_ok(int32_t d) { return d == 64 || d == 128; }

constexpr int64_t kInt = 0x7fffffff, kHalf = (int64_t)1 << 30;

// workspace: a word for timeouts, the parts, then one Join per worker
constexpr size_t kHead = 256;
size_t part_bytes(Workers w, int d) { return (size_t)w.count * 2 * w.rows * part_floats(d) * 4; }

}  // namespace

extern "C" size_t qwm_paged_block_bytes(int32_t head_dim, int32_t page_tokens) {
  return dim_ok(head_dim) && page_shift(page_tokens) >= 0 ? (size_t)block_bytes(head_dim, page_tokens) : 0;
}

extern "C" qwm_status qwm_qk_norm_rope(const qwm_qk_norm_rope_args* a, void* stream) {
  if (!a || !dtype_ok(a->dtype) || a->rows < 0 || a->rows > kInt || a->q_heads < 1 || a->k_heads < 0 ||
      a->q_heads > 65536 || a->k_heads > 65536 || a->axes < 1 || a->axes > 4 || a->rot < 16 || a->rot % 16 ||
      a->n_positions < 1 || a->n_positions > kInt || !(a->eps >= 0.f))
    return QWM_ERR_INVALID_ARG;
  if (!dim_ok(a->head_dim)) return QWM_ERR_UNSUPPORTED;
  if (a->rot > a->head_dim) return QWM_ERR_INVALID_ARG;
  int64_t pairs = 0;
  for (int i = 0; i < a->axes; ++i) {
    if (a->sections[i] < 0) return QWM_ERR_INVALID_ARG;
    pairs += a->sections[i];
  }
  if (a->axes > 1 && pairs != a->rot / 2) return QWM_ERR_INVALID_ARG;
  if (a->rows == 0) return QWM_OK;
  const int e = esize(a->dtype);
  if (!rows_ok(a->q, a->rows, a->q_heads, a->head_dim, e, false) ||
      !rows_ok(a->q_out, a->rows, a->q_heads, a->head_dim, e, true))
    return QWM_ERR_INVALID_ARG;
  if (a->k_heads > 0 && (!rows_ok(a->k, a->rows, a->k_heads, a->head_dim, e, false) ||
                         !rows_ok(a->k_out, a->rows, a->k_heads, a->head_dim, e, true)))
    return QWM_ERR_INVALID_ARG;
  if (!a->cos_sin || !aligned(a->cos_sin, 16) || !a->positions || !words(a->positions, a->status) ||
      !aligned(a->q_weight, 16) || !aligned(a->k_weight, 16))
    return QWM_ERR_INVALID_ARG;
  if (fault_injected("launch")) return QWM_ERR_CUDA;
  NvtxRange range("qwm_qk_norm_rope");
  return cuda_status(launch_qk_norm_rope(*a, S(stream)));
}

extern "C" qwm_status qwm_paged_plan(const qwm_paged_plan_args* a, void* stream) {
  if (!a || a->requests < 1 || a->max_blocks < 1 || a->rows < 0 || a->rows > kInt || a->n_pages < 1 ||
      a->n_pages > kInt || page_shift(a->page_tokens) < 0)
    return QWM_ERR_INVALID_ARG;
  if (a->requests > kMaxRequests) return QWM_ERR_UNSUPPORTED;
  if (!a->kv_len || !a->new_len || !a->free_pages || !a->free_count || !a->block_table || !a->kv_len_out ||
      !a->free_count_out || !a->cu_rows || (a->rows > 0 && (!a->slots || !a->positions)) || !aligned(a->slots, 8) ||
      !words(a->kv_len, a->new_len, a->free_pages, a->free_count, a->block_table, a->kv_len_out, a->free_count_out,
             a->cu_rows, a->positions, a->status))
    return QWM_ERR_INVALID_ARG;
  if (fault_injected("launch")) return QWM_ERR_CUDA;
  NvtxRange range("qwm_paged_plan");
  return cuda_status(launch_plan(*a, page_shift(a->page_tokens), S(stream)));
}

extern "C" qwm_status qwm_paged_release(const qwm_paged_release_args* a, void* stream) {
  if (!a || a->requests < 1 || a->max_blocks < 1 || a->n_pages < 1 || a->n_pages > kInt ||
      page_shift(a->page_tokens) < 0)
    return QWM_ERR_INVALID_ARG;
  if (a->requests > kMaxRequests) return QWM_ERR_UNSUPPORTED;
  if (!a->keep_len || !a->kv_len || !a->block_table || !a->free_pages || !a->free_count ||
      !words(a->keep_len, a->kv_len, a->block_table, a->free_pages, a->free_count, a->status))
    return QWM_ERR_INVALID_ARG;
  if (fault_injected("launch")) return QWM_ERR_CUDA;
  NvtxRange range("qwm_paged_release");
  return cuda_status(launch_release(*a, page_shift(a->page_tokens), S(stream)));
}

extern "C" qwm_status qwm_paged_append(const qwm_paged_append_args* a, void* stream) {
  if (!a || !dtype_ok(a->dtype) || a->rows < 0 || a->rows > kInt || a->kv_heads < 1 || a->kv_heads > 65536 ||
      a->n_pages < 1 || a->n_pages > kInt)
    return QWM_ERR_INVALID_ARG;
  const int shift = page_shift(a->page_tokens);
  if (!dim_ok(a->head_dim) || shift < 0) return QWM_ERR_UNSUPPORTED;
  if (a->rows == 0) return QWM_OK;
  const int e = esize(a->dtype);
  if (!rows_ok(a->k, a->rows, a->kv_heads, a->head_dim, e, false) ||
      !rows_ok(a->v, a->rows, a->kv_heads, a->head_dim, e, false))
    return QWM_ERR_INVALID_ARG;
  if ((a->k_hat.ptr && !rows_ok(a->k_hat, a->rows, a->kv_heads, a->head_dim, e, true)) ||
      (a->v_hat.ptr && !rows_ok(a->v_hat, a->rows, a->kv_heads, a->head_dim, e, true)))
    return QWM_ERR_INVALID_ARG;
  if (!a->pool || !aligned(a->pool, 16) || !a->slots || !aligned(a->slots, 8) || !words(a->status))
    return QWM_ERR_INVALID_ARG;
  if (a->rows * a->kv_heads > kInt) return QWM_ERR_UNSUPPORTED;
  if (fault_injected("launch")) return QWM_ERR_CUDA;
  NvtxRange range("qwm_paged_append");
  return cuda_status(launch_append(*a, shift, S(stream)));
}

namespace {
size_t attend_workspace(int32_t head_dim, int bits) {
  if (!dim_ok(head_dim)) return 0;
  size_t n = 0, w = 0;
  for (const Workers& x : {simt_workers(1), simt_workers(64), mma_workers(1, bits, false, head_dim), mma_workers(16, bits, false, head_dim), tc_workers()}) {
    const size_t b = part_bytes(x, head_dim);
    n = b > n ? b : n;
    w = (size_t)x.count > w ? (size_t)x.count : w;
  }
  return kHead + ((n + 255) & ~(size_t)255) + w * sizeof(Join);
}
}  // namespace

extern "C" size_t qwm_paged_attend_workspace_bytes(int32_t head_dim) { return attend_workspace(head_dim, 4); }
extern "C" size_t qwm_paged8_attend_workspace_bytes(int32_t head_dim) { return attend_workspace(head_dim, 8); }

extern "C" int32_t qwm_paged_attend_kernel_for(int32_t dtype, int32_t heads, int32_t kv_heads, int64_t max_new) {
  if (!dtype_ok(dtype) || heads < 1 || kv_heads < 1 || heads % kv_heads || max_new < 0) return -1;
  if (dtype == QWM_F32) return 1;
  // Kernel 2 reads the pages once for 16 rows of a key/value head, kernel 3 once
  // for 256, of which few rows leave most of its tensor work and softmax empty.
  // Measured, kernel 2 against 3 in us, d = 128: 48 ragged requests (200 to 16,380
  // tokens, 32 heads over 8) 106 and 324 at 4 rows, 149 and 325 at 16, 279 and 325
  // at 20, 281 and 327 at 32, where it reads twice, 411 and 327 at 36; four
  // requests of up to 1,000 tokens 17 and 29 at 32; one of 98,280 tokens 80 and 95
  // at 30.
  return max_new <= 32 && max_new * (heads / kv_heads) <= 32 ? 2 : 3;   // the product stays small
}

namespace {
// Either cache's attention; table_heads: tables a request has.
qwm_status attend(const qwm_paged_attend_args* a, int bits, int table_heads, const char* name, void* stream) {
  if (!dtype_ok(a->dtype) || a->rows < 0 || a->rows > kInt || a->heads < 1 || a->heads > 65536 ||
      a->kv_heads < 1 || a->kv_heads > a->heads || a->heads % a->kv_heads || a->requests < 0 || a->max_blocks < 1 ||
      a->n_pages < 1 || a->n_pages > kInt || a->window < 0 || (a->window > 0 && !a->causal) || a->max_new < 0 ||
      a->kernel < 0 || a->kernel > 3 || !(fabsf(a->scale) < INFINITY))
    return QWM_ERR_INVALID_ARG;
  const int shift = page_shift(a->page_tokens), d = a->head_dim;
  if (!dim_ok(d) || shift < 0) return QWM_ERR_UNSUPPORTED;
  const int group = a->heads / a->kv_heads, block = bits == 4 ? block_bytes(d, a->page_tokens) : block8_bytes(d, a->page_tokens);
  // positions and the rows of one kv head's problem are kept in 32 bits
  if (a->rows * group > kHalf || (int64_t)a->max_blocks * a->page_tokens > kHalf ||
      (int64_t)a->kv_heads * block > kInt)
    return QWM_ERR_UNSUPPORTED;
  if (a->rows == 0 || a->requests == 0) return QWM_OK;
  const int e = esize(a->dtype);
  if (!rows_ok(a->q, a->rows, a->heads, d, e, false) || !rows_ok(a->out, a->rows, a->heads, d, e, true))
    return QWM_ERR_INVALID_ARG;
  if (!a->pool || !aligned(a->pool, 16) || !a->block_table || !a->kv_len || !a->cu_rows || !a->workspace ||
      !aligned(a->workspace, 256) || a->workspace_bytes < attend_workspace(d, bits) ||
      !words(a->block_table, a->kv_len, a->cu_rows, a->lse, a->status))
    return QWM_ERR_INVALID_ARG;
  // keys and values of 8 bits are exact in float16, so that kernel 2 does float32 too,
  // with two terms of each query and weight: three windowed requests of 30 to 260
  // tokens 25.0 us, 47.6 on the CUDA cores
  const bool f32 = a->dtype == QWM_F32;
  const int k = a->kernel ? a->kernel : f32 && bits == 8 ? 2 : qwm_paged_attend_kernel_for(a->dtype, a->heads, a->kv_heads, a->max_new);
  if (f32 && k != 1 && !(k == 2 && bits == 8)) return QWM_ERR_UNSUPPORTED;
  if (fault_injected("launch")) return QWM_ERR_CUDA;
  NvtxRange range(name);
  const int64_t max_rows = (a->max_new < 1 ? 1 : a->max_new > a->rows ? a->rows : a->max_new) * group;
  const Workers w = k == 1 ? simt_workers(max_rows) : k == 2 ? mma_workers(max_rows, bits, f32, d) : tc_workers();
  AttendArgs x;
  memset(&x, 0, sizeof(x));
  x.q = a->q.ptr;
  x.q_row = a->q.row_stride;
  x.q_head = a->q.head_stride;
  x.out = a->out.ptr;
  x.o_row = a->out.row_stride;
  x.o_head = a->out.head_stride;
  x.lse = a->lse;
  x.pool = (const uint8_t*)a->pool;
  x.table = a->block_table;
  x.kv_len = a->kv_len;
  x.cu = a->cu_rows;
  x.status = a->status;
  x.timeout = a->status ? a->status : (uint32_t*)a->workspace;
  x.wait_cycles = injected_wait_cycles(tcx::kWaitCycles);
  x.part = (float*)((uint8_t*)a->workspace + kHead);
  x.join = (Join*)((uint8_t*)a->workspace + kHead + ((part_bytes(w, d) + 255) & ~(size_t)255));
  x.rows = a->rows;
  x.n_pages = (int32_t)a->n_pages;
  x.heads = a->heads;
  x.kv_heads = a->kv_heads;
  x.group = group;
  fast_division(group, &x.group_mul, &x.group_shift);
  x.page = a->page_tokens;
  x.page_shift = shift;
  x.block = block;
  x.bits = bits;
  x.table_h = table_heads > 1 ? a->max_blocks : 0;
  x.table_b = (int64_t)table_heads * a->max_blocks;
  x.requests = a->requests;
  x.max_blocks = a->max_blocks;
  x.causal = a->causal != 0;
  // a window as long as the tables hides nothing
  x.window = a->window >= (int64_t)a->max_blocks * a->page_tokens ? 0 : a->window;
  const float scale = a->scale > 0.f ? a->scale : 1.0f / sqrtf((float)d);
  x.scale_log2 = scale * 1.4426950408889634f;
  x.magic = 0x64006400u;
  return cuda_status(k == 1 ? launch_attend_simt(x, d, a->dtype == QWM_BF16, max_rows, S(stream))
                     : k == 2 ? launch_attend_mma(x, d, f32, max_rows, S(stream))
                              : launch_attend_tc(x, d, max_rows, S(stream)));
}
}  // namespace

extern "C" qwm_status qwm_paged_attend(const qwm_paged_attend_args* a, void* stream) {
  return a ? attend(a, 4, 1, "qwm_paged_attend", stream) : QWM_ERR_INVALID_ARG;
}

extern "C" qwm_status qwm_paged8_attend(const qwm_paged8_attend_args* a, void* stream) {
  if (!a || (a->table_heads != 1 && a->table_heads != a->attend.kv_heads) || a->reserved != 0) return QWM_ERR_INVALID_ARG;
  return attend(&a->attend, 8, a->table_heads, "qwm_paged8_attend", stream);
}

extern "C" size_t qwm_paged8_block_bytes(int32_t head_dim, int32_t page_tokens) {
  return dim_ok(head_dim) && page_shift(page_tokens) >= 0 ? (size_t)block8_bytes(head_dim, page_tokens) : 0;
}

namespace {
// what the 8-bit cache's calls ask of a step's requests: 0 or the status
template <class A>
qwm_status step_status(const A& a) {
  if (a.requests < 0 || a.max_blocks < 1 || a.kv_heads < 1 || a.kv_heads > 65536 || a.n_pages < 1 || a.n_pages > kInt)
    return QWM_ERR_INVALID_ARG;
  if (!dim_ok(a.head_dim) || page_shift(a.page_tokens) < 0 || a.requests > kMaxRequests ||
      (int64_t)a.max_blocks * a.page_tokens > kHalf)
    return QWM_ERR_UNSUPPORTED;
  return QWM_OK;
}
// whether n words at p and m words at q share none
bool apart(const int32_t* p, int64_t n, const int32_t* q, int64_t m) {
  return (uintptr_t)p + 4 * n <= (uintptr_t)q || (uintptr_t)q + 4 * m <= (uintptr_t)p;
}
template <class A>
bool step_pointers_ok(const A& a) {
  return a.block_table && a.kv_len && a.cu_rows && words(a.block_table, a.kv_len, a.cu_rows, a.status);
}
}  // namespace

extern "C" qwm_status qwm_paged8_append(const qwm_paged8_append_args* a, void* stream) {
  if (!a || !dtype_ok(a->dtype) || a->rows < 0 || a->rows > kInt) return QWM_ERR_INVALID_ARG;
  const qwm_status s = step_status(*a);
  if (s != QWM_OK || a->rows == 0 || a->requests == 0) return s;
  const int e = esize(a->dtype);
  if (!rows_ok(a->k, a->rows, a->kv_heads, a->head_dim, e, false) ||
      !rows_ok(a->v, a->rows, a->kv_heads, a->head_dim, e, false) ||
      (a->k_hat.ptr && !rows_ok(a->k_hat, a->rows, a->kv_heads, a->head_dim, e, true)) ||
      (a->v_hat.ptr && !rows_ok(a->v_hat, a->rows, a->kv_heads, a->head_dim, e, true)) || !a->pool || !aligned(a->pool, 16) ||
      !step_pointers_ok(*a))
    return QWM_ERR_INVALID_ARG;
  if (fault_injected("launch")) return QWM_ERR_CUDA;
  NvtxRange range("qwm_paged8_append");
  return cuda_status(launch_append8(*a, page_shift(a->page_tokens), S(stream)));
}

extern "C" qwm_status qwm_paged8_read(const qwm_paged8_read_args* a, void* stream) {
  if (!a || !dtype_ok(a->dtype) || a->rows < 0 || a->rows > kInt) return QWM_ERR_INVALID_ARG;
  const qwm_status s = step_status(*a);
  if (s != QWM_OK || a->rows == 0 || a->requests == 0) return s;
  const int e = esize(a->dtype);
  if (!rows_ok(a->k, a->rows, a->kv_heads, a->head_dim, e, true) ||
      !rows_ok(a->v, a->rows, a->kv_heads, a->head_dim, e, true) || !a->pool || !aligned(a->pool, 16) || !step_pointers_ok(*a))
    return QWM_ERR_INVALID_ARG;
  if (fault_injected("launch")) return QWM_ERR_CUDA;
  NvtxRange range("qwm_paged8_read");
  return cuda_status(launch_read8(*a, page_shift(a->page_tokens), S(stream)));
}

extern "C" qwm_status qwm_paged8_bounds(const qwm_paged8_bounds_args* a, void* stream) {
  if (!a || a->max_new < 0) return QWM_ERR_INVALID_ARG;
  const qwm_status s = step_status(*a);
  if (s != QWM_OK || a->requests == 0) return s;
  if (a->kv_heads > 65535) return QWM_ERR_UNSUPPORTED;
  if (!a->pool || !aligned(a->pool, 16) || !a->bounds || !aligned(a->bounds, 16) || !step_pointers_ok(*a))
    return QWM_ERR_INVALID_ARG;
  if (fault_injected("launch")) return QWM_ERR_CUDA;
  NvtxRange range("qwm_paged8_bounds");
  return cuda_status(launch_bounds8(*a, page_shift(a->page_tokens), S(stream)));
}

extern "C" size_t qwm_paged8_select_workspace_bytes(int64_t rows, int32_t heads, int32_t head_dim, int32_t requests, int32_t kv_heads,
                                                    int32_t max_blocks) {
  if (rows < 0 || rows > kInt || heads < 1 || !dim_ok(head_dim) || requests < 0 || kv_heads < 1 || max_blocks < 1) return 0;
  return select8_keys(requests, kv_heads, max_blocks) + select8_units(rows, heads) + (size_t)(rows * heads) * head_dim;
}

extern "C" qwm_status qwm_paged8_select(const qwm_paged8_select_args* a, void* stream) {
  if (!a || !dtype_ok(a->dtype) || a->rows < 0 || a->rows > kInt || a->heads < 1 || a->heads > 65536 || a->width < 1 ||
      a->sink < 0)
    return QWM_ERR_INVALID_ARG;
  const qwm_status s = step_status(*a);
  if (s == QWM_ERR_INVALID_ARG || a->heads % a->kv_heads) return QWM_ERR_INVALID_ARG;
  if (s != QWM_OK || a->requests == 0) return s;
  if (a->kv_heads > 65535 || a->rows * (a->heads / a->kv_heads) > kHalf || a->rows * a->heads > (int64_t)1 << 36)
    return QWM_ERR_UNSUPPORTED;
  if ((a->rows > 0 && !rows_ok(a->q, a->rows, a->heads, a->head_dim, esize(a->dtype), false)) || !a->bounds ||
      !aligned(a->bounds, 16) || !a->pages || !a->len_out ||
      !apart(a->len_out, a->requests, a->kv_len, a->requests) || !apart(a->len_out, a->requests, a->cu_rows, a->requests + 1) || !words(a->pages, a->len_out) ||
      !a->workspace || !aligned(a->workspace, 256) ||
      a->workspace_bytes < qwm_paged8_select_workspace_bytes(a->rows, a->heads, a->head_dim, a->requests, a->kv_heads, a->max_blocks) ||
      !step_pointers_ok(*a))
    return QWM_ERR_INVALID_ARG;
  if (fault_injected("launch")) return QWM_ERR_CUDA;
  NvtxRange range("qwm_paged8_select");
  return cuda_status(launch_select8(*a, page_shift(a->page_tokens), S(stream)));
}
