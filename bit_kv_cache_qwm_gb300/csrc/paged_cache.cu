// The paged cache's bookkeeping (qwm_paged_plan, qwm_paged_release) and its
// 4-bit quantiser (qwm_paged_append).
#include <cooperative_groups.h>

#include "paged_internal.cuh"
#include "paged_launch.cuh"

namespace cg = cooperative_groups;

namespace qwm {
namespace paged {
namespace {

constexpr int kPlanNt = 1024;

__device__ __forceinline__ int pages_of(int64_t tokens, int shift) { return (int)((tokens + (1 << shift) - 1) >> shift); }

// Exclusive prefix sums of (x, y) over the CTA's threads; *sx, *sy: the totals.
__device__ __forceinline__ void scan2(int64_t& x, int64_t& y, int64_t* sx, int64_t* sy) {
  __shared__ int64_t wx[32], wy[32];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int64_t x0 = x, y0 = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, x, o), b = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) x += a, y += b;
  }
  __syncthreads();
  if (lane == 31) wx[wid] = x, wy[wid] = y;
  __syncthreads();
  if (wid == 0) {
    int64_t a = lane < nw ? wx[lane] : 0, b = lane < nw ? wy[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t c = __shfl_up_sync(0xffffffffu, a, o), d = __shfl_up_sync(0xffffffffu, b, o);
      if (lane >= o) a += c, b += d;
    }
    wx[lane] = a, wy[lane] = b;
  }
  __syncthreads();
  const int64_t bx = wid ? wx[wid - 1] : 0, by = wid ? wy[wid - 1] : 0;
  *sx = wx[nw - 1], *sy = wy[nw - 1];
  x += bx - x0, y += by - y0;
}

// The largest b with first[b] <= i (first ascending, first[0] <= i).
__device__ __forceinline__ int find(const int32_t* first, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Every CTA scans the lengths for itself (a few loads a thread), then all
// write rows and table entries, CTA 0 the rest.  Where an output is an input
// (kv_len_out = kv_len) the CTAs are one cluster that meets once all have read
// it; otherwise nothing joins them and there is one for every 1024 rows.  The
// prefix sums stay in shared memory: a row finds its request by bisection.
// Bound by latency: the loads of the lengths, the scan, the page ids: 4 us for
// 48 requests, 5 us for 240 requests and 98,280 rows.
__global__ void __launch_bounds__(kPlanNt) paged_plan_kernel(const qwm_paged_plan_args a, int shift, bool in_place) {
  extern __shared__ int32_t plan_sm[];
  int32_t* row_of = plan_sm;                 // first row of each request
  int32_t* page_of = row_of + a.requests;    // first new page
  int32_t* len_of = page_of + a.requests;    // cached tokens
  __shared__ int32_t count_sh;
  __shared__ int bad_sh, full_sh;
  const int tid = threadIdx.x, rank = blockIdx.x, ctas = gridDim.x;
  wait_for_kernel_ahead();
  if (tid == 0) bad_sh = full_sh = 0, count_sh = *a.free_count;
  __syncthreads();
  int64_t rows = 0, pages = 0;
  for (int b0 = 0; b0 < a.requests; b0 += kPlanNt) {
    const int b = b0 + tid;
    int64_t x = 0, y = 0;
    int len = 0;
    if (b < a.requests) {
      len = a.kv_len[b];
      const int add = a.new_len[b];
      if (len < 0 || add < 0) {
        bad_sh = 1;
      } else {
        const int64_t total = ((int64_t)len + add + (1 << shift) - 1) >> shift;
        x = add;
        y = total - pages_of(len, shift);
        // a length beyond int32 does not fit its output either
        if (total > a.max_blocks || (int64_t)len + add > 0x7fffffff) full_sh = 1;
      }
    }
    int64_t sx, sy;
    scan2(x, y, &sx, &sy);
    if (b < a.requests) {
      row_of[b] = (int32_t)(rows + x);
      page_of[b] = (int32_t)(pages + y);
      len_of[b] = len;
    }
    rows += sx;
    pages += sy;
  }
  __syncthreads();
  const int count = count_sh;
  const bool bad = bad_sh != 0 || count < 0 || count > a.n_pages;
  const bool ok = !bad && !full_sh && rows <= a.rows && pages <= count;
  if (in_place && ctas > 1) cg::this_cluster().sync();
  else __syncthreads();
  if (rank == 0) {
    for (int b = tid; b < a.requests; b += kPlanNt) {
      const int next = b + 1 < a.requests ? row_of[b + 1] : (int32_t)rows;
      a.kv_len_out[b] = len_of[b] + (ok ? next - row_of[b] : 0);
      a.cu_rows[b] = ok ? row_of[b] : 0;
    }
    if (tid == 0) {
      a.cu_rows[a.requests] = ok ? (int32_t)rows : 0;
      *a.free_count_out = count - (ok ? (int32_t)pages : 0);
      if (!ok) flag(a.status, bad ? QWM_DEV_BOUNDS : QWM_DEV_CAPACITY);
    }
  }
  const int first = rank * kPlanNt + tid, step = ctas * kPlanNt;
  const int used = ok ? (int)rows : 0;
  if (ok) {
    for (int i = first; i < (int)pages; i += step) {
      const int b = find(page_of, a.requests, i);
      int pg = a.free_pages[count - 1 - i];
      if (pg < 0 || pg >= a.n_pages) {
        flag(a.status, QWM_DEV_BOUNDS);
        pg = -1;
      }
      a.block_table[(int64_t)b * a.max_blocks + pages_of(len_of[b], shift) + (i - page_of[b])] = pg;
    }
  }
  for (int64_t t = first; t < a.rows; t += step) {
    int64_t slot = -1;
    int pos = -1;
    if (t < used) {
      const int b = find(row_of, a.requests, (int)t);
      pos = len_of[b] + (int)t - row_of[b];
      const int held = pages_of(len_of[b], shift), j = pos >> shift;
      // pages held before the call are in the table, the new ones on the stack
      const int pg = j < held ? a.block_table[(int64_t)b * a.max_blocks + j]
                              : a.free_pages[count - 1 - (page_of[b] + j - held)];
      if (pg >= 0 && pg < a.n_pages) slot = ((int64_t)pg << shift) + (pos & ((1 << shift) - 1));
      else flag(a.status, QWM_DEV_BOUNDS);
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
  }
}

// One CTA, a warp a request: the pages behind keep_len are counted (ids in
// range), the counts summed up in the order of the requests, and if the stack
// holds them all, pushed.  Bound by latency.
__global__ void __launch_bounds__(kPlanNt) paged_release_kernel(const qwm_paged_release_args a, int shift) {
  extern __shared__ int32_t first_sm[];   // pages given up by each request, then their first place
  __shared__ int32_t count_sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  wait_for_kernel_ahead();
  if (tid == 0) count_sh = *a.free_count;
  // entries [keep, held) of a request's table; false where keep_len is out of range
  auto range = [&](int b, int* keep, int* held) {
    const int len = a.kv_len[b], want = a.keep_len[b];
    if (want < 0 || want > len || pages_of(len, shift) > a.max_blocks) return false;
    *keep = pages_of(want, shift);
    *held = pages_of(len, shift);
    return true;
  };
  for (int b = warp; b < a.requests; b += kPlanNt / 32) {
    int keep = 0, held = 0, n = 0;
    const bool ok = range(b, &keep, &held);
    if (!ok && lane == 0) flag(a.status, QWM_DEV_BOUNDS);
    for (int j = keep + lane; ok && j < held; j += 32) {
      const int pg = a.block_table[(int64_t)b * a.max_blocks + j];
      if (pg >= 0 && pg < a.n_pages) ++n;
      else flag(a.status, QWM_DEV_BOUNDS);
    }
    n = (int)__reduce_add_sync(0xffffffffu, (unsigned)n);
    if (lane == 0) first_sm[b] = n;
  }
  __syncthreads();
  const int count = count_sh;
  int64_t total = 0;
  for (int b0 = 0; b0 < a.requests; b0 += kPlanNt) {
    const int b = b0 + tid;
    int64_t x = b < a.requests ? first_sm[b] : 0, y = 0, sx, sy;
    scan2(x, y, &sx, &sy);
    // beyond int32 only where it does not fit, and is not used
    if (b < a.requests) first_sm[b] = (int32_t)(total + x);
    total += sx;
  }
  __syncthreads();
  if (count < 0 || count > a.n_pages || total + count > a.n_pages) {
    if (tid == 0) flag(a.status, QWM_DEV_CAPACITY);
    return;
  }
  for (int b = warp; b < a.requests; b += kPlanNt / 32) {
    int keep = 0, held = 0;
    if (!range(b, &keep, &held)) continue;
    int put = count + first_sm[b];
    for (int j0 = keep; j0 < held; j0 += 32) {
      const int j = j0 + lane;
      int32_t* e = a.block_table + (int64_t)b * a.max_blocks + j;
      const int pg = j < held ? *e : -1;
      const bool good = pg >= 0 && pg < a.n_pages;
      const uint32_t who = __ballot_sync(0xffffffffu, good);
      if (good) a.free_pages[put + __popc(who & ((1u << lane) - 1))] = pg;
      if (j < held) *e = -1;
      put += __popc(who);
    }
    __syncwarp();
    if (lane == 0) a.kv_len[b] = a.keep_len[b];
  }
  if (tid == 0) *a.free_count = (int32_t)(count + total);
}

// ---- append
//
// A thread takes 16 channels of one row and head, of k and then of v (32 or 64
// bytes each, loaded together; 8 bytes of codes out); the 2 threads of a group
// of 32 channels share its range by a shuffle (bf16: minimum and negated
// maximum in one register).  The definition divides once a channel: here the
// quotient over 15 is formed with a reciprocal and saturated to [0, 1], which
// is the clamp; where 15 times it comes within 2^-14 of a tie between two
// codes, farther than its error of 2^-17 (15 times four roundings and the
// reciprocal's), the thread divides after all, so the codes are those of the
// definition.  Adding 1.5 2^23 rounds to the nearest even integer and leaves
// the code in the low bits.  A group's range over 15 is Markstein's corrected
// quotient (IBM J. Res. Dev. 34, 1990): q = R c, q + (R - 15 q) c with
// c = f32(1/15) and fused multiply-adds, the correctly rounded R / 15.
// Bound by HBM (2 or 4 bytes a channel in, 0.625 out, 2 or 4 more for x_hat)
// and by the instructions (69% of the issue slots): 4,680 rows of 24 heads, d =
// 128, bf16 with x_hat, 25.6 us (5.2 TB/s); with a division a channel 71 us, with
// 8 channels a thread and scalar ranges 35 us.  A step of 48 rows takes 3.5 us.
__device__ __forceinline__ void store8(float* p, const float2* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float2* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[i].x, x[i].y);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kAppendNt = 128, kAppendCtas = 8, kCh = 16;
constexpr float kClamp = 60000.f, kRound = 12582912.f;

// kCh channels as loaded, and the range of the group's 32 (2 lanes): NaN when
// a channel is NaN
template <class T>
struct Raw;
template <>
struct Raw<float> {
  float4 u[4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = load_global(reinterpret_cast<const float4*>(p) + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void get(float2* x) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = make_float2(u[i].x, u[i].y), x[2 * i + 1] = make_float2(u[i].z, u[i].w);
  }
  __device__ __forceinline__ static float min_nan(float x, float y) {
    float z;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
    return z;
  }
  __device__ __forceinline__ static float max_nan(float x, float y) {
    float z;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
    return z;
  }
  __device__ __forceinline__ void range(float* mn, float* mx) const {
    float l = u[0].x, h = u[0].x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      l = min_nan(l, min_nan(min_nan(u[i].x, u[i].y), min_nan(u[i].z, u[i].w)));
      h = max_nan(h, max_nan(max_nan(u[i].x, u[i].y), max_nan(u[i].z, u[i].w)));
    }
    *mn = min_nan(l, __shfl_xor_sync(0xffffffffu, l, 1));
    *mx = max_nan(h, __shfl_xor_sync(0xffffffffu, h, 1));
  }
};
template <>
struct Raw<__nv_bfloat16> {
  uint4 u[2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    u[0] = load_global(reinterpret_cast<const uint4*>(p));
    u[1] = load_global(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { u[0] = u[1] = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float2* x) const {
    const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  __device__ __forceinline__ void range(float* mn, float* mx) const {
    auto b = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    __nv_bfloat162 l = b(u[0].x), h = l;
    const uint32_t w[7] = {u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
    for (int i = 0; i < 7; ++i) l = __hmin2_nan(l, b(w[i])), h = __hmax2_nan(h, b(w[i]));
    // (minimum, -maximum): one minimum serves both
    l = __halves2bfloat162(__hmin_nan(__low2bfloat16(l), __high2bfloat16(l)),
                           __hneg(__hmax_nan(__low2bfloat16(h), __high2bfloat16(h))));
    l = __hmin2_nan(l, __shfl_xor_sync(0xffffffffu, l, 1));
    *mn = __low2float(l), *mx = -__high2float(l);
  }
};

// Quantises the thread's channels of its group; x receives x_hat.  Whole warps
// call this.
template <class T>
__device__ __forceinline__ uint2 quantise(const Raw<T>& raw, float2* x, __half2* par, uint32_t* bits) {
  float mn, mx;
  raw.range(&mn, &mx);
  raw.get(x);
  // NaN, infinite or beyond the clamp: the group starts again from mended channels
  if (__any_sync(0xffffffffu, !(mn >= -kClamp && mx <= kClamp))) {
    float lo = kClamp, hi = -kClamp;
#pragma unroll
    for (int k = 0; k < kCh; ++k) {
      float& v = (k & 1) ? x[k >> 1].y : x[k >> 1].x;
      if (!(v == v)) {
        v = 0.f;
        *bits |= QWM_DEV_NAN;
      }
      if (fabsf(v) > kClamp) {
        v = copysignf(kClamp, v);
        *bits |= QWM_DEV_SATURATED;
      }
      lo = fminf(lo, v), hi = fmaxf(hi, v);
    }
    mn = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, 1));
    mx = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, 1));
  }
  constexpr float k15th = 1.0f / 15.0f;
  const float span = __fsub_rn(mx, mn), part = __fmul_rn(span, k15th);
  const __half zh = __float2half_rn(mn), sh = __float2half_rn(__fmaf_rn(__fmaf_rn(-15.f, part, span), k15th, part));
  *par = __halves2half2(zh, sh);
  const float z = __half2float(zh), s = __half2float(sh);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  r = s > 0.f ? r * k15th : 0.f;   // scale 0: every quotient and code 0
  const float2 z2 = make_float2(-z, -z), k15 = make_float2(15.f, 15.f), round2 = make_float2(kRound, kRound);
  const float2 minus2 = make_float2(-1.f, -1.f), s2 = make_float2(-s, -s), zz = make_float2(z, z);
  float2 c[kCh / 2];   // minus the codes
  uint32_t y[kCh];
  float far = 0.f;
#pragma unroll
  for (int k = 0; k < kCh / 2; ++k) {
    const float2 t = __fadd2_rn(x[k], z2);
    const float2 q = make_float2(__saturatef(t.x * r), __saturatef(t.y * r));
    const float2 v = __ffma2_rn(q, k15, round2);
    c[k] = __ffma2_rn(v, minus2, round2);
    const float2 d = __ffma2_rn(q, k15, c[k]);
    far = fmaxf(far, fmaxf(fabsf(d.x), fabsf(d.y)));
    y[2 * k] = __float_as_uint(v.x), y[2 * k + 1] = __float_as_uint(v.y);
  }
  // y = bits of 1.5 2^23 + code, 0x4b400000 + code: their sums with weights
  // 16^k, less that of the constant
  uint2 code = make_uint2(y[7], y[15]);
#pragma unroll
  for (int k = 6; k >= 0; --k) code.x = (code.x << 4) + y[k], code.y = (code.y << 4) + y[8 + k];
  code.x -= 0x3f400000u, code.y -= 0x3f400000u;
  if (far > 0.5f - 6.1035e-5f) {
    code = make_uint2(0, 0);
#pragma unroll
    for (int k = 0; k < kCh; ++k) {
      const float v = (k & 1) ? x[k >> 1].y : x[k >> 1].x;
      const float e = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(v, z), s)), 0.f), 15.f);
      if (k & 1) c[k >> 1].y = -e;
      else c[k >> 1].x = -e;
      (k < 8 ? code.x : code.y) |= (uint32_t)e << (4 * (k & 7));
    }
  }
#pragma unroll
  for (int k = 0; k < kCh / 2; ++k) x[k] = __ffma2_rn(c[k], s2, zz);
  return code;
}

template <int D, class T>
__global__ void __launch_bounds__(kAppendNt, kAppendCtas) paged_append_kernel(const qwm_paged_append_args a, int shift, uint32_t heads_mul,
                                                                 uint32_t heads_shift) {
  constexpr int L = D / kCh, G = D / 32;
  wait_for_kernel_ahead();
  const uint32_t unit = blockIdx.x * (kAppendNt / L) + threadIdx.x / L;
  const int wd = threadIdx.x % L, page = 1 << shift;
  const bool live = unit < (uint32_t)(a.rows * a.kv_heads);
  const uint32_t t = live ? (uint32_t)(((uint64_t)unit * heads_mul) >> heads_shift) : 0;
  const int h = live ? (int)(unit - t * a.kv_heads) : 0;
  // the channels do not wait for the slot: every row may be read
  Raw<T> raw[2];
  raw[0].load((const T*)a.k.ptr + t * a.k.row_stride + h * a.k.head_stride + kCh * wd);
  raw[1].load((const T*)a.v.ptr + t * a.v.row_stride + h * a.v.head_stride + kCh * wd);
  int64_t slot = live ? load_global(reinterpret_cast<const long long*>(a.slots) + t) : -1;
  uint32_t bits = 0;
  if (slot >= (a.n_pages << shift)) {
    bits = QWM_DEV_BOUNDS;
    slot = -1;
  }
  if (slot < 0) raw[0].zero(), raw[1].zero();   // a row without a slot: zeros
  const int at = (int)(slot & (page - 1));
  uint8_t* block = (uint8_t*)a.pool + ((slot >> shift) * a.kv_heads + h) * (int64_t)block_bytes(D, page);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float2 x[kCh / 2];
    __half2 par;
    const uint2 code = quantise(raw[half], x, &par, &bits);
    if (slot >= 0) {
      uint8_t* dst = block + half * (block_bytes(D, page) / 2);
      *reinterpret_cast<uint2*>(dst + at * (D / 2) + 8 * wd) = code;
      if ((wd & 1) == 0) *reinterpret_cast<__half2*>(dst + page * (D / 2) + (at * G + wd / 2) * 4) = par;
    }
    const qwm_rows& hat = half ? a.v_hat : a.k_hat;
    if (hat.ptr && live) {
      T* p = (T*)hat.ptr + t * hat.row_stride + h * hat.head_stride + kCh * wd;
      store8(p, x);
      store8(p + 8, x + 4);
    }
  }
  if (bits) flag(a.status, bits);
}

}  // namespace

cudaError_t launch_plan(const qwm_paged_plan_args& a, int shift, cudaStream_t st) {
  static SmemLimit limit;
  const bool in_place = a.kv_len_out == a.kv_len || a.free_count_out == a.free_count;
  const int64_t want = (a.rows + kPlanNt - 1) / kPlanNt, most = in_place ? 8 : 2 * sm_count();
  const unsigned ctas = (unsigned)(want < 1 ? 1 : want < most ? want : most);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kPlanNt, 1, 1);
  cfg.dynamicSmemBytes = (size_t)a.requests * 12;
  cfg.stream = st;
  cudaLaunchAttribute attr[2] = {early_launch()};
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = in_place && ctas > 1 ? 2 : 1;
  // 48 KB without a raised limit hold the prefix sums and the kernel's own shared
  // memory up to 4,052 requests only: the limit is raised whatever their number
  return launch_smem(limit, kMaxRequests * 12, paged_plan_kernel, cfg, a, shift, in_place);
}

cudaError_t launch_release(const qwm_paged_release_args& a, int shift, cudaStream_t st) {
  return launch_early(paged_release_kernel, dim3(1, 1, 1), kPlanNt, (size_t)a.requests * 4, st, a, shift);   // 32 KB at most
}

cudaError_t launch_append(const qwm_paged_append_args& a, int shift, cudaStream_t st) {
  const int per = kAppendNt / (a.head_dim / kCh);
  const dim3 grid((unsigned)((a.rows * a.kv_heads + per - 1) / per), 1, 1);
  uint32_t mul, by;
  fast_division(a.kv_heads, &mul, &by);
  const bool bf = a.dtype == QWM_BF16;
  auto kern = a.head_dim == 64 ? (bf ? paged_append_kernel<64, __nv_bfloat16> : paged_append_kernel<64, float>)
                               : (bf ? paged_append_kernel<128, __nv_bfloat16> : paged_append_kernel<128, float>);
  return launch_early(kern, grid, kAppendNt, 0, st, a, shift, mul, by);
}

}  // namespace paged
}  // namespace qwm
