// The paged 8-bit cache's quantiser (qwm_paged8_append), its inverse
// (qwm_paged8_read) and the bounds of its pages (qwm_paged8_bounds).
#include "paged_internal.cuh"
#include "paged_launch.cuh"

namespace qwm {
namespace paged {
namespace {

// The requests of a step, as every kernel here reads them.
struct Steps {
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* cu;
  uint32_t* status;
  int64_t rows;        // of the caller's tensors; -1: there are none
  int32_t n_pages, requests, max_blocks, shift;
  bool by_row;         // units are rows
};

// Request b: its rows row0 ... are the tokens first ... n - 1.
struct Step {
  int row0, first, n;
  bool good;
};

__device__ __forceinline__ __half load_half(const void* p) {
  uint16_t x;
  asm volatile("ld.global.b16 %0, [%1];" : "=h"(x) : "l"(p));
  return __ushort_as_half(x);
}
__device__ __forceinline__ int load_cu(const Steps& s, int b) { return load_global(s.cu + b); }

__device__ __forceinline__ Step load_step(const Steps& s, int b) {
  const int most = s.rows < 0 ? 0x7fffffff : (int)s.rows;
  int lo = load_cu(s, b), hi = load_cu(s, b + 1), n = load_global(s.kv_len + b);
  const int64_t cap64 = (int64_t)s.max_blocks << s.shift;
  const int cap = cap64 < 0x7fffff00 ? (int)cap64 : 0x7fffff00;
  Step x;
  x.good = lo >= 0 && hi >= lo && hi <= most && n >= 0 && n <= cap && hi - lo <= n;
  lo = max(lo, 0);
  hi = max(min(hi, most), lo);
  n = min(max(n, 0), cap);
  x.row0 = lo, x.first = n - (hi - lo), x.n = n;
  return x;
}

// Work is dealt out by blocks of 16 slots: request b takes the units from
// cu[b] / 16 + 2 b up to the next one's, no fewer than the blocks that its rows
// can lie in; or, where that makes fewer (single tokens), a unit is a row and the
// first row in a block has it.  The request of a unit, found by a whole warp, 32
// guesses at a time, whatever the values in cu.
__device__ __forceinline__ int unit_of(const Steps& s, int b) {
  const int most = (int)s.rows, row = min(max(load_cu(s, b), 0), most);
  return s.by_row ? row : row / kScaleSlots + 2 * b;
}
__device__ __forceinline__ int find_request(const Steps& s, int unit) {
  const int lane = threadIdx.x & 31;
  int lo = 0, span = s.requests;
  while (span > 1) {
    const int step = (span + 31) / 32, at = lane * step;
    const uint32_t ok = __ballot_sync(0xffffffffu, at < span && unit_of(s, lo + min(at, span - 1)) <= unit);
    const int k = ok ? 31 - __clz(ok) : 0;
    lo += k * step;
    span = min(step, span - k * step);
  }
  return lo;
}

// a warp's block of 16 slots of one head
struct Block {
  Step s;
  int n0;              // its first token
  int at;              // its first slot in the page
  int lo, hi;          // its rows are tokens n0 + lo ... n0 + hi - 1
  bool any, known;     // whether there are rows, whether the page's id is in range
  int64_t page;
};
__device__ __forceinline__ Block find_block(const Steps& s, int unit) {
  Block x;
  // a token for every request (8,192 appends 80 us, 143 with blocks as units and the
  // search), else the search
  int b = unit;
  bool guess = false;
  if (s.by_row && unit < s.requests) {
    x.s = load_step(s, b);
    guess = x.s.row0 == unit && x.s.first < x.s.n;
  }
  if (!guess) {
    b = find_request(s, unit);
    x.s = load_step(s, b);
  }
  int64_t n0;
  if (s.by_row) {
    const int64_t n = (int64_t)x.s.first + unit - x.s.row0;   // the row's token
    n0 = n & ~(int64_t)(kScaleSlots - 1);
    x.any = n >= x.s.first && n < x.s.n && (n == n0 || n == x.s.first);
  } else {
    n0 = ((int64_t)(x.s.first >> 4) + unit - unit_of(s, b)) * kScaleSlots;
    // units ahead of the first request's, in a slice of a step, are no request's
    x.any = n0 < x.s.n && n0 + kScaleSlots > x.s.first && x.s.first < x.s.n;
  }
  x.n0 = x.any ? (int)n0 : 0;
  x.lo = max(x.s.first - x.n0, 0), x.hi = min(x.s.n - x.n0, kScaleSlots);
  x.at = x.n0 & ((1 << s.shift) - 1);
  x.page = -1;
  if (x.any && x.n0 >= 0) x.page = load_global(s.table + (int64_t)b * s.max_blocks + (x.n0 >> s.shift));
  x.known = x.page >= 0 && x.page < s.n_pages;
  return x;
}
// what the calls report of the requests
__device__ __forceinline__ void check_requests(const Steps& s) {
  if (blockIdx.y) return;
  for (int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; b < s.requests; b += (int64_t)gridDim.x * blockDim.x)
    if (!load_step(s, (int)b).good) flag(s.status, QWM_DEV_BOUNDS);
}

constexpr int kNt = 256, kWarps = kNt / 32;

// 8 channels of a row as they lie in memory
template <class T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = load_global(reinterpret_cast<const uint4*>(p)); }
  // bits of the largest magnitude as float32
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = 0x7fff7fffu;
    const uint32_t x = __vmaxu2(__vmaxu2(u.x & m, u.y & m), __vmaxu2(u.z & m, u.w & m));
    return max(x << 16, x & 0xffff0000u);
  }
  __device__ __forceinline__ void get(float* x) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  __device__ __forceinline__ void put(const float* x) {   // of values that bf16 holds
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (__float_as_uint(x[2 * i]) >> 16) | (__float_as_uint(x[2 * i + 1]) & 0xffff0000u);
    u = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = u; }
};
template <>
struct Raw<float> {
  uint4 u[2];
  __device__ __forceinline__ void zero() { u[0] = u[1] = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const float* p) {
    u[0] = load_global(reinterpret_cast<const uint4*>(p));
    u[1] = load_global(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = 0x7fffffffu;
    return max(max(max(u[0].x & m, u[0].y & m), max(u[0].z & m, u[0].w & m)),
               max(max(u[1].x & m, u[1].y & m), max(u[1].z & m, u[1].w & m)));
  }
  __device__ __forceinline__ void get(float* x) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[4 * i] = __uint_as_float(u[i].x), x[4 * i + 1] = __uint_as_float(u[i].y);
      x[4 * i + 2] = __uint_as_float(u[i].z), x[4 * i + 3] = __uint_as_float(u[i].w);
    }
  }
  __device__ __forceinline__ void put(const float* x) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      u[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]),
                        __float_as_uint(x[4 * i + 3]));
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<uint4*>(p)[0] = u[0];
    reinterpret_cast<uint4*>(p)[1] = u[1];
  }
};

__device__ __forceinline__ uint32_t to_e4m3(float a, float b) {   // a in the lower byte
  uint16_t y;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(y) : "f"(b), "f"(a));
  return y;
}
__device__ __forceinline__ uint32_t to_e4m3(uint32_t x) {
  uint16_t y;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float power(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// code x scale of 8 channels
template <class T>
__device__ __forceinline__ Raw<T> decode8(uint2 code, __half2 scale) {
  const uint32_t h[4] = {e4m3_lo(code.x), e4m3_hi(code.x), e4m3_lo(code.y), e4m3_hi(code.y)};
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = mul_f16x2(h[i], scale);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    x[2 * i] = f.x, x[2 * i + 1] = f.y;
  }
  Raw<T> r;
  r.put(x);
  return r;
}

// A warp quantises the block of 16 slots of one head, of K or of V: its lanes
// load all its rows (8 channels a piece), the scale is a maximum over the warp,
// and the codes go out as the rows came in.  Where the block holds earlier tokens
// and the scale grows, their codes are moved first.
// Bound by HBM (2 or 4 bytes a channel in, 1 out, 2 or 4 more for x_hat) in a
// chunk: 4,680 rows of 24 heads, d = 128, with x_hat, in bf16 24.9 us (5.8 TB/s), in
// float32 44 us (5.9 TB/s); by the chain of loads (lengths, page, rows and scale) in a
// step of single tokens: 2.8 us for 48 rows of 8 heads, one call behind another.
template <int D, class T>
__global__ void __launch_bounds__(kNt) paged8_append_kernel(const qwm_paged8_append_args a, const Steps s) {
  constexpr int L = D / 8, RS = 32 / L, NP = kScaleSlots / RS;
  wait_for_kernel_ahead();
  const int lane = threadIdx.x & 31, job = blockIdx.y * kWarps + (threadIdx.x >> 5), h = job >> 1, half = job & 1;
  check_requests(s);
  if (h >= a.kv_heads) return;
  const Block b = find_block(s, blockIdx.x);
  if (!b.any) return;
  if (!b.known) {
    if (lane == 0) flag(s.status, QWM_DEV_BOUNDS);
    return;
  }
  const qwm_rows& in = half ? a.v : a.k;
  const int page = 1 << s.shift, piece = lane % L, r0 = lane / L;
  uint8_t* block = (uint8_t*)a.pool + (b.page * a.kv_heads + h) * (int64_t)block8_bytes(D, page);
  uint8_t* codes = block + half * page * D + b.at * D + 8 * piece;
  __half* place = reinterpret_cast<__half*>(block + 2 * page * D) + b.at / kScaleSlots * 2 + half;
  const int64_t row = b.s.row0 + b.n0 - b.s.first;   // of the block's first slot
  Raw<T> raw[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int r = r0 + i * RS;
    if (r >= b.lo && r < b.hi) raw[i].load((const T*)in.ptr + (row + r) * in.row_stride + h * in.head_stride + 8 * piece);
    else raw[i].zero();
  }
  const bool before = b.lo > 0;
  float had = before ? __half2float(load_half(place)) : 0.f;
  auto largest = [&]() {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NP; ++i) m = max(m, raw[i].top());
    return __reduce_max_sync(0xffffffffu, m);
  };
  uint32_t top = largest();
  if (top > __float_as_uint(kClamp8)) {   // NaN, infinite or beyond the clamp
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      float x[8];
      raw[i].get(x);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (x[k] != x[k]) x[k] = 0.f, bits |= QWM_DEV_NAN;
        if (fabsf(x[k]) > kClamp8) x[k] = copysignf(kClamp8, x[k]), bits |= QWM_DEV_SATURATED;
      }
      raw[i].put(x);
    }
    if (bits) flag(s.status, bits);
    top = largest();
  }
  // 448 = 1.75 2^8
  const int e = min(max((int)(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u), kScaleLow), kScaleHigh);
  float scale = power(e);
  if (before) {
    // no append leaves another; whatever the bytes are, the new ones are sound
    had = had >= power(kScaleLow) ? fminf(had, power(kScaleHigh)) : power(kScaleLow);
    if (scale > had) {
      const __half2 by = __float2half2_rn(had / scale);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int r = r0 + i * RS;
        if (r < b.lo) {
          uint2* p = reinterpret_cast<uint2*>(codes + r * D);
          const uint2 c = load_global(p);
          uint2 m;
          m.x = to_e4m3(mul_f16x2(e4m3_lo(c.x), by)) | to_e4m3(mul_f16x2(e4m3_hi(c.x), by)) << 16;
          m.y = to_e4m3(mul_f16x2(e4m3_lo(c.y), by)) | to_e4m3(mul_f16x2(e4m3_hi(c.y), by)) << 16;
          *p = m;
        }
      }
    } else {
      scale = had;
    }
  }
  if (lane == 0) *place = __float2half_rn(scale);
  const float inv = 1.f / scale;
  const __half2 scale2 = __float2half2_rn(scale);
  const qwm_rows& hat = half ? a.v_hat : a.k_hat;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int r = r0 + i * RS;
    float x[8];
    raw[i].get(x);
    uint2 c;
    c.x = to_e4m3(x[0] * inv, x[1] * inv) | to_e4m3(x[2] * inv, x[3] * inv) << 16;
    c.y = to_e4m3(x[4] * inv, x[5] * inv) | to_e4m3(x[6] * inv, x[7] * inv) << 16;
    if (r >= b.lo && r < b.hi) {
      *reinterpret_cast<uint2*>(codes + r * D) = c;
      if (hat.ptr) decode8<T>(c, scale2).store((T*)hat.ptr + (row + r) * hat.row_stride + h * hat.head_stride + 8 * piece);
    }
  }
}

// The same walk the other way: a warp reads the block of 16 slots of one head, of
// K or of V.  Bound by HBM (1 byte a channel in, 2 or 4 out): 98,280 tokens of 8
// heads, d = 128, to bf16 91 us (6.6 TB/s).
template <int D, class T>
__global__ void __launch_bounds__(kNt) paged8_read_kernel(const qwm_paged8_read_args a, const Steps s) {
  constexpr int L = D / 8, RS = 32 / L, NP = kScaleSlots / RS;
  wait_for_kernel_ahead();
  const int lane = threadIdx.x & 31, job = blockIdx.y * kWarps + (threadIdx.x >> 5), h = job >> 1, half = job & 1;
  check_requests(s);
  if (h >= a.kv_heads) return;
  const Block b = find_block(s, blockIdx.x);
  if (!b.any) return;
  if (!b.known && lane == 0) flag(s.status, QWM_DEV_BOUNDS);
  const qwm_rows& out = half ? a.v : a.k;
  const int page = 1 << s.shift, piece = lane % L, r0 = lane / L;
  const uint8_t* block = (const uint8_t*)a.pool + ((b.known ? b.page : 0) * a.kv_heads + h) * (int64_t)block8_bytes(D, page);
  const uint8_t* codes = block + half * page * D + b.at * D + 8 * piece;
  const int64_t row = b.s.row0 + b.n0 - b.s.first;
  uint2 c[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) c[i] = load_global(reinterpret_cast<const uint2*>(codes + (r0 + i * RS) * D));
  const __half scale = load_half(block + 2 * page * D + (b.at / kScaleSlots * 2 + half) * 2);
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int r = r0 + i * RS;
    Raw<T> x = decode8<T>(c[i], __half2half2(scale));
    if (!b.known) x.zero();
    if (r >= b.lo && r < b.hi) x.store((T*)out.ptr + (row + r) * out.row_stride + h * out.head_stride + 8 * piece);
  }
}

// A CTA takes a page and a head: a warp its blocks of 16 slots in turn, a lane 16
// channels of every fourth (d = 64: eighth) row; maxima and minima in float16,
// exact.  Bound by the chain of loads; the keys of a step's pages are few: 3 us for 48
// single tokens, 7 for the 38 pages of a chunk.  (A warp a page and head where pages
// have up to 64 tokens takes 5 for the single tokens: 16 divisions a lane.)
constexpr int kBoundsNt = 128;

template <int D>
__global__ void __launch_bounds__(kBoundsNt) paged8_bounds_kernel(const qwm_paged8_bounds_args a, const Steps s) {
  constexpr int L = D / 16, RS = 32 / L, NP = kScaleSlots / RS;
  __shared__ __half high_sh[kBoundsNt / 32][D], low_sh[kBoundsNt / 32][D];
  __shared__ float top_sh[kBoundsNt / 32];
  wait_for_kernel_ahead();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, h = blockIdx.y, b = blockIdx.z;
  const Step st = load_step(s, b);
  if (!st.good && tid == 0 && h == 0 && blockIdx.x == 0) flag(s.status, QWM_DEV_BOUNDS);
  if (st.first >= st.n) return;
  const int page = 1 << s.shift, last = (st.n - 1) >> s.shift, piece = lane % L, r0 = lane / L;
  for (int j = (max(st.first, 0) >> s.shift) + blockIdx.x; j <= last; j += gridDim.x) {
    const int id = load_global(s.table + (int64_t)b * s.max_blocks + j);
    if (id < 0 || id >= s.n_pages) {
      if (tid == 0) flag(s.status, QWM_DEV_BOUNDS);
      continue;
    }
    const int live = min(st.n - (j << s.shift), page);
    const uint8_t* block = (const uint8_t*)a.pool + ((int64_t)id * a.kv_heads + h) * block8_bytes(D, page);
    __half2 high[8], low[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) high[k] = __float2half2_rn(-INFINITY), low[k] = __float2half2_rn(INFINITY);
    for (int t = warp * kScaleSlots; t < live; t += kBoundsNt / 32 * kScaleSlots) {
      uint4 c[NP];
#pragma unroll
      for (int i = 0; i < NP; ++i) c[i] = load_global(reinterpret_cast<const uint4*>(block + (t + r0 + i * RS) * D + 16 * piece));
      const __half2 scale = __half2half2(load_half(block + 2 * page * D + t / kScaleSlots * 4));
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if (t + r0 + i * RS >= live) continue;
        const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t x = mul_f16x2((k & 1) ? e4m3_hi(w[k >> 1]) : e4m3_lo(w[k >> 1]), scale);
          const __half2 v = *reinterpret_cast<const __half2*>(&x);
          high[k] = __hmax2(high[k], v), low[k] = __hmin2(low[k], v);
        }
      }
    }
#pragma unroll
    for (int o = L; o < 32; o <<= 1)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        high[k] = __hmax2(high[k], __shfl_xor_sync(0xffffffffu, high[k], o));
        low[k] = __hmin2(low[k], __shfl_xor_sync(0xffffffffu, low[k], o));
      }
    if (lane < L) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        *reinterpret_cast<__half2*>(&high_sh[warp][16 * piece + 2 * k]) = high[k];
        *reinterpret_cast<__half2*>(&low_sh[warp][16 * piece + 2 * k]) = low[k];
      }
    }
    __syncthreads();
    float hi = 0.f, lo = 0.f, top = 0.f;
    if (tid < D) {
      hi = __half2float(high_sh[0][tid]), lo = __half2float(low_sh[0][tid]);
#pragma unroll
      for (int k = 1; k < kBoundsNt / 32; ++k) {
        hi = fmaxf(hi, __half2float(high_sh[k][tid]));
        lo = fminf(lo, __half2float(low_sh[k][tid]));
      }
      top = fmaxf(fabsf(hi), fabsf(lo));
    }
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    if (lane == 0) top_sh[warp] = top;
    __syncthreads();
    top = fmaxf(fmaxf(top_sh[0], top_sh[1]), fmaxf(top_sh[2], top_sh[3]));
    const float unit = __fdiv_rn(top, 127.f), by = unit > 0.f ? unit : 1.f;
    uint8_t* out = (uint8_t*)a.bounds + ((int64_t)id * a.kv_heads + h) * (2 * D + 16);
    if (tid < D) {
      out[tid] = (uint8_t)(int8_t)rintf(__fdiv_rn(hi, by));
      out[D + tid] = (uint8_t)(int8_t)rintf(__fdiv_rn(lo, by));
    }
    if (tid < 4) reinterpret_cast<float*>(out + 2 * D)[tid] = tid ? 0.f : unit;
    __syncthreads();   // the shared arrays are read
  }
}

template <class A>
Steps steps_of(const A& a, int64_t rows, int shift) {
  return Steps{a.block_table, a.kv_len, a.cu_rows, a.status, rows, (int32_t)a.n_pages, a.requests, a.max_blocks, shift,
               rows >= 0 && rows <= rows / kScaleSlots + 2 * (int64_t)a.requests};
}

template <class A>
dim3 unit_grid(const A& a) {
  const int64_t blocks = a.rows / kScaleSlots + 2 * (int64_t)a.requests;
  return dim3((unsigned)(a.rows < blocks ? a.rows : blocks), (unsigned)((2 * a.kv_heads + kWarps - 1) / kWarps), 1);
}

}  // namespace

cudaError_t launch_append8(const qwm_paged8_append_args& a, int shift, cudaStream_t st) {
  const bool bf = a.dtype == QWM_BF16;
  auto kern = a.head_dim == 64 ? (bf ? paged8_append_kernel<64, __nv_bfloat16> : paged8_append_kernel<64, float>)
                               : (bf ? paged8_append_kernel<128, __nv_bfloat16> : paged8_append_kernel<128, float>);
  return launch_early(kern, unit_grid(a), kNt, 0, st, a, steps_of(a, a.rows, shift));
}

cudaError_t launch_read8(const qwm_paged8_read_args& a, int shift, cudaStream_t st) {
  const bool bf = a.dtype == QWM_BF16;
  auto kern = a.head_dim == 64 ? (bf ? paged8_read_kernel<64, __nv_bfloat16> : paged8_read_kernel<64, float>)
                               : (bf ? paged8_read_kernel<128, __nv_bfloat16> : paged8_read_kernel<128, float>);
  return launch_early(kern, unit_grid(a), kNt, 0, st, a, steps_of(a, a.rows, shift));
}

cudaError_t launch_bounds8(const qwm_paged8_bounds_args& a, int shift, cudaStream_t st) {
  // no more rows than the tables hold, which also keeps the sum below in range
  const int64_t page = (int64_t)1 << shift, all = a.max_blocks * page, most = a.max_new < 1 ? 1 : a.max_new < all ? a.max_new : all;
  int64_t pages = (most + page - 2) / page + 1;   // that so many rows can lie in
  pages = pages < a.max_blocks ? pages : a.max_blocks;
  const dim3 grid((unsigned)pages, (unsigned)a.kv_heads, (unsigned)a.requests);
  return launch_early(a.head_dim == 64 ? paged8_bounds_kernel<64> : paged8_bounds_kernel<128>, grid, kBoundsNt, 0, st, a,
                      steps_of(a, -1, shift));
}

}  // namespace paged
}  // namespace qwm
