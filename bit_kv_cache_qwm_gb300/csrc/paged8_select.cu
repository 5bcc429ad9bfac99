// Which pages a step reads (qwm_paged8_select): the score of every earlier page
// for every key/value head, then the pages with the highest scores.
//
//   S(page, row) = sum_c x_c^+ high_c + sum_c x_c^- low_c,   x^+ = max(x, 0), x^- = min(x, 0)
//
// two products of whole numbers of at most 7 bits, which float16 holds and
// float32 sums exactly in any order: mma.m16n8k16, 16 pages by 8 rows.
#include "paged_internal.cuh"
#include "paged_launch.cuh"

namespace qwm {
namespace paged {
namespace {

constexpr int kNt = 256, kWarps = kNt / 32, kPages = 16 * kWarps;

// A request of the call: its rows, its pages (count in all, those from `tail` on
// are the step's own) and how many of them are kept.
struct Pages {
  int row0, first, n, count, tail, kept;
  bool good;
};
__device__ __forceinline__ Pages load_pages(const qwm_paged8_select_args& a, int shift, int b) {
  int lo = load_global(a.cu_rows + b), hi = load_global(a.cu_rows + b + 1), n = load_global(a.kv_len + b);
  const int64_t cap64 = (int64_t)a.max_blocks << shift;
  const int cap = cap64 < 0x7fffff00 ? (int)cap64 : 0x7fffff00, most = (int)a.rows;
  Pages p;
  p.good = lo >= 0 && hi >= lo && hi <= most && n >= 0 && n <= cap && hi - lo <= n;
  lo = max(lo, 0);
  hi = max(min(hi, most), lo);
  n = min(max(n, 0), cap);
  p.row0 = lo, p.first = n - (hi - lo), p.n = n;
  p.count = (int)(((int64_t)n + (1 << shift) - 1) >> shift);
  p.tail = max(p.first, 0) >> shift;
  p.kept = min(p.count, a.width);
  return p;
}

__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }

// four signed bytes as float16: 1024 + (byte + 128) less 1152
__device__ __forceinline__ void whole(uint32_t x, uint32_t* lo, uint32_t* hi) {
  const uint32_t u = x ^ 0x80808080u;
  const __half2 off = __float2half2_rn(1152.f);
  *lo = h2u(__hsub2(u2h(__byte_perm(u, 0x64646464u, 0x4140)), off));
  *hi = h2u(__hsub2(u2h(__byte_perm(u, 0x64646464u, 0x4342)), off));
}

__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int N>
__device__ __forceinline__ void load_row(const float* p, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const float4 u = load_global(reinterpret_cast<const float4*>(p) + i);
    x[4 * i] = u.x, x[4 * i + 1] = u.y, x[4 * i + 2] = u.z, x[4 * i + 3] = u.w;
  }
}
template <int N>
__device__ __forceinline__ void load_row(const __nv_bfloat16* p, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N / 8; ++i) {
    const uint4 u = load_global(reinterpret_cast<const uint4*>(p) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) x[8 * i + 2 * k] = __uint_as_float(w[k] << 16), x[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}

// A CTA scores 128 pages of one request and head, a warp 16 of them, whose bounds
// stay in its registers.  Its warps turn 8 rows each (a row a query head of a
// token) into whole numbers, share them as MMA operands, and go through all 64;
// lane (g, c) of a warp has channels c d/4 ... of row g, and of pages g and g + 8.
template <int D, class T>
__global__ void __launch_bounds__(kNt) paged8_score_kernel(const qwm_paged8_select_args a, int shift) {
  constexpr int C = D / 4, KS = D / 16;
  __shared__ __align__(16) uint4 rows_sh[kWarps][KS][32];   // b0, b1 of x^+, then of x^-
  __shared__ float unit_sh[kWarps * 8];
  wait_for_kernel_ahead();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int h = blockIdx.y, b = blockIdx.z, group = a.heads / a.kv_heads;
  const Pages p = load_pages(a, shift, b);
  // the step's own pages, and all where all are kept, need no score
  if (p.first >= p.n || p.count <= a.width || (int)blockIdx.x * kPages >= p.tail) return;
  const int j0 = blockIdx.x * kPages + 16 * warp;
  uint32_t high[KS][4], low[KS][4];
  float unit[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int j = j0 + g + 8 * x;
    int id = j < p.tail ? load_global(a.block_table + (int64_t)b * a.max_blocks + j) : -1;
    if (id < 0 || id >= a.n_pages) {
      if (j < p.tail && c == 0) flag(a.status, QWM_DEV_BOUNDS);
      id = -1;
    }
    unit[x] = __int_as_float(0x7fffffff);   // such a page's scores are NaN
    const uint8_t* src = (const uint8_t*)a.bounds + ((int64_t)(id < 0 ? 0 : id) * a.kv_heads + h) * (2 * D + 16);
    if (id >= 0) unit[x] = load_global(reinterpret_cast<const float*>(src + 2 * D));
#pragma unroll
    for (int q = 0; q < C / 16; ++q) {
      const uint4 u = load_global(reinterpret_cast<const uint4*>(src + c * C) + q), v = load_global(reinterpret_cast<const uint4*>(src + D + c * C) + q);
      const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        whole(uw[i], &high[4 * q + i][x], &high[4 * q + i][2 + x]);
        whole(vw[i], &low[4 * q + i][x], &low[4 * q + i][2 + x]);
      }
    }
  }
  float best[2] = {-INFINITY, -INFINITY};
  const int64_t rows = (int64_t)(p.n - p.first) * group;
  for (int64_t r0 = 0; r0 < rows; r0 += 8 * kWarps) {
    const int64_t r = r0 + 8 * warp + g;
    if (r0 + 8 * warp < rows) {
      float x[C];
      const int64_t tok = r / group;
      if (r < rows) {
        load_row(static_cast<const T*>(a.q.ptr) + (p.row0 + tok) * a.q.row_stride + (h * group + r - tok * group) * a.q.head_stride + c * C, x);
      } else {
#pragma unroll
        for (int i = 0; i < C; ++i) x[i] = 0.f;
      }
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        x[i] = x[i] == x[i] ? fminf(fmaxf(x[i], -3.402823466e38f), 3.402823466e38f) : 0.f;
        top = fmaxf(top, fabsf(x[i]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float u = top >= 7.888609052e-31f ? __fdiv_rn(top, 127.f) : 0.f;   // 2^-100
      const __half2 zero = __float2half2_rn(0.f);
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        __half2 w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float y[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) y[e] = u > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(x[4 * i + 2 * k + e], u)), -127.f), 127.f) : 0.f;
          w[k] = __floats2half2_rn(y[0], y[1]);
        }
        rows_sh[warp][i][lane] = make_uint4(h2u(__hmax2(w[0], zero)), h2u(__hmax2(w[1], zero)), h2u(__hmin2(w[0], zero)),
                                            h2u(__hmin2(w[1], zero)));
      }
      // a row that is not there is NaN, which no maximum takes
      if (c == 0) unit_sh[8 * warp + g] = r < rows ? u : __int_as_float(0x7fffffff);
    }
    __syncthreads();
    const int blocks = (int)min((rows - r0 + 7) / 8, (int64_t)kWarps);
    if (j0 < p.tail) {
      for (int y = 0; y < blocks; ++y) {
        float s[4] = {0.f, 0.f, 0.f, 0.f}, t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          const uint4 w = rows_sh[y][i][lane];
          mma(s, high[i], w.x, w.y);
          mma(t, low[i], w.z, w.w);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float u = unit_sh[8 * y + 2 * c + k];
#pragma unroll
          for (int x = 0; x < 2; ++x) best[x] = fmaxf(best[x], __fmul_rn(__fmul_rn(s[2 * x + k] + t[2 * x + k], unit[x]), u));
        }
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    best[x] = fmaxf(best[x], __shfl_xor_sync(0xffffffffu, best[x], 1));
    best[x] = fmaxf(best[x], __shfl_xor_sync(0xffffffffu, best[x], 2));
    const int j = j0 + g + 8 * x;
    if (c == 0 && j < p.tail) static_cast<float*>(a.workspace)[((int64_t)b * a.kv_heads + h) * a.max_blocks + j] = best[x];
  }
}

// One CTA a request and head.  The scores become keys that order like them; the
// least key kept is found digit by digit (8 bits, counted from the highest bit in
// which the keys differ, so that a digit's counts spread), then every thread
// writes those of its range of pages.  Keys stay in shared memory where they fit.
// Bound by the latency of its barriers.
constexpr int kSelNt = 512, kSelWarps = kSelNt / 32, kKeys = 16384;

__device__ __forceinline__ uint32_t key_of(float s) {   // NaN below all, -0 as 0
  const uint32_t u = __float_as_uint(s + 0.f);
  return s != s ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// exclusive sums of (x, y) over the CTA
__device__ __forceinline__ void scan2(int& x, int& y, int2* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, x0 = x, y0 = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int p = __shfl_up_sync(0xffffffffu, x, o), q = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) x += p, y += q;
  }
  if (lane == 31) sums[warp] = make_int2(x, y);
  __syncthreads();
  x -= x0, y -= y0;
  for (int w = 0; w < warp; ++w) x += sums[w].x, y += sums[w].y;
}

__global__ void __launch_bounds__(kSelNt) paged8_select_kernel(const qwm_paged8_select_args a, int shift) {
  extern __shared__ uint32_t keys_sh[];
  __shared__ uint32_t count_sh[256], least_sh, most_sh;
  __shared__ int digit_sh, left_sh;
  __shared__ int2 sums_sh[kSelWarps];
  wait_for_kernel_ahead();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, h = blockIdx.x, b = blockIdx.y;
  const Pages p = load_pages(a, shift, b);
  const bool any = p.first < p.n, fits = p.count - p.tail <= p.kept;
  if (h == 0 && tid == 0) {
    if (!p.good) flag(a.status, QWM_DEV_BOUNDS);
    if (any && !fits) flag(a.status, QWM_DEV_CAPACITY);
    a.len_out[b] = any && fits ? (int)(p.n - ((int64_t)(p.count - p.kept) << shift)) : 0;
  }
  const int kept = any && fits ? p.kept : 0;
  int32_t* out = a.pages + ((int64_t)b * a.kv_heads + h) * a.width;
  const int32_t* table = a.block_table + (int64_t)b * a.max_blocks;
  for (int i = kept + tid; i < a.width; i += kSelNt) out[i] = -1;
  if (kept == 0) return;
  if (kept == p.count) {
    for (int i = tid; i < kept; i += kSelNt) out[i] = load_global(table + i);
    return;
  }
  const int own = p.count - p.tail, sink = min(min(a.sink, p.tail), kept - own);
  for (int i = tid; i < own; i += kSelNt) out[kept - own + i] = load_global(table + p.tail + i);
  for (int i = tid; i < sink; i += kSelNt) out[i] = load_global(table + i);
  // of pages sink ... tail - 1, the `left` with the highest keys
  const int n = p.tail - sink, want = kept - own - sink;
  if (want == 0) return;
  const float* score = static_cast<const float*>(a.workspace) + ((int64_t)b * a.kv_heads + h) * a.max_blocks + sink;
  const bool staged = n <= kKeys;
  if (tid == 0) least_sh = 0xffffffffu, most_sh = 0;
  __syncthreads();
  uint32_t least = 0xffffffffu, most = 0;
  for (int i = tid; i < n; i += kSelNt) {
    const uint32_t k = key_of(load_global(score + i));
    if (staged) keys_sh[i] = k;
    least = min(least, k), most = max(most, k);
  }
  least = __reduce_min_sync(0xffffffffu, least), most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) atomicMin(&least_sh, least), atomicMax(&most_sh, most);
  __syncthreads();
  least = least_sh, most = most_sh;
  auto key = [&](int i) { return (staged ? keys_sh[i] : key_of(load_global(score + i))) - least; };
  int bits = 32 - __clz(most - least), left = want;
  uint32_t found = 0;   // the digits so far, of the least key kept
  while (bits > 0) {
    const int down = max(bits - 8, 0), width = bits - down;
    if (tid < 256) count_sh[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kSelNt) {
      const uint32_t k = key(i);
      if ((uint64_t)k >> bits == found) atomicAdd(&count_sh[(k >> down) & ((1u << width) - 1)], 1u);
    }
    __syncthreads();
    if (warp == 0) {
      // lane 0 has the highest 8 digits
      uint32_t mine[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) mine[i] = count_sh[255 - 8 * lane - i], sum += mine[i];
      uint32_t upto = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      uint32_t before = upto - sum;
      if (before < (uint32_t)left && (uint32_t)left <= upto) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (before < (uint32_t)left && (uint32_t)left <= before + mine[i]) {
            digit_sh = 255 - 8 * lane - i;
            left_sh = left - (int)before;
          }
          before += mine[i];
        }
      }
    }
    __syncthreads();
    found = (found << width) | (uint32_t)digit_sh;
    left = left_sh;
    bits = down;
  }
  // keys above `found` are kept, and the first `left` of those equal to it
  const int per = (n + kSelNt - 1) / kSelNt, i0 = min(tid * per, n), i1 = min(i0 + per, n);
  int above = 0, equal = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key(i);
    above += k > found, equal += k == found;
  }
  scan2(above, equal, sums_sh);
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key(i);
    if (k > found || (k == found && equal < left)) out[sink + above + min(equal, left)] = load_global(table + sink + i);
    above += k > found, equal += k == found;
  }
}

}  // namespace

cudaError_t launch_select8(const qwm_paged8_select_args& a, int shift, cudaStream_t st) {
  const bool bf = a.dtype == QWM_BF16;
  if (a.max_blocks > a.width) {   // else all pages are kept
    const dim3 grid((unsigned)(((int64_t)a.max_blocks + kPages - 1) / kPages), (unsigned)a.kv_heads, (unsigned)a.requests);
    auto kern = a.head_dim == 64 ? (bf ? paged8_score_kernel<64, __nv_bfloat16> : paged8_score_kernel<64, float>)
                                 : (bf ? paged8_score_kernel<128, __nv_bfloat16> : paged8_score_kernel<128, float>);
    const cudaError_t e = launch_early(kern, grid, kNt, 0, st, a, shift);
    if (e != cudaSuccess) return e;
  }
  static SmemLimit limit;
  const int keys = a.max_blocks < kKeys ? a.max_blocks : kKeys;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.kv_heads, (unsigned)a.requests, 1);
  cfg.blockDim = dim3(kSelNt, 1, 1);
  cfg.dynamicSmemBytes = (size_t)keys * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {early_launch()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return launched(launch_smem(limit, kKeys * 4, paged8_select_kernel, cfg, a, shift));
}

}  // namespace paged
}  // namespace qwm
