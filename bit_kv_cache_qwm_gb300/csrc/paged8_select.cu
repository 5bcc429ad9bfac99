// Which pages a step reads (qwm_paged8_select): the score of every earlier page
// for every key/value head, then the pages with the highest scores.
//
//   S(page, row) = sum_c x_c^+ high_c + sum_c x_c^- low_c,   x^+ = max(x, 0), x^- = min(x, 0)
//
// two products of whole numbers of at most 7 bits, which float16 holds and
// float32 sums exactly in any order: mma.m16n8k16, 16 pages by 8 rows.
#include "paged_internal.cuh"
#include "paged_launch.cuh"
#include "tcgen05_util.cuh"

namespace qwm {
namespace paged {
namespace {

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

// A lane's channels of a row: 16 of every 64, so that four lanes load 64 neighbours
template <int N>
__device__ __forceinline__ void load_row(const float* p, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const float4 u = load_global(reinterpret_cast<const float4*>(p) + (i >> 2) * 16 + (i & 3));
    x[4 * i] = u.x, x[4 * i + 1] = u.y, x[4 * i + 2] = u.z, x[4 * i + 3] = u.w;
  }
}
template <int N>
__device__ __forceinline__ void load_row(const __nv_bfloat16* p, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N / 8; ++i) {
    const uint4 u = load_global(reinterpret_cast<const uint4*>(p) + (i >> 1) * 8 + (i & 1));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) x[8 * i + 2 * k] = __uint_as_float(w[k] << 16), x[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}

// A score's key: keys order as scores do, NaN below all, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float s) {
  const uint32_t u = __float_as_uint(s + 0.f);
  return s != s ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Where maxima over scores start, and what those of a page without bounds stay: NaN,
// which no maximum takes and whose key is below that of -infinity, the score that an
// infinite query can have on every page.
__device__ __forceinline__ float no_score() { return __int_as_float(0x7fffffff); }

// A query row as whole numbers (four lanes share a row, d/4 channels each; `src`: the
// lane's first, nullptr for a row of zeros) and its unit.  A number y comes as the
// float kWhole + y, whose low bits it is.
// The definition divides once a channel.  Here a product with 1/unit, off by less
// than 2 10^-5 (127 times 2^-23, and the quotient's own rounding), gives the same
// whole number unless it comes within 3 10^-5 of a tie, where the warp divides after
// all.  The largest quotient is 127 but for its rounding, so none passes 127.
constexpr float kWhole = 12582912.f;   // 1.5 2^23: a sum with it is rounded to the nearest even

template <int D, class T>
__device__ __forceinline__ float whole_row(const T* src, float2 (&v)[D / 8]) {
  constexpr int C = D / 4;
  float x[C];
  if (src) {
    load_row(src, x);
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) x[i] = 0.f;
  }
  float top = 0.f;
  float2 sum = make_float2(0.f, 0.f);   // NaN where a channel is NaN or infinite
#pragma unroll
  for (int i = 0; i < C; i += 2) {
    top = fmaxf(fmaxf(top, fabsf(x[i])), fabsf(x[i + 1]));
    sum = __ffma2_rn(make_float2(x[i], x[i + 1]), make_float2(0.f, 0.f), sum);
  }
  if (__any_sync(0xffffffffu, !(sum.x + sum.y == 0.f))) {
    top = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      x[i] = x[i] == x[i] ? fminf(fmaxf(x[i], -3.402823466e38f), 3.402823466e38f) : 0.f;
      top = fmaxf(top, fabsf(x[i]));
    }
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const bool some = top >= 7.888609052e-31f;   // 2^-100
  const float u = some ? __fdiv_rn(top, 127.f) : 0.f, inv = some ? __frcp_rn(u) : 0.f;
  float far = 0.f;
#pragma unroll
  for (int i = 0; i < C / 2; ++i) {
    const float2 q = __fmul2_rn(make_float2(x[2 * i], x[2 * i + 1]), make_float2(inv, inv));
    v[i] = __fadd2_rn(q, make_float2(kWhole, kWhole));
    const float2 d = __fadd2_rn(q, __fadd2_rn(make_float2(kWhole, kWhole), make_float2(-v[i].x, -v[i].y)));
    far = fmaxf(fmaxf(far, fabsf(d.x)), fabsf(d.y));
  }
  if (__any_sync(0xffffffffu, far > 0.49997f)) {
#pragma unroll
    for (int i = 0; i < C; ++i) ((i & 1) ? v[i >> 1].y : v[i >> 1].x) = kWhole + (some ? rintf(__fdiv_rn(x[i], u)) : 0.f);
  }
  return u;
}

// Row r of a request and head (a query head of a token) as MMA operands of x^+ and
// of x^-, and the row's unit (NaN where there is no such row: no maximum takes it).
template <int D, class T>
__device__ __forceinline__ float row_operands(const qwm_paged8_select_args& a, const Pages& p, int h, int group, int64_t r, int64_t rows,
                                              uint4 (&w)[D / 16]) {
  const int64_t tok = r / group;
  const T* src = static_cast<const T*>(a.q.ptr) + (p.row0 + tok) * a.q.row_stride + (h * group + r - tok * group) * a.q.head_stride +
                 16 * (threadIdx.x & 3);
  float2 v[D / 8];
  const float u = whole_row<D, T>(r < rows ? src : nullptr, v);
  const __half2 zero = __float2half2_rn(0.f);
  const float2 less = make_float2(-kWhole, -kWhole);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    const __half2 v0 = __float22half2_rn(__fadd2_rn(v[2 * i], less)), v1 = __float22half2_rn(__fadd2_rn(v[2 * i + 1], less));
    w[i] = make_uint4(h2u(__hmax2(v0, zero)), h2u(__hmax2(v1, zero)), h2u(__hmin2(v0, zero)), h2u(__hmin2(v1, zero)));
  }
  return r < rows ? u : __int_as_float(0x7fffffff);
}

// The bounds of 16 pages as a warp loads them: lane (g, c) has channels 16 c ... and
// 64 + 16 c ... of pages g and g + 8.
template <int D>
struct Tile {
  static constexpr int Q = D / 64;
  uint4 high[2][Q], low[2][Q];
  float unit[2];

  // ids of pages g and g + 8; < 0: no page, whose scores are NaN
  __device__ __forceinline__ void load(const qwm_paged8_select_args& a, int h, const int* id) {
    const int c = threadIdx.x & 3;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint8_t* src = (const uint8_t*)a.bounds + ((int64_t)max(id[x], 0) * a.kv_heads + h) * (2 * D + 16);
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        high[x][q] = load_global(reinterpret_cast<const uint4*>(src + 16 * c) + 4 * q);
        low[x][q] = load_global(reinterpret_cast<const uint4*>(src + D + 16 * c) + 4 * q);
      }
      unit[x] = load_global(reinterpret_cast<const float*>(src + 2 * D));
      if (id[x] < 0) unit[x] = __int_as_float(0x7fffffff);
    }
  }
  // operands of step i: 4 channels of each lane
  __device__ __forceinline__ static void operand(const uint4 (&b)[2][Q], int i, uint32_t* f) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint4& u = b[x][i >> 2];
      whole((i & 3) == 0 ? u.x : (i & 3) == 1 ? u.y : (i & 3) == 2 ? u.z : u.w, &f[x], &f[2 + x]);
    }
  }
};

__device__ __forceinline__ int page_id(const qwm_paged8_select_args& a, int b, int j, int tail) {
  int id = j < tail ? load_global(a.block_table + (int64_t)b * a.max_blocks + j) : -1;
  if (id >= a.n_pages || id < 0) {
    if (j < tail) flag(a.status, QWM_DEV_BOUNDS);
    id = -1;
  }
  return id;
}

// the larger of two scores; a page's scores over rows 2 c, 2 c + 1 of the lanes
__device__ __forceinline__ void take(float* best, const float* s, const float* t, const float* unit, float u0, float u1) {
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int k = 0; k < 2; ++k)
      best[x] = fmaxf(best[x], __fmul_rn(__fmul_rn(s[2 * x + k] + t[2 * x + k], unit[x]), k ? u1 : u0));
}

// ---- few rows: a step of single tokens
//
// A warp has 8 rows in its registers and goes through tiles of 16 pages, the next
// tile's bounds on their way; their ids come first, together.  More rows take
// another walk each 8.  Bound by latency (lengths, ids, bounds, each waits for the one
// before, and the rows' conversion): 48 requests of 515 pages on average 17 to 20 us,
// one of 5,850 pages 10.
constexpr int kFewNt = 128, kFewWarps = kFewNt / 32, kMostTiles = 8;

template <int D, class T>
__global__ void __launch_bounds__(kFewNt) paged8_score_few_kernel(const qwm_paged8_select_args a, int shift, int tiles) {
  constexpr int KS = D / 16;
  wait_for_kernel_ahead();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int h = blockIdx.y, b = blockIdx.z, group = a.heads / a.kv_heads;
  const Pages p = load_pages(a, shift, b);
  const int j0 = 16 * (blockIdx.x * kFewWarps + warp) * tiles;
  // the step's own pages, and all where all are kept, need no score
  if (p.first >= p.n || p.count <= a.width || j0 >= p.tail) return;
  const int mine = min(tiles, (p.tail - j0 + 15) / 16);
  int ids[kMostTiles / 2];   // loaded together, then looked at
  const int32_t* table = a.block_table + (int64_t)b * a.max_blocks + j0 + lane;
#pragma unroll
  for (int i = 0; i < kMostTiles / 2; ++i) ids[i] = j0 + 32 * i + lane < p.tail ? load_global(table + 32 * i) : -1;
#pragma unroll
  for (int i = 0; i < kMostTiles / 2; ++i)
    if (ids[i] < 0 || ids[i] >= a.n_pages) {
      if (2 * i < mine && j0 + 32 * i + lane < p.tail && (lane < 16 || 2 * i + 1 < mine)) flag(a.status, QWM_DEV_BOUNDS);
      ids[i] = -1;
    }
  uint32_t* keys = static_cast<uint32_t*>(a.workspace) + ((int64_t)b * a.kv_heads + h) * a.max_blocks;
  const int64_t rows = (int64_t)(p.n - p.first) * group;
  auto fetch = [&](Tile<D>& t, int i) {
    int two = ids[0];
#pragma unroll
    for (int k = 1; k < kMostTiles / 2; ++k) two = (i >> 1) == k ? ids[k] : two;
    const int id[2] = {__shfl_sync(0xffffffffu, two, 16 * (i & 1) + g), __shfl_sync(0xffffffffu, two, 16 * (i & 1) + g + 8)};
    t.load(a, h, id);
  };
  for (int64_t r0 = 0; r0 < rows; r0 += 8) {
    Tile<D> next;
    fetch(next, 0);
    uint4 w[KS];
    const float u = row_operands<D, T>(a, p, h, group, r0 + g, rows, w);
    const float u0 = __shfl_sync(0xffffffffu, u, 8 * c), u1 = __shfl_sync(0xffffffffu, u, 8 * c + 4);
    for (int i = 0; i < mine; ++i) {
      const Tile<D> t = next;
      if (i + 1 < mine) fetch(next, i + 1);
      float s[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t f[4];
        Tile<D>::operand(t.high, k, f);
        mma(s, f, w[k].x, w[k].y);
        Tile<D>::operand(t.low, k, f);
        mma(v, f, w[k].z, w[k].w);
      }
      float best[2] = {no_score(), no_score()};
      take(best, s, v, t.unit, u0, u1);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        best[x] = fmaxf(best[x], __shfl_xor_sync(0xffffffffu, best[x], 1));
        best[x] = fmaxf(best[x], __shfl_xor_sync(0xffffffffu, best[x], 2));
        const int j = j0 + 16 * i + g + 8 * x;
        if (c == 0 && j < p.tail) {
          uint32_t k = key_of(best[x]);
          if (r0) k = max(k, keys[j]);
          keys[j] = k;
        }
      }
    }
  }
}

// ---- many rows: drafts, prompts and chunks
//
// First every row of q becomes whole numbers in int8 with its unit (and the keys are
// cleared): a row is used by every tile of pages.
constexpr int kRowsNt = 256;

template <int D, class T>
__global__ void __launch_bounds__(kRowsNt) paged8_rows_kernel(const qwm_paged8_select_args a, uint8_t* whole_rows, float* units,
                                                              int64_t n_keys) {
  wait_for_kernel_ahead();
  const int64_t at = (int64_t)blockIdx.x * kRowsNt + threadIdx.x, rows = a.rows * a.heads;
  for (int64_t i = at; i < n_keys; i += (int64_t)gridDim.x * kRowsNt) static_cast<uint32_t*>(a.workspace)[i] = 0;
  const int64_t r = at >> 2, t = r >> 31 ? r / a.heads : (uint32_t)r / (uint32_t)a.heads;
  const int c = threadIdx.x & 3;
  if ((at & ~(int64_t)31) >= 4 * rows) return;
  float2 v[D / 8];
  const float u = whole_row<D, T>(r < rows ? static_cast<const T*>(a.q.ptr) + t * a.q.row_stride + (r - t * a.heads) * a.q.head_stride + 16 * c
                                           : nullptr, v);
  if (r >= rows) return;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 x = v[8 * i + 2 * k], y = v[8 * i + 2 * k + 1];
      w[k] = __byte_perm(__byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x0040),
                         __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x0040), 0x5410);
    }
    *reinterpret_cast<uint4*>(whole_rows + r * D + 64 * i + 16 * c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (c == 0) units[r] = u;
}

// Then the products on the 5th-generation tensor cores: M = 128 pages (thread = page =
// TMEM lane, so that a page's maximum over the rows stays in its thread), N = up to
// 128 rows, K = 2 d.  A CTA keeps a tile of pages as the operand in TMEM and goes
// through its rows: while one tile of rows is multiplied, warps 8-15 turn the next
// one's bytes into the operand in shared memory, and warps 0-7 take the maxima of the
// one before (four its first 64 rows, four the others) into the keys, by atomicMax,
// whose order does not matter.
// The chunk of 4,680 rows and 24 heads over 767 pages: 51 us, 1.3 a step, and 18 for
// the rows' kernel.  Bound by the three parts' hand-over once a step (51 us without
// the MMAs, half a microsecond of each step, are 44, without the maxima 40, without
// the rows' conversion 44).  On mma.sync 250 us, with the pages streamed past a tile of
// rows and both converted in the kernel 113.
constexpr int kManyNt = 512, kTile = 128;
constexpr uint32_t kColPages = 256;

template <int D>
struct Lay {
  static constexpr int op = kTile * 2 * D * 2;   // 128 rows of x^+ and x^- in float16
  static constexpr int bytes = 2 * op + 1024;    // two, and room to align
};

// byte offset of 8 channels (chunk) of a row in an operand of SW128 atoms of 64 elements
__device__ __forceinline__ int op_off(int row, int chunk) {
  return (chunk >> 3) * 16384 + (row >> 3) * 1024 + (row & 7) * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

template <int D>
__global__ void __launch_bounds__(kManyNt, 1) paged8_score_many_kernel(const qwm_paged8_select_args a, int shift, const uint8_t* whole_rows,
                                                                       const float* units, int page_parts, uint32_t group_mul,
                                                                       uint32_t group_shift, int64_t wait_cycles) {
  using namespace tcx;
  extern __shared__ uint8_t sm_raw[];
  uint8_t* sm = sm_raw + ((1024 - (su32(sm_raw) & 1023)) & 1023);
  __shared__ __align__(8) uint64_t done[2], drained;       // a step complete, by its parity; nothing left in the pipe
  // by step mod 4 and page tile mod 4: those of step s + 1 are written while s - 1 is read
  __shared__ __align__(16) float unit_row[4][kTile];       // NaN: no such row
  __shared__ float unit_page[4][kTile];
  __shared__ uint32_t tmem_sh, nowhere;
  __shared__ volatile int abort_sh, late_sh;
  wait_for_kernel_ahead();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int h = blockIdx.y, b = blockIdx.z, group = a.heads / a.kv_heads;
  const Pages p = load_pages(a, shift, b);
  if (p.first >= p.n || p.count <= a.width) return;
  // this CTA's tiles: pages p0, p0 + page_parts, ..., rows r0, r0 + row_parts, ...
  const int rows = (p.n - p.first) * group, row_tiles = (rows + kTile - 1) / kTile, page_tiles = (p.tail + kTile - 1) / kTile;
  const int row_parts = (int)gridDim.x / page_parts, p0 = (int)blockIdx.x % page_parts, r0 = (int)blockIdx.x / page_parts;
  if (p0 >= page_tiles || r0 >= row_tiles) return;
  const int nr = (row_tiles - r0 + row_parts - 1) / row_parts, np = (page_tiles - p0 + page_parts - 1) / page_parts, steps = nr * np;
  if (tid == 0) {
    abort_sh = late_sh = 0, nowhere = 0;
    bar_init(&done[0], 1);
    bar_init(&done[1], 1);
    bar_init(&drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(su32(&tmem_sh)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_sh;
  uint32_t* status = a.status ? a.status : &nowhere;
  // both roles take the same steps and meet before them and at the end of each
  auto meet = []() { asm volatile("bar.sync 1, %0;" ::"n"(kManyNt) : "memory"); };
  auto complete = [&](int s) { return warp_all(bar_wait(&done[s & 1], (s >> 1) & 1, &abort_sh, status, wait_cycles)); };

  if (warp >= 8) {
    // ---- the operands.  Rows: 16 a warp; a load takes 64 bytes of eight rows, and the
    // eight lanes of a store phase have two rows, whose swizzles differ.
    const int w = warp - 8;
    uint4 raw[2][D / 64];
    float unit = 0.f;
    int ri = 0;             // the row tile on its way
    auto fetch = [&]() {
      const int base = (r0 + ri * row_parts) * kTile + 16 * w;
      auto at = [&](int r) {   // of a row of the request and head, in the caller's order
        const int tok = (int)(((uint64_t)(uint32_t)r * group_mul) >> group_shift);
        return (int64_t)(p.row0 + tok) * a.heads + h * group + r - tok * group;
      };
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = base + 8 * k + g;
        const uint8_t* src = whole_rows + at(min(r, rows - 1)) * D + 16 * c;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) raw[k][i] = load_global(reinterpret_cast<const uint4*>(src + 64 * i));
      }
      const int r = base + (lane & 15);
      unit = load_global(units + at(min(r, rows - 1)));
      if (r >= rows) unit = __int_as_float(0x7fffffff);
      if (++ri == nr) ri = 0;
    };
    auto expand = [&](int s) {
      if (lane < 16) unit_row[s & 3][16 * w + lane] = unit;
      uint8_t* to = sm + (s & 1) * Lay<D>::op;
      const __half2 zero = __float2half2_rn(0.f);
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const uint32_t u[4] = {raw[k][i].x, raw[k][i].y, raw[k][i].z, raw[k][i].w};
          const int row = 16 * w + 8 * k + g;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t f[4];
            whole(u[2 * e], &f[0], &f[1]);
            whole(u[2 * e + 1], &f[2], &f[3]);
            const int chunk = 2 * (c + 4 * i) + e;
            *reinterpret_cast<uint4*>(to + op_off(row, chunk)) = make_uint4(h2u(__hmax2(u2h(f[0]), zero)), h2u(__hmax2(u2h(f[1]), zero)),
                                                                            h2u(__hmax2(u2h(f[2]), zero)), h2u(__hmax2(u2h(f[3]), zero)));
            *reinterpret_cast<uint4*>(to + op_off(row, D / 8 + chunk)) = make_uint4(h2u(__hmin2(u2h(f[0]), zero)), h2u(__hmin2(u2h(f[1]), zero)),
                                                                                    h2u(__hmin2(u2h(f[2]), zero)), h2u(__hmin2(u2h(f[3]), zero)));
          }
        }
      fence_async_smem();
      fetch();
    };
    // Pages: warps 8-11, a thread a page = a TMEM lane, 64 bounds at a time
    auto pages = [&](int pi) {
      if (w < 4) {
        const int page = 32 * w + lane, id = page_id(a, b, (p0 + pi * page_parts) * kTile + page, p.tail);
        const uint8_t* src = (const uint8_t*)a.bounds + ((int64_t)max(id, 0) * a.kv_heads + h) * (2 * D + 16);
        const uint32_t to = tmem + ((uint32_t)(32 * w) << 16) + kColPages;
        __syncwarp();   // the stores below are the warp's
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint32_t f[32];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint4 u = load_global(reinterpret_cast<const uint4*>(src + 64 * i) + q);
            whole(u.x, &f[8 * q], &f[8 * q + 1]);
            whole(u.y, &f[8 * q + 2], &f[8 * q + 3]);
            whole(u.z, &f[8 * q + 4], &f[8 * q + 5]);
            whole(u.w, &f[8 * q + 6], &f[8 * q + 7]);
          }
          tmem_st32(to + 32 * i, f);
        }
        unit_page[pi & 3][page] = id < 0 ? __int_as_float(0x7fffffff) : load_global(reinterpret_cast<const float*>(src + 2 * D));
        tmem_wait_st();
        fence_before();
      }
    };
    fetch();
    pages(0);
    expand(0);
    meet();
    for (int s = 0, pi = 0, left = nr; s <= steps; ++s) {
      if (s > 0) complete(s - 1);
      if (s + 1 < steps) {
        if (--left == 0) {   // the next step is the next page tile's first
          left = nr;
          complete(s);       // reads this one's operand
          fence_after();
          pages(++pi);
        }
        expand(s + 1);
      }
      meet();
    }
  } else {
    // ---- products and maxima
    uint32_t* keys = static_cast<uint32_t*>(a.workspace) + ((int64_t)b * a.kv_heads + h) * a.max_blocks;
    const int page = tid & (kTile - 1), i0 = 64 * (warp >> 2);
    // rows of the operand of row tile i, in 32s
    auto width = [&](int i) { return min((rows - (r0 + i * row_parts) * kTile + 31) & ~31, kTile); };
    meet();
    fence_after();
    for (int s = 0, ri = 0, pi = 0, before = 0, pi_before = 0; s <= steps; ++s) {
      if (s < steps && warp == 0) {
        const bool go = !__any_sync(0xffffffffu, abort_sh != 0);
        if (go && elect_one()) {
          const uint32_t idesc = (1u << 4) | ((uint32_t)(width(ri) / 8) << 17) | (8u << 24);
          const uint32_t ra = su32(sm + (s & 1) * Lay<D>::op);
#pragma unroll
          for (int k = 0; k < 2 * D / 16; ++k)
            mma_ts(tmem + 128u * (s & 1), tmem + kColPages + 8 * k, desc_sw128(ra + (k >> 2) * 16384 + (k & 3) * 32), idesc, k > 0);
          commit(&done[s & 1]);
        }
        __syncwarp();
      }
      if (s > 0) {
        // the largest score of each page over half of the rows of step s - 1
        const bool ok = complete(s - 1);
        fence_after();
        const int v = s - 1, n = min(width(before), i0 + 64), j = (p0 + pi_before * page_parts) * kTile + page;
        const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 128u * (v & 1);
        const float2 up = make_float2(unit_page[pi_before & 3][page], unit_page[pi_before & 3][page]);
        float best = no_score();
#pragma unroll 1
        for (int i = i0; i < n; i += 32) {
          uint32_t x[32];
          tmem_ld32(at + i, x);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            const float4 r = *reinterpret_cast<const float4*>(&unit_row[v & 3][i + k]);
            const float2 y = __fmul2_rn(__fmul2_rn(make_float2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), up), make_float2(r.x, r.y));
            const float2 z = __fmul2_rn(__fmul2_rn(make_float2(__uint_as_float(x[k + 2]), __uint_as_float(x[k + 3])), up), make_float2(r.z, r.w));
            best = max3f(max3f(best, y.x, y.y), z.x, z.y);
          }
        }
        if (ok && j < p.tail && i0 < n) atomicMax(keys + j, key_of(best));
        fence_before();
      }
      before = ri, pi_before = pi;
      if (++ri == nr) ri = 0, ++pi;
      meet();
      fence_after();
    }
  }
  // after a wait that ran out MMAs may still be on their way
  if (warp == 0) {
    if (elect_one()) commit(&drained);
    __syncwarp();
    bar_wait(&drained, 0, &late_sh, status);
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

template <int D>
cudaError_t launch_many(const qwm_paged8_select_args& a, int shift, const uint8_t* whole_rows, const float* units, cudaStream_t st) {
  static SmemLimit limit;
  const int64_t pairs = (int64_t)a.requests * a.kv_heads, want = (sm_count() + pairs - 1) / pairs;   // CTAs for each
  const int64_t pages = ((int64_t)a.max_blocks + kTile - 1) / kTile, parts = want < pages ? want : pages;
  // of rows only where the pages are too few, by the rows of an average request
  const int64_t rows = (a.rows * (a.heads / a.kv_heads) / a.requests + kTile - 1) / kTile, more = (want + parts - 1) / parts;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(parts * (more < rows ? more : rows < 1 ? 1 : rows)), (unsigned)a.kv_heads, (unsigned)a.requests);
  cfg.blockDim = dim3(kManyNt, 1, 1);
  cfg.dynamicSmemBytes = Lay<D>::bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {early_launch()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  uint32_t mul, by;
  fast_division(a.heads / a.kv_heads, &mul, &by);
  return launched(launch_smem(limit, cfg.dynamicSmemBytes, paged8_score_many_kernel<D>, cfg, a, shift, whole_rows, units, (int)parts, mul,
                              by, injected_wait_cycles(tcx::kWaitCycles)));
}

// ---- the choice
//
// One CTA a request and head.  The least key kept is found digit by digit (8 bits,
// counted from the highest bit in which the keys differ, so that a digit's counts
// spread); once no more than kFew are left in question, a thread each counts those
// ahead of its own instead.  Then every thread writes those of its range of pages.
// Keys stay in registers where kE a thread are enough, else they are read again for
// every step.  Bound by the latency of its barriers: 6 to 8 us.
constexpr int kE = 8, kFew = 128;

// exclusive sum of x over the CTA
template <int NT>
__device__ __forceinline__ int scan(int x, int* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, x0 = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int p = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += p;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int before = lane < warp ? sums[lane] : 0;
  before = (int)__reduce_add_sync(0xffffffffu, (unsigned)before);
  return x - x0 + before;
}

template <int NT>
__global__ void __launch_bounds__(NT) paged8_select_kernel(const qwm_paged8_select_args a, int shift) {
  __shared__ uint32_t count_sh[256], least_sh, most_sh, found_sh;
  __shared__ int digit_sh, left_sh, in_sh, index_sh;
  __shared__ int sums_sh[NT / 32];
  __shared__ uint2 some_sh[kFew];   // (key, index) of those in question
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
  for (int i = kept + tid; i < a.width; i += NT) out[i] = -1;
  if (kept == 0) return;
  if (kept == p.count) {
    for (int i = tid; i < kept; i += NT) out[i] = load_global(table + i);
    return;
  }
  const int own = p.count - p.tail, sink = min(min(a.sink, p.tail), kept - own);
  for (int i = tid; i < own; i += NT) out[kept - own + i] = load_global(table + p.tail + i);
  for (int i = tid; i < sink; i += NT) out[i] = load_global(table + i);
  // of pages sink ... tail - 1, the `left` with the highest keys
  const int n = p.tail - sink, want = kept - own - sink;
  if (want == 0) return;
  const uint32_t* keys = static_cast<const uint32_t*>(a.workspace) + ((int64_t)b * a.kv_heads + h) * a.max_blocks + sink;
  // a thread's range of pages
  const int per = (n + NT - 1) / NT, i0 = min(tid * per, n), i1 = min(i0 + per, n);
  const bool held = per <= kE;
  uint32_t mine[kE];
  if (held) {
#pragma unroll
    for (int e = 0; e < kE; ++e) mine[e] = i0 + e < i1 ? load_global(keys + i0 + e) : 0u;
  }
  auto each = [&](auto f) {   // f(key, index) over the thread's range
    if (held) {
#pragma unroll
      for (int e = 0; e < kE; ++e)
        if (i0 + e < i1) f(mine[e], i0 + e);
    } else {
      for (int i = i0; i < i1; ++i) f(load_global(keys + i), i);
    }
  };
  if (tid == 0) least_sh = 0xffffffffu, most_sh = 0;
  __syncthreads();
  uint32_t least = 0xffffffffu, most = 0;
  each([&](uint32_t k, int) { least = min(least, k), most = max(most, k); });
  least = __reduce_min_sync(0xffffffffu, least), most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) atomicMin(&least_sh, least), atomicMax(&most_sh, most);
  __syncthreads();
  least = least_sh, most = most_sh;
  int bits = 32 - __clz(most - least), left = want, in = n;
  uint32_t found = 0;   // the digits so far, of the least key kept
  while (bits > 0 && in > kFew) {
    const int down = max(bits - 8, 0), width = bits - down;
    for (int i = tid; i < 256; i += NT) count_sh[i] = 0;
    __syncthreads();
    each([&](uint32_t k, int) {
      k -= least;
      if ((uint64_t)k >> bits == found) atomicAdd(&count_sh[(k >> down) & ((1u << width) - 1)], 1u);
    });
    __syncthreads();
    if (warp == 0) {
      // lane 0 has the highest 8 digits
      uint32_t has[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) has[i] = count_sh[255 - 8 * lane - i], sum += has[i];
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
          if (before < (uint32_t)left && (uint32_t)left <= before + has[i]) {
            digit_sh = 255 - 8 * lane - i;
            left_sh = left - (int)before;
            in_sh = (int)has[i];
          }
          before += has[i];
        }
      }
    }
    __syncthreads();
    found = (found << width) | (uint32_t)digit_sh;
    left = left_sh, in = in_sh;
    bits = down;
  }
  // Of the `in` keys that start with `found`, `left` are kept.  Those above are kept
  // all.  `last`: the last page kept among those of the least key kept.
  int last = 0x7fffffff;
  if (in > left) {
    if (in <= kFew) {
      int m = 0;
      each([&](uint32_t k, int) { m += (uint64_t)(k - least) >> bits == found; });
      int at = scan<NT>(m, sums_sh);
      each([&](uint32_t k, int i) {
        if ((uint64_t)(k - least) >> bits == found) some_sh[at++] = make_uint2(k - least, (uint32_t)i);
      });
      __syncthreads();
      if (tid < in) {
        const uint2 x = some_sh[tid];
        int ahead = 0;   // the list is in the order of the pages
        for (int i = 0; i < in; ++i) {
          const uint32_t k = some_sh[i].x;
          ahead += k > x.x || (k == x.x && i < tid);
        }
        if (ahead == left - 1) found_sh = x.x, index_sh = (int)x.y;
      }
      __syncthreads();
      found = found_sh, last = index_sh;
    } else {   // all of one key: the first `left` of them
      int m = 0;
      each([&](uint32_t k, int) { m += k - least == found; });
      int at = scan<NT>(m, sums_sh);
      each([&](uint32_t k, int i) {
        if (k - least == found && at++ == left - 1) index_sh = i;
      });
      __syncthreads();
      last = index_sh;
    }
    bits = 0;
  }
  auto keep = [&](uint32_t k, int i) {
    const uint64_t y = (uint64_t)(k - least) >> bits;
    return y > found || (y == found && i <= last);
  };
  int m = 0;
  each([&](uint32_t k, int i) { m += keep(k, i); });
  __syncthreads();
  int at = sink + scan<NT>(m, sums_sh);
  each([&](uint32_t k, int i) {
    if (keep(k, i)) out[at++] = load_global(table + sink + i);
  });
}

template <int NT>
cudaError_t launch_choice(const qwm_paged8_select_args& a, int shift, cudaStream_t st) {
  return launch_early(paged8_select_kernel<NT>, dim3((unsigned)a.kv_heads, (unsigned)a.requests, 1), NT, 0, st, a, shift);
}

}  // namespace

cudaError_t launch_select8(const qwm_paged8_select_args& a, int shift, cudaStream_t st) {
  const bool bf = a.dtype == QWM_BF16, wide = a.head_dim == 128;
  if (a.max_blocks > a.width) {   // else all pages are kept
    const int64_t pairs = (int64_t)a.requests * a.kv_heads, sms = sm_count();
    const dim3 grid(1, (unsigned)a.kv_heads, (unsigned)a.requests);
    cudaError_t e;
    // Up to 8 rows a request and key/value head, on the mean, the first kernel: it goes
    // through the bounds once for every 8.  Whole selections at 4 query heads a key/value
    // head, few against many, us: 48 requests of 200 to 32,760 tokens 22 and 55 at 8
    // rows, 38 and 54 at 16, 54 and 55 at 20, 69 and 55 at 32; one of 374,400 15 and 25, 20
    // and 22, 25 and 23, 29 and 22; six of 2,000 to 8,000 10 and 13, 13 and 13, 16 and 13,
    // 19 and 13.  The mean misleads where a prompt comes with many single tokens: 1,000 of
    // 2,000 tokens and 900 rows over 30,000 take 4.2 ms together, 0.08 and 0.03 apart.
    if (a.rows * (a.heads / a.kv_heads) <= 8 * (int64_t)a.requests) {
      // tiles of 16 pages for a warp: as many as leave no more than the 16 warps an SM
      // that fit at once
      const int64_t all = ((int64_t)a.max_blocks + 15) / 16, fair = (all * pairs + 16 * sms - 1) / (16 * sms);
      const int tiles = (int)(fair < 1 ? 1 : fair < kMostTiles ? fair : kMostTiles);
      dim3 g = grid;
      g.x = (unsigned)((all + kFewWarps * tiles - 1) / (kFewWarps * tiles));
      auto kern = wide ? (bf ? paged8_score_few_kernel<128, __nv_bfloat16> : paged8_score_few_kernel<128, float>)
                       : (bf ? paged8_score_few_kernel<64, __nv_bfloat16> : paged8_score_few_kernel<64, float>);
      e = launch_early(kern, g, kFewNt, 0, st, a, shift, tiles);
    } else {
      // behind the keys: the rows' units, then the rows
      float* units = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + select8_keys(a.requests, a.kv_heads, a.max_blocks));
      uint8_t* rows = reinterpret_cast<uint8_t*>(units) + select8_units(a.rows, a.heads);
      auto kern = wide ? (bf ? paged8_rows_kernel<128, __nv_bfloat16> : paged8_rows_kernel<128, float>)
                       : (bf ? paged8_rows_kernel<64, __nv_bfloat16> : paged8_rows_kernel<64, float>);
      const int64_t ctas = (4 * a.rows * a.heads + kRowsNt - 1) / kRowsNt;
      e = launch_early(kern, dim3((unsigned)ctas, 1, 1), kRowsNt, 0, st, a, rows, units, pairs * a.max_blocks);
      if (e != cudaSuccess) return e;
      e = wide ? launch_many<128>(a, shift, rows, units, st) : launch_many<64>(a, shift, rows, units, st);
    }
    if (e != cudaSuccess) return e;
  }
  return a.max_blocks <= 256 * kE ? launch_choice<256>(a, shift, st) : launch_choice<1024>(a, shift, st);
}

}  // namespace paged
}  // namespace qwm
