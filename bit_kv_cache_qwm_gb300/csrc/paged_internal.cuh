// Shared declarations of the paged caches: the block layouts, the work
// partition of the attention kernels and their partial results.
#pragma once

#include <math.h>

#include <atomic>

#include "qwm_internal.cuh"

namespace qwm {
namespace paged {

constexpr int kMaxRequests = 8192;

inline __host__ __device__ int block_bytes(int d, int page) { return page * (d + d / 4); }

// ---- the 8-bit cache: codes of K and of V, then the scales of each 16 slots
constexpr int kScaleSlots = 16, kScaleLow = -15, kScaleHigh = 7;
constexpr float kClamp8 = 57344.f;   // 448 2^kScaleHigh
inline __host__ __device__ int block8_bytes(int d, int page) { return 2 * page * d + (page >= 64 ? page / 4 : 16); }

// A selection's workspace: keys of all pages, and of many rows their units and bytes.
inline size_t select8_keys(int64_t requests, int64_t kv_heads, int64_t max_blocks) { return ((size_t)(requests * kv_heads * max_blocks) * 4 + 255) & ~(size_t)255; }
inline size_t select8_units(int64_t rows, int64_t heads) { return ((size_t)(rows * heads) * 4 + 255) & ~(size_t)255; }

// two e4m3 codes (the lower or the upper half of x) as float16, exact; 64 a clock
// and SM, a third of the instructions of moving the bits into place
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t x) {
  uint32_t y;
  asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %1;\ncvt.rn.f16x2.e4m3x2 %0, l;\n}" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t x) {
  uint32_t y;
  asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %1;\ncvt.rn.f16x2.e4m3x2 %0, h;\n}" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t x, __half2 s) {
  const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&x), s);
  return *reinterpret_cast<const uint32_t*>(&y);
}

// x / d = x mul >> shift for every x < 2^31: mul = ceil(2^(31 + l) / d) with 2^l >= d
inline void fast_division(int d, uint32_t* mul, uint32_t* shift) {
  int l = 0;
  while (((int64_t)1 << l) < d) ++l;
  *shift = 31 + l;
  *mul = (uint32_t)((((uint64_t)1 << (31 + l)) + d - 1) / d);
}

// What every attention kernel reads of a call.
struct AttendArgs {
  const void* q;
  int64_t q_row, q_head;         // element strides
  void* out;
  int64_t o_row, o_head;
  float* lse;
  const uint8_t* pool;
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* cu;
  uint32_t* status;
  uint32_t* timeout;             // word for the bit of a bounded wait that ran out (never null)
  int64_t wait_cycles;           // limit of a bounded wait
  float* part;                   // [workers][2][tile rows][part_floats(d)]
  struct Join* join;             // [workers]
  int64_t rows;
  int32_t n_pages;
  int32_t heads, kv_heads, group;
  uint32_t group_mul, group_shift;   // x / group = x group_mul >> group_shift for x < 2^31
  int32_t page, page_shift, block;
  int32_t requests, max_blocks;
  int32_t causal, window;
  float scale_log2;              // softmax scale * log2(e)
  uint32_t magic;                // 1024 twice in float16
  int32_t bits;                  // of a channel's code: 4 or 8
  int64_t table_b, table_h;      // 8 bits: strides of a request's and of a head's table
};

// The two encodings, as the kernels are told them.
struct Int4 {
  static constexpr int kBits = 4;
};
struct E4m3 {
  static constexpr int kBits = 8;
};

// the table that a key/value head of a request reads by
template <class F>
__device__ __forceinline__ const int32_t* table_of(const AttendArgs& a, int b, int h) {
  if constexpr (F::kBits == 8) return a.table + b * a.table_b + h * a.table_h;
  else return a.table + (int64_t)b * a.max_blocks;
}

// A row of a partial result: O[d] unnormalised, running maximum (log2
// domain), sum, pad to 16 bytes.
inline __host__ __device__ constexpr int part_floats(int d) { return d + 4; }

// An item whose tiles are spread over several workers: the worker it starts
// in records it, the join kernel adds up the parts in the order of the
// workers (first: the starting worker's part 1, then part 0 of each later
// one), so the result does not depend on timing.
struct Join {
  int32_t last;        // last worker with a part, -1: nothing to join
  int32_t q_row0;      // first row of q of the request
  int32_t head;        // kv head
  int32_t row0, rows;  // first row of the item in its request's problem, its rows
  int32_t pad[3];
};

__device__ __forceinline__ void flag(uint32_t* status, uint32_t bit) {
  if (status) atomicOr(status, bit);
}

// What a row's sum of weights, l = sum exp2(x_n - m), gives: the factor of O and
// the log-sum-exp.  0 is the sum of a row that sees nothing; NaN (a row of NaN
// in q) stays NaN in both.
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float log_sum(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// Queries become float16 after an exact scaling of each row by 2^-e that brings
// its largest entry (exponent ex; -127 for zeros and subnormals) to [2^14, 2^15),
// up or down: entries down to 2^-31 of the largest keep all their bits.  e stays
// where both factors are normal floats: at -126 a subnormal row lands above
// 2^-8.  e is kept with 127 added, in a byte.
__device__ __forceinline__ int row_exponent(int ex) { return max(ex - 14, -126); }
// what the products of such a row are multiplied with; never 0, which would turn
// a hidden token's -inf into NaN (2^-126 times a product is 0 in every logit)
__device__ __forceinline__ float row_factor(const AttendArgs& a, int e127) {
  return fmaxf(a.scale_log2 * __uint_as_float((uint32_t)e127 << 23), 1.1754944e-38f);
}

// A value's parameters (float16 zero, scale) where some row does not see the
// token: its weight 0 there must not meet NaN or infinity, which bytes that no
// append wrote may stand for.  Parameters with a value outside float16 count as 0.
__device__ __forceinline__ uint32_t hidden_params(uint32_t par) {
  const __half2 x = *reinterpret_cast<const __half2*>(&par);
  const __half most = __hfma(__habs(__high2half(x)), __float2half(15.f), __habs(__low2half(x)));
  return __hle(most, __float2half(65504.f)) ? par : 0u;
}

// The same for 8 bits: codes that are NaN count as 0, scales beyond those that an
// append leaves (or NaN) as 0.
__device__ __forceinline__ uint32_t known_codes(uint32_t x) {
  return x & ~__vcmpeq4(x & 0x7f7f7f7fu, 0x7f7f7f7fu);
}
__device__ __forceinline__ uint32_t known_scales(uint32_t par) {
  const __half2 x = *reinterpret_cast<const __half2*>(&par);
  const uint32_t ok = __hle2_mask(__habs2(x), __float2half2_rn(128.f));   // false for NaN
  return par & ok;
}

// Kernels 2 and 3 form exp2's argument as s c - m from a maximum m rounded to
// float32.  Up to 2^23 that leaves it within 1/2 and P (at most 2^15 else) in
// float16; beyond, a row's weights could overflow or all vanish, so its sum is
// made NaN.  `none`: m of a row that has seen nothing.
constexpr float kFarLogit = 8388608.f;
__device__ __forceinline__ float near_sum(float m, float l, float none) {
  return m != none && !(fabsf(m) <= kFarLogit) ? __int_as_float(0x7fffffff) : l;
}

__device__ __forceinline__ int div_group(const AttendArgs& a, int x) {
  return (int)(((uint64_t)(uint32_t)x * a.group_mul) >> a.group_shift);
}

// One request as the kernels see it, with lengths clamped to what the tables hold.
struct Request {
  int32_t row0;     // first row of q
  int32_t n_new;    // query tokens
  int32_t n;        // cached tokens
  int32_t rows;     // n_new * group: rows of one kv head's problem, token-major
};

__device__ __forceinline__ Request load_request(const AttendArgs& a, int b) {
  int lo = a.cu[b], hi = a.cu[b + 1], n = a.kv_len[b];
  const int64_t cap64 = (int64_t)a.max_blocks * a.page;
  const int cap = cap64 < 0x7fffff00 ? (int)cap64 : 0x7fffff00;
  const int64_t rows = a.rows;
  if (lo < 0 || hi < lo || hi > rows || n < 0 || n > cap) {
    flag(a.status, QWM_DEV_BOUNDS);
    lo = lo < 0 ? 0 : lo;
    hi = hi > rows ? (int)rows : hi;
    hi = hi < lo ? lo : hi;
    n = n < 0 ? 0 : n > cap ? cap : n;
  }
  Request r;
  r.row0 = lo;
  r.n_new = hi - lo;
  r.n = n;
  r.rows = r.n_new * a.group;
  return r;
}

// Token range [lo, hi) that the tokens tok0 .. tok1 of a request's query see
// between them (empty: lo = hi = 0).
__device__ __forceinline__ void visible(const AttendArgs& a, const Request& r, int tok0, int tok1, int* lo, int* hi) {
  int l = 0, h = r.n;
  if (a.causal) {
    const int base = r.n - r.n_new;
    h = min(h, base + tok1 + 1);
    if (a.window > 0) l = max(0, base + tok0 - a.window + 1);
  }
  if (h <= l) l = h = 0;
  *lo = l;
  *hi = h;
}

// ---- the partition of a call's work over `workers` CTAs
//
// The work is a list of items (request, kv head, block of R rows), each a run
// of tiles of TK tokens that its rows see; an item that sees nothing has one
// tile, so that it is visited and its rows are written.  An item weighs its
// tiles and C more, the cost of starting and ending it in units of a tile
// (measured for each kernel).  The list's weight is dealt to the workers in
// equal contiguous shares whatever the lengths are: no worker waits for
// another, and a long request is split exactly as far as the machine needs.
// A share cuts at most its first and its last item.  Shares weigh more than C,
// so every one has a tile; one that ends inside an item's C leaves the item to
// the next.
template <int R, int TK, int C>
struct Walker {
  int64_t n, done;     // the share's weight, and what of it has been handed out
  int64_t item_at;     // weight of the current item's start, from the share's
  // the current item
  int b, h, rt;
  Request rq;
  int t0, t1;          // its tiles
  int lo, hi;          // its visible tokens
  int from, to;        // the tiles of it that are this worker's
  int rows;            // valid rows of the item

  __device__ int row_tiles() const { return (rq.rows + R - 1) / R; }

  __device__ static void tiles_of(const AttendArgs& a, const Request& r, int rt, int* lo, int* hi, int* t0, int* t1) {
    const int first = rt * R, last = min(r.rows, first + R) - 1;
    visible(a, r, div_group(a, first), div_group(a, last), lo, hi);
    *t0 = *lo / TK;
    *t1 = *hi > *lo ? (*hi + TK - 1) / TK : *t0 + 1;
  }

  // weight of one kv head of a request
  __device__ static int64_t head_tiles(const AttendArgs& a, const Request& r) {
    const int nrt = (r.rows + R - 1) / R;
    if (nrt == 0) return 0;
    int lo, hi, t0, t1;
    if (!a.causal) {
      tiles_of(a, r, 0, &lo, &hi, &t0, &t1);
      return (int64_t)nrt * (t1 - t0 + C);
    }
    int64_t s = (int64_t)nrt * C;
    for (int i = 0; i < nrt; ++i) {
      tiles_of(a, r, i, &lo, &hi, &t0, &t1);
      s += t1 - t0;
    }
    return s;
  }

  // The share's piece of the item, which starts `skip` into its weight; false
  // when it has no tile.
  __device__ bool item(const AttendArgs& a, int skip) {
    tiles_of(a, rq, rt, &lo, &hi, &t0, &t1);
    item_at = done - skip;
    const int all = t1 - t0 + C;
    const int end = (int)min((int64_t)all, n - done + skip);
    done += end - skip;
    from = t0 + max(0, skip - C);
    to = t0 + max(0, end - C);
    rows = min(R, rq.rows - rt * R);
    return to > from;
  }

  // the same by a whole warp
  __device__ static int64_t head_tiles_warp(const AttendArgs& a, const Request& r) {
    if (!a.causal) return head_tiles(a, r);
    const int nrt = (r.rows + R - 1) / R;
    int64_t s = 0;
    for (int i = threadIdx.x & 31; i < nrt; i += 32) {
      s += C;
      int lo, hi, t0, t1;
      tiles_of(a, r, i, &lo, &hi, &t0, &t1);
      s += t1 - t0;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
  }

  // To the first item of a share (whole warps call this): it starts `skip`
  // into the weight of request b0, whose kv heads weigh `per` each.
  __device__ void start(const AttendArgs& a, int b0, int64_t skip, int64_t per, int64_t weight) {
    b = b0;
    rq = load_request(a, b);
    n = weight;
    done = 0;
    h = (int)(skip / per);
    skip -= h * per;
    const int nrt = row_tiles(), lane = threadIdx.x & 31;
    for (int base = 0;; base += 32) {
      int l, u, x0 = 0, x1 = 0;
      if (base + lane < nrt) tiles_of(a, rq, base + lane, &l, &u, &x0, &x1);
      const int64_t mine = base + lane < nrt ? x1 - x0 + C : 0;
      int64_t sum = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, sum > skip);
      const int64_t before = sum - mine;
      if (past) {
        const int f = __ffs(past) - 1;
        rt = base + f;
        skip -= __shfl_sync(0xffffffffu, before, f);
        break;
      }
      skip -= __shfl_sync(0xffffffffu, sum, 31);
    }
    item(a, (int)skip);
  }

  __device__ bool next(const AttendArgs& a) {
    if (done >= n) return false;
    if (++rt >= row_tiles()) {
      rt = 0;
      if (++h >= a.kv_heads) {
        h = 0;
        do {
          if (++b >= a.requests) return false;
          rq = load_request(a, b);
        } while (rq.rows == 0);
      }
    }
    return item(a, 0);
  }

  __device__ bool begins() const { return from == t0; }
  __device__ bool ends() const { return to == t1; }
  // where the item ends in the whole list's weight
  __device__ int64_t end_of(int64_t share_first) const { return share_first + item_at + (t1 - t0) + C; }
};

// The share of worker `w` of `workers`: where it starts and what it weighs.  Called by all threads of a CTA of NT threads; the sums over the
// requests are made by every CTA for itself (a few loads per thread).
struct Share {
  int b;
  int workers;         // those with work: no more than have a tile each
  int64_t skip, per, n, first, total;
};

template <int R, int TK, int C, int NT>
__device__ Share find_share(const AttendArgs& a, int w, int workers) {
  constexpr int NW = NT / 32;
  __shared__ int64_t warp_sum[NW];
  __shared__ int64_t chunk_base, found_skip, found_per;
  __shared__ int found_b;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  Share s;
  s.b = s.workers = 0;
  s.skip = s.n = s.first = s.total = 0;
  s.per = 0;
  auto active = [](int64_t total, int workers) {
    const int64_t most = total / (C + 1);
    return most < workers ? (int)most : workers;
  };
  if (a.requests <= NW) {
    // a warp for each request: with few requests these may be long
    int64_t per = 0;
    if (wid < a.requests) per = Walker<R, TK, C>::head_tiles_warp(a, load_request(a, wid));
    if (lane == 0) warp_sum[wid] = per;
    __syncthreads();
    for (int b = 0; b < a.requests; ++b) s.total += warp_sum[b] * a.kv_heads;
    s.workers = active(s.total, workers);
    if (w < s.workers) {
      s.first = s.total * w / s.workers;
      s.n = s.total * (w + 1) / s.workers - s.first;
      int64_t at = 0;
      for (int b = 0; b < a.requests; ++b) {
        const int64_t x = warp_sum[b] * a.kv_heads;
        if (s.first < at + x) {
          s.b = b;
          s.skip = s.first - at;
          s.per = warp_sum[b];
          break;
        }
        at += x;
      }
    }
    return s;
  }
  for (int pass = 0; pass < 2; ++pass) {
    if (tid == 0) {
      chunk_base = 0;
      found_b = -1;
    }
    __syncthreads();
    const int64_t want = s.first;
    for (int b0 = 0; b0 < a.requests; b0 += NT) {
      const int b = b0 + tid;
      int64_t mine = 0;
      if (b < a.requests) mine = Walker<R, TK, C>::head_tiles(a, load_request(a, b)) * a.kv_heads;
      int64_t x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) warp_sum[wid] = x;
      __syncthreads();
      int64_t before = chunk_base, all = 0;
      for (int i = 0; i < NT / 32; ++i) {
        if (i < wid) before += warp_sum[i];
        all += warp_sum[i];
      }
      const int64_t at = before + x - mine;
      if (pass == 1 && want >= at && want < at + mine) {
        found_b = b;
        found_skip = want - at;
        found_per = mine / a.kv_heads;
      }
      // one pass finds both when the requests fit one chunk
      if (pass == 0 && a.requests <= NT) {
        const int act = active(all, workers);
        const int64_t f = act ? all * w / act : 0;
        if (f >= at && f < at + mine) {
          found_b = b;
          found_skip = f - at;
          found_per = mine / a.kv_heads;
        }
      }
      __syncthreads();
      if (tid == 0) chunk_base += all;
      __syncthreads();
    }
    if (pass == 0) {
      s.total = chunk_base;
      s.workers = active(s.total, workers);
      if (w < s.workers) {
        s.first = s.total * w / s.workers;
        s.n = s.total * (w + 1) / s.workers - s.first;
      }
      if (a.requests <= NT) break;
      __syncthreads();
    }
  }
  s.b = found_b;
  s.skip = found_skip;
  s.per = found_per;
  __syncthreads();
  return s;
}

// The last worker that has a tile of the item that ends at `end` of the
// whole list's weight.
__device__ __forceinline__ int last_worker(const Share& s, int64_t end) {
  // the worker w with first(w) <= end - 1 < first(w + 1), first(w) = floor(total w / workers)
  int64_t w = ((end - 1) * s.workers + s.workers - 1) / s.total;
  if (w >= s.workers) w = s.workers - 1;
  while (w > 0 && s.total * w / s.workers > end - 1) --w;
  while (w + 1 < s.workers && s.total * (w + 1) / s.workers <= end - 1) ++w;
  return (int)w;
}

// What a worker writes for the join kernel: `last` of an item that starts in
// its share and ends in another's, -1 when there is none.
template <class W>
__device__ __forceinline__ void record_join(const AttendArgs& a, int worker, const W& it, int last, int R) {
  Join j;
  j.last = last;
  j.q_row0 = it.rq.row0;
  j.head = it.h;
  j.row0 = it.rt * R;
  j.rows = it.rows;
  j.pad[0] = j.pad[1] = j.pad[2] = 0;
  a.join[worker] = j;
}

__device__ __forceinline__ float* part_row(const AttendArgs& a, int worker, int slot, int R, int r, int d) {
  return a.part + (((int64_t)worker * 2 + slot) * R + r) * part_floats(d);
}

// A load of memory that the kernel ahead may have written: not one the compiler
// may take for constant and move ahead of wait_for_kernel_ahead.
template <class T>
__device__ __forceinline__ T load_global(const T* p) {
  static_assert(sizeof(T) == 4 || sizeof(T) == 8 || sizeof(T) == 16, "a vector");
  T x;
  if constexpr (sizeof(T) == 4) {
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(reinterpret_cast<uint32_t&>(x)) : "l"(p));
  } else if constexpr (sizeof(T) == 8) {
    uint2& u = reinterpret_cast<uint2&>(x);
    asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(u.x), "=r"(u.y) : "l"(p));
  } else {
    uint4& u = reinterpret_cast<uint4&>(x);
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
  }
  return x;
}

// Every kernel of the paged cache is launched so that its CTAs may be placed
// while the kernel ahead of it on the stream runs out (of which it sees nothing
// before it has ended), and lets the next one do the same: a step is a row of
// short kernels, and this hides a launch's latency between two of them (single
// token steps called one after another: append 6.1 -> 3.3 us, plan 6.1 -> 3.7,
// norm and rotation 4.1 -> 2.2; captured, 0.3 to 0.7 us each).  Comes first in a
// kernel, before any access to memory.
__device__ __forceinline__ void wait_for_kernel_ahead() {
  cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();
}

// ---- launchers
inline cudaLaunchAttribute early_launch() {
  cudaLaunchAttribute x = {};
  x.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  x.val.programmaticStreamSerializationAllowed = 1;
  return x;
}
// A launch's result; an error is reported by this call alone, not left for the
// caller's next look at the runtime's last error.
inline cudaError_t launched(cudaError_t e) {
  const cudaError_t last = cudaGetLastError();
  return e != cudaSuccess ? e : last;
}
template <class... P, class... A>
cudaError_t launch_early(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {early_launch()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return launched(cudaLaunchKernelEx(&cfg, kern, args...));
}
struct Workers {
  int count;   // CTAs that share the work
  int rows;    // rows of one item
};
int sm_count();   // of the current device
// Launch `kern` with more dynamic shared memory than 48 KB.  The limit (the
// most the kernel ever asks for) is set on its first launch on a device, and
// once more if a launch fails: a reset of the device forgets it.
struct SmemLimit {
  std::atomic<uint8_t> set[64] = {};
};
template <class K, class... A>
cudaError_t launch_smem(SmemLimit& lim, size_t most, K kern, cudaLaunchConfig_t& cfg, const A&... args) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  for (int attempt = 0; attempt < 2; ++attempt) {
    if (dev >= 64 || attempt == 1 || !lim.set[dev].load(std::memory_order_acquire)) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
      if (e != cudaSuccess) return e;
      if (dev < 64) lim.set[dev].store(1, std::memory_order_release);
    }
    e = cudaLaunchKernelEx(&cfg, kern, args...);
    if (e == cudaSuccess) break;
    cudaGetLastError();   // a failed first launch is not the error of the second
  }
  return e;
}
Workers simt_workers(int64_t max_rows);
cudaError_t launch_attend_simt(const AttendArgs& a, int d, bool bf16, int64_t max_rows, cudaStream_t st);
Workers mma_workers(int64_t max_rows, int bits, bool f32, int d);
cudaError_t launch_attend_mma(const AttendArgs& a, int d, bool f32, int64_t max_rows, cudaStream_t st);
Workers tc_workers();
cudaError_t launch_attend_tc(const AttendArgs& a, int d, int64_t max_rows, cudaStream_t st);
// joins the parts of the items that were cut; max_rows: the rows of a
// request's longest problem as the host knows them (any value is correct)
cudaError_t launch_attend_join(const AttendArgs& a, int d, bool bf16, Workers w, int64_t max_rows, cudaStream_t st);

}  // namespace paged
}  // namespace qwm
