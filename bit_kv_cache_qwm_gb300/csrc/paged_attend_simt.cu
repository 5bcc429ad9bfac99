// qwm_paged_attend in float32 on the CUDA cores (kernel 1): the kernel of
// float32 calls, right for every case, and the cross-check of the others.
//
//   s_n = q . k_hat_n,  k_hat = zero + code scale;   online softmax in the exp2
//   domain;   O = sum_n p_n v_hat_n / sum_n p_n.
//
// A worker (CTA) walks the tiles of 64 tokens that the partition deals to it.
// Per tile it dequantises K and V into shared memory (float32, rows padded so
// that the reads of different keys fall into different banks), sends for the
// next tile's packed bytes (without that the page ids' and the codes' latency
// lay between every two tiles: 38 us of the windowed batch below), and every
// thread computes RT rows x KT keys of S and RT rows x CT channels of O from
// registers, two float32 multiply-adds an instruction (S: even and odd channels
// apart, O: neighbouring channels).  Items have R = 64 rows, or 8 when no
// request has more than 8 (single-token steps: with 64 the arithmetic on absent
// rows would be 8 times the work on present ones).  Bound by the float32 FMA
// rate and the shared-memory reads beside it (96 wavefronts to 128 cycles of
// FMA a step of 4 channels), with two warps a scheduler to overlap them.
// Measured: three windowed requests (30 to 260 rows, 1,001 tokens visible, 8
// heads over 4, d = 64) 33 us (32 before values that some row does not see were
// checked), of one-wide multiply-adds and scalar reads of V
// 35 us; 2,048 rows over 10,240 tokens 1.22 ms (32 TFLOP/s), at d = 128 2.08 ms
// (37).  Two CTAs an SM (128 registers) bring the long d = 64 case to 1.09 ms,
// but the short one to 37.5 us and d = 128, which spills, to 2.46 ms.
#include "paged_internal.cuh"

namespace qwm {
namespace paged {
namespace {

constexpr int kTk = 64, kNt = 256, kItem = 1, kCtas64 = 1;

template <int D, int R>
struct Shape {
  static constexpr int TX = R == 64 ? 16 : 32;   // threads along the keys (and channels) of a row group
  static constexpr int TY = kNt / TX;
  static constexpr int RT = R / TY, KT = kTk / TX, CT = D / TX;
  static constexpr int CW = CT < 4 ? CT : 4;     // channels of a thread that are neighbours
  static constexpr int LD = D + 4, LP = kTk + 4;
  static constexpr int floats = (R + kTk) * LD + kTk * D + R * LP;
};

__device__ __forceinline__ void load8(const float* p, float* x) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// channel j of a thread
template <class S>
__device__ __forceinline__ int channel(int tx, int j) { return (j / S::CW) * S::TX * S::CW + tx * S::CW + j % S::CW; }

__device__ __forceinline__ void load_run(const float* p, float2 (&x)[2]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  x[0] = make_float2(a.x, a.y), x[1] = make_float2(a.z, a.w);
}
__device__ __forceinline__ void load_run(const float* p, float2 (&x)[1]) { x[0] = *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ void store_pair(float* p, float2 x) { *reinterpret_cast<float2*>(p) = x; }
__device__ __forceinline__ void store_pair(__nv_bfloat16* p, float2 x) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x.x, x.y);
}

// Eight channels of a token, codes and parameters as loaded, and what they stand
// for.
template <class F>
struct Piece;
template <>
struct Piece<Int4> {
  uint32_t code, par;
  __device__ __forceinline__ void zero() { code = par = 0; }
  template <int D>
  __device__ __forceinline__ void load(const uint8_t* blk, int page, int half, int s, int wd) {
    blk += half * page * (D / 2 + D / 8);
    code = load_global(reinterpret_cast<const uint32_t*>(blk + s * (D / 2) + wd * 4));
    par = load_global(reinterpret_cast<const uint32_t*>(blk + page * (D / 2) + (s * (D / 32) + wd / 4) * 4));
  }
  // in a tile of which some row does not see every token
  __device__ __forceinline__ void hide() { par = hidden_params(par); }
  __device__ __forceinline__ void get(int, float* v) const {
    const __half2 p = *reinterpret_cast<const __half2*>(&par);
    const float z = __low2float(p), sc = __high2float(p);
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = fmaf((float)((code >> (4 * c)) & 15u), sc, z);
  }
};
template <>
struct Piece<E4m3> {
  uint2 code;
  uint32_t par;   // K's and V's scale
  __device__ __forceinline__ void zero() { code = make_uint2(0, 0), par = 0; }
  template <int D>
  __device__ __forceinline__ void load(const uint8_t* blk, int page, int half, int s, int wd) {
    code = load_global(reinterpret_cast<const uint2*>(blk + (half * page + s) * D + wd * 8));
    par = load_global(reinterpret_cast<const uint32_t*>(blk + 2 * page * D + s / kScaleSlots * 4));
  }
  __device__ __forceinline__ void hide() {
    code.x = known_codes(code.x), code.y = known_codes(code.y);
    par = known_scales(par);
  }
  __device__ __forceinline__ void get(int half, float* v) const {
    const __half2 p = *reinterpret_cast<const __half2*>(&par);
    const float sc = half ? __high2float(p) : __low2float(p);
    const uint32_t h[4] = {e4m3_lo(code.x), e4m3_hi(code.x), e4m3_lo(code.y), e4m3_hi(code.y)};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[c]));
      v[2 * c] = f.x * sc, v[2 * c + 1] = f.y * sc;
    }
  }
};

template <int D, int R, class T, class F>
__global__ void __launch_bounds__(kNt) paged_attend_simt_kernel(const AttendArgs a) {
  using S = Shape<D, R>;
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;                       // [R][LD], scaled by scale * log2(e)
  float* Ks = Qs + R * S::LD;           // [kTk][LD]
  float* Vs = Ks + kTk * S::LD;         // [kTk][D]
  float* Ps = Vs + kTk * D;             // [R][LP]
  __shared__ uint8_t live_sh[kTk];      // the tile's tokens that are there
  const int tid = threadIdx.x, tx = tid % S::TX, ty = tid / S::TX;
  const int w = blockIdx.x;
  wait_for_kernel_ahead();
  const Share sh = find_share<R, kTk, kItem, kNt>(a, w, (int)gridDim.x);
  if (tid == 0) a.join[w].last = -1;
  if (sh.n == 0) return;
  Walker<R, kTk, kItem> it;
  it.start(a, sh.b, sh.skip, sh.per, sh.n);
  do {
    const int row0 = it.rt * R;
    __syncthreads();   // the previous item's reads of Qs are done
    for (int i = tid; i < R * (D / 8); i += kNt) {
      const int r = i / (D / 8), c = (i % (D / 8)) * 8;
      float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (r < it.rows) {
        const int tok = div_group(a, row0 + r), head = it.h * a.group + (row0 + r) - div_group(a, row0 + r) * a.group;
        load8((const T*)a.q + (int64_t)(it.rq.row0 + tok) * a.q_row + head * a.q_head + c, x);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) Qs[r * S::LD + c + k] = x[k] * a.scale_log2;
    }
    float2 o[S::RT][S::CT / 2];
    float m[S::RT], l[S::RT];
    int top[S::RT], bottom[S::RT];      // a row sees bottom <= n < top
#pragma unroll
    for (int i = 0; i < S::RT; ++i) {
      const int r = ty * S::RT + i, tok = div_group(a, row0 + r);
      m[i] = -INFINITY;
      l[i] = 0.f;
      top[i] = it.hi, bottom[i] = it.lo;
      if (a.causal) {
        const int pos = it.rq.n - it.rq.n_new + tok;
        top[i] = min(it.hi, pos + 1);
        if (a.window > 0) bottom[i] = max(it.lo, pos - a.window + 1);
      }
      if (r >= it.rows) top[i] = 0;
#pragma unroll
      for (int j = 0; j < S::CT / 2; ++j) o[i][j] = make_float2(0.f, 0.f);
    }
    // every row of the item sees the tokens bottom_max <= n < top_min
    int top_min = it.hi, bottom_max = it.lo;
    if (a.causal) {
      const int at = it.rq.n - it.rq.n_new;
      top_min = at + div_group(a, row0) + 1;
      if (a.window > 0) bottom_max = at + div_group(a, row0 + it.rows - 1) - a.window + 1;
    }
    // the next tile's packed bytes, on their way during this one's arithmetic:
    // thread's code words i = tid, tid + 256, ... of [half][token][word]
    constexpr int IT = 2 * kTk * (D / 8) / kNt;
    Piece<F> got[IT];
    uint32_t live = 0;
    auto fetch = [&](int n0) {
      live = 0;
#pragma unroll
      for (int x = 0; x < IT; ++x) {
        const int i = tid + x * kNt, half = i / (kTk * (D / 8)), rem = i % (kTk * (D / 8));
        const int k = rem / (D / 8), wd = rem % (D / 8), n = n0 + k;
        got[x].zero();
        if (n < it.lo || n >= it.hi) continue;
        const int pg = load_global(table_of<F>(a, it.b, it.h) + (n >> a.page_shift));
        if (pg < 0 || pg >= a.n_pages) {
          if (half == 0 && wd == 0) flag(a.status, QWM_DEV_BOUNDS);
          continue;
        }
        live |= 1u << x;
        const int s = n & (a.page - 1);
        got[x].template load<D>(a.pool + ((int64_t)pg * a.kv_heads + it.h) * a.block, a.page, half, s, wd);
      }
    };
    fetch(it.from * kTk);
    for (int t = it.from; t < it.to; ++t) {
      const int n0 = t * kTk;
      __syncthreads();   // the previous tile's reads are done
#pragma unroll
      for (int x = 0; x < IT; ++x) {
        const int i = tid + x * kNt, half = i / (kTk * (D / 8)), rem = i % (kTk * (D / 8));
        const int k = rem / (D / 8), wd = rem % (D / 8);
        if (half && (n0 + kTk > top_min || n0 < bottom_max)) got[x].hide();
        float v[8];
        got[x].get(half, v);
        float* dst = half ? Vs + k * D + wd * 8 : Ks + k * S::LD + wd * 8;
        *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(dst + 4) = make_float4(v[4], v[5], v[6], v[7]);
        if (half == 0 && wd == 0) live_sh[k] = (live >> x) & 1;
      }
      __syncthreads();
      if (t + 1 < it.to) fetch(n0 + kTk);
      float s[S::RT][S::KT];
      float2 s2[S::RT][S::KT];   // even and odd channels
#pragma unroll
      for (int i = 0; i < S::RT; ++i)
#pragma unroll
        for (int j = 0; j < S::KT; ++j) s2[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
      for (int c = 0; c < D; c += 4) {
        float4 kv[S::KT];
#pragma unroll
        for (int j = 0; j < S::KT; ++j) kv[j] = *reinterpret_cast<const float4*>(Ks + (tx + S::TX * j) * S::LD + c);
#pragma unroll
        for (int i = 0; i < S::RT; ++i) {
          const float4 qv = *reinterpret_cast<const float4*>(Qs + (ty * S::RT + i) * S::LD + c);
#pragma unroll
          for (int j = 0; j < S::KT; ++j)
            s2[i][j] = __ffma2_rn(make_float2(qv.x, qv.y), make_float2(kv[j].x, kv[j].y),
                                  __ffma2_rn(make_float2(qv.z, qv.w), make_float2(kv[j].z, kv[j].w), s2[i][j]));
        }
      }
#pragma unroll
      for (int i = 0; i < S::RT; ++i)
#pragma unroll
        for (int j = 0; j < S::KT; ++j) s[i][j] = s2[i][j].x + s2[i][j].y;
#pragma unroll
      for (int i = 0; i < S::RT; ++i) {
        float mx = m[i];
#pragma unroll
        for (int j = 0; j < S::KT; ++j) {
          const int n = n0 + tx + S::TX * j;
          const bool sees = n >= bottom[i] && n < top[i] && live_sh[tx + S::TX * j];
          s[i][j] = sees ? s[i][j] : -INFINITY;
          mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int d = S::TX / 2; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d, S::TX));
        const float ref = mx == -INFINITY ? 0.f : mx, corr = exp2f(m[i] - ref);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < S::KT; ++j) {
          const float p = exp2f(s[i][j] - ref);
          Ps[(ty * S::RT + i) * S::LP + tx + S::TX * j] = p;
          sum += p;
        }
#pragma unroll
        for (int d = S::TX / 2; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d, S::TX);
        l[i] = fmaf(l[i], corr, sum);
        m[i] = mx;
#pragma unroll
        for (int j = 0; j < S::CT / 2; ++j) o[i][j] = __fmul2_rn(o[i][j], make_float2(corr, corr));
      }
      __syncwarp();   // a row's P is written and read by the same warp
#pragma unroll 2
      for (int n = 0; n < kTk; n += 4) {
        float4 p[S::RT];
#pragma unroll
        for (int i = 0; i < S::RT; ++i) p[i] = *reinterpret_cast<const float4*>(Ps + (ty * S::RT + i) * S::LP + n);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int j = 0; j < S::CT; j += S::CW) {
            float2 v[S::CW / 2];
            load_run(Vs + (n + k) * D + channel<S>(tx, j), v);
#pragma unroll
            for (int i = 0; i < S::RT; ++i) {
              const float pk = k == 0 ? p[i].x : k == 1 ? p[i].y : k == 2 ? p[i].z : p[i].w;
#pragma unroll
              for (int x = 0; x < S::CW / 2; ++x) o[i][j / 2 + x] = __ffma2_rn(make_float2(pk, pk), v[x], o[i][j / 2 + x]);
            }
          }
      }
    }
    const bool whole = it.begins() && it.ends();
    const int slot = it.begins() ? 1 : 0;
#pragma unroll
    for (int i = 0; i < S::RT; ++i) {
      const int r = ty * S::RT + i;
      if (r >= it.rows) continue;
      if (whole) {
        const int64_t tok = it.rq.row0 + div_group(a, row0 + r);
        const int head = it.h * a.group + (row0 + r) - div_group(a, row0 + r) * a.group;
        const float inv = inverse_sum(l[i]);
        T* dst = (T*)a.out + tok * a.o_row + head * a.o_head;
#pragma unroll
        for (int j = 0; j < S::CT; j += 2) {
          const float2 y = __fmul2_rn(o[i][j / 2], make_float2(inv, inv));
          store_pair(dst + channel<S>(tx, j), y);
        }
        if (a.lse && tx == 0) a.lse[tok * a.heads + head] = log_sum(m[i], l[i]);
      } else {
        float* dst = part_row(a, w, slot, R, r, D);
#pragma unroll
        for (int j = 0; j < S::CT; j += 2) store_pair(dst + channel<S>(tx, j), o[i][j / 2]);
        if (tx == 0) dst[D] = m[i], dst[D + 1] = l[i];
      }
    }
    if (tid == 0 && it.begins() && !it.ends()) {
      record_join(a, w, it, last_worker(sh, it.end_of(sh.first)), R);
    }
  } while (it.next(a));
}

// Joins the parts of a cut item, in the order of the workers.  With few parts
// a warp takes a row; with many (one long request over the whole machine) a
// CTA does: its threads fetch the parts' maxima and sums together, then groups
// of D/4 lanes add up the parts' O with the factors from shared memory, so
// that neither waits for one part at a time.  Bound by latency.
constexpr int kJoinNt = 256, kFewParts = 8, kPartsAtOnce = 256, kEarlyParts = 8;
static_assert(kPartsAtOnce == kJoinNt, "a thread has a part");

template <int D, class T>
__device__ __forceinline__ void join_store(const AttendArgs& a, const Join& j, int r, int ch, float4 o, float m, float l) {
  const int y = j.row0 + r, tok = div_group(a, y);
  const int head = j.head * a.group + y - tok * a.group;
  const int64_t row = j.q_row0 + tok;
  const float inv = inverse_sum(l);
  T* dst = (T*)a.out + row * a.o_row + head * a.o_head + ch;
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(dst) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  } else {
    const __nv_bfloat162 b0 = __floats2bfloat162_rn(o.x * inv, o.y * inv), b1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
  }
  if (a.lse && ch == 0) a.lse[row * a.heads + head] = log_sum(m, l);
}

template <int D, class T>
__global__ void __launch_bounds__(kJoinNt, 3) paged_attend_join_kernel(const AttendArgs a, int R) {
  constexpr int L = D / 4, NG = kJoinNt / L;
  __shared__ __align__(16) float4 sum[NG][L];
  __shared__ float factor[kPartsAtOnce];
  __shared__ float red[kJoinNt / 32];
  wait_for_kernel_ahead();
  const int w = blockIdx.x, tid = threadIdx.x, g = tid / L, c = tid % L;
  const Join j = a.join[w];
  if (j.last < 0) return;
  const int parts = j.last - w + 1;
  if (parts <= kFewParts) {
    for (int r = blockIdx.y * NG + g; r < j.rows; r += gridDim.y * NG) {
      float4 v[kFewParts];
      float2 ml[kFewParts];
#pragma unroll
      for (int x = 0; x < kFewParts; ++x)
        if (x < parts) {
          const float* p = part_row(a, w + x, x == 0 ? 1 : 0, R, r, D);
          v[x] = *reinterpret_cast<const float4*>(p + 4 * c);
          ml[x] = *reinterpret_cast<const float2*>(p + D);
        }
      float m = -INFINITY;
#pragma unroll
      for (int x = 0; x < kFewParts; ++x)
        if (x < parts) m = fmaxf(m, ml[x].x);
      const float ref = m == -INFINITY ? 0.f : m;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      float l = 0.f;
#pragma unroll
      for (int x = 0; x < kFewParts; ++x)
        if (x < parts) {
          const float f = exp2f(ml[x].x - ref);
          o.x = fmaf(v[x].x, f, o.x), o.y = fmaf(v[x].y, f, o.y), o.z = fmaf(v[x].z, f, o.z), o.w = fmaf(v[x].w, f, o.w);
          l = fmaf(ml[x].y, f, l);
        }
      join_store<D, T>(a, j, r, 4 * c, o, m, l);
    }
    return;
  }
  // the row's maximum over all parts, then the parts in chunks
  auto reduce = [&](float v, bool max) {
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      const float y = __shfl_xor_sync(0xffffffffu, v, d);
      v = max ? fmaxf(v, y) : v + y;
    }
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < kJoinNt / 32; ++i) v = max ? fmaxf(v, red[i]) : v + red[i];
    return v;
  };
  for (int r = blockIdx.y; r < j.rows; r += gridDim.y) {
    auto part = [&](int x) { return part_row(a, w + x, x == 0 ? 1 : 0, R, r, D); };
    // the first parts' O, maxima and sums are on their way together
    float4 early[kEarlyParts];
#pragma unroll
    for (int u = 0; u < kEarlyParts; ++u)
      if (g + u * NG < parts) early[u] = *reinterpret_cast<const float4*>(part(g + u * NG) + 4 * c);
    float2 mine = make_float2(-INFINITY, 0.f);
    if (tid < parts) mine = *reinterpret_cast<const float2*>(part(tid) + D);
    float m = mine.x;
    for (int x = tid + kJoinNt; x < parts; x += kJoinNt) m = fmaxf(m, part(x)[D]);
    m = reduce(m, true);
    const float ref = m == -INFINITY ? 0.f : m;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    auto add = [&](const float4& v, float f) {
      o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
    };
    for (int x0 = 0; x0 < parts; x0 += kPartsAtOnce) {
      const int n = min(kPartsAtOnce, parts - x0);
      __syncthreads();
      if (tid < n) {
        const float2 ml = x0 == 0 ? mine : *reinterpret_cast<const float2*>(part(x0 + tid) + D);
        const float f = exp2f(ml.x - ref);
        factor[tid] = f;
        l = fmaf(ml.y, f, l);
      }
      __syncthreads();
      int x = g;
      if (x0 == 0) {
#pragma unroll
        for (int u = 0; u < kEarlyParts; ++u)
          if (g + u * NG < n) add(early[u], factor[g + u * NG]);
        x += kEarlyParts * NG;
      }
#pragma unroll 8
      for (; x < n; x += NG) add(*reinterpret_cast<const float4*>(part(x0 + x) + 4 * c), factor[x]);
    }
    sum[g][c] = o;
    l = reduce(l, false);   // its barriers publish the groups' sums
    if (g == 0) {
#pragma unroll
      for (int i = 1; i < NG; ++i) {
        const float4 v = sum[i][c];
        o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
      }
      join_store<D, T>(a, j, r, 4 * c, o, m, l);
    }
    __syncthreads();
  }
}

template <int D, int R, class T, class F>
cudaError_t launch_simt(const AttendArgs& a, int workers, cudaStream_t st) {
  static SmemLimit limit;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)workers, 1, 1);
  cfg.blockDim = dim3(kNt, 1, 1);
  cfg.dynamicSmemBytes = Shape<D, R>::floats * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {early_launch()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return launch_smem(limit, cfg.dynamicSmemBytes, paged_attend_simt_kernel<D, R, T, F>, cfg, a);
}

template <class T, class F>
cudaError_t launch_simt_t(const AttendArgs& a, int d, Workers w, cudaStream_t st) {
  if (w.rows == 64) return d == 64 ? launch_simt<64, 64, T, F>(a, w.count, st) : launch_simt<128, 64, T, F>(a, w.count, st);
  return d == 64 ? launch_simt<64, 8, T, F>(a, w.count, st) : launch_simt<128, 8, T, F>(a, w.count, st);
}

}  // namespace

int sm_count() {
  static std::atomic<int> known[64];   // 0: not asked yet
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 152;
  if (dev < 64 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) return 152;
  if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

Workers simt_workers(int64_t max_rows) {
  const int sms = sm_count();
  return max_rows <= 8 ? Workers{2 * sms, 8} : Workers{kCtas64 * sms, 64};
}

cudaError_t launch_attend_simt(const AttendArgs& a, int d, bool bf16, int64_t max_rows, cudaStream_t st) {
  const Workers w = simt_workers(max_rows);
  const cudaError_t e = a.bits == 8 ? (bf16 ? launch_simt_t<__nv_bfloat16, E4m3>(a, d, w, st) : launch_simt_t<float, E4m3>(a, d, w, st))
                                    : (bf16 ? launch_simt_t<__nv_bfloat16, Int4>(a, d, w, st) : launch_simt_t<float, Int4>(a, d, w, st));
  return e != cudaSuccess ? e : launch_attend_join(a, d, bf16, w, max_rows, st);
}

cudaError_t launch_attend_join(const AttendArgs& a, int d, bool bf16, Workers w, int64_t max_rows, cudaStream_t st) {
  const int rows = max_rows < 1 ? 1 : max_rows < w.rows ? (int)max_rows : w.rows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)w.count, (unsigned)(rows < 16 ? rows : 16), 1);
  cfg.blockDim = dim3(kJoinNt, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {early_launch()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kern = bf16 ? (d == 64 ? paged_attend_join_kernel<64, __nv_bfloat16> : paged_attend_join_kernel<128, __nv_bfloat16>)
                   : (d == 64 ? paged_attend_join_kernel<64, float> : paged_attend_join_kernel<128, float>);
  return launched(cudaLaunchKernelEx(&cfg, kern, a, w.rows));
}

}  // namespace paged
}  // namespace qwm
