// qwm_qk_norm_rope: RMS norm of every query and key head and the rotary
// position encoding in one pass over the data.
//
//   x' = x (mean(x^2) + eps)^(-1/2) w;   (a, b) -> (a cos - b sin, b cos + a sin)
//
// A warp takes one row and some or all of its heads: D/8 lanes hold a head, 2
// or 4 heads a step.  A rotating lane holds both channels of four pairs (two
// pieces of four channels, rot/2 apart or, for adjacent pairs, side by side),
// so no channel has to travel between lanes; the others hold eight channels
// behind the rotated ones, which they only weigh (cos 1).  A lane keeps four cos
// and sin for all heads of the row, multiplied by the weight once for the queries
// and once for the keys:
//   out_a = inv (a (w_a c) - b (w_b s)),  out_b = inv (b (w_b c) + a (w_a s))
// in two-wide float32 arithmetic; the mean square is a shuffle sum.  The table
// is read once a row; its loads do not hold up the first heads' loads.
// Bound by HBM (every element is read and written once) and, in bf16, by the
// ~60 instructions of a step: with pairs in lanes apart (8 shuffles), per-head
// addresses from the strides and scalar arithmetic a step took 215.  4,680 rows
// of 48 heads, d = 128, bf16: 23.4 us (5.0 TB/s; 34 us with those 215), 32,760
// rows of 16 heads, d = 64, float32: 48 us (5.7 TB/s).
#include "paged_internal.cuh"
#include "paged_launch.cuh"

namespace qwm {
namespace paged {
namespace {

constexpr int kRopeNt = 128;

// four channels as loaded
template <class T>
struct Vec4;
template <>
struct Vec4<float> {
  float4 u;
  __device__ __forceinline__ void load(const float* p) { u = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void get(float2* x) const { x[0] = make_float2(u.x, u.y), x[1] = make_float2(u.z, u.w); }
  __device__ __forceinline__ static void store(float* p, float2 a, float2 b) {
    *reinterpret_cast<float4*>(p) = make_float4(a.x, a.y, b.x, b.y);
  }
};
template <>
struct Vec4<__nv_bfloat16> {
  uint2 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void get(float2* x) const {
    x[0] = make_float2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
    x[1] = make_float2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
  }
  __device__ __forceinline__ static void store(__nv_bfloat16* p, float2 a, float2 b) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(a.x, a.y), y = __floats2bfloat162_rn(b.x, b.y);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  }
};

// steps whose loads are in flight together, and whether the next ones are sent
// for before these are worked on: in bf16 the chunk takes 25.5 us without, in
// float32, where they are twice the registers, 48 us without and 55 us with
constexpr int kAhead = 3;
template <class T>
constexpr bool kEarly = sizeof(T) == 2;

// ADJ: pairs are adjacent channels
template <int D, bool ADJ, class T>
__global__ void __launch_bounds__(kRopeNt, sizeof(T) == 2 ? 6 : 5) qk_norm_rope_kernel(const qwm_qk_norm_rope_args a, int splits,
                                                                                     int per_split) {
  constexpr int L = D / 8, PER = 32 / L;
  wait_for_kernel_ahead();
  const int lane = threadIdx.x % L, sub = (threadIdx.x & 31) / L, heads = a.q_heads + a.k_heads;
  const int64_t unit = (int64_t)blockIdx.x * (kRopeNt / 32) + (threadIdx.x >> 5);
  const int64_t t = splits == 1 ? unit : unit / splits;
  if (t >= a.rows) return;
  const int h0 = (int)(unit - t * splits) * per_split, h1 = min(heads, h0 + per_split);
  // this lane's two pieces of four channels
  const int half = a.rot / 2;
  const bool turned = 4 * lane < half;
  const int o0 = ADJ || !turned ? 8 * lane : 4 * lane, o1 = ADJ || !turned ? o0 + 4 : o0 + half;
  // the row's positions: one negative or beyond the table leaves the row alone
  int pos[4] = {0, 0, 0, 0};
#pragma unroll
  for (int x = 0; x < 4; ++x)
    if (x < a.axes) pos[x] = load_global(a.positions + t * a.axes + x);
  float2 co[2] = {make_float2(1.f, 1.f), make_float2(1.f, 1.f)}, si[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  bool first = true, dead = false;
  auto run = [&](const qwm_rows& in, const qwm_rows& out, const T* weight, int n0, int n1) {
    const T* src = (const T*)in.ptr + t * in.row_stride + (int64_t)(n0 + sub) * in.head_stride;
    T* dst = (T*)out.ptr + t * out.row_stride + (int64_t)(n0 + sub) * out.head_stride;
    const int64_t src_step = PER * in.head_stride, dst_step = PER * out.head_stride;
    float2 ca[2], sa[2], cb[2], sb[2];   // w_a c, w_a s, w_b c, -w_b s
    bool ready = false;
    Vec4<T> next[kAhead][2];
    auto fetch = [&](int n) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (n + u * PER + sub < n1) {
          next[u][0].load(src + u * src_step + o0);
          next[u][1].load(src + u * src_step + o1);
        }
      src += kAhead * src_step;
    };
    if (kEarly<T>) fetch(n0);
    for (int n = n0; n < n1; n += kAhead * PER) {
      if (!kEarly<T>) fetch(n);
      if (first) {
        first = false;
        bool skip = false, over = false;
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (x < a.axes) {
            skip |= pos[x] < 0;
            over |= pos[x] >= a.n_positions;
          }
        if (skip || over) {
          if (!skip && h0 == 0 && (threadIdx.x & 31) == 0) flag(a.status, QWM_DEV_BOUNDS);
          dead = true;
          return;
        }
        if (turned) {
          const int p0 = 4 * lane, e0 = a.sections[0], e1 = e0 + a.sections[1], e2 = e1 + a.sections[2];
          auto axis = [&](int p) { return a.axes == 1 || p < e0 ? 0 : p < e1 ? 1 : p < e2 ? 2 : 3; };
          auto row = [&](int x) {
            return a.cos_sin + (int64_t)(x == 0 ? pos[0] : x == 1 ? pos[1] : x == 2 ? pos[2] : pos[3]) * a.rot;
          };
          const int x0 = axis(p0);
          if (x0 == axis(p0 + 3)) {
            // rot is a multiple of 16, so the vectors are aligned
            const float* r = row(x0) + p0;
            const float4 c = load_global(reinterpret_cast<const float4*>(r)), z = load_global(reinterpret_cast<const float4*>(r + half));
            co[0] = make_float2(c.x, c.y), co[1] = make_float2(c.z, c.w);
            si[0] = make_float2(z.x, z.y), si[1] = make_float2(z.z, z.w);
          } else {
            float c[4], z[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float* r = row(axis(p0 + k)) + p0 + k;
              c[k] = load_global(r);
              z[k] = load_global(r + half);
            }
            co[0] = make_float2(c[0], c[1]), co[1] = make_float2(c[2], c[3]);
            si[0] = make_float2(z[0], z[1]), si[1] = make_float2(z[2], z[3]);
          }
        }
      }
      if (!ready) {
        ready = true;
        float2 w0[2] = {make_float2(1.f, 1.f), make_float2(1.f, 1.f)}, w1[2] = {make_float2(1.f, 1.f), make_float2(1.f, 1.f)};
        if (weight) {
          Vec4<T> x;
          x.load(weight + o0);
          x.get(w0);
          x.load(weight + o1);
          x.get(w1);
        }
        if (ADJ) {
          // pairs (x0, x1), (x2, x3) of both pieces: a = (0, 2 | 4, 6), b = (1, 3 | 5, 7)
          const float2 p[2] = {w0[0], w0[1]}, q[2] = {w1[0], w1[1]};
          w0[0] = make_float2(p[0].x, p[1].x), w0[1] = make_float2(q[0].x, q[1].x);
          w1[0] = make_float2(p[0].y, p[1].y), w1[1] = make_float2(q[0].y, q[1].y);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          ca[k] = __fmul2_rn(w0[k], co[k]);
          sa[k] = __fmul2_rn(w0[k], si[k]);
          cb[k] = __fmul2_rn(w1[k], co[k]);
          sb[k] = __fmul2_rn(make_float2(-w1[k].x, -w1[k].y), si[k]);
        }
      }
      Vec4<T> v[kAhead][2];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) v[u][0] = next[u][0], v[u][1] = next[u][1];
      if (kEarly<T>) fetch(n + kAhead * PER);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (n + u * PER >= n1) break;   // the whole warp
        float2 x[2], y[2];
        v[u][0].get(x);
        v[u][1].get(y);
        float2 s2 = __fmul2_rn(x[0], x[0]);
        s2 = __ffma2_rn(x[1], x[1], s2);
        s2 = __ffma2_rn(y[0], y[0], s2);
        s2 = __ffma2_rn(y[1], y[1], s2);
        float ss = s2.x + s2.y;
#pragma unroll
        for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, L);
        const float inv = rsqrtf(fmaf(ss, 1.0f / D, a.eps));
        const float2 i2 = make_float2(inv, inv);
        if (ADJ) {
          const float2 p[2] = {x[0], x[1]}, q[2] = {y[0], y[1]};
          x[0] = make_float2(p[0].x, p[1].x), x[1] = make_float2(q[0].x, q[1].x);
          y[0] = make_float2(p[0].y, p[1].y), y[1] = make_float2(q[0].y, q[1].y);
        }
        float2 r[2], z[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          x[k] = __fmul2_rn(x[k], i2);
          y[k] = __fmul2_rn(y[k], i2);
          if (turned) {
            r[k] = __ffma2_rn(x[k], ca[k], __fmul2_rn(y[k], sb[k]));
            z[k] = __ffma2_rn(y[k], cb[k], __fmul2_rn(x[k], sa[k]));
          } else {   // no product with a sine of 0: infinity times 0 is NaN
            r[k] = __fmul2_rn(x[k], ca[k]);
            z[k] = __fmul2_rn(y[k], cb[k]);
          }
        }
        if (ADJ) {
          const float2 p[2] = {r[0], r[1]}, q[2] = {z[0], z[1]};
          r[0] = make_float2(p[0].x, q[0].x), r[1] = make_float2(p[0].y, q[0].y);
          z[0] = make_float2(p[1].x, q[1].x), z[1] = make_float2(p[1].y, q[1].y);
        }
        if (n + u * PER + sub < n1) {
          Vec4<T>::store(dst + u * dst_step + o0, r[0], r[1]);
          Vec4<T>::store(dst + u * dst_step + o1, z[0], z[1]);
        }
      }
      dst += kAhead * dst_step;
    }
  };
  if (h0 < a.q_heads) run(a.q, a.q_out, (const T*)a.q_weight, h0, min(h1, a.q_heads));
  if (h1 > a.q_heads && !dead) run(a.k, a.k_out, (const T*)a.k_weight, max(h0, a.q_heads) - a.q_heads, h1 - a.q_heads);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const qwm_qk_norm_rope_args& a, cudaStream_t st) {
  // a warp takes a whole row when the rows alone fill the machine with 32
  // warps an SM, else fewer heads, down to one step (4,680 rows: one warp a row
  // 25.5 us, two, as here, 23.6, three 27.7, which read the table and the
  // weights once more each)
  const int step = 32 / (a.head_dim / 8), heads = a.q_heads + a.k_heads, steps = (heads + step - 1) / step;
  const int64_t want = ((int64_t)sm_count() * 32 + a.rows - 1) / a.rows;
  const int split = (int)(want < steps ? want : steps), per = (steps + split - 1) / split * step;
  const int splits = (heads + per - 1) / per;
  const dim3 grid((unsigned)((a.rows * splits + kRopeNt / 32 - 1) / (kRopeNt / 32)), 1, 1);
  const bool bf = a.dtype == QWM_BF16;
  auto kern = a.head_dim == 64
                  ? (a.interleaved ? (bf ? qk_norm_rope_kernel<64, true, __nv_bfloat16> : qk_norm_rope_kernel<64, true, float>)
                                   : (bf ? qk_norm_rope_kernel<64, false, __nv_bfloat16> : qk_norm_rope_kernel<64, false, float>))
                  : (a.interleaved ? (bf ? qk_norm_rope_kernel<128, true, __nv_bfloat16> : qk_norm_rope_kernel<128, true, float>)
                                   : (bf ? qk_norm_rope_kernel<128, false, __nv_bfloat16> : qk_norm_rope_kernel<128, false, float>));
  return launch_early(kern, grid, kRopeNt, 0, st, a, splits, per);
}

}  // namespace paged
}  // namespace qwm
