// qwm_qk_norm_rope: RMS norm of every query and key head and the rotary
// position encoding in one pass over the data.
//
//   x' = x (mean(x^2) + eps)^(-1/2) w;   (a, b) -> (a cos - b sin, b cos + a sin)
//
// A warp takes one row and some or all of its heads: D/8 lanes hold a head, 8
// channels each (16 bytes of bf16), 2 or 4 heads a step, four steps' loads in
// flight.  A lane keeps its cos and sin for all heads of the row, so the table
// is read once a row (a group of lanes for each head read it 16 times, more
// bytes from L1 than the data: 64 us on the chunk below); its loads follow the
// first heads' loads, which do not depend on the position.  The mean square is
// a shuffle sum.  Pairs half the rotated width apart sit in lanes R/16 apart
// and meet by one shuffle a channel; adjacent pairs sit in the same lane.
// Bound by HBM: every element is read and written once.
#include "paged_internal.cuh"
#include "paged_launch.cuh"

namespace qwm {
namespace paged {
namespace {

constexpr int kRopeNt = 256;

template <class T>
struct Vec8;
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};
template <>
struct Vec8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float* x) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
__device__ __forceinline__ void store8(float* p, const float* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// steps whose loads are in flight together
constexpr int kAhead = 4;

template <int D, class T>
__global__ void __launch_bounds__(kRopeNt) qk_norm_rope_kernel(const qwm_qk_norm_rope_args a, int splits, int per_split) {
  constexpr int L = D / 8, PER = 32 / L;
  const int lane = threadIdx.x % L, sub = (threadIdx.x & 31) / L, heads = a.q_heads + a.k_heads;
  const int64_t unit = (int64_t)blockIdx.x * (kRopeNt / 32) + (threadIdx.x >> 5);
  const int64_t t = unit / splits;
  if (t >= a.rows) return;
  const int h0 = (int)(unit - t * splits) * per_split, h1 = min(heads, h0 + per_split);
  const int half = a.rot / 2, ch = 8 * lane;
  // the row's positions: one negative or beyond the table leaves the row alone
  int pos[4] = {0, 0, 0, 0};
  bool skip = false, out = false;
#pragma unroll
  for (int x = 0; x < 4; ++x)
    if (x < a.axes) pos[x] = __ldg(a.positions + t * a.axes + x);
  Vec8<T> v[kAhead];
  auto load = [&](int hb) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int h = hb + u * PER + sub;
      if (h < h1) {
        const bool key = h >= a.q_heads;
        v[u].load((const T*)(key ? a.k.ptr : a.q.ptr) + t * (key ? a.k.row_stride : a.q.row_stride) +
                  (key ? (h - a.q_heads) * a.k.head_stride : h * a.q.head_stride) + ch);
      }
    }
  };
  load(h0);
#pragma unroll
  for (int x = 0; x < 4; ++x)
    if (x < a.axes) {
      skip |= pos[x] < 0;
      out |= pos[x] >= a.n_positions;
    }
  if (skip || out) {
    if (!skip && h0 == 0 && (threadIdx.x & 31) == 0) flag(a.status, QWM_DEV_BOUNDS);
    return;
  }
  // the cos and sin of this lane's channels: 4 pairs (interleaved) or 8
  const bool turned = ch < a.rot, low = ch < half;
  float co[8], si[8];
  if (turned) {
    const int p0 = a.interleaved ? ch / 2 : low ? ch : ch - half;
    const int e0 = a.sections[0], e1 = e0 + a.sections[1], e2 = e1 + a.sections[2];
    auto axis = [&](int p) { return a.axes == 1 || p < e0 ? 0 : p < e1 ? 1 : p < e2 ? 2 : 3; };
    auto row = [&](int x) {
      return a.cos_sin + (int64_t)(x == 0 ? pos[0] : x == 1 ? pos[1] : x == 2 ? pos[2] : pos[3]) * a.rot;
    };
    const int last = a.interleaved ? 3 : 7, x0 = axis(p0);
    if (x0 == axis(p0 + last)) {
      // rot is a multiple of 16, so the vectors are aligned
      const float* r = row(x0) + p0;
      const float4 c0 = __ldg(reinterpret_cast<const float4*>(r)), s0 = __ldg(reinterpret_cast<const float4*>(r + half));
      co[0] = c0.x, co[1] = c0.y, co[2] = c0.z, co[3] = c0.w, si[0] = s0.x, si[1] = s0.y, si[2] = s0.z, si[3] = s0.w;
      if (!a.interleaved) {
        const float4 c1 = __ldg(reinterpret_cast<const float4*>(r + 4)), s1 = __ldg(reinterpret_cast<const float4*>(r + half + 4));
        co[4] = c1.x, co[5] = c1.y, co[6] = c1.z, co[7] = c1.w, si[4] = s1.x, si[5] = s1.y, si[6] = s1.z, si[7] = s1.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k <= last) {
          const float* r = row(axis(p0 + k)) + p0 + k;
          co[k] = __ldg(r);
          si[k] = __ldg(r + half);
        }
    }
  }
  // lane of a pair's other half: half / 8 lanes away
  const int mate = !turned ? lane : low ? lane + half / 8 : lane - half / 8;
  const float sign = low ? -1.f : 1.f;
  Vec8<T> wq, wk;
  if (a.q_weight) wq.load((const T*)a.q_weight + ch);
  if (a.k_weight && h1 > a.q_heads) wk.load((const T*)a.k_weight + ch);
  for (int hb = h0; hb < h1; hb += kAhead * PER) {
    if (hb > h0) load(hb);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int h = hb + u * PER + sub;
      if (hb + u * PER >= h1) break;   // the whole warp
      const bool key = h >= a.q_heads;
      float x[8], y[8];
      v[u].get(x);
      float ss = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(x[k], x[k], ss);
#pragma unroll
      for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, L);
      const float inv = rsqrtf(ss * (1.0f / D) + a.eps);
      if (key ? a.k_weight : a.q_weight) {
        if (key) wk.get(y);
        else wq.get(y);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] *= inv * y[k];
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] *= inv;
      }
      if (a.interleaved) {
        if (turned) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float p = x[2 * k], q = x[2 * k + 1];
            x[2 * k] = p * co[k] - q * si[k];
            x[2 * k + 1] = q * co[k] + p * si[k];
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = __shfl_sync(0xffffffffu, x[k], mate, L);
        if (turned) {
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = fmaf(x[k], co[k], sign * (y[k] * si[k]));
        }
      }
      if (h < h1)
        store8((T*)(key ? a.k_out.ptr : a.q_out.ptr) + t * (key ? a.k_out.row_stride : a.q_out.row_stride) +
                   (key ? (h - a.q_heads) * a.k_out.head_stride : h * a.q_out.head_stride) + ch, x);
    }
  }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const qwm_qk_norm_rope_args& a, cudaStream_t st) {
  // a warp takes a whole row when the rows alone fill the machine with 32
  // warps an SM, else fewer heads, down to one step
  const int step = 32 / (a.head_dim / 8), heads = a.q_heads + a.k_heads, steps = (heads + step - 1) / step;
  const int64_t want = ((int64_t)sm_count() * 32 + a.rows - 1) / a.rows;
  const int split = (int)(want < steps ? want : steps), per = (steps + split - 1) / split * step;
  const int splits = (heads + per - 1) / per;
  const dim3 grid((unsigned)((a.rows * splits + kRopeNt / 32 - 1) / (kRopeNt / 32)), 1, 1);
  const bool bf = a.dtype == QWM_BF16;
  auto kern = a.head_dim == 64 ? (bf ? qk_norm_rope_kernel<64, __nv_bfloat16> : qk_norm_rope_kernel<64, float>)
                               : (bf ? qk_norm_rope_kernel<128, __nv_bfloat16> : qk_norm_rope_kernel<128, float>);
  kern<<<grid, kRopeNt, 0, st>>>(a, splits, per);
  return cudaGetLastError();
}

}  // namespace paged
}  // namespace qwm
