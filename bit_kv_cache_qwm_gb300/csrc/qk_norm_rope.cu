// qwm_qk_norm_rope: RMS norm of every query and key head and the rotary
// position encoding in one pass over the data.
//
//   x' = x (mean(x^2) + eps)^(-1/2) w;   (a, b) -> (a cos - b sin, b cos + a sin)
//
// D/8 lanes hold one head, 8 channels each (16 bytes of bf16), the mean square
// is a shuffle sum over them.  Pairs half the rotated width apart sit in lanes
// R/16 apart and meet by one shuffle per channel; adjacent pairs sit in the
// same lane.  A lane keeps its cos and sin in registers for all heads of a
// row, so the table is read once per row and group of lanes.  Bound by HBM:
// every element is read and written once.
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

template <int D, class T>
__global__ void __launch_bounds__(kRopeNt) qk_norm_rope_kernel(const qwm_qk_norm_rope_args a) {
  constexpr int L = D / 8, PER = kRopeNt / L;
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x % L, heads = a.q_heads + a.k_heads;
  const int half = a.rot / 2;
  // the row's positions: one negative or beyond the table leaves the row alone
  int pos[4] = {0, 0, 0, 0};
  bool skip = false, out = false;
#pragma unroll
  for (int x = 0; x < 4; ++x)
    if (x < a.axes) {
      pos[x] = a.positions[t * a.axes + x];
      skip |= pos[x] < 0;
      out |= pos[x] >= a.n_positions;
    }
  if (skip || out) {
    if (!skip && blockIdx.y == 0 && threadIdx.x == 0) flag(a.status, QWM_DEV_BOUNDS);
    return;
  }
  // the cos and sin of this lane's channels: 4 pairs (interleaved) or 8
  const int ch = 8 * lane;
  const bool turned = ch < a.rot;
  float co[8], si[8];
  if (turned) {
    const int p0 = a.interleaved ? ch / 2 : ch % half;
    const int n = a.interleaved ? 4 : 8;
    const int e0 = a.sections[0], e1 = e0 + a.sections[1], e2 = e1 + a.sections[2];
    auto row = [&](int p) {
      const int64_t r = a.axes == 1 || p < e0 ? pos[0] : p < e1 ? pos[1] : p < e2 ? pos[2] : pos[3];
      return a.cos_sin + r * a.rot;
    };
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k < n) {
        const float* r = row(p0 + k);
        co[k] = r[p0 + k];
        si[k] = r[half + p0 + k];
      }
    }
  }
  const bool low = ch < half;
  // the lanes of one head: its group leaves the loop as a whole
  const uint32_t mask = (L == 16 ? 0xffffu : 0xffu) << ((threadIdx.x & 31) / L * L);
  for (int hh = blockIdx.y * PER + threadIdx.x / L; hh < heads; hh += gridDim.y * PER) {
    const bool key = hh >= a.q_heads;
    const int h = key ? hh - a.q_heads : hh;
    const qwm_rows in = key ? a.k : a.q, dst = key ? a.k_out : a.q_out;
    const T* weight = (const T*)(key ? a.k_weight : a.q_weight);
    Vec8<T> v;
    v.load((const T*)in.ptr + t * in.row_stride + h * in.head_stride + ch);
    float x[8], y[8];
    v.get(x);
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fmaf(x[k], x[k], ss);
#pragma unroll
    for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(mask, ss, o, L);
    const float inv = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
    if (weight) {
      Vec8<T> wv;
      wv.load(weight + ch);
      wv.get(y);
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
      // lane of the pair's other half: half / 8 lanes away
      const int mate = turned ? (low ? lane + half / 8 : lane - half / 8) : lane;
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = __shfl_sync(mask, x[k], mate, L);
      if (turned) {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = low ? x[k] * co[k] - y[k] * si[k] : x[k] * co[k] + y[k] * si[k];
      }
    }
    store8((T*)dst.ptr + t * dst.row_stride + h * dst.head_stride + ch, x);
  }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const qwm_qk_norm_rope_args& a, cudaStream_t st) {
  const int per = kRopeNt / (a.head_dim / 8), heads = a.q_heads + a.k_heads;
  const int64_t groups = (heads + per - 1) / per;
  const dim3 grid((unsigned)a.rows, (unsigned)(groups < 65535 ? groups : 65535), 1);
  const bool bf = a.dtype == QWM_BF16;
  auto kern = a.head_dim == 64 ? (bf ? qk_norm_rope_kernel<64, __nv_bfloat16> : qk_norm_rope_kernel<64, float>)
                               : (bf ? qk_norm_rope_kernel<128, __nv_bfloat16> : qk_norm_rope_kernel<128, float>);
  kern<<<grid, kRopeNt, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace paged
}  // namespace qwm
