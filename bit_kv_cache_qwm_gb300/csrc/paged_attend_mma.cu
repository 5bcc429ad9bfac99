// qwm_paged_attend for few rows (kernel 2, bf16): single-token steps and short
// drafts, where the pages are read once and everything else must keep up.
//
//   s_n = q . k_hat_n;  O = sum_n exp2(s_n - m) v_hat_n, running maximum m
//
// A worker (CTA) walks the tiles of 64 tokens that the partition deals to it.
// One producer warp copies the packed tiles (160 bytes a token at d = 128)
// into a ring of shared-memory stages with bulk copies, one mbarrier a stage;
// it holds the next 64 page ids in registers, so the table's latency is not
// on the copies' path.  Four consumer warps take 16 tokens of every tile each,
// with their own running maximum, and meet at the end of an item only.
//
// A consumer keeps everything in registers.  Both products are formed
// transposed with mma.m16n8k16 (float16 in, float32 out), the 16 tokens or
// channels on the long side and the 8 query rows on the short one:
//   S^T[16 tokens][8 rows]  = K_hat[16][d] Q^T      d/16 MMAs
//   O^T[d][8 rows]         += V_hat^T[d][16] P^T    d/16 MMAs
// so that a step of 5 or 8 query heads a key/value head does not pay for 16
// rows.  Channels are contracted in the order in which the codes lie in
// memory: a lane takes one run of codes of its token in one load, and Q is
// laid out to match.  P^T is S^T transposed in 8 x 8 blocks (movmatrix).
// A code c becomes float16 by one mask that puts it into the mantissa of 1024
// (1024 + c, or 1024 + 16 c for the upper nibble of a byte), one exact
// subtraction (or fused multiply by 1/16), and c scale + zero by one fused
// multiply-add: the only rounding of k_hat and v_hat.  Q is float16 scaled per
// row by a power of two (exact).  The rows' sums and O are float32; O is
// rescaled only when a row's maximum grows by more than 2^8 (P <= 2^8).
// Tokens outside a request (or on a page out of range) have their logits
// replaced and their value parameters zeroed, so garbage bytes do no harm.
//
// Bound by HBM: 1.25 d bytes a token; about 18 instructions a token and warp
// leave the issue slots about as busy as the memory.
#include "paged_internal.cuh"
#include "tcgen05_util.cuh"

namespace qwm {
namespace paged {
namespace {

using namespace tcx;

constexpr int kTk = 64, kCw = 4, kNt = (kCw + 1) * 32, kStages = 4, kItem = 2;
constexpr float kNone = -3.0e38f;   // running maximum of a row that has seen nothing

template <int D>
struct Stage {
  static constexpr int G = D / 32;
  static constexpr int kcode = 0, kpar = kTk * D / 2, vcode = kpar + kTk * G * 4, vpar = vcode + kTk * D / 2;
  static constexpr int bytes = vpar + kTk * G * 4;
};
template <int D, int NB>
struct Smem {
  static constexpr int LD = D + 4;                          // rows 2 c of a store phase 8 banks apart
  static constexpr int merge = kStages * Stage<D>::bytes;   // float [kCw][8 NB][LD]
  static constexpr int stat = merge + kCw * 8 * NB * LD * 4;
  static constexpr int bytes = stat + kCw * 8 * NB * 8;     // float2 (m, l) [kCw][8 NB]
};

__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }

// c scale + zero for the lower (upper) nibbles of bytes 0 and 2 of x
__device__ __forceinline__ uint32_t dq_lo(uint32_t x, __half2 s, __half2 z) {
  const __half2 c = __hsub2(u2h((x & 0x000f000fu) | 0x64006400u), __float2half2_rn(1024.f));
  return h2u(__hfma2(c, s, z));
}
__device__ __forceinline__ uint32_t dq_hi(uint32_t x, __half2 s, __half2 z) {
  const __half2 c = __hfma2(u2h((x & 0x00f000f0u) | 0x64006400u), __float2half2_rn(0.0625f), __float2half2_rn(-64.f));
  return h2u(__hfma2(c, s, z));
}
// the token of a block of 8 that column (or row) n of a fragment holds: the
// lanes of a load phase then meet even and odd 64-byte rows
__device__ __forceinline__ int token_of(int n) { return (n & 1) ? 4 + ((n >> 1) ^ 1) : n >> 1; }

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kCw * 32) : "memory"); }

template <int D, int NB>
__global__ void __launch_bounds__(kNt, NB == 1 ? 3 : 2) paged_attend_mma_kernel(const AttendArgs a) {
  constexpr int R = 8 * NB, G = D / 32, KW = D / 32, VW = D / 64, MB = D / 16;
  using St = Stage<D>;
  using Sm = Smem<D, NB>;
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages];
  __shared__ uint32_t vmask[kStages];
  __shared__ volatile int abort_sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, w = blockIdx.x;
  if (tid == 0) {
    abort_sh = 0;
    for (int i = 0; i < kStages; ++i) {
      bar_init(&full[i], 1);
      bar_init(&empty[i], kCw);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    a.join[w].last = -1;
  }
  const Share sh = find_share<R, kTk, kItem, kNt>(a, w, (int)gridDim.x);   // has block barriers
  cudaTriggerProgrammaticLaunchCompletion();   // the join kernel may be made ready
  if (sh.n == 0) return;
  Walker<R, kTk, kItem> it(a);
  it.start(sh.b, sh.skip, sh.per, sh.n);
  int st = 0;
  uint32_t phase = 0;

  if (warp == kCw) {
    // ------------------------------------------------------------ producer
    const int run = a.page < kTk ? a.page : kTk;        // tokens of one copy
    const int r = lane >> 2, sec = lane & 3;
    const bool code = (sec & 1) == 0;
    const int per = code ? D / 2 : G * 4;               // bytes a token in this section
    const int src_off = (sec & 2 ? a.block / 2 : 0) + (code ? 0 : a.page * (D / 2));
    const int dst_off = (sec == 0 ? St::kcode : sec == 1 ? St::kpar : sec == 2 ? St::vcode : St::vpar) + r * run * per;
    const uint32_t bytes = (uint32_t)(run * per);
    int issued = 0;
    bool ok = true;
    do {
      const int32_t* row = a.table + (int64_t)it.b * a.max_blocks;
      int base = (it.from * kTk) >> a.page_shift;
      auto ids = [&](int p) { return p + lane < a.max_blocks ? row[p + lane] : -1; };
      int cur = ids(base), nxt = ids(base + 32);
      for (int t = it.from; t < it.to && ok; ++t) {
        const int n = t * kTk + r * run, p = (t * kTk) >> a.page_shift;
        if (p >= base + 32) {
          base += 32;
          cur = nxt;
          nxt = ids(base + 32);
        }
        const bool need = r * run < kTk && n < it.hi && n + run > it.lo;
        const int pg = __shfl_sync(0xffffffffu, cur, ((n >> a.page_shift) - base) & 31);
        const bool good = need && pg >= 0 && pg < a.n_pages;
        if (need && !good && sec == 0) flag(a.status, QWM_DEV_BOUNDS);
        const uint32_t who = __ballot_sync(0xffffffffu, good);
        if (issued >= kStages) ok = warp_all(bar_wait(&empty[st], phase ^ 1, &abort_sh, a.timeout));
        if (!ok) break;
        if (lane == 0) {
          uint32_t m = 0;      // a bit for every 16 tokens
          for (int s = 0; s < 4; ++s)
            if (who >> ((s * 16 / run) * 4) & 1) m |= 1u << s;
          vmask[st] = m;
          bar_expect_tx(&full[st], (uint32_t)(__popc(who) / 4) * (uint32_t)(run * (D + D / 4)));
        }
        __syncwarp();
        if (good) {
          const uint8_t* src = a.pool + ((int64_t)pg * a.kv_heads + it.h) * a.block + src_off + (n & (a.page - 1)) * per;
          bulk_g2s(sm + st * St::bytes + dst_off, src, bytes, &full[st]);
        }
        ++issued;
        if (++st == kStages) st = 0, phase ^= 1;
      }
    } while (ok && it.next());
    // after a timeout: no copy of ours may land in memory that is given back
    if (!ok && lane == 0)
      for (int i = 0; i < (issued < kStages ? issued : kStages); ++i) {
        const int s = (st + kStages - 1 - i) % kStages;
        const uint32_t ph = (uint32_t)(((issued - 1 - i) / kStages) & 1);
        const long long t0 = clock64();
        while (!bar_test(&full[s], ph) && clock64() - t0 < kWaitCycles) {}
      }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int g = lane >> 2, c = lane & 3;
  const int tok0 = token_of(g);                  // this lane's key of a block of 8
  const int ta = token_of(2 * c), tb = token_of(2 * c + 1);   // its value tokens
  float* merge = reinterpret_cast<float*>(sm + Sm::merge);
  float2* stat = reinterpret_cast<float2*>(sm + Sm::stat);
  do {
    // Q^T fragments: row g of each block of 8, in the order of the codes
    uint32_t qf[NB][MB][2];
    float c2[NB][2];       // logit factor of rows 2 c and 2 c + 1
    int top[NB][2], bottom[NB][2];
    int top_min = it.hi, bottom_max = it.lo;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int rr = it.rt * R + nb * 8 + g;
      const bool live = nb * 8 + g < it.rows;
      float x[D / 4];
      float mx = 0.f;
      const int tok = live ? div_group(a, rr) : 0, head = live ? it.h * a.group + rr - div_group(a, rr) * a.group : 0;
      const uint4* src = reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.q + (int64_t)(it.rq.row0 + tok) * a.q_row +
                                                       head * a.q_head + c * (D / 4));
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 u = live ? src[i] : make_uint4(0, 0, 0, 0);
        const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[8 * i + 2 * k] = __uint_as_float(v[k] << 16);
          x[8 * i + 2 * k + 1] = __uint_as_float(v[k] & 0xffff0000u);
          mx = max3f(mx, fabsf(x[8 * i + 2 * k]), fabsf(x[8 * i + 2 * k + 1]));
        }
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int ex = (int)((__float_as_uint(mx) >> 23) & 0xffu) - 127;
      const int e = ex > 14 ? ex - 14 : 0;
      const float qs = __uint_as_float((uint32_t)(127 - e) << 23);   // 2^-e: the largest entry below 2^15
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        const float* y = x + 8 * i;
        qf[nb][2 * i][0] = h2u(__floats2half2_rn(y[0] * qs, y[4] * qs));
        qf[nb][2 * i][1] = h2u(__floats2half2_rn(y[1] * qs, y[5] * qs));
        qf[nb][2 * i + 1][0] = h2u(__floats2half2_rn(y[2] * qs, y[6] * qs));
        qf[nb][2 * i + 1][1] = h2u(__floats2half2_rn(y[3] * qs, y[7] * qs));
      }
      const float f = a.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        c2[nb][k] = __shfl_sync(0xffffffffu, f, (2 * c + k) * 4);
        const int r2 = it.rt * R + nb * 8 + 2 * c + k;
        top[nb][k] = it.hi, bottom[nb][k] = it.lo;
        if (a.causal) {
          const int pos = it.rq.n - it.rq.n_new + div_group(a, r2);
          top[nb][k] = min(it.hi, pos + 1);
          if (a.window > 0) bottom[nb][k] = max(it.lo, pos - a.window + 1);
        }
      }
    }
    if (a.causal) {
      const int first = div_group(a, it.rt * R), last = div_group(a, it.rt * R + it.rows - 1), at = it.rq.n - it.rq.n_new;
      top_min = min(it.hi, at + first + 1);
      if (a.window > 0) bottom_max = max(it.lo, at + last - a.window + 1);
    }
    float o[NB][MB][4], m[NB][2], l[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int j = 0; j < MB; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[nb][j][k] = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) m[nb][k] = kNone, l[nb][k] = 0.f;
    }
    for (int t = it.from; t < it.to; ++t) {
      bar_wait(&full[st], phase, &abort_sh, a.timeout);
      const uint8_t* tile = sm + st * St::bytes;
      const int n0 = t * kTk + 16 * warp;
      const bool have = (vmask[st] >> warp) & 1;
      if (have && n0 < it.hi && n0 + 16 > it.lo) {
        const bool whole = n0 + 16 <= top_min && n0 >= bottom_max;
        // ---- S^T
        float s[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.f;
        {
          uint32_t kw[2][KW];
          __half2 ks[2], kz[2];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int row = 16 * warp + 8 * b + tok0;
            if constexpr (D == 128) {
              const uint4 u = *reinterpret_cast<const uint4*>(tile + St::kcode + row * 64 + 16 * c);
              kw[b][0] = u.x, kw[b][1] = u.y, kw[b][2] = u.z, kw[b][3] = u.w;
            } else {
              const uint2 u = *reinterpret_cast<const uint2*>(tile + St::kcode + row * 32 + 8 * c);
              kw[b][0] = u.x, kw[b][1] = u.y;
            }
            const __half2 par = *reinterpret_cast<const __half2*>(tile + St::kpar + (row * G + c * G / 4) * 4);
            kz[b] = __low2half2(par);
            ks[b] = __high2half2(par);
          }
#pragma unroll
          for (int i = 0; i < KW; ++i) {
            uint32_t f[4], f2[4];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              f[b] = dq_lo(kw[b][i], ks[b], kz[b]);
              f[2 + b] = dq_hi(kw[b][i], ks[b], kz[b]);
              const uint32_t up = kw[b][i] >> 8;
              f2[b] = dq_lo(up, ks[b], kz[b]);
              f2[2 + b] = dq_hi(up, ks[b], kz[b]);
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              mma(s[nb], f, qf[nb][2 * i][0], qf[nb][2 * i][1]);
              mma(s[nb], f2, qf[nb][2 * i + 1][0], qf[nb][2 * i + 1][1]);
            }
          }
        }
        // ---- softmax: s[nb][2 b + k] is token 8 b + token_of(g), row 2 c + k
        uint32_t pf[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = s[nb][i] * c2[nb][i & 1];
          if (!whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int n = n0 + 8 * (i >> 1) + tok0;
              if (n < bottom[nb][i & 1] || n >= top[nb][i & 1]) x[i] = -INFINITY;
            }
          }
          const float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
          if (__any_sync(0xffffffffu, mx0 > m[nb][0] + 8.f || mx1 > m[nb][1] + 8.f)) {
            // rare: the rows' maxima over the 16 tokens, and O rescaled
            float u0 = mx0, u1 = mx1;
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              u0 = fmaxf(u0, __shfl_xor_sync(0xffffffffu, u0, d));
              u1 = fmaxf(u1, __shfl_xor_sync(0xffffffffu, u1, d));
            }
            u0 = fmaxf(u0, m[nb][0]);
            u1 = fmaxf(u1, m[nb][1]);
            const float f0 = ex2(m[nb][0] - u0), f1 = ex2(m[nb][1] - u1);
            m[nb][0] = u0, m[nb][1] = u1;
            l[nb][0] *= f0, l[nb][1] *= f1;
#pragma unroll
            for (int j = 0; j < MB; ++j) {
              o[nb][j][0] *= f0, o[nb][j][1] *= f1;
              o[nb][j][2] *= f0, o[nb][j][3] *= f1;
            }
          }
          float p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) p[i] = ex2(x[i] - m[nb][i & 1]);
          l[nb][0] += p[0] + p[2];
          l[nb][1] += p[1] + p[3];
          pf[nb][0] = transpose8(h2u(__floats2half2_rn(p[0], p[1])));
          pf[nb][1] = transpose8(h2u(__floats2half2_rn(p[2], p[3])));
        }
        // ---- O^T: tokens ta, tb (columns 2 c, 2 c + 1) of both blocks of 8
        uint32_t f[MB][4];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int r0 = 16 * warp + 8 * b + ta, r1 = 16 * warp + 8 * b + tb;
          uint32_t v0[VW], v1[VW];
          if constexpr (D == 128) {
            const uint2 u0 = *reinterpret_cast<const uint2*>(tile + St::vcode + r0 * 64 + 8 * g);
            const uint2 u1 = *reinterpret_cast<const uint2*>(tile + St::vcode + r1 * 64 + 8 * g);
            v0[0] = u0.x, v0[1] = u0.y, v1[0] = u1.x, v1[1] = u1.y;
          } else {
            v0[0] = *reinterpret_cast<const uint32_t*>(tile + St::vcode + r0 * 32 + 4 * g);
            v1[0] = *reinterpret_cast<const uint32_t*>(tile + St::vcode + r1 * 32 + 4 * g);
          }
          uint32_t p0 = *reinterpret_cast<const uint32_t*>(tile + St::vpar + (r0 * G + g * G / 8) * 4);
          uint32_t p1 = *reinterpret_cast<const uint32_t*>(tile + St::vpar + (r1 * G + g * G / 8) * 4);
          if (!whole) {
            // tokens outside the request: their bytes may be anything
            const int x0 = n0 + 8 * b + ta, x1 = n0 + 8 * b + tb;
            if (x0 < it.lo || x0 >= it.hi) p0 = 0;
            if (x1 < it.lo || x1 >= it.hi) p1 = 0;
          }
          const __half2 z = u2h(__byte_perm(p0, p1, 0x5410)), sc = u2h(__byte_perm(p0, p1, 0x7632));
          // f[j][2 b]: channel row g, f[j][2 b + 1]: channel row g + 8 of block j
#pragma unroll
          for (int q = 0; q < VW; ++q)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              // byte y of both tokens into bytes 0 and 2
              const uint32_t x = __byte_perm(v0[q], v1[q], y * 0x0011 + (4 + y) * 0x1100);
              const uint32_t lo = dq_lo(x, sc, z), hi = dq_hi(x, sc, z);
              if constexpr (D == 128) {
                f[2 * y][2 * b + q] = lo;
                f[2 * y + 1][2 * b + q] = hi;
              } else {
                f[(2 * y) & 3][2 * b + (y >> 1)] = lo;
                f[(2 * y + 1) & 3][2 * b + (y >> 1)] = hi;
              }
            }
        }
#pragma unroll
        for (int j = 0; j < MB; ++j)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma(o[nb][j], f[j], pf[nb][0], pf[nb][1]);
      }
      __syncwarp();
      if (lane == 0) bar_arrive(&empty[st]);
      if (++st == kStages) st = 0, phase ^= 1;
    }
    // ---- the warps' parts of the item meet
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nb][k] += __shfl_xor_sync(0xffffffffu, l[nb][k], d);
        const int r = nb * 8 + 2 * c + k;
        if (g == 0) stat[warp * R + r] = make_float2(m[nb][k], l[nb][k]);
        // rows g and g + 8 of block j are the channels (2 MB) g + j and
        // (2 MB) g + MB + j, kept at 16 j + 2 g and 16 j + 2 g + 1
        float* row = merge + (warp * R + r) * Sm::LD;
#pragma unroll
        for (int j = 0; j < MB; ++j)
          *reinterpret_cast<float2*>(row + 16 * j + 2 * g) = make_float2(o[nb][j][k], o[nb][j][2 + k]);
      }
    }
    consumers_sync();
    {
      const bool all = it.begins() && it.ends();
      const int slot = it.begins() ? 1 : 0;
      for (int i = tid; i < it.rows * (D / 4); i += kCw * 32) {
        const int r = i / (D / 4), ch = 4 * (i % (D / 4));
        float mx = kNone;
#pragma unroll
        for (int x = 0; x < kCw; ++x) mx = fmaxf(mx, stat[x * R + r].x);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll
        for (int x = 0; x < kCw; ++x) {
          const float2 ml = stat[x * R + r];
          const float f = ex2(ml.x - mx);
          const float* y = merge + (x * R + r) * Sm::LD + 16 * (ch % MB) + ch / MB;
          v.x = fmaf(y[0], f, v.x), v.y = fmaf(y[16], f, v.y), v.z = fmaf(y[32], f, v.z), v.w = fmaf(y[48], f, v.w);
          sum = fmaf(ml.y, f, sum);
        }
        if (all) {
          const int rr = it.rt * R + r;
          const int64_t tok = it.rq.row0 + div_group(a, rr);
          const int head = it.h * a.group + rr - div_group(a, rr) * a.group;
          const float inv = sum > 0.f ? 1.f / sum : 0.f;
          const __nv_bfloat162 b0 = __floats2bfloat162_rn(v.x * inv, v.y * inv), b1 = __floats2bfloat162_rn(v.z * inv, v.w * inv);
          *reinterpret_cast<uint2*>((__nv_bfloat16*)a.out + tok * a.o_row + head * a.o_head + ch) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
          if (a.lse && ch == 0) a.lse[tok * a.heads + head] = sum > 0.f ? (mx + log2f(sum)) * 0.69314718055994531f : -INFINITY;
        } else {
          float* dst = part_row(a, w, slot, R, r, D);
          *reinterpret_cast<float4*>(dst + ch) = v;
          if (ch == 0) dst[D] = mx, dst[D + 1] = sum;
        }
      }
      if (tid == 0 && it.begins() && !it.ends()) {
        record_join(a, w, it, last_worker(sh, it.end_of(sh.first)), R);
      }
    }
    consumers_sync();
  } while (it.next());
}

template <int D, int NB>
cudaError_t launch_mma(const AttendArgs& a, int workers, cudaStream_t st) {
  static SmemLimit limit;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)workers, 1, 1);
  cfg.blockDim = dim3(kNt, 1, 1);
  cfg.dynamicSmemBytes = Smem<D, NB>::bytes;
  cfg.stream = st;
  return launch_smem(limit, cfg.dynamicSmemBytes, paged_attend_mma_kernel<D, NB>, cfg, a);
}

}  // namespace

Workers mma_workers(int64_t max_rows) {
  const int sms = sm_count();
  return max_rows <= 8 ? Workers{3 * sms, 8} : Workers{2 * sms, 16};
}

cudaError_t launch_attend_mma(const AttendArgs& a, int d, int64_t max_rows, cudaStream_t st) {
  const Workers w = mma_workers(max_rows);
  const cudaError_t e = w.rows == 8 ? (d == 64 ? launch_mma<64, 1>(a, w.count, st) : launch_mma<128, 1>(a, w.count, st))
                                    : (d == 64 ? launch_mma<64, 2>(a, w.count, st) : launch_mma<128, 2>(a, w.count, st));
  return e != cudaSuccess ? e : launch_attend_join(a, d, true, w, max_rows, st);
}

}  // namespace paged
}  // namespace qwm
