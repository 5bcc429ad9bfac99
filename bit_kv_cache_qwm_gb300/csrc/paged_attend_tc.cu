// qwm_paged_attend for many rows (kernel 3, bf16): prompts and chunks, on the
// 5th-generation tensor cores.
//
//   S = Q K_hat^T,  P = exp2(S - m),  O += P V_hat   (float16 operands, float32 sums)
//
// A worker (one CTA an SM) walks items of 256 rows (two M = 128 query tiles a,
// b of one request and key/value head; the rows of a head group follow one
// another token by token) and tiles of 128 tokens.  Warp roles (16 warps):
//   warps 0-3 / 4-7  softmax of query tile a / b, thread = row = TMEM lane:
//                    per tile the online softmax in the exp2 domain with O
//                    rescaled only when the maximum grows by more than 2^8 (P <=
//                    2^15), P
//                    in float16 over the first 64 columns of S; at the item's
//                    end O from TMEM to memory.
//   warps 8-11       producers, thread = token: the packed codes (64 + 64
//                    bytes at d = 128) and parameters of the next tile are
//                    loaded into registers one tile ahead, its page id two
//                    tiles ahead, and dequantised into two-stage K and V tiles
//                    (one 16-byte store a code word, no bank conflicts: the
//                    eight rows of a store phase differ in the swizzle).
//   warp 12          MMA issuer and TMEM owner.
//   warps 13-15      query loaders: an item's queries (float16, SW128 K-major)
//                    as soon as the last S of the item before is complete, so
//                    its first S runs while that one's O is stored.
// Tensor order: S_a(0) S_b(0), then per tile t
//   PV_a(t) S_a(t+1) PV_b(t) S_b(t+1)
// so while one query tile's 16 MMAs run (1.25K cycles at d = 128) the other's
// softmax has the time for P; S_g(t+1) follows PV_g(t) in the pipe, which keeps
// P_g(t), lying over S_g, until it has been read.  PV_g is issued in three
// parts as P's keys are written.  K and V are double-buffered so that the
// producers are never waited for.
// Handoffs between threads are named barriers (K and V of a stage written, P
// parts written), which do not queue behind the operand reads in the
// shared-memory pipe; the tensor pipe's completions arrive on mbarriers.
// Every mbarrier wait is bounded.  Named barriers cannot be, and the mbarriers
// are what keeps their feeders (producers, softmax) from arriving twice before
// the issuer has taken the first arrival.  So once a wait has run out every role
// still goes through its loop with all arrivals, the issuer without issuing, and
// a feeder whose wait has failed follows the issuer's count of finished tiles
// from then on (its mbarriers stand still, and a parity two phases behind reads
// as done).  A tile's arrivals need no more than the tile before to be finished,
// so this always goes on; tests/test_paged_handoffs.py runs the hand-offs in
// random orders.  The rows of an item that ends after a wait has run out are
// NaN, the status bit is set, and the TMEM is freed after what is in flight.
// Channel order of all operands within 8 channels: 0 4 1 5 2 6 3 7, the order
// in which masks of a code word give float16 pairs.
// TMEM columns: S_a [0,128), S_b [128,256), O_a [256,256+d), O_b [384,384+d).
// Bound by the tensor pipe and the softmax between its MMAs.  Measured at d =
// 128: 4,680 queries over 32,760 tokens, 24 heads, not causal, called back to
// back 1.43 ms (1.32 PFLOP/s; the power cap holds the clock down), ten calls in a
// graph after a pause 1.35 to 1.40 each; four ragged prompts of 900 to 4,096
// tokens, 32 heads over 8, causal, 0.42 ms (0.95 PFLOP/s of the visible
// products), where an item has some 18 tiles and its first S, its end and its
// causal edge cost about 5 more.  Of these 0.42 ms the rows' scales up as well as
// down take 5 us, the check of values that some row does not see 2.
// In a graph, before those two, the first without the producers' stores took 1.22
// ms, without exponentials 1.30 and without either 1.18 (these three with the
// queries loaded by the softmax warps, then 1.43 in all: the loads shared their
// registers); with the producers loading the queries 1.55, the prompts 0.51.
// What an item weighs in tiles when work is dealt out (kItem): the prompts took
// 0.57 ms at 0, 0.45 at 3, 0.42 at 4 to 6 (then 0.41 in all).
#include "paged_internal.cuh"
#include "tcgen05_util.cuh"

namespace qwm {
namespace paged {
namespace {

using namespace tcx;

constexpr int kTk = 128, kRows = 256, kNt = 16 * 32, kProd = 8, kMma = 12, kLoad = 13, kItem = 6;
constexpr uint32_t kColO = 256;
constexpr float kNone = -3.0e38f;
// Where a row's maximum is x0 when it is taken, m = x0 - 7, and it is taken again
// when a logit passes x0 + 8: P <= 2^15 stays inside float16, and a token of a
// long cache is lost only below 2^-25 / 2^7 of the largest weight
constexpr float kBelow = 7.f, kGrow = 8.f;
// an item's queries are scaled by 2^kUp together where their bf16 bits allow it
constexpr int kUp = 6;
constexpr uint32_t kFitLow = (127 - 2 - kUp) << 7, kFitHigh = (127 + 15 - kUp) << 7;
// float16 x float16 -> float32, M = 128; N = 128 keys, or N = d channels with an MN-major B
constexpr uint32_t kIdescS = (1u << 4) | (16u << 17) | (8u << 24);

template <int D>
struct Lay {
  static constexpr int op = 128 * D * 2;              // one operand tile
  static constexpr int k = 2 * op, v = k + 2 * op;    // after Q_a, Q_b
  static constexpr int stage = v + 2 * op;            // 32 rows x 128 bytes for each softmax warp
  static constexpr int bytes = stage + kProd * 4096 + 1024;   // and room to align
  static constexpr uint32_t idesc_pv = (1u << 4) | (1u << 16) | ((uint32_t)(D / 8) << 17) | (8u << 24);
};

// named barriers: K stage s written (1 + s), V stage s written (3 + s), P_g in
// three parts (5 + g, 7 + g, 9 + g); softmax group g (11 + g), query
// loaders (13)
constexpr int kNbK = 1, kNbV = 3, kNbP1 = 5, kNbP2 = 7, kNbP3 = 9, kNbS = 11, kNbQ = 13;
constexpr int kLoaders = (kNt / 32 - kLoad) * 32;   // threads
__device__ __forceinline__ void nb_arrive(int id) { asm volatile("bar.arrive %0, 160;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void nb_sync(int id) { asm volatile("bar.sync %0, 160;" ::"r"(id) : "memory"); }
// a softmax group meets (the barrier that also takes a vote makes the better code
// around the loop's wait: 48 ragged single tokens on this kernel 320 us, with the
// plain one 332)
__device__ __forceinline__ void group_meet(int g, bool v) {
  asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %0, 0;\nbar.red.and.pred q, %1, 128, p;\n}"
               ::"r"((uint32_t)v), "r"(kNbS + g) : "memory");
}
__device__ __forceinline__ void group_sync(int g) { asm volatile("bar.sync %0, 128;" ::"r"(kNbS + g) : "memory"); }

// what a wait that does not end at once needs
struct Waits {
  volatile int abort;      // a wait has run out
  volatile int finished;   // tiles that the issuer has taken all arrivals of
  uint32_t* status;
  long long limit;
};

// until the issuer has finished `tiles` tiles
__device__ __noinline__ void follow(const Waits* w, int tiles) {
  const long long t0 = clock64();
  while (w->finished < tiles && clock64() - t0 < kWaitCycles) {
  }
}

__device__ __noinline__ bool wait_long(bool ok, uint64_t* bar, uint32_t par, Waits* w, int tiles) {
  if (ok && bar_wait(bar, par, &w->abort, w->status, w->limit)) return true;
  follow(w, tiles);
  return false;
}
// The phase of parity `par` of an mbarrier; false when the wait for it, or one
// before (not ok), ran out: then the issuer has finished `tiles` tiles.  What is
// not the first look is out of line, so that it costs the loops no registers.
__device__ __forceinline__ bool wait_for(bool ok, uint64_t* bar, uint32_t par, Waits* w, int tiles) {
  if (ok) {
    uint32_t done;
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
                 "selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(done) : "r"(su32(bar)), "r"(par) : "memory");
    if (done) return true;
  }
  return wait_long(ok, bar, par, w, tiles);
}

__device__ __forceinline__ bool loaders_all(bool v) {
  uint32_t r;
  asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbar.red.and.pred q, %2, %3, p;\n"
               "selp.u32 %0, 1, 0, q;\n}"
               : "=r"(r) : "r"((uint32_t)v), "n"(kNbQ), "n"(kLoaders) : "memory");
  return r != 0;
}

// byte offset of 16-byte chunk `chunk` of row `row` in an operand tile of
// SW128 atoms of 64 elements
__device__ __forceinline__ int op_off(int row, int chunk) {
  return (chunk >> 3) * 16384 + (row >> 3) * 1024 + (row & 7) * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }
__device__ __forceinline__ uint32_t dq_lo(uint32_t x, __half2 s, __half2 z) {
  const __half2 c = __hsub2(u2h((x & 0x000f000fu) | 0x64006400u), __float2half2_rn(1024.f));
  return h2u(__hfma2(c, s, z));
}
__device__ __forceinline__ uint32_t dq_hi(uint32_t x, __half2 s, __half2 z) {
  const __half2 c = __hfma2(u2h((x & 0x00f000f0u) | 0x64006400u), __float2half2_rn(0.0625f), __float2half2_rn(-64.f));
  return h2u(__hfma2(c, s, z));
}

// one token's packed codes and parameters of K or V
template <int D>
struct Packed {
  uint4 code[D / 32];
  uint32_t par[D / 32];

  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* params) {
    if (codes) {
#pragma unroll
      for (int i = 0; i < D / 32; ++i) code[i] = load_global(reinterpret_cast<const uint4*>(codes) + i);
      if constexpr (D == 128) {
        const uint4 u = load_global(reinterpret_cast<const uint4*>(params));
        par[0] = u.x, par[1] = u.y, par[2] = u.z, par[3] = u.w;
      } else {
        const uint2 u = load_global(reinterpret_cast<const uint2*>(params));
        par[0] = u.x, par[1] = u.y;
      }
    } else {   // a token outside the request: zeros
#pragma unroll
      for (int i = 0; i < D / 32; ++i) code[i] = make_uint4(0, 0, 0, 0), par[i] = 0;
    }
  }
  __device__ __forceinline__ void hide() {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) par[i] = hidden_params(par[i]);
  }
  __device__ __forceinline__ void store(uint8_t* tile, int row) const {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const __half2 z = __low2half2(u2h(par[i])), s = __high2half2(u2h(par[i]));
      const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4*>(tile + op_off(row, 4 * i + j)) =
            make_uint4(dq_lo(w[j], s, z), dq_hi(w[j], s, z), dq_lo(w[j] >> 8, s, z), dq_hi(w[j] >> 8, s, z));
    }
  }
};

// keys key0 ... of a tile in v: those from hi on become -inf (P = 0)
template <int N>
__device__ __forceinline__ void hide_keys(uint32_t* v, int key0, int hi) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = key0 + k < hi ? v[k] : 0xff800000u;
}

// P of the 16 Q keys key0 ... of a tile held in v (float16 pairs into TMEM
// columns key0 / 2 ...).  Returns the sum.
template <int Q>
__device__ __forceinline__ float exp_keys(const uint32_t* v, int key0, float2 c2, float2 mv, uint32_t taddr) {
  float2 ps = make_float2(0.f, 0.f);
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    uint32_t pk[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int k0 = 16 * q + 2 * k;
      const float2 arg = __ffma2_rn(make_float2(__uint_as_float(v[k0]), __uint_as_float(v[k0 + 1])), c2, mv);
      const float2 pp = make_float2(ex2(arg.x), ex2(arg.y));
      ps = __fadd2_rn(ps, pp);
      pk[k] = h2u(__floats2half2_rn(pp.x, pp.y));
    }
    tmem_st8(taddr + key0 / 2 + 8 * q, pk);
  }
  return ps.x + ps.y;
}

__device__ __forceinline__ float max64(const uint32_t* v) {
  float a = -INFINITY, b = -INFINITY;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    a = max3f(a, __uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]));
    b = max3f(b, __uint_as_float(v[4 * k + 2]), __uint_as_float(v[4 * k + 3]));
  }
  return fmaxf(a, b);
}

// The row's logits of tokens below `lo` of the tile, and of those whose bit in
// `bad` is set, become -inf in place.  Rare and out of line: it must not cost
// the tile loop its registers.
__device__ __noinline__ void mend_logits(uint32_t sbase, const uint32_t* bad, int lo) {
#pragma unroll 1
  for (int cb = 0; cb < 8; ++cb) {
    const int below = min(max(lo - 16 * cb, 0), 16);
    const uint32_t bits = (bad[cb >> 1] >> (16 * (cb & 1))) | ((1u << below) - 1);
    uint32_t x[16];
    tmem_ld16(sbase + 16 * cb, x);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (bits >> k & 1) x[k] = 0xff800000u;
    tmem_st16(sbase + 16 * cb, x);
  }
  tmem_wait_st();
}

template <int D>
__global__ void __launch_bounds__(kNt, 1) paged_attend_tc_kernel(const AttendArgs a) {
  using L = Lay<D>;
  using W = Walker<kRows, kTk, kItem>;
  extern __shared__ uint8_t sm_raw[];
  uint8_t* sm = sm_raw + ((1024 - (su32(sm_raw) & 1023)) & 1023);
  __shared__ __align__(8) uint64_t bars[11];
  __shared__ uint32_t tmem_base_sh;
  __shared__ Waits waits;
  __shared__ volatile int late_sh;       // the last wait for the tensor pipe ran out
  // tokens of a tile on a page out of range, a word for each producer warp.
  // Four tiles deep: a slot is written again after S(u + 2) is complete, which
  // every softmax thread's P(u + 1) precedes
  __shared__ __align__(16) uint32_t bad_sh[4][4];
  uint64_t* s_done = &bars[0];    // [2] S_g complete
  uint64_t* pv_done = &bars[2];   // [2] O_g of the item complete
  uint64_t* k_free = &bars[4];    // [2] K stage read by both query tiles
  uint64_t* v_free = &bars[6];    // [2]
  uint64_t* q_ready = &bars[8];   // Q_a and Q_b of the item written
  uint64_t* q_free = &bars[9];    // all S of the item complete
  uint64_t* drained = &bars[10];  // nothing left in the tensor pipe
  // what the softmax needs of an item besides its logits, two items deep (a
  // slot is written again when all S of the item in between are complete)
  __shared__ uint8_t row_exp_sh[2][kRows];   // Q was scaled by 2^(127 - this)
  __shared__ uint32_t bad_item_sh[2];        // some page of the item is out of range
  const int tid = threadIdx.x, warp = tid >> 5, w = blockIdx.x;
  wait_for_kernel_ahead();

  if (tid == 0) {
    waits.abort = waits.finished = late_sh = 0;
    waits.status = a.timeout;
    waits.limit = a.wait_cycles;
    for (int i = 0; i < 8; ++i) bar_init(&bars[i], 1);
    bar_init(q_ready, kLoaders);
    bar_init(q_free, 1);
    bar_init(drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    a.join[w].last = -1;
  }
  const Share sh = find_share<kRows, kTk, kItem, kNt>(a, w, (int)gridDim.x);   // has block barriers
  if (sh.n == 0) return;
  if (warp == kMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(su32(&tmem_base_sh)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_base_sh;
  W it;
  it.start(a, sh.b, sh.skip, sh.per, sh.n);

  if (warp < kProd) {
    // ------------------------------------------------------------ softmax
    const int g = warp >> 2, i = tid & 127, lane = tid & 31;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t sbase = tmem + lane_base + 128u * g, obase = tmem + lane_base + kColO + 128u * g;
    uint8_t* stage = sm + L::stage + warp * 4096;
    int u = 0, slot_in = 0;
    while (true) {
      int top = it.hi, bottom = it.lo, top_min = it.hi, bottom_max = it.lo;
      if (a.causal) {
        const int at = it.rq.n - it.rq.n_new, pos = at + div_group(a, it.rt * kRows + 128 * g + i);
        top = min(it.hi, pos + 1);
        top_min = min(it.hi, at + div_group(a, it.rt * kRows + 128 * g) + 1);
        if (a.window > 0) {
          bottom = max(it.lo, pos - a.window + 1);
          bottom_max = max(it.lo, at + div_group(a, it.rt * kRows + min(it.rows, 128 * g + 128) - 1) - a.window + 1);
        }
      }
      // tiles that start below mend_until hold tokens that a row must not see
      // left of its window, or (any tile of the item) on a page out of range
      int mend_until = bottom_max;
      float c2 = 0.f;
      float m_run = kNone, l_run = 0.f;
      for (int t = it.from; t < it.to; ++t, ++u) {
        const int n0 = t * kTk, hi = top - n0;
        const bool full = n0 + kTk <= top_min;
        // one warp of the group polls the mbarrier, the others wait for it.  When a
        // wait had run out before, this one may have read a stale parity: it
        // follows the issuer too.
        auto arrived = [&]() {
          const int gone = waits.abort;
          wait_for(true, &s_done[g], u & 1, &waits, u);
          if (gone) follow(&waits, u);
          return true;
        };
        group_meet(g, (warp & 3) != 0 || arrived());
        fence_after();
        if (t == it.from) {
          c2 = row_factor(a, row_exp_sh[slot_in][128 * g + i]);
          if (bad_item_sh[slot_in]) mend_until = 0x7fffffff;
          slot_in ^= 1;
        }
        if (n0 < mend_until) mend_logits(sbase, bad_sh[u & 3], bottom - n0);
        uint32_t v[64];
        tmem_ld64(sbase + 64, v);
        tmem_wait_ld();
        if (!full) hide_keys<64>(v, 64, hi);
        float mx = max64(v);
        tmem_ld64(sbase, v);
        tmem_wait_ld();
        if (!full) hide_keys<64>(v, 0, hi);
        mx = fmaxf(mx, max64(v));
        const float mnew = mx * c2 - kBelow;
        const bool need = mnew > m_run + kGrow;
        // S_g(t) follows PV_g(t-1) in the tensor pipe's order, so O_g is complete
        if (t > it.from && __any_sync(0xffffffffu, need)) {
          const float corr = need ? ex2(m_run - mnew) : 1.f;
#pragma unroll 1
          for (int cb = 0; cb < D / 16; ++cb) {
            uint32_t o[16];
            tmem_ld16(obase + 16 * cb, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * corr);
            tmem_st16(obase + 16 * cb, o);
          }
          l_run *= corr;
        }
        if (need) m_run = mnew;
        const float2 c2v = make_float2(c2, c2), mv = make_float2(-m_run, -m_run);
        float ps = exp_keys<4>(v, 0, c2v, mv, sbase);
        tmem_wait_st();
        fence_before();
        nb_arrive(kNbP1 + g);
#pragma unroll 1
        for (int hq = 0; hq < 2; ++hq) {
          uint32_t x[32];
          tmem_ld32(sbase + 64 + 32 * hq, x);
          tmem_wait_ld();
          if (!full) hide_keys<32>(x, 64 + 32 * hq, hi);
          ps += exp_keys<2>(x, 64 + 32 * hq, c2v, mv, sbase);
          if (hq == 0) {
            tmem_wait_st();
            fence_before();
            nb_arrive(kNbP2 + g);
          }
        }
        tmem_wait_st();
        l_run += ps;
        fence_before();
        nb_arrive(kNbP3 + g);
      }
      // what the item's end needs
      const bool all = it.begins() && it.ends();
      const int slot = it.begins() ? 1 : 0, rows = it.rows - 128 * g, y0 = it.rt * kRows + 128 * g;
      const int64_t q_row0 = it.rq.row0;
      const int head0 = it.h * a.group;
      if (tid == 0 && it.begins() && !it.ends()) record_join(a, w, it, last_worker(sh, it.end_of(sh.first)), kRows);
      const bool more = it.next(a);
      // O is lost when any wait of the CTA has run out by now (waits.abort below)
      if ((warp & 3) == 0) wait_for(true, &pv_done[g], slot_in ^ 1, &waits, 0);
      group_sync(g);
      fence_after();
      l_run = waits.abort == 0 ? near_sum(m_run, l_run, kNone) : __int_as_float(0x7fffffff);
      // ---- O of the item by way of shared memory, 128 bytes a row at a time,
      // so that a row is stored by neighbouring lanes.  Column p of 8 holds
      // channel (p / 2) + 4 (p % 2).
      const float inv = inverse_sum(l_run);
      const int per = all ? 64 : 32;   // channels of a round: bf16 rows, or float32 parts
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += per) {
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          if (all) {
            uint32_t x[16];
            tmem_ld16(obase + c0 + 16 * q, x);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t o[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                // channels 2 k, 2 k + 1 are in columns 2 (2 k % 4) + (k > 1), + 2
                const int c = 8 * e + 2 * ((2 * k) & 3) + (k >> 1);
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(x[c]) * inv, __uint_as_float(x[c + 2]) * inv);
                o[k] = *reinterpret_cast<const uint32_t*>(&b2);
              }
              *reinterpret_cast<uint4*>(stage + lane * 128 + (((2 * q + e) ^ (lane & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
            }
          } else {
            uint32_t x[8];
            tmem_ld8(obase + c0 + 8 * q, x);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 2; ++e)
              *reinterpret_cast<uint4*>(stage + lane * 128 + (((2 * q + e) ^ (lane & 7)) << 4)) =
                  make_uint4(x[e], x[e + 2], x[e + 4], x[e + 6]);
          }
        }
        __syncwarp();
        uint4 piece[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int y = 4 * k + (lane >> 3);
          piece[k] = *reinterpret_cast<const uint4*>(stage + y * 128 + (((lane & 7) ^ (y & 7)) << 4));
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = 32 * (warp & 3) + 4 * k + (lane >> 3);
          if (r < rows) {
            const uint4 x = piece[k];
            if (all) {
              const int tok = div_group(a, y0 + r);
              *reinterpret_cast<uint4*>((__nv_bfloat16*)a.out + (q_row0 + tok) * a.o_row +
                                        (int64_t)(head0 + y0 + r - tok * a.group) * a.o_head + c0 + 8 * (lane & 7)) = x;
            } else {
              *reinterpret_cast<uint4*>(part_row(a, w, slot, kRows, 128 * g + r, D) + c0 + 4 * (lane & 7)) = x;
            }
          }
        }
        __syncwarp();
      }
      if (i < rows) {
        if (!all) {
          float* part = part_row(a, w, slot, kRows, 128 * g + i, D);
          part[D] = m_run, part[D + 1] = l_run;
        } else if (a.lse) {
          const int tok = div_group(a, y0 + i);
          a.lse[(q_row0 + tok) * a.heads + head0 + y0 + i - tok * a.group] = log_sum(m_run, l_run);
        }
      }
      fence_before();   // the reads of O come before the next item's MMAs
      if (!more) break;
    }
  } else if (warp < kMma) {
    // ------------------------------------------------------------ producers
    const int p = tid - kProd * 32;
    constexpr int G = D / 32;
    Packed<D> kp, vp;
    int t = it.from;        // the tile whose page id is in flight
    int pg = -1, n = 0, h = 0;
    bool in = false, more = true;
    // the page id of this thread's token of tile t of the current item
    auto lookup = [&]() {
      n = t * kTk + p;
      h = it.h;
      in = n >= it.lo && n < it.hi;
      pg = in ? load_global(a.table + (int64_t)it.b * a.max_blocks + (n >> a.page_shift)) : -1;
    };
    auto advance = [&]() {
      if (++t < it.to) return true;
      if (!it.next(a)) return false;
      t = it.from;
      return true;
    };
    const uint8_t* blk = nullptr;
    int s = 0;
    uint32_t bad = 0;
    auto resolve = [&]() {
      const bool good = in && pg >= 0 && pg < a.n_pages;
      if (in && !good) flag(a.status, QWM_DEV_BOUNDS);
      bad = __ballot_sync(0xffffffffu, in && !good);
      s = n & (a.page - 1);
      blk = good ? a.pool + ((int64_t)pg * a.kv_heads + h) * a.block : nullptr;
    };
    auto load = [&](Packed<D>& x, int half) {
      const uint8_t* b = blk ? blk + half * (a.block / 2) : nullptr;
      x.load(b ? b + s * (D / 2) : nullptr, b ? b + a.page * (D / 2) + s * (G * 4) : nullptr);
    };
    lookup();
    resolve();
    load(kp, 0);
    load(vp, 1);
    more = advance();
    if (more) lookup();
    bool ok = true;         // no wait of this thread has run out
    // the stage of tile u was read by tile u - 2
    auto wait_free = [&](uint64_t* bar, uint32_t par, int u) {
      ok = wait_for(ok, bar, par, &waits, u - 1);
    };
    for (int u = 0;; ++u) {
      const int st = u & 1;
      const uint32_t par = (uint32_t)(((u >> 1) - 1) & 1);
      const bool have = more;
      if (u >= 2) wait_free(&k_free[st], par, u);
      kp.store(sm + L::k + st * L::op, p);
      if ((p & 31) == 0) bad_sh[u & 3][p >> 5] = bad;
      fence_async_smem();
      nb_arrive(kNbK + st);
      if (have) {
        resolve();
        load(kp, 0);
      }
      if (u >= 2) wait_free(&v_free[st], par, u);
      if (a.causal) vp.hide();   // in every tile: to tell those with hidden tokens apart is no faster
      vp.store(sm + L::v + st * L::op, p);
      fence_async_smem();
      nb_arrive(kNbV + st);
      if (!have) break;
      load(vp, 1);
      more = advance();
      if (more) lookup();
    }
  } else if (warp == kMma) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t q0 = su32(sm), k0 = su32(sm + L::k), v0 = su32(sm + L::v);
    int u = 0;
    uint32_t q_par = 0;
    bool ok = true;
    auto issue_s = [&](int g, int st, bool last) {
      if (elect_one()) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const uint32_t ko = (j >> 2) * 16384 + (j & 3) * 32;
          mma_ss(tmem + 128u * g, desc_sw128(q0 + g * L::op + ko), desc_sw128(k0 + st * L::op + ko), kIdescS, j > 0);
        }
        commit(&s_done[g]);
        if (g == 1) commit(&k_free[st]);
        if (g == 1 && last) commit(q_free);
      }
      __syncwarp();
    };
    auto issue_pv = [&](int g, int st, int j0, int j1, bool first) {
      if (elect_one()) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j >= j0 && j < j1)
            mma_ts(tmem + kColO + 128u * g, tmem + 128u * g + 8 * j, desc_sw128_mn(v0 + st * L::op + 2048 * j), L::idesc_pv,
                   (first && j == 0) ? 0u : 1u);
      }
      __syncwarp();
    };
    do {
      nb_sync(kNbK + (u & 1));
      ok = warp_all(bar_wait(q_ready, q_par, &waits.abort, a.timeout, a.wait_cycles)) && ok;
      q_par ^= 1;
      fence_after();
      if (ok) {
        issue_s(0, u & 1, false);
        issue_s(1, u & 1, it.from + 1 == it.to);
      }
      for (int t = it.from; t < it.to; ++t, ++u) {
        const int st = u & 1;
        const bool last = t + 1 == it.to;
        ok = ok && !__any_sync(0xffffffffu, waits.abort != 0);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          nb_sync(kNbP1 + g);
          if (g == 0) nb_sync(kNbV + st);
          fence_after();
          if (ok) issue_pv(g, st, 0, 4, t == it.from);
          nb_sync(kNbP2 + g);
          fence_after();
          if (ok) issue_pv(g, st, 4, 6, false);
          nb_sync(kNbP3 + g);
          fence_after();
          if (ok) {
            issue_pv(g, st, 6, 8, false);
            if (elect_one()) {
              if (last) commit(&pv_done[g]);
              if (g == 1) commit(&v_free[st]);
            }
            __syncwarp();
          }
          if (!last) {
            if (g == 0) {
              nb_sync(kNbK + (st ^ 1));
              fence_after();
            }
            if (ok) issue_s(g, st ^ 1, t + 2 == it.to);
          }
        }
        if ((tid & 31) == 0) waits.finished = u + 1;
      }
    } while (it.next(a));
    // after a wait that ran out MMAs may still be on their way
    if (elect_one()) commit(drained);
    __syncwarp();
    bar_wait(drained, 0, &late_sh, a.timeout);
  } else {
    // ------------------------------------------------------------ query loaders
    // The queries of an item to float16 in the order (0, 4), (1, 5), (2, 6),
    // (3, 7) into the Q tiles, CH lanes a row, rows behind the item's zero, as
    // soon as all S of the item before are complete.  All rows are scaled by
    // 2^6, which suits entries below 2^9; if one is larger, or the largest of 8
    // neighbours (other than zeros) below 2^-8, the rows are read again and each
    // scaled by the power of two that suits it (row_exponent).  So an entry loses
    // bits only below 2^-23, and no more than 2^-31: 2^-23 of the largest of its
    // neighbours.  The softmax is told the rows' scales.  Also: whether any
    // page of the item is out of range.
    constexpr int CH = D / 8, STEP = kLoaders / CH;
    const int p = tid - kLoad * 32, cl = p % CH;
    int slot_out = 0;
    uint32_t free_par = 0;
    bool more = true, first = true, ok = true;
    while (more) {
      auto row_of = [&](int y) {
        const int x = it.rt * kRows + y, tok = div_group(a, x);
        return (const __nv_bfloat16*)a.q + (int64_t)(it.rq.row0 + tok) * a.q_row + (int64_t)(it.h * a.group + x - tok * a.group) * a.q_head;
      };
      auto place = [&](int y) { return sm + (y >> 7) * L::op + op_off(y & 127, cl); };
      bool good = true;
      const int last = (min(it.hi, it.to * kTk) - 1) >> a.page_shift;
#pragma unroll 1
      for (int x = (max(it.lo, it.from * kTk) >> a.page_shift) + p; x <= last; x += kLoaders) {
        const int id = load_global(a.table + (int64_t)it.b * a.max_blocks + x);
        good = good && id >= 0 && id < a.n_pages;
      }
      // on their way to L2 before the tiles are free
#pragma unroll 1
      for (int y = p >> 1; y < it.rows; y += kLoaders / 2)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(row_of(y) + (D / 2) * (p & 1)));
      if (!first) {
        ok = wait_for(ok, q_free, free_par, &waits, 0);
        free_par ^= 1;
      }
      first = false;
      for (int y = p; y < kRows; y += kLoaders) row_exp_sh[slot_out][y] = 127 - kUp;
#pragma unroll 2
      for (int y = p / CH; y < kRows; y += STEP) {
        const bool live = y < it.rows;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(su32(place(y))),
                     "l"(live ? row_of(y) + 8 * cl : (const __nv_bfloat16*)a.q), "r"(live ? 16 : 0) : "memory");
      }
      cp_async_wait_all();
      // a thread converts the pieces it has copied
      auto store = [&](int y, float2 x0, float2 x1, float2 x2, float2 x3) {
        *reinterpret_cast<uint4*>(place(y)) = make_uint4(h2u(__floats2half2_rn(x0.x, x2.x)), h2u(__floats2half2_rn(x0.y, x2.y)),
                                                         h2u(__floats2half2_rn(x1.x, x3.x)), h2u(__floats2half2_rn(x1.y, x3.y)));
      };
      auto pair = [](uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); };
      auto largest = [](uint4 x) {   // the bits of the largest magnitude
        uint32_t m;   // a NaN wins
        asm("{\n.reg .b32 s, t;\nmax.NaN.xorsign.abs.bf16x2 s, %1, %2;\nmax.NaN.xorsign.abs.bf16x2 t, %3, %4;\n"
            "max.NaN.xorsign.abs.bf16x2 s, s, t;\nand.b32 %0, s, 0x7fff7fff;\n}"
            : "=r"(m) : "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w));
        return max(m & 0xffffu, m >> 16);
      };
      const __nv_bfloat162 up2 = __float2bfloat162_rn((float)(1 << kUp));
      auto up = [&](uint32_t w) {
        const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), up2);
        return pair(*reinterpret_cast<const uint32_t*>(&x));
      };
      uint32_t high = 0, low = 0xffffffffu;
#pragma unroll 4
      for (int y = p / CH; y < kRows; y += STEP) {
        const uint4 x = *reinterpret_cast<const uint4*>(place(y));
        store(y, up(x.x), up(x.y), up(x.z), up(x.w));
        const uint32_t m = largest(x);
        high = max(high, m), low = min(low, m - 1);   // zeros are no limit
      }
      const bool all_fit = loaders_all(high < kFitHigh && low >= kFitLow - 1), all_good = loaders_all(good);
      if (!all_fit) {
        // CH lanes share a row; the rows of a step need not divide 256
#pragma unroll 1
        for (int y0 = 0; y0 < kRows; y0 += STEP) {
          const int y = y0 + p / CH;
          const bool live = y < it.rows;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (live) v = *reinterpret_cast<const uint4*>(row_of(y) + 8 * cl);
          uint32_t m = largest(v);
#pragma unroll
          for (int o = CH / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          const int e = row_exponent((int)(m >> 7) - 127);
          if (live) {
            const float qs = __uint_as_float((uint32_t)(127 - e) << 23);
            auto by = [&](uint32_t w) {
              const float2 x = pair(w);
              return make_float2(x.x * qs, x.y * qs);
            };
            store(y, by(v.x), by(v.y), by(v.z), by(v.w));
            if (cl == 0) row_exp_sh[slot_out][y] = (uint8_t)(127 + e);
          }
        }
      }
      if (p == 0) bad_item_sh[slot_out] = !all_good;
      slot_out ^= 1;
      fence_async_smem();
      bar_arrive(q_ready);
      more = it.next(a);
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kMma) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

template <int D>
cudaError_t launch_tc(const AttendArgs& a, int workers, cudaStream_t st) {
  static SmemLimit limit;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)workers, 1, 1);
  cfg.blockDim = dim3(kNt, 1, 1);
  cfg.dynamicSmemBytes = Lay<D>::bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {early_launch()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return launch_smem(limit, cfg.dynamicSmemBytes, paged_attend_tc_kernel<D>, cfg, a);
}

}  // namespace

Workers tc_workers() { return Workers{sm_count(), kRows}; }

cudaError_t launch_attend_tc(const AttendArgs& a, int d, int64_t max_rows, cudaStream_t st) {
  const Workers w = tc_workers();
  const cudaError_t e = d == 64 ? launch_tc<64>(a, w.count, st) : launch_tc<128>(a, w.count, st);
  return e != cudaSuccess ? e : launch_attend_join(a, d, true, w, max_rows, st);
}

}  // namespace paged
}  // namespace qwm
