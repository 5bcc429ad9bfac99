// qwm_paged_attend for few rows (kernel 2, bf16): single-token steps and short
// drafts, where the pages are read once and everything else must keep up.
//
//   s_n = q . k_hat_n;  O = sum_n exp2(s_n - m) v_hat_n, running maximum m
//
// A worker (a CTA of four warps) walks the tiles of 128 tokens that the
// partition deals to it; a warp takes 32 tokens of each, with its own running
// maximum, and the warps meet at the end of an item only.  Every warp copies
// its own packed bytes (2.5 KB a block of 16 tokens at d = 128, five 16-byte
// asynchronous copies a lane) into its own ring of shared memory, so that no
// barrier stands between the copies and the arithmetic; the page ids of 32
// tiles are loaded at once, a step before the first is needed.  (Measured on
// the ragged batch of 48 requests: one producer warp a CTA with bulk copies
// 155 us, where a thread issues one copy at a time and pages of 16 tokens make
// 16 a tile; loads to registers two blocks ahead 143 us, too few bytes in
// flight; this with 16 tokens a step 118 us, with 32 103 us: half the control
// and address instructions, two independent chains of MMAs.)
//
// Both products are formed transposed with mma.m16n8k16 (float16 in, float32
// out), the 16 tokens or channels on the long side and the 8 query rows on the
// short one:
//   S^T[16 tokens][8 rows]  = K_hat[16][d] Q^T      d/16 MMAs
//   O^T[d][8 rows]         += V_hat^T[d][16] P^T    d/16 MMAs
// so that a step of 5 or 8 query heads a key/value head does not pay for 16
// rows.  Channels are contracted in the order in which the codes lie in
// memory, and Q is laid out to match.  P^T is S^T transposed in 8 x 8 blocks
// (movmatrix).  A code c becomes float16 by one mask that puts it into the
// mantissa of 1024 (1024 + c, or 1024 + 16 c for the upper nibble of a byte),
// one exact subtraction (or fused multiply by 1/16), and c scale + zero by one
// fused multiply-add: the only rounding of k_hat and v_hat.  Q is float16 scaled
// per row by a power of two, up or down (row_exponent).  The rows' sums and O are
// float32; O is rescaled only when a row's maximum grows by more than 2^8 (P <= 2^15).
// Tokens outside a request (or on a page out of range) have their logits
// replaced and their value parameters zeroed, so garbage bytes do no harm.
//
// Bound by the latency of chains: the ~26 instructions a token and warp, half of
// them the codes' way to float16, lie behind one another (copy, conversion, MMA,
// softmax, MMA), and 12 warps an SM fill neither the issue slots (61%) nor HBM
// (4.6 TB/s, 68% of a copy) with them: that batch (8 K tokens on average, 32
// query heads over 8, d = 128, pages of 16) takes 103 us, the same copies without
// arithmetic 84; 40% fewer float16 instructions in the conversions were no faster.
// One request of 98,280 tokens (40 heads over 8) takes 35 us, 8 to 10 of them
// the start, the first ids and copies, and the join.
//
// 8 bits (E4m3): codes become float16 by a conversion of two, exact; K's scale of 16
// tokens is behind the product, one multiply a logit, V's in the operand.  Half the
// instructions a byte, so the pages' way from HBM is the bound: that batch takes 143
// us (5.9 TB/s in all; reads of blocks of 4,112 bytes in random order reach 6.1 TB/s
// with 64 KB in flight an SM and 6.5 to 6.7 with 128), that request 42.
//
// float32 (8 bits alone, whose keys and values float16 holds): q and P as two
// float16 terms each, so two MMAs for one, and a step's 16 tokens of O summed apart.
// Three windowed requests (30 to 260 rows, 8 heads over 4, d = 64) 25 us, on the CUDA
// cores 48; 2,048 rows over 10,240 tokens 412 us (d = 128: 820), 1,206 (2,293) there.
#include "paged_internal.cuh"
#include "tcgen05_util.cuh"

namespace qwm {
namespace paged {
namespace {

using namespace tcx;

constexpr int kCw = 4, kNt = kCw * 32, kItem = 2;
// CTAs an SM (of 8 rows), a warp's stages, the blocks of 16 tokens in one, and the
// bits of a note on each
template <class F>
struct Plan;
template <>
struct Plan<Int4> {
  static constexpr int kCtas = 3, kStages = 2, kSub = 2, kNote = 1, kTk = 16 * kSub * kCw;
};
template <>
struct Plan<E4m3> {
  static constexpr int kCtas = 3, kStages = 2, kSub = 1, kNote = 4, kTk = 16 * kSub * kCw;
};
constexpr float kNone = -3.0e38f;   // running maximum of a row that has seen nothing
// Where a row's maximum is x0 when it is taken, m = x0 - 7, and it is taken again
// when a logit passes x0 + 8: P <= 2^15 stays inside float16, and a token of a
// long cache is lost only below 2^-25 / 2^7 of the largest weight
constexpr float kBelow = 7.f, kGrow = 8.f;

__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same from a zero sum
__device__ __forceinline__ void mma0(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }

// Two values as float16 pairs, each: one, or in float32 two that add up to them but
// for 2^-22 of either (22 of 24 bits).
template <int TERMS, class Put>
__device__ __forceinline__ void split(float x, float y, Put put) {
  const __half2 h = __floats2half2_rn(x, y);
  put(0, h2u(h));
  if constexpr (TERMS == 2) {
    const float2 f = __half22float2(h);
    put(1, h2u(__floats2half2_rn(x - f.x, y - f.y)));
  }
}

// c scale + zero for the lower (upper) nibbles of bytes 0 and 2 of x.  `magic`
// (1024 twice in float16) comes from the call's arguments: with a mask and a
// register one instruction puts the codes into place, with two constants known
// to the compiler it takes two.
__device__ __forceinline__ uint32_t dq_lo(uint32_t x, __half2 s, __half2 z, uint32_t magic) {
  const __half2 c = __hsub2(u2h((x & 0x000f000fu) | magic), __float2half2_rn(1024.f));
  return h2u(__hfma2(c, s, z));
}
__device__ __forceinline__ uint32_t dq_hi(uint32_t x, __half2 s, __half2 z, uint32_t magic) {
  const __half2 c = __hfma2(u2h((x & 0x00f000f0u) | magic), __float2half2_rn(0.0625f), __float2half2_rn(-64.f));
  return h2u(__hfma2(c, s, z));
}
// the token of a block of 8 that column (or row) n of a fragment holds: the
// lanes of a load phase then meet even and odd rows of codes
__device__ __forceinline__ int token_of(int n) { return (n & 1) ? 4 + ((n >> 1) ^ 1) : n >> 1; }

// 16 tokens of one head as they lie in a ring stage
template <int D, class F>
struct Stage;
template <int D>
struct Stage<D, Int4> {
  static constexpr int G = D / 32;
  static constexpr int kcode = 0, kpar = 8 * D, vcode = kpar + 64 * G, vpar = vcode + 8 * D, bytes = vpar + 64 * G;
  static constexpr int copies = (bytes / 16 + 31) / 32;   // of 16 bytes, a lane

  // Where a lane's copies come from: byte cst + mul x (first token's slot) of
  // the page's block, for 16-byte piece 32 k + lane of the stage.
  struct Source {
    int cst[copies], mul[copies];
    __device__ __forceinline__ void init(int page, int block, int lane) {
      const int half = block / 2;
#pragma unroll
      for (int k = 0; k < copies; ++k) {
        const int o = 16 * (32 * k + lane);
        const bool value = o >= vcode;
        const int x = value ? o - vcode : o;
        const bool code = x < kpar;
        cst[k] = (code ? x : page * (D / 2) + x - kpar) + (value ? half : 0);
        mul[k] = code ? D / 2 : 4 * G;
      }
    }
  };
  __device__ __forceinline__ static void copy(uint32_t stage, const uint8_t* blk, int at, const Source& src, int lane) {
#pragma unroll
    for (int k = 0; k < copies; ++k)
      if (32 * k + 32 <= bytes / 16 || 32 * k + lane < bytes / 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(stage + 512 * k),
                     "l"(blk + (uint32_t)(src.cst[k] + at * src.mul[k])) : "memory");
  }
};

// 8 bits: K and V lie as in memory, line for line of 128 bytes: a block starts on 16
// bytes, so its first piece is at 16 `off` in the first line, and the last `off`
// pieces lie ahead of it.  The pieces of a line are swapped so that neither the
// loads of keys (8 lanes: half of two rows of opposite parity) nor those of values
// (two pieces of four rows that follow one another) meet in a bank.  Swapped row by
// row instead, over the lines, a copy falls into twice the requests to L2: one
// request of 98,280 tokens 47.9 us, the ragged batch 164, with these 42.6 and 142.
template <int D>
struct Stage<D, E4m3> {
  static constexpr int vcode = 16 * D, scale = 32 * D, bytes = 32 * D + 16;
  // where place s of K or V lies
  __device__ __forceinline__ static int k_place(int s) { return (D == 128 ? s ^ (s >> 3 & 1) : s) << 4; }
  __device__ __forceinline__ static int v_place(int s) { return (D == 128 ? s ^ (s >> 2 & 6) : s ^ (s >> 2 & 2)) << 4; }
  // where piece x of row `row` of the first 8 lies; row + 8 is half the places on
  __device__ __forceinline__ static int place(int row, int x, uint32_t off) { return (row * (D / 16) + x + (int)off) & (D - 1); }
  static constexpr int kRow8 = 8 * D;   // to be xored
  struct Source {
    int values, scales;
    __device__ __forceinline__ void init(int page, int, int) { values = page * D, scales = 2 * page * D; }
  };
  __device__ __forceinline__ static uint32_t offset(const uint8_t* blk) { return (uint32_t)((uintptr_t)blk >> 4) & 7; }
  __device__ __forceinline__ static void copy(uint32_t stage, const uint8_t* blk, int at, const Source& src, int lane) {
    const int piece = lane - (int)offset(blk), wrap = piece < 0 ? 16 * D : 0;
    const uint8_t* kb = blk + (at * D + 16 * piece);
    const uint8_t* vb = kb + src.values;
    const uint32_t kd = stage + k_place(lane), vd = stage + vcode + v_place(lane);   // four lines on, the swaps are the same
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int o = i ? 512 * i : wrap;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(kd + 512 * i), "l"(kb + o) : "memory");
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(vd + 512 * i), "l"(vb + o) : "memory");
    }
    if (lane == 0)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(stage + scale), "l"(blk + (src.scales + at / 4)) : "memory");
  }
};

// The blocks of one warp, in order, ahead of the arithmetic.  Its walker is in
// shared memory: registers hold only what every block needs.
template <int D, class F, class W>
struct Ahead {
  using St = Stage<D, F>;
  static constexpr int kSub = Plan<F>::kSub, kTk = Plan<F>::kTk, kNote = Plan<F>::kNote;
  W* walker;
  int t, to, base;       // next tile; end of the item's; first tile of the ids
  int lo, hi, ids[kSub];
  const int32_t* row;
  const uint8_t* head;   // pool + the head's offset in a page
  uint32_t page_bytes;   // of all heads
  typename St::Source src;
  bool more;

  __device__ __forceinline__ void fetch_ids(const AttendArgs& a, int warp, int lane) {
    base = t;
#pragma unroll
    for (int x = 0; x < kSub; ++x) {
      const int n = (t + lane) * kTk + 16 * (kSub * warp + x);
      const bool in = t + lane < to && n < hi && n + 16 > lo;
      ids[x] = in ? load_global(row + (n >> a.page_shift)) : -2;
      if (in && (ids[x] < 0 || ids[x] >= a.n_pages)) {
        flag(a.status, QWM_DEV_BOUNDS);
        ids[x] = -2;
      }
    }
  }
  __device__ __forceinline__ void open(const AttendArgs& a, const W& w, int warp, int lane) {
    t = w.from, to = w.to, lo = w.lo, hi = w.hi;
    row = table_of<F>(a, w.b, w.h);
    head = a.pool + (int64_t)w.h * a.block;
    fetch_ids(a, warp, lane);
  }
  // Copies the next block into a stage (one commit group, also when there is
  // nothing to copy); returns a note for each 16 tokens: a bit whether there are
  // any, and with 8 bits their offset.
  __device__ __forceinline__ uint32_t copy(const AttendArgs& a, uint32_t stage, int warp, int lane) {
    uint32_t have = 0;
    if (more) {
#pragma unroll
      for (int x = 0; x < kSub; ++x) {
        const int pg = __shfl_sync(0xffffffffu, ids[x], t - base);
        if (pg >= 0) {
          const uint8_t* blk = head + (uint64_t)(uint32_t)pg * page_bytes;
          if constexpr (F::kBits == 8) have |= (1u | St::offset(blk) << 1) << (kNote * x);
          else have |= 1u << x;
          St::copy(stage + x * St::bytes, blk,
                         (t * kTk + 16 * (kSub * warp + x)) & (a.page - 1), src, lane);
        }
      }
      // on to the next block; its id is on the way before it is asked for
      if (++t == to) {
        W w = *walker;
        more = w.next(a);
        __syncwarp();
        if (more) {
          if (lane == 0) *walker = w;
          open(a, w, warp, lane);
        }
        __syncwarp();
      } else if (t == base + 32) {
        fetch_ids(a, warp, lane);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return have;
  }
};

template <int D, int NB, class F>
struct Smem {
  static constexpr int LD = D + 4;                          // rows 2 c of a store phase 8 banks apart
  static constexpr int merge = kCw * Plan<F>::kStages * Plan<F>::kSub * Stage<D, F>::bytes;   // float [kCw][8 NB][LD]
  static constexpr int stat = merge + kCw * 8 * NB * LD * 4;
  static constexpr int bytes = stat + kCw * 8 * NB * 8;     // float2 (m, l) [kCw][8 NB]
};

template <int D, int NB, class F, class T>
__global__ void __launch_bounds__(kNt, NB == 1 && sizeof(T) == 2 ? Plan<F>::kCtas : 2) paged_attend_mma_kernel(const AttendArgs a) {
  constexpr int TERMS = sizeof(T) == 4 ? 2 : 1;
  static_assert(TERMS == 1 || F::kBits == 8, "float32 needs keys and values that float16 holds");
  constexpr int R = 8 * NB, KW = D / 32, MB = D / 16;
  constexpr int kStages = Plan<F>::kStages, kSub = Plan<F>::kSub, kTk = Plan<F>::kTk, kNote = Plan<F>::kNote;
  constexpr uint32_t kNotes = (1u << kNote * kSub) - 1, kLive = kNotes / ((1u << kNote) - 1);   // of a stage; their first bits
  static_assert(kNote * kSub * kStages < 32, "the notes fit a register");
  using Sm = Smem<D, NB, F>;
  using St = Stage<D, F>;
  using W = Walker<R, kTk, kItem>;
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ W ahead_sh[kCw];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, w = blockIdx.x;
  wait_for_kernel_ahead();
  if (tid == 0) a.join[w].last = -1;
  const Share sh = find_share<R, kTk, kItem, kNt>(a, w, (int)gridDim.x);   // has block barriers
  if (sh.n == 0) return;
  W it;
  it.start(a, sh.b, sh.skip, sh.per, sh.n);
  if (lane == 0) ahead_sh[warp] = it;
  __syncwarp();
  Ahead<D, F, W> ahead;
  ahead.walker = &ahead_sh[warp];
  ahead.more = true;
  ahead.page_bytes = (uint32_t)(a.kv_heads * a.block);
  ahead.src.init(a.page, a.block, lane);
  ahead.open(a, it, warp, lane);
  // the warp's stages; 4 bits: copies of a lane start 16 bytes a lane into one
  const uint8_t* ring = sm + warp * kStages * kSub * St::bytes;
  const uint32_t ring_at = su32(ring) + (F::kBits == 4 ? 16 * lane : 0);
  // the item's queries, sent for ahead of the copies, which they would queue
  // behind (2 to 3 us of a first item)
  uint4 qraw[NB][KW * TERMS];
  auto load_q = [&]() {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int r = nb * 8 + (lane >> 2), rr = it.rt * R + r, tok = div_group(a, rr);
      const uint4* src = reinterpret_cast<const uint4*>((const T*)a.q + (int64_t)(it.rq.row0 + tok) * a.q_row +
                                                       (int64_t)(it.h * a.group + rr - tok * a.group) * a.q_head + (lane & 3) * (D / 4));
#pragma unroll
      for (int i = 0; i < KW * TERMS; ++i) qraw[nb][i] = r < it.rows ? src[i] : make_uint4(0, 0, 0, 0);
    }
  };
  load_q();
  uint32_t have = 0;     // notes for each stage: which 16 tokens there are
  for (int i = 0; i < kStages; ++i) have |= ahead.copy(a, ring_at + i * kSub * St::bytes, warp, lane) << (kNote * kSub * i);
  int st = 0;
  bool more = true;

  const int g = lane >> 2, c = lane & 3;
  const int tok0 = token_of(g), ta = token_of(2 * c), tb = token_of(2 * c + 1);   // this lane's key, its values
  const uint32_t magic = a.magic;
  float* merge = reinterpret_cast<float*>(sm + Sm::merge);
  float2* stat = reinterpret_cast<float2*>(sm + Sm::stat);
  do {
    // Q^T fragments: row g of each block of 8, in the order of the codes
    uint32_t qf[TERMS][NB][MB][2];
    float c2[NB][2];       // logit factor of rows 2 c and 2 c + 1
    int top[NB][2], bottom[NB][2];
    int top_min = it.hi, bottom_max = it.lo;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float x[D / 4];
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < KW * TERMS; ++i) {
        const uint4 u = qraw[nb][i];
        const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (TERMS == 2) {
            x[4 * i + k] = __uint_as_float(v[k]);
          } else {
            x[8 * i + 2 * k] = __uint_as_float(v[k] << 16);
            x[8 * i + 2 * k + 1] = __uint_as_float(v[k] & 0xffff0000u);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < D / 4; i += 2) mx = max3f(mx, fabsf(x[i]), fabsf(x[i + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int ex = (int)((__float_as_uint(mx) >> 23) & 0xffu) - 127;
      const int e = row_exponent(ex);
      const float qs = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        const float* y = x + 8 * i;
        constexpr bool nibbles = F::kBits == 4;   // else the channels follow one another
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float y0 = y[nibbles ? k : 2 * k] * qs, y1 = y[nibbles ? k + 4 : 2 * k + 1] * qs;
          split<TERMS>(y0, y1, [&](int term, uint32_t h) { qf[term][nb][2 * i + (k >> 1)][k & 1] = h; });
        }
      }
      const float f = row_factor(a, 127 + e);
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
      const int n0 = t * kTk + 16 * kSub * warp;                   // the step's first token
      const uint32_t note = (have >> (kNote * kSub * st)) & kNotes, live = note & kLive;
      // every row sees all of them
      const bool whole = live == kLive && n0 + 16 * kSub <= top_min && n0 >= bottom_max;
      const uint8_t* x0 = ring + st * kSub * St::bytes;
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();
      if (live) {
        // ---- S^T
        float s[NB][kSub][4];
#pragma unroll
        for (int e = 0; e < kSub; ++e) {
          const uint8_t* x = x0 + e * St::bytes;
          float s2[NB][4];   // two sums: half the chain of dependent MMAs
          if constexpr (F::kBits == 8) {
            uint32_t kw[2][2 * KW];
#pragma unroll
            for (int i = 0; i < KW / 2; ++i) {
              const int at = St::k_place(St::place(tok0, c * (KW / 2) + i, note >> (kNote * e + 1) & 7));
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                const uint4 u = *reinterpret_cast<const uint4*>(x + (at ^ b * St::kRow8));
                kw[b][4 * i] = u.x, kw[b][4 * i + 1] = u.y, kw[b][4 * i + 2] = u.z, kw[b][4 * i + 3] = u.w;
              }
            }
#pragma unroll
            for (int i = 0; i < 2 * KW; ++i) {
              const uint32_t f[4] = {e4m3_lo(kw[0][i]), e4m3_lo(kw[1][i]), e4m3_hi(kw[0][i]), e4m3_hi(kw[1][i])};
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                float* to = (i & 1) ? s2[nb] : s[nb][e];
                if (i < 2) mma0(to, f, qf[0][nb][i][0], qf[0][nb][i][1]);
                else mma(to, f, qf[0][nb][i][0], qf[0][nb][i][1]);
                if constexpr (TERMS == 2) mma(to, f, qf[1][nb][i][0], qf[1][nb][i][1]);
              }
            }
          } else {
            uint32_t kw[2][KW];
            __half2 ks[2], kz[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const int row = 8 * b + tok0;
              if constexpr (D == 128) {
                const uint4 u = *reinterpret_cast<const uint4*>(x + St::kcode + row * 64 + 16 * c);
                kw[b][0] = u.x, kw[b][1] = u.y, kw[b][2] = u.z, kw[b][3] = u.w;
              } else {
                const uint2 u = *reinterpret_cast<const uint2*>(x + St::kcode + row * 32 + 8 * c);
                kw[b][0] = u.x, kw[b][1] = u.y;
              }
              const __half2 par = *reinterpret_cast<const __half2*>(x + St::kpar + (row * St::G + c * St::G / 4) * 4);
              kz[b] = __low2half2(par);
              ks[b] = __high2half2(par);
            }
#pragma unroll
            for (int i = 0; i < KW; ++i) {
              uint32_t f[4], f2[4];
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                f[b] = dq_lo(kw[b][i], ks[b], kz[b], magic);
                f[2 + b] = dq_hi(kw[b][i], ks[b], kz[b], magic);
                const uint32_t up = kw[b][i] >> 8;
                f2[b] = dq_lo(up, ks[b], kz[b], magic);
                f2[2 + b] = dq_hi(up, ks[b], kz[b], magic);
              }
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                if (i == 0) {
                  mma0(s[nb][e], f, qf[0][nb][0][0], qf[0][nb][0][1]);
                  mma0(s2[nb], f2, qf[0][nb][1][0], qf[0][nb][1][1]);
                } else {
                  mma(s[nb][e], f, qf[0][nb][2 * i][0], qf[0][nb][2 * i][1]);
                  mma(s2[nb], f2, qf[0][nb][2 * i + 1][0], qf[0][nb][2 * i + 1][1]);
                }
              }
            }
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[nb][e][i] += s2[nb][i];
          if constexpr (F::kBits == 8) {   // the block's scale, behind the product
            const float ks = __half2float(*reinterpret_cast<const __half*>(x + St::scale));
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[nb][e][i] *= ks;
          }
        }
        // ---- softmax: s[nb][e][2 b + k] is token 16 e + 8 b + tok0, row 2 c + k
        uint32_t pf[TERMS][NB][kSub][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if (!whole) {
#pragma unroll
            for (int e = 0; e < kSub; ++e)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int n = n0 + 16 * e + 8 * (i >> 1) + tok0;
                if (n < bottom[nb][i & 1] || n >= top[nb][i & 1] || !(live >> (kNote * e) & 1)) s[nb][e][i] = -INFINITY;
              }
          }
          float mx0 = fmaxf(s[nb][0][0], s[nb][0][2]), mx1 = fmaxf(s[nb][0][1], s[nb][0][3]);
#pragma unroll
          for (int e = 1; e < kSub; ++e) {
            mx0 = max3f(mx0, s[nb][e][0], s[nb][e][2]);
            mx1 = max3f(mx1, s[nb][e][1], s[nb][e][3]);
          }
          mx0 = fmaf(mx0, c2[nb][0], -kBelow);
          mx1 = fmaf(mx1, c2[nb][1], -kBelow);
          if (__any_sync(0xffffffffu, mx0 > m[nb][0] + kGrow || mx1 > m[nb][1] + kGrow)) {
            // rare: the rows' maxima over the tokens, and O rescaled
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, d));
              mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, d));
            }
            // a row that does not need it keeps its maximum, so its bits do
            // not depend on its neighbours
            mx0 = mx0 > m[nb][0] + kGrow ? mx0 : m[nb][0];
            mx1 = mx1 > m[nb][1] + kGrow ? mx1 : m[nb][1];
            const float f0 = ex2(m[nb][0] - mx0), f1 = ex2(m[nb][1] - mx1);
            m[nb][0] = mx0, m[nb][1] = mx1;
            l[nb][0] *= f0, l[nb][1] *= f1;
#pragma unroll
            for (int j = 0; j < MB; ++j) {
              o[nb][j][0] *= f0, o[nb][j][1] *= f1;
              o[nb][j][2] *= f0, o[nb][j][3] *= f1;
            }
          }
#pragma unroll
          for (int e = 0; e < kSub; ++e) {
            float p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = ex2(fmaf(s[nb][e][i], c2[nb][i & 1], -m[nb][i & 1]));
            l[nb][0] += p[0] + p[2];
            l[nb][1] += p[1] + p[3];
            split<TERMS>(p[0], p[1], [&](int term, uint32_t h) { pf[term][nb][e][0] = transpose8(h); });
            split<TERMS>(p[2], p[3], [&](int term, uint32_t h) { pf[term][nb][e][1] = transpose8(h); });
          }
        }
        // ---- O^T: tokens ta, tb (columns 2 c, 2 c + 1) of both blocks of 8
#pragma unroll
        for (int e = 0; e < kSub; ++e) {
          const uint8_t* x = x0 + e * St::bytes;
          if constexpr (F::kBits == 8) {
            uint32_t v0[2][D / 32], v1[2][D / 32];
            uint32_t par = *reinterpret_cast<const uint32_t*>(x + St::scale);
            const uint32_t off = note >> (kNote * e + 1) & 7;
            const int at0 = St::v_place(St::place(ta, g * D / 128, off)), at1 = St::v_place(St::place(tb, g * D / 128, off));
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const int r0 = 8 * b + ta, r1 = 8 * b + tb;
              const uint8_t* x0 = x + St::vcode + (at0 ^ b * St::kRow8);
              const uint8_t* x1 = x + St::vcode + (at1 ^ b * St::kRow8);
              if constexpr (D == 128) {
                const uint4 u0 = *reinterpret_cast<const uint4*>(x0);
                const uint4 u1 = *reinterpret_cast<const uint4*>(x1);
                v0[b][0] = u0.x, v0[b][1] = u0.y, v0[b][2] = u0.z, v0[b][3] = u0.w;
                v1[b][0] = u1.x, v1[b][1] = u1.y, v1[b][2] = u1.z, v1[b][3] = u1.w;
              } else {
                const uint2 u0 = *reinterpret_cast<const uint2*>(x0 + 8 * (g & 1));
                const uint2 u1 = *reinterpret_cast<const uint2*>(x1 + 8 * (g & 1));
                v0[b][0] = u0.x, v0[b][1] = u0.y, v1[b][0] = u1.x, v1[b][1] = u1.y;
              }
              if (!whole) {
                // tokens outside the request, on no page, or hidden from some row:
                // their bytes may be anything
                const int y0 = n0 + 16 * e + r0, y1 = n0 + 16 * e + r1;
                const bool got = live >> (kNote * e) & 1, in0 = got && y0 >= it.lo && y0 < it.hi, in1 = got && y1 >= it.lo && y1 < it.hi;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                  v0[b][i] = in0 ? known_codes(v0[b][i]) : 0u;
                  v1[b][i] = in1 ? known_codes(v1[b][i]) : 0u;
                }
              }
            }
            if (!whole) par = known_scales(par);
            const __half2 vs = __high2half2(u2h(par));
            // as below: byte j of the lane's channels is row g of block j, byte MB + j
            // row g + 8
#pragma unroll
            for (int y = 0; y < MB / 2; ++y) {
              uint32_t f[2][4];
#pragma unroll
              for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  const int word = (y >> 1) + MB / 4 * q;
                  const uint32_t v = __byte_perm(v0[b][word], v1[b][word], (y & 1) ? 0x7362 : 0x5140);
                  f[0][2 * b + q] = mul_f16x2(e4m3_lo(v), vs);
                  f[1][2 * b + q] = mul_f16x2(e4m3_hi(v), vs);
                }
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                  if constexpr (TERMS == 2) {
                    // summed up apart: the tensor cores' sums are cut off, these rounded
                    float part[4];
                    mma0(part, f[j], pf[0][nb][e][0], pf[0][nb][e][1]);
                    mma(part, f[j], pf[1][nb][e][0], pf[1][nb][e][1]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[nb][2 * y + j][k] += part[k];
                  } else {
                    mma(o[nb][2 * y + j], f[j], pf[0][nb][e][0], pf[0][nb][e][1]);
                  }
                }
            }
          } else {
            uint32_t v0[2][D / 64], v1[2][D / 64];
            __half2 vz[2], vs[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const int r0 = 8 * b + ta, r1 = 8 * b + tb;
              if constexpr (D == 128) {
                const uint2 u0 = *reinterpret_cast<const uint2*>(x + St::vcode + r0 * 64 + 8 * g);
                const uint2 u1 = *reinterpret_cast<const uint2*>(x + St::vcode + r1 * 64 + 8 * g);
                v0[b][0] = u0.x, v0[b][1] = u0.y, v1[b][0] = u1.x, v1[b][1] = u1.y;
              } else {
                v0[b][0] = *reinterpret_cast<const uint32_t*>(x + St::vcode + r0 * 32 + 4 * g);
                v1[b][0] = *reinterpret_cast<const uint32_t*>(x + St::vcode + r1 * 32 + 4 * g);
              }
              uint32_t p0 = *reinterpret_cast<const uint32_t*>(x + St::vpar + (r0 * St::G + g * St::G / 8) * 4);
              uint32_t p1 = *reinterpret_cast<const uint32_t*>(x + St::vpar + (r1 * St::G + g * St::G / 8) * 4);
              if (!whole) {
                // tokens outside the request, on no page, or hidden from some row:
                // their bytes may be anything
                const int y0 = n0 + 16 * e + r0, y1 = n0 + 16 * e + r1;
                const bool got = live >> (kNote * e) & 1;
                p0 = !got || y0 < it.lo || y0 >= it.hi ? 0u : hidden_params(p0);
                p1 = !got || y1 < it.lo || y1 >= it.hi ? 0u : hidden_params(p1);
              }
              vz[b] = u2h(__byte_perm(p0, p1, 0x5410));
              vs[b] = u2h(__byte_perm(p0, p1, 0x7632));
            }
            // two blocks j of 16 channels at a time: f[.][2 b] is channel row g,
            // f[.][2 b + 1] row g + 8 (d = 128: of the two words; d = 64: of the
            // two halves of the one)
#pragma unroll
            for (int y = 0; y < MB / 2; ++y) {
              uint32_t f[2][4];
#pragma unroll
              for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  // byte y (or y + 2) of both tokens into bytes 0 and 2
                  const int word = D == 128 ? q : 0, byte = D == 128 ? y : y + 2 * q;
                  const uint32_t v = __byte_perm(v0[b][word], v1[b][word], byte * 0x0011 + (4 + byte) * 0x1100);
                  f[0][2 * b + q] = dq_lo(v, vs[b], vz[b], magic);
                  f[1][2 * b + q] = dq_hi(v, vs[b], vz[b], magic);
                }
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) mma(o[nb][2 * y + j], f[j], pf[0][nb][e][0], pf[0][nb][e][1]);
            }
          }
        }
      }
      // the stage is read: the step kStages on takes it
      __syncwarp();
      have = (have & ~(kNotes << (kNote * kSub * st))) |
             (ahead.copy(a, ring_at + st * kSub * St::bytes, warp, lane) << (kNote * kSub * st));
      if (++st == kStages) st = 0;
    }
    // ---- the warps' parts of the item meet
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nb][k] += __shfl_xor_sync(0xffffffffu, l[nb][k], d);
        const int r = nb * 8 + 2 * c + k;
        if (g == 0) stat[warp * R + r] = make_float2(m[nb][k], near_sum(m[nb][k], l[nb][k], kNone));
        // rows g and g + 8 of block j are the channels (2 MB) g + j and
        // (2 MB) g + MB + j, kept at 16 j + 2 g and 16 j + 2 g + 1
        float* row = merge + (warp * R + r) * Sm::LD;
#pragma unroll
        for (int j = 0; j < MB; ++j)
          *reinterpret_cast<float2*>(row + 16 * j + 2 * g) = make_float2(o[nb][j][k], o[nb][j][2 + k]);
      }
    }
    __syncthreads();
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
          const float inv = inverse_sum(sum);
          T* dst = (T*)a.out + tok * a.o_row + head * a.o_head + ch;
          if constexpr (TERMS == 2) {
            *reinterpret_cast<float4*>(dst) = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
          } else {
            const __nv_bfloat162 b0 = __floats2bfloat162_rn(v.x * inv, v.y * inv), b1 = __floats2bfloat162_rn(v.z * inv, v.w * inv);
            *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
          }
          if (a.lse && ch == 0) a.lse[tok * a.heads + head] = log_sum(mx, sum);
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
    more = it.next(a);
    __syncthreads();
    if (more) load_q();
  } while (more);
}

template <int D, int NB, class F, class T>
cudaError_t launch_mma(const AttendArgs& a, int workers, cudaStream_t st) {
  static SmemLimit limit;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)workers, 1, 1);
  cfg.blockDim = dim3(kNt, 1, 1);
  cfg.dynamicSmemBytes = Smem<D, NB, F>::bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {early_launch()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return launch_smem(limit, cfg.dynamicSmemBytes, paged_attend_mma_kernel<D, NB, F, T>, cfg, a);
}

// float32 at d = 128 has no registers for 16 rows
Workers workers_of(int64_t max_rows, int bits, bool f32, int d) {
  const int sms = sm_count();
  if (max_rows <= 8) return Workers{(f32 ? 2 : bits == 8 ? Plan<E4m3>::kCtas : Plan<Int4>::kCtas) * sms, 8};
  return Workers{2 * sms, f32 && d == 128 ? 8 : 16};
}

template <int D, class F, class T>
cudaError_t launch_rows(const AttendArgs& a, Workers w, cudaStream_t st) {
  if constexpr (sizeof(T) == 4 && D == 128) return launch_mma<D, 1, F, T>(a, w.count, st);
  else return w.rows == 8 ? launch_mma<D, 1, F, T>(a, w.count, st) : launch_mma<D, 2, F, T>(a, w.count, st);
}

template <class F, class T>
cudaError_t launch_dim(const AttendArgs& a, int d, Workers w, cudaStream_t st) {
  return d == 64 ? launch_rows<64, F, T>(a, w, st) : launch_rows<128, F, T>(a, w, st);
}

}  // namespace

Workers mma_workers(int64_t max_rows, int bits, bool f32, int d) { return workers_of(max_rows, bits, f32, d); }

cudaError_t launch_attend_mma(const AttendArgs& a, int d, bool f32, int64_t max_rows, cudaStream_t st) {
  const Workers w = workers_of(max_rows, a.bits, f32, d);
  const cudaError_t e = f32 ? launch_dim<E4m3, float>(a, d, w, st)
                        : a.bits == 8 ? launch_dim<E4m3, __nv_bfloat16>(a, d, w, st) : launch_dim<Int4, __nv_bfloat16>(a, d, w, st);
  return e != cudaSuccess ? e : launch_attend_join(a, d, !f32, w, max_rows, st);
}

}  // namespace paged
}  // namespace qwm
