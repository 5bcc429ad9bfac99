/*
 * libqwm -- the QuantWM 2-bit KV cache on one GB300 GPU (sm_103a).
 *
 * C ABI of the data-parallel hot path of QuantWM ("QuantWM: Temporally
 * Consistent 2-Bit KV Cache Quantization for World Models and Video
 * Generation", Abstract; the roboind article on QuantWM, sections "Step 1" and
 * "Step 2"):
 *
 *   qwm_calibrate  historical-query sensitivity s_c = mean q_c^2 and the PSAC
 *                  basis U_r (top-r eigenvectors of Q_hist^T Q_hist);
 *   qwm_append     QSAC centroid choice, INT2 quantisation and 2-bit packing of
 *                  the key residual and of the value, PSAC coefficients
 *                  e = U_r (k - k_hat);
 *   qwm_attend     softmax attention of a query chunk over every cached token,
 *                  logit = q.k_hat + (q U_r^T).e.
 *
 * Conventions shared by every call
 *   - The caller owns every device buffer (cache, state, workspace, inputs,
 *     outputs); the library owns only the host handle qwm_ctx.
 *   - Device pointers are plain CUDA device addresses on the device that was
 *     current at qwm_create.  Tensors are dense and row-major:
 *     keys, values, queries and outputs are [heads][rows][head_dim] in the
 *     configured dtype (float32 or bfloat16).
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Compute calls are asynchronous on that stream; calls on one
 *     context must be ordered (one stream, or events between streams).  One
 *     exception: the eigen-solver of qwm_calibrate runs on a stream the
 *     context owns (see qwm_calibrate); every later call that reads what it
 *     writes makes its own stream wait for it first.
 *   - Errors found on the host (arguments, sizes, capacity, call order) are
 *     returned before any launch and leave the context unchanged.  A CUDA
 *     launch error returns QWM_ERR_CUDA.  Conditions found on the device (an
 *     eigen-solver that did not converge, a float16 parameter that saturated)
 *     set bits of a device status word read by qwm_get_status.
 *   - Every entry point is thread-compatible: one context must not be used by
 *     two host threads at once.
 */
#ifndef QWM_H
#define QWM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  QWM_OK = 0,
  QWM_ERR_INVALID_ARG = 1,     /* null pointer, bad size or shape             */
  QWM_ERR_UNSUPPORTED = 2,     /* valid but not built (e.g. head_dim 96)      */
  QWM_ERR_CAPACITY = 3,        /* cache tiles or basis versions exhausted     */
  QWM_ERR_NOT_CALIBRATED = 4,  /* append/attend before calibrate/centroids    */
  QWM_ERR_NOT_CONVERGED = 5,   /* device: eigen-solver hit its iteration cap  */
  QWM_ERR_CUDA = 6,            /* a CUDA runtime call or launch failed        */
  QWM_ERR_OOM = 7,             /* host allocation failed                      */
  QWM_ERR_DEVICE = 8           /* device: other status bits set (see below)   */
} qwm_status;

typedef enum { QWM_F32 = 0, QWM_BF16 = 1 } qwm_dtype;

/* Test hooks, read from the environment at every call:
 *   QWM_FAULT_INJECT=oom     qwm_create returns QWM_ERR_OOM after its argument
 *                            checks, before any CUDA call, creating nothing;
 *   QWM_FAULT_INJECT=launch  qwm_set_centroids, qwm_calibrate,
 *                            qwm_set_calibration, qwm_append, qwm_attend,
 *                            qwm_dequantize, qwm_kmeans, qwm_qk_norm_rope and
 *                            the qwm_paged_ calls return QWM_ERR_CUDA
 *                            after their argument checks and before launching
 *                            anything; the context is left unchanged.
 * A library built with -DQWM_DEBUG_BOUNDS (libqwm_dbg.so) checks every
 * centroid index it reads from the cache against n_centroids; one out of range
 * sets QWM_DEV_BOUNDS in the status word and is read as 0.
 * qwm_calibrate, qwm_append, qwm_attend, qwm_qk_norm_rope and the qwm_paged_
 * calls each open an NVTX range of their own name (recorded only under a
 * profiler). */

/* device status word bits (qwm_get_status / qwm_peek_status_bits) */
#define QWM_DEV_NOT_CONVERGED 0x1u  /* calibrate: residual above tolerance at max_iter */
#define QWM_DEV_SATURATED     0x2u  /* append: a float16 zero or scale saturated at 65504 */
#define QWM_DEV_TIMEOUT       0x4u  /* a bounded device wait ran out; the kernel left early */
#define QWM_DEV_BOUNDS        0x8u  /* QWM_DEBUG_BOUNDS builds only: a cache slot named a
                                       centroid index >= n_centroids (read as 0); in every
                                       build: an index, length or position on the device that
                                       a paged call was handed was out of range (see there) */
#define QWM_DEV_NAN           0x10u /* paged append: a NaN was stored as 0 */
#define QWM_DEV_CAPACITY      0x20u /* paged plan or release: the request did not fit; nothing
                                       was changed */

typedef struct {
  int32_t heads;         /* H >= 1                                              */
  int32_t head_dim;      /* d: 64 or 128                                        */
  int32_t group;         /* channels per quantisation group: must be 32         */
  int32_t rank;          /* PSAC rank r, 0 <= r <= d                            */
  int32_t n_centroids;   /* C, 1 <= C <= 1024                                   */
  int32_t dtype;         /* qwm_dtype of keys, values, queries, centroids, out  */
  int64_t max_tokens;    /* cache capacity in token slots (rounded up to 128);
                            every append starts a new 128-slot tile             */
  int32_t max_versions;  /* basis slots: versions alive at once, the current
                            one included (>= 1)                                 */
  int32_t max_iter;      /* eigen-solver iteration cap (>= 1)                   */
  int32_t oversample;    /* extra subspace columns of the eigen-solver (>= 0)   */
  int32_t max_hist;      /* largest n_h a calibrate call may pass (>= 1)        */
} qwm_config;

/* Sizes and byte offsets derived from a config (qwm_sizes). */
typedef struct {
  size_t cache_bytes;      /* H * max_tiles * tile_bytes                        */
  size_t state_bytes;      /* calibration, centroids, bases, tile table, status */
  size_t workspace_bytes;  /* calibrate scratch, then the few-row attention's   */
                           /* partial results (bf16, d = 128)                    */
  size_t tile_bytes;       /* bytes of one 128-slot tile of one head            */
  size_t bytes_per_token;  /* tile_bytes / 128                                  */
  int64_t max_tiles;       /* tiles per head                                    */
  /* offsets of the sections inside one tile */
  size_t off_idx, off_kcode, off_kqp, off_e, off_vcode, off_vqp;
  /* offsets of the arrays inside the state buffer */
  size_t st_status, st_s, st_w, st_lambda, st_energy, st_centroids, st_basis, st_tiles, st_iters;
  size_t st_centroids_f32;  /* float32 copy of bf16 centroids (= st_centroids for f32) */
  size_t st_centroids_f16;  /* float16 copy of bf16 centroids at d = 128, the channels of
                               every 16-channel block in the order 0, 8, 1, 9, ..., 7, 15
                               (= st_centroids when unused)                         */
} qwm_layout;

typedef struct qwm_ctx qwm_ctx;

/* Human-readable name of a status code (static string). */
const char* qwm_status_string(qwm_status s);

/* Validate `cfg` and compute every size and offset.  No CUDA call.
 * Cache layout: [H][max_tiles][tile_bytes]; one tile holds 128 token slots as
 *   idx   u8 (C <= 256) or u16       [128]
 *   kcode 2-bit K residual codes     [128][d/4]   channel c in byte c/4, bits 2(c%4)
 *   kqp   fp16 (zero, scale) of K    [128][d/32][2]
 *   e     fp16 PSAC coefficients     [128][r]
 *   vcode 2-bit V codes              [128][d/4]
 *   vqp   fp16 (zero, scale) of V    [128][d/32][2]
 * State tile table: int32 pairs (basis slot, valid slots) per tile; a basis
 * slot holds the U of one live basis version. */
qwm_status qwm_sizes(const qwm_config* cfg, qwm_layout* out);

/* Bind a context to caller-owned device buffers of at least the sizes from
 * qwm_sizes (256-byte aligned).  Zeroes the state buffer (synchronously).
 * The buffers must outlive the context.  *out receives the handle. */
qwm_status qwm_create(const qwm_config* cfg, void* d_cache, void* d_state, void* d_workspace,
                      qwm_ctx** out);

/* Release the host handle (device buffers stay with the caller); waits for
 * the context's own stream first.  NULL is a no-op. */
qwm_status qwm_destroy(qwm_ctx* ctx);

/* Self-test of the bounded device waits: one warp waits on an mbarrier that
 * nothing arrives at, with the wait of the attention kernels limited to
 * limit_cycles SM cycles (1 .. 2^32); when it runs out it ORs QWM_DEV_TIMEOUT
 * into *d_status (a caller-owned, caller-zeroed device word) and the kernel
 * returns, leaving the CUDA context usable.  Asynchronous on `stream`. */
qwm_status qwm_selftest_wait_timeout(int64_t limit_cycles, uint32_t* d_status, void* stream);

/* Copy the high-precision centroids [H][C][d] (configured dtype, device) into
 * the state.  QSAC chooses among these ("each Key is assigned to a
 * clustering center ... the center retaining high accuracy", roboind
 * article, "Step 1").  Asynchronous on `stream`, except for bf16 caches at
 * d = 128: there the call also builds the float16 copy that attention
 * kernel 6 reads and waits for `stream` once to learn whether every centroid
 * fits the float16 range (|C| < 65520); when one does not, kernel 6 is not
 * used for this context. */
qwm_status qwm_set_centroids(qwm_ctx* ctx, const void* d_centroids, void* stream);

/* Calibrate from n_h historical queries [H][n_h][d] (device, configured dtype):
 * s_c = mean q_c^2, group weights w_g = sum of s over the group, and the PSAC
 * basis U_r = top-r eigenvectors of Q_hist^T Q_hist (rows, descending
 * eigenvalue; the largest-magnitude entry of each is positive) by block
 * subspace iteration with Rayleigh-Ritz ("the energy of historical queries
 * tends to be concentrated in a few directions", roboind article "Step 2").
 * Opens a new basis version: later appends store coefficients in it.
 * Needs 1 <= n_h <= max_hist.  Asynchronous; non-convergence within max_iter
 * sets QWM_DEV_NOT_CONVERGED and keeps the best basis found.
 * Streams: the Gram sums, s and the group weights are computed on `stream`;
 * the eigen-solver then runs on a stream owned by the context, after them.
 * Later calls on the context that read its results (the coefficient step of
 * qwm_append, qwm_attend, qwm_calibrate, qwm_set_calibration,
 * qwm_get_calibration, qwm_get_status, qwm_peek_status_bits,
 * qwm_dequantize) make their stream wait for it, so the quantisation of the
 * next qwm_append, which needs only the group weights, overlaps it.  Code
 * that reads the basis in the state buffer directly must first issue one of
 * those calls on its stream.  Under CUDA graph capture, end the capture
 * after such a call (it joins the context's stream back into the graph). */
qwm_status qwm_calibrate(qwm_ctx* ctx, const void* d_q_hist, int64_t n_h, void* stream);

/* Calibration for callers that cannot allocate device memory.  (The QuantWM
 * pages have no counterpart of this entry point; it only changes where the
 * scratch lives.)  Some callers cannot call cudaMalloc at all: a plugin whose
 * host application owns all device memory through its own pool, or a code
 * path that must not allocate or free because cudaMalloc/cudaFree may
 * synchronise the device.  This call needs no context and no workspace: it
 * computes the same sensitivity s [H][d], basis U [H][r][d], eigenvalues
 * lambda [H][r] and energy [H] as qwm_calibrate (all float32, caller-owned
 * device buffers; U and lambda may be NULL when rank is 0) from q_hist
 * [H][n_h][d] (dtype QWM_F32 or QWM_BF16), with its scratch (Gram partial
 * sums, A^2, eigen-solver buffers) in one 8 MiB array compiled into the
 * library, which every GPU that loads the library keeps until the process
 * exits.
 *   - Limit: one split of partial sums (H*d*d floats) plus A^2 (H*d*d floats)
 *     must fit in 8 MiB; when rank + oversample > 64 the whole-matrix solver
 *     needs no A^2 but spills 6*d*(d+1) floats per head at d = 128.  Larger
 *     requests return QWM_ERR_CAPACITY before any launch.  That is up to 63
 *     heads at d = 128 (18 when rank + oversample > 64) and 255 at d = 64.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress) once for that device and its current context;
 *     make that first call before any stream capture.  A new context on the
 *     device (after cudaDeviceReset, for instance) has a new driver id, and
 *     the first call in it looks the address up again (also before any
 *     capture).  No call allocates or frees memory.
 *   - All calls share the one array: calls that overlap on the GPU (two
 *     streams, or two host threads) race and corrupt each other's results;
 *     order them.  Nothing in the array needs to start at zero except the
 *     status word, which the call clears itself.
 *   - d_status (optional, caller-zeroed) receives QWM_DEV_NOT_CONVERGED when
 *     the eigen-solver hits max_iter.  With d_status NULL that bit goes to a
 *     word of the shared array and is not reported: a caller that needs to
 *     know about non-convergence passes d_status.  Asynchronous on `stream`. */
qwm_status qwm_calibrate_static(int32_t heads, int32_t head_dim, int32_t rank, int32_t dtype,
                                int32_t max_iter, int32_t oversample, const void* d_q_hist,
                                int64_t n_h, float* d_s, float* d_U, float* d_lambda,
                                float* d_energy, uint32_t* d_status, void* stream);

/* Install a calibration computed elsewhere: s [H][d] and U [H][r][d] (host
 * float32).  Opens a new basis version like qwm_calibrate.  Synchronous. */
qwm_status qwm_set_calibration(qwm_ctx* ctx, const float* h_s, const float* h_U, void* stream);

/* Read the current calibration back (host float32, any pointer may be NULL):
 * s [H][d], U [H][r][d], lambda [H][r], energy [H] = sum(lambda)/trace.
 * Synchronous. */
qwm_status qwm_get_calibration(qwm_ctx* ctx, float* h_s, float* h_U, float* h_lambda,
                               float* h_energy, void* stream);

/* Append one chunk of n tokens: keys and values [H][n][d] (device).  For each
 * key: QSAC j* = argmin_j sum_g w_g (range_g(k - C_j)/3)^2/12 (float32
 * decision, lowest j on a tie), the residual k - C_j* and the value are
 * quantised per 32-channel group to INT2 with fp16 zero = min and
 * scale = range/3, packed 4 codes a byte, and e = U_r (k - k_hat) is stored
 * as r fp16 values (QuantWM Abstract; roboind article "Step 1", "Step 2").
 * Occupies ceil(n/128) new tiles; slots past n in the last tile are zeroed
 * and masked in attention.  n = 0 is a no-op.  Needs a calibration and
 * centroids.  Asynchronous: the quantisation runs at once on `stream`, the
 * coefficients e after the eigen-solver of the last qwm_calibrate (two
 * kernels; the second rebuilds k - k_hat from the tile with the same float32
 * operations). */
qwm_status qwm_append(qwm_ctx* ctx, const void* d_k, const void* d_v, int64_t n, void* stream);

/* Attention of M query rows [H][M][d] over every cached token:
 *   O = softmax(scale * (q.k_hat_n + (q U_t(n)^T).e_n)) V_hat
 * with U_t(n) the basis version the token was appended under ("the current
 * Query matching score with the Historical Key determines how the model
 * allocates attention", roboind article, "The key to a smaller error").
 * softmax_scale <= 0 selects 1/sqrt(d).  Output [H][M][d] in the configured
 * dtype (device).  The cache must hold at least one token.  Asynchronous. */
qwm_status qwm_attend(qwm_ctx* ctx, const void* d_q, int64_t M, float softmax_scale, void* d_out,
                      void* stream);

/* Drop every segment (append call) after the first n_segments, freeing their
 * tiles.  Host bookkeeping only; no device work. */
qwm_status qwm_rewind(qwm_ctx* ctx, int32_t n_segments);

/* Synchronise `stream`, read and clear the device status word.  Returns
 * QWM_ERR_NOT_CONVERGED or QWM_ERR_DEVICE when bits were set, else QWM_OK. */
qwm_status qwm_get_status(qwm_ctx* ctx, void* stream);

/* Same as qwm_get_status but returns the raw bits in *bits. */
qwm_status qwm_peek_status_bits(qwm_ctx* ctx, uint32_t* bits, void* stream);

/* Lloyd's k-means that builds the centroids QSAC assigns keys to ("each Key is
 * assigned to a clustering center", roboind article, "Step 1").  keys
 * [H][n][d] (dtype), d_init_rows [H][C] int32 (device; the starting keys,
 * e.g. the first C entries of a seeded permutation), `iters` iterations:
 * assignment to the nearest centroid in float32 squared distance (lowest
 * index on a tie), update to the float64 mean of the assigned keys rounded to
 * float32, an empty cluster keeps its centroid.  Output [H][C][d] in dtype
 * (nearest even), ready for qwm_set_centroids.  d_workspace: at least
 * qwm_kmeans_workspace_bytes(...) bytes, 256-byte aligned, caller-owned.
 * Asynchronous. */
size_t qwm_kmeans_workspace_bytes(int32_t heads, int32_t head_dim, int32_t n_centroids, int64_t n);
qwm_status qwm_kmeans(int32_t heads, int32_t head_dim, int32_t dtype, int32_t n_centroids,
                      const void* d_keys, int64_t n, const int32_t* d_init_rows, int32_t iters,
                      void* d_centroids, void* d_workspace, void* stream);

/* Centroid assignment of later appends: 0 = QSAC (default; the
 * sensitivity-weighted residual-range score), 1 = nearest centroid (squared
 * distance), the baseline the roboind article's "Step 1" describes for QVG and
 * that QSAC replaces.  For comparisons (the attention-shift diagnostics). */
qwm_status qwm_set_assignment(qwm_ctx* ctx, int32_t mode);

/* The cache in float32 for analysis: k_hat [H][n_tiles*128][d] =
 * C[j] + zero + code*scale, v_hat [H][n_tiles*128][d] = zero + code*scale,
 * e [H][n_tiles*128][r] (the stored fp16 coefficients; may be NULL when
 * r = 0), slot s of tile t at row t*128 + s; pad slots are zero.  Caller-owned
 * device buffers.  Asynchronous. */
qwm_status qwm_dequantize(qwm_ctx* ctx, float* d_khat, float* d_vhat, float* d_e, void* stream);

/* Attention kernel choice: 0 = automatic (bf16 and d = 128: for M <= 64 and
 * r <= 32 kernel 5, or kernel 7 when 16 < M and kernel 6 applies; else kernel
 * 6 when r <= 16 and the centroids fit float16, kernel 4 when r <= 16, kernel
 * 3 when r <= 32; otherwise kernel 2 where it applies, else kernel 1), 1 =
 * float32 CUDA-core kernel, 2 = bf16
 * mma.sync kernel, 3 = bf16 tcgen05 kernel with 128 query rows per CTA, 4 =
 * bf16 tcgen05 kernel with 256 query rows per CTA (r <= 16; the key as two
 * bf16 terms), 5 = bf16 kernel for at most 64 query rows (split over the
 * cache tiles, partial results in the context workspace, merged by a second
 * kernel), 6 = tcgen05 kernel with 256 query rows per CTA and the key split
 * into its float16 centroid row and float16 residual (r <= 16, centroids
 * within the float16 range; queries are scaled per row by a power of two
 * into that range), 7 = kernel 6 with one 128-row query tile per CTA and the
 * cache tiles split over CTAs, merged by kernel 5's second kernel (M <= 64;
 * partial results in the context workspace).  An explicit choice the
 * configuration (or M) does not support makes qwm_attend return
 * QWM_ERR_UNSUPPORTED. */
qwm_status qwm_set_attend_kernel(qwm_ctx* ctx, int32_t kernel);

/* The attention kernel qwm_attend runs for more than 64 query rows (1 to 4,
 * or 6; automatic resolved). */
int32_t qwm_resolved_attend_kernel(const qwm_ctx* ctx);

/* The attention kernel qwm_attend runs for M query rows (1 to 7). */
int32_t qwm_attend_kernel_for(const qwm_ctx* ctx, int64_t M);

int64_t qwm_num_tokens(const qwm_ctx* ctx);    /* valid tokens cached        */
int64_t qwm_num_tiles(const qwm_ctx* ctx);     /* tiles in use per head      */
int32_t qwm_num_segments(const qwm_ctx* ctx);  /* append calls kept          */
int32_t qwm_version(const qwm_ctx* ctx);       /* current basis version, -1 before any */

/* ------------------------------------------------------------------------
 * The paged 4-bit cache: many requests of different lengths in one pool of
 * pages, without calibration or centroids (an extension; the QuantWM pages
 * describe the 2-bit cache above only).  A serving step is
 *   qwm_paged_plan      once a step: new pages, slots and positions of its rows;
 * and in every layer
 *   qwm_qk_norm_rope    RMS norm of each query and key head, and rotation;
 *   qwm_paged_append    INT4 quantisation of the new keys and values into pages;
 *   qwm_paged_attend    attention of the new rows over their requests' pages;
 * and qwm_paged_release when requests end or are cut back.
 *
 * These calls keep nothing between calls and need no context.  Every pointer
 * in the argument structs is a device address on the current device, aligned to
 * its type at least (QWM_ERR_INVALID_ARG otherwise); all
 * lengths, tables and counts live on the device, so a step can be captured
 * into a CUDA graph and replayed with other lengths.  Calls are asynchronous
 * on `stream`, allocate nothing and write only what is documented, so calls
 * on different streams (or graphs replayed at the same time) are independent
 * as long as they share no buffer that one of them writes, workspaces
 * included.  `status`, where a struct has it, is an optional device word
 * (caller-zeroed) into which the call ORs QWM_DEV_ bits.
 *
 * Pool: [n_pages][kv_heads][block], one pool per layer.  A block holds
 * page_tokens slots (16, 32, 64, 128 or 256) of one key/value head:
 *   K codes   [slot][d/2]       4-bit codes, channel c in byte c/2, bits 4 (c mod 2)
 *   K params  [slot][d/32][2]   fp16 (zero, scale) of each group of 32 channels
 *   V codes, V params           the same for the value
 * qwm_paged_block_bytes = page_tokens (d + d/4) bytes.  Token n of request b
 * is in slot n mod page_tokens of page block_table[b][n / page_tokens]. */

/* Rows of a caller's tensor [rows][heads][head_dim]: element (t, h, c) is at
 * ptr + t row_stride + h head_stride + c (strides in elements, so views of a
 * fused projection and [heads][rows][head_dim] tensors both fit).  ptr and
 * strides must be multiples of 16 bytes (QWM_ERR_INVALID_ARG otherwise);
 * strides are not negative, and those of an output must not let two elements
 * share an address. */
typedef struct {
  void* ptr;
  int64_t row_stride, head_stride;
} qwm_rows;

/* RMS norm of every head of q and k with the rotary position encoding in the
 * same pass:
 *   x' = x (mean(x^2) + eps)^(-1/2) w     (float32; w = 1 where a weight is NULL)
 *   pair j of the rot/2 rotated pairs: (a, b) -> (a cos - b sin, b cos + a sin)
 * with channels (j, j + rot/2), or (2j, 2j + 1) when interleaved, and cos, sin
 * = cos_sin[p][j], cos_sin[p][rot/2 + j] at p = positions[t][axis(j)].  Pairs
 * are dealt to the axes in order: the first sections[0] to axis 0 and so on
 * (one axis takes all).  Channels from rot on are normed, not rotated.  One
 * rounding to the dtype at the end.  Outputs may be the inputs (in place; the
 * same pointer and strides), else must not overlap them.
 * A row with a negative position on any axis is padding: its outputs are left
 * as they were.  So is a row with a position >= n_positions, which also sets
 * QWM_DEV_BOUNDS. */
typedef struct {
  qwm_rows q, k, q_out, k_out;   /* dtype; k ignored when k_heads = 0           */
  const void* q_weight;          /* [head_dim] dtype, or NULL                   */
  const void* k_weight;
  const float* cos_sin;          /* [n_positions][rot]: rot/2 cos, rot/2 sin;
                                    16-byte aligned                             */
  const int32_t* positions;      /* [rows][axes]                                */
  uint32_t* status;              /* or NULL                                     */
  int64_t rows, n_positions;
  int32_t dtype, head_dim;       /* QWM_F32 or QWM_BF16; 64 or 128              */
  int32_t q_heads, k_heads;      /* >= 1, >= 0                                  */
  int32_t rot;                   /* rotated channels: a multiple of 16, <= d    */
  int32_t axes;                  /* 1 to 4                                      */
  int32_t sections[4];           /* pairs of each axis; sum rot/2               */
  int32_t interleaved;
  float eps;                     /* >= 0                                        */
} qwm_qk_norm_rope_args;
qwm_status qwm_qk_norm_rope(const qwm_qk_norm_rope_args* a, void* stream);

/* Block tables, slots and positions of a step from the lengths of its
 * requests.  Request b holds kv_len[b] tokens in ceil(kv_len[b] / page_tokens)
 * pages and brings new_len[b] >= 0 tokens.  Pages come off the top of a stack
 * (free_pages[0 .. free_count)) in the order of the requests: the i-th new
 * page of the call is free_pages[free_count - 1 - i].  Writes
 *   kv_len_out[b]   kv_len[b] + new_len[b]
 *   cu_rows[b]      first row of request b; cu_rows[requests] = rows in use
 *   block_table     the entries of the new pages, no others
 *   free_count_out  pages left
 *   slots[t]        page * page_tokens + slot of row t, -1 for rows not in use
 *   positions[t]    the row's position in its request, -1 for rows not in use
 * The call changes all or nothing: when the pages run out, a request would
 * outgrow max_blocks, the new rows exceed `rows`, or a length is negative, it
 * sets QWM_DEV_CAPACITY (QWM_DEV_BOUNDS for a negative length or free_count
 * outside [0, n_pages]), copies kv_len and free_count, sets cu_rows to 0 and
 * every slot and position to -1, and leaves block_table alone.  A page id
 * outside [0, n_pages) sets QWM_DEV_BOUNDS and its rows get slot -1.
 * kv_len_out may be kv_len, free_count_out may be free_count; other outputs
 * overlap nothing.  At most 8192 requests (QWM_ERR_UNSUPPORTED above). */
typedef struct {
  const int32_t* kv_len;         /* [requests]                                  */
  const int32_t* new_len;        /* [requests]                                  */
  const int32_t* free_pages;     /* [n_pages]                                   */
  const int32_t* free_count;     /* [1]                                         */
  int32_t* block_table;          /* [requests][max_blocks]                      */
  int32_t* kv_len_out;           /* [requests]                                  */
  int32_t* free_count_out;       /* [1]                                         */
  int32_t* cu_rows;              /* [requests + 1]                              */
  int64_t* slots;                /* [rows]                                      */
  int32_t* positions;            /* [rows]                                      */
  uint32_t* status;              /* or NULL                                     */
  int64_t rows, n_pages;         /* rows < 2^31, n_pages < 2^31                 */
  int32_t requests, max_blocks, page_tokens;
} qwm_paged_plan_args;
qwm_status qwm_paged_plan(const qwm_paged_plan_args* a, void* stream);

/* Cut request b back to keep_len[b] tokens (0 ends it) and push the pages it
 * no longer needs on the free stack, requests in order, a request's pages in
 * order; their table entries become -1.  kv_len, block_table, free_pages and
 * free_count are updated in place.  keep_len[b] outside [0, kv_len[b]] keeps
 * the request as it is and sets QWM_DEV_BOUNDS; a page id outside
 * [0, n_pages) is not pushed and sets it too.  When the stack would pass
 * n_pages (a page released twice) nothing is changed and QWM_DEV_CAPACITY is
 * set.  No references are counted: a page that several tables name (a shared
 * prefix, which the attention reads like any other) would be pushed once for
 * each, so such pages stay out of this call.  At most 8192 requests. */
typedef struct {
  const int32_t* keep_len;       /* [requests]                                  */
  int32_t* kv_len;               /* [requests]                                  */
  int32_t* block_table;          /* [requests][max_blocks]                      */
  int32_t* free_pages;           /* [n_pages]                                   */
  int32_t* free_count;           /* [1]                                         */
  uint32_t* status;              /* or NULL                                     */
  int64_t n_pages;
  int32_t requests, max_blocks, page_tokens;
} qwm_paged_release_args;
qwm_status qwm_paged_release(const qwm_paged_release_args* a, void* stream);

/* Bytes of one block, or 0 for a head_dim or page_tokens that is not built. */
size_t qwm_paged_block_bytes(int32_t head_dim, int32_t page_tokens);

/* Quantise keys and values [rows][kv_heads][d] into the slots of a plan.  For
 * each group of 32 channels, in float32, one IEEE operation at a time:
 *   NaN -> 0 (QWM_DEV_NAN), then clamped to +-60000 (QWM_DEV_SATURATED), so
 *   that every value a page stands for is finite in fp16;
 *   mn, mx = min, max;  zero = f16(mn);  scale = f16(f32(mx - mn) / 15)
 *   code = 0 if scale = 0, else clamp(rint(f32(f32(x - zero) / scale)), 0, 15)
 *   x_hat = zero + code scale
 * k_hat and v_hat (optional; dtype, rows like the inputs) receive x_hat
 * rounded to the dtype; they overlap neither the inputs nor each other.  A row
 * with slot -1 (any negative slot) stores nothing, and its k_hat and v_hat are
 * 0; so does a slot >= n_pages page_tokens, which sets QWM_DEV_BOUNDS.  The slots of one call must differ
 * (those of a plan do): of two rows with the same slot, which one's bytes end
 * up there is undefined. */
typedef struct {
  qwm_rows k, v;
  qwm_rows k_hat, v_hat;         /* ptr NULL: not wanted                        */
  void* pool;                    /* 16-byte aligned                             */
  const int64_t* slots;          /* [rows]                                      */
  uint32_t* status;              /* or NULL                                     */
  int64_t rows, n_pages;
  int32_t dtype, head_dim, kv_heads, page_tokens;
} qwm_paged_append_args;
qwm_status qwm_paged_append(const qwm_paged_append_args* a, void* stream);

/* Attention of the rows of a plan over their requests' pages.  Row
 * cu_rows[b] + i is query i of request b, at position
 * P = kv_len[b] - (cu_rows[b + 1] - cu_rows[b]) + i (kv_len with the new
 * tokens, as a plan leaves it), and sees the tokens n < kv_len[b] with n <= P
 * when causal and n > P - window when window > 0 (window needs causal):
 *   O = softmax(scale q . k_hat_n) v_hat_n,   lse = log sum exp(scale q . k_hat_n)
 * Query head h reads key/value head h / (heads / kv_heads).  A row that sees
 * no token gets O = 0 and lse = -inf; one with NaN in q gets NaN in both.
 * Tokens that a row does not see have no effect on it, whatever bytes their
 * slots hold; a row that sees a token whose slot no append has written may get
 * any value, NaN included.  Rows outside cu_rows[0 .. requests] are left as they
 * were.
 * Kernels 2 and 3 take logits scale q . k_hat up to 2^22 in magnitude; a row
 * that meets a larger one may have NaN in O and lse (kernel 1 takes any).
 * When a bounded device wait of kernel 3 runs out, which no input makes it do,
 * the call still ends: the rows that were not done have NaN in O and lse, and
 * QWM_DEV_TIMEOUT is set in `status`, where there is one.
 * A page id outside [0, n_pages) hides its tokens, a kv_len outside
 * [0, max_blocks page_tokens] is clamped to it and cu_rows that decrease or
 * leave [0, rows] are clamped; each sets QWM_DEV_BOUNDS.
 * max_new is the longest request's row count as the host knows it: it chooses
 * the kernel and never changes what is computed (too large a value costs time:
 * 48 single tokens given as many rows 323 us, as one 106).  A step of single tokens and
 * prompts is better made in two calls, each over its range of requests
 * (block_table, kv_len and cu_rows from the range's first entry on, q and out
 * whole), so that either gets its kernel.
 * kernel: 0 = automatic; 1 = float32 CUDA-core kernel (the choice for
 * float32); 2 = bf16 mma.sync kernel that streams the pages once for every 16
 * rows (the choice for heads / kv_heads times max_new up to 32); 3 = bf16
 * tcgen05 kernel with 256 rows per CTA.  All split long requests over CTAs and join the parts in a second
 * kernel, in a fixed order.  QWM_ERR_UNSUPPORTED: 2 and 3 with float32, more
 * than 2^30 rows times heads / kv_heads, max_blocks page_tokens above 2^30. */
typedef struct {
  qwm_rows q, out;               /* out may be q (in place)                     */
  float* lse;                    /* [rows][heads], or NULL                      */
  const void* pool;              /* 16-byte aligned                             */
  const int32_t* block_table;    /* [requests][max_blocks]                      */
  const int32_t* kv_len;         /* [requests]                                  */
  const int32_t* cu_rows;        /* [requests + 1]                              */
  uint32_t* status;              /* or NULL                                     */
  void* workspace;               /* 256-byte aligned                            */
  size_t workspace_bytes;        /* >= qwm_paged_attend_workspace_bytes         */
  int64_t rows, n_pages, max_new;
  int32_t dtype, head_dim, heads, kv_heads, page_tokens;
  int32_t requests, max_blocks;
  int32_t causal, window;
  float scale;                   /* <= 0: 1/sqrt(d)                             */
  int32_t kernel;
} qwm_paged_attend_args;
qwm_status qwm_paged_attend(const qwm_paged_attend_args* a, void* stream);

/* Bytes of workspace that any call with this head_dim needs on the current
 * device, whatever its lengths and kernel (0 for a head_dim that is not built):
 * 41 MB at 128 channels, of which a step of single tokens uses 4. */
size_t qwm_paged_attend_workspace_bytes(int32_t head_dim);

/* The kernel (1 to 3) that the automatic choice runs. */
int32_t qwm_paged_attend_kernel_for(int32_t dtype, int32_t heads, int32_t kv_heads, int64_t max_new);

#ifdef __cplusplus
}
#endif
#endif /* QWM_H */
