/*
 * fa.h -- C ABI of libfa, exact attention for NVIDIA GB300 (sm_103a).
 *
 * Computes, for every batch element b and head h (the plain definition of
 * attention: "FlashAttention: Fast and Memory-Efficient Exact Attention with
 * IO-Awareness", summary page, "Problem and motivation"; scale on the scores
 * as in the GitHub issue "Fewer matrix multiplications, same results"):
 *
 *     S   = scale * Q K^T      (entries of invisible keys are -inf)
 *     P   = softmax(S)         (row-wise, with the row maximum subtracted)
 *     O   = P V
 *     lse = ln sum_j exp(S_ij)  (natural log; the only statistic kept)
 *
 * tile by tile with the online-softmax recurrence (blog review "From Online
 * Softmax to FlashAttention", "Algorithm FlashAttention (Tiling)"; summary
 * page, "Method": running max m, running denominator l, rescaled output), so
 * the N x N score matrix never reaches device memory, and the backward pass
 * recomputes P on chip from Q, K and lse (summary page, "Key ideas:
 * recomputation in the backward pass").
 *
 * Conventions shared by every call:
 *   - Tensors are dense row-major [B, H, N, d] (d contiguous) in DEVICE
 *     memory, 16-byte aligned; lse and D are fp32 [B, H, N].  The *_ex
 *     calls take Q, K, V, O, dO, dQ, dK, dV in any layout whose d elements of
 *     a row are contiguous (fa_layout), and dropout (fa_dropout); lse and D
 *     stay dense.  The caller owns
 *     every buffer; the library allocates nothing.
 *   - bf16 calls take bf16 (uint16 storage) Q, K, V, O, dO, dQ, dK, dV and
 *     accumulate in fp32.  *_fp32 calls take fp32 everywhere.
 *   - d must be 64 or 128; N >= 1 (any N: ragged tails are masked); B >= 1,
 *     H >= 1, B*H <= 65535; scale must be positive and finite.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Calls
 *     are asynchronous with respect to the host, like cuBLAS: a returned
 *     FA_OK means the work was enqueued.
 *   - Argument errors are detected on the host before anything is launched
 *     (and before any CUDA runtime call), and reported through the return
 *     value only.
 *   - Masking: `causal` keeps keys j <= i (queries and keys share indices).
 *     `mask` may add key padding (keys j >= kv_len[b] are invisible) or a
 *     block-sparse tile mask (tile (i/128, j/128) visible iff
 *     block_mask[(i/128)*T + j/128] != 0, T = ceil(N/128); summary page,
 *     "Extension: block-sparse FlashAttention").  causal combines with either
 *     (intersection).  A query row with no visible key gets O = 0,
 *     lse = -inf and contributes no gradient.
 */
#ifndef FA_H_
#define FA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1,  /* null pointer, non-positive size, bad mask kind  */
  FA_ERR_UNSUPPORTED = 2,  /* valid but not implemented (d not 64/128, ...)   */
  FA_ERR_ALIGNMENT = 3,    /* a tensor pointer is not 16-byte aligned         */
  FA_ERR_WORKSPACE = 4,    /* workspace missing or smaller than required      */
  FA_ERR_CUDA = 5,         /* a CUDA runtime/driver call failed               */
  FA_ERR_TIMEOUT = 6,      /* a kernel gave up waiting (see fa_get_device_status) */
  FA_ERR_PAGE = 7          /* a block table named a page outside the cache, or a row  */
                           /* past its capacity (see fa_get_device_status)            */
} fa_status;

typedef enum {
  FA_MASK_NONE = 0,
  FA_MASK_KEY_PADDING = 1,
  FA_MASK_BLOCK_SPARSE = 2
} fa_mask_kind;

typedef struct {
  int kind;                  /* an fa_mask_kind                                     */
  const int32_t* kv_len;     /* KEY_PADDING: device int32 [B]; values are clamped   */
                             /* to 0..N (0 = every key of the batch is padding)     */
  const uint8_t* block_mask; /* BLOCK_SPARSE: device uint8 [T*T], T = ceil(N/128)   */
                             /* <= 4096 (N <= 524288; FA_ERR_UNSUPPORTED beyond)    */
  int block_size;            /* BLOCK_SPARSE: tile edge of block_mask, must be 128  */
  const int32_t* tile_order; /* BLOCK_SPARSE, optional (NULL: the default order):    */
                             /* the work order fa_block_mask_order wrote for this   */
                             /* block_mask; device int32, 4-byte aligned            */
} fa_mask;

/* Work order of a block-sparse mask.  The kernels skip the tiles the mask
 * hides (summary page, "Extension: block-sparse FlashAttention": only the
 * nonzero blocks are visited) and give each CTA one tile row or column, so a
 * row or column that sees far more tiles than the rest (a global token) ends
 * the kernel alone if the grid takes it last.  This call writes, on `stream`,
 * fa_block_mask_order_len(T) int32 to tile_order:
 *   [0, T)              query tiles, most visible key tiles first
 *   [T, 2T)             key tiles, most query tiles that see them first
 * counting with the causal restriction when causal = 1; ties keep the lower
 * index first.  Passed as fa_mask.tile_order, the kernels take their tiles in
 * that order; every tile is still computed exactly once and the results are
 * bit-identical to the default order's.  The buffer must be this call's
 * output (any other permutation of each part is also correct; contents that
 * are not permutations leave output tiles unwritten or written twice -- the
 * kernels only clamp entries to [0, T)).  Recompute it when the mask changes;
 * it costs one small launch per mask.
 *   block_mask : device uint8 [T*T].   T : 1..4096.   causal : 0 or 1.
 * Argument errors come back before any CUDA runtime call. */
int fa_block_mask_order_len(int T); /* 2T + (T+1)/2, or 0 when T is out of range */
fa_status fa_block_mask_order(const uint8_t* block_mask, int T, int causal, int32_t* tile_order,
                              void* stream);

/* Forward pass, bf16 in/out.
 *   q, k, v : [B,H,N,d] bf16 inputs.   o : [B,H,N,d] bf16 output.
 *   lse     : [B,H,N] fp32 output, natural-log log-sum-exp of each score row
 *             (-inf for a row with no visible key).
 *   scale   : multiplies Q K^T (1/sqrt(d) for standard attention).
 *   causal  : 0 or 1.   mask : NULL for none.
 * Summary page "Method" (block statistics m, l and the rescaled output) and
 * blog review "Algorithm FlashAttention (Tiling)". */
fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                 int N, int d, float scale, int causal, const fa_mask* mask, void* stream);

/* Bytes of device workspace fa_bwd / fa_bwd_fp32 need: D (fp32 [B,H,N]),
 * padded to 256 bytes, then 256 bytes for the counter from which the backward
 * kernel's CTAs take their units of work.  0 on bad sizes. */
size_t fa_bwd_workspace_size(int B, int H, int N, int d);

/* Backward pass, bf16.  Given the forward's inputs, its outputs o and lse,
 * and the output gradient dO, writes dq, dk, dv ([B,H,N,d] bf16) for the loss
 * whose gradient with respect to O is dO.  P is recomputed from q, k, lse
 * (summary page, "Key ideas: recomputation in the backward pass"); the
 * gradient formulas (dV = P^T dO, dP = dO V^T, D = rowsum(dO o O),
 * dS = P o (dP - D), dQ = scale dS K, dK = scale dS^T Q) are the textbook
 * derivative, which the pages do not write out.
 *   workspace : device, >= fa_bwd_workspace_size(B,H,N,d) bytes, 16-byte
 *               aligned; contents on entry are ignored.
 * Runs fa_bwd_preprocess, fa_bwd_dkdv and fa_bwd_dq on `stream`. */
fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dO,
                 const float* lse, void* dq, void* dk, void* dv, void* workspace,
                 size_t workspace_bytes, int B, int H, int N, int d, float scale, int causal,
                 const fa_mask* mask, void* stream);

/* The three steps of fa_bwd, exposed for timing each kernel on its own.
 * fa_bwd_preprocess: D[b,h,i] = sum_c dO[b,h,i,c] * O[b,h,i,c] (fp32 [B,H,N]).
 * fa_bwd_dkdv: recomputes P and dS tile by tile for each 128-key tile and
 *   writes dk, dv (bf16 [B,H,N,d]).  D as left by the preprocess.
 * fa_bwd_dq: recomputes P and dS tile by tile for each 128-query tile and
 *   writes dq (bf16 [B,H,N,d]); each row of dq is summed by one CTA in fp32,
 *   so dq is the same bit for bit from run to run.
 * fa_bwd_dkdv and fa_bwd_dq read the same inputs and write disjoint outputs:
 *   they may run in either order, or concurrently on two streams. */
fa_status fa_bwd_preprocess(const void* o, const void* dO, float* D, int B, int H, int N, int d,
                            void* stream);
fa_status fa_bwd_dkdv(const void* q, const void* k, const void* v, const void* dO,
                      const float* lse, const float* D, void* dk, void* dv, int B, int H, int N,
                      int d, float scale, int causal, const fa_mask* mask, void* stream);
fa_status fa_bwd_dq(const void* q, const void* k, const void* v, const void* dO, const float* lse,
                    const float* D, void* dq, int B, int H, int N, int d, float scale, int causal,
                    const fa_mask* mask, void* stream);

/* fp32 twins of fa_fwd / fa_bwd: identical argument meaning with fp32
 * tensors everywhere (CUDA cores, no tensor cores; for small fp32 workloads). */
fa_status fa_fwd_fp32(const float* q, const float* k, const float* v, float* o, float* lse, int B,
                      int H, int N, int d, float scale, int causal, const fa_mask* mask,
                      void* stream);
fa_status fa_bwd_fp32(const float* q, const float* k, const float* v, const float* o,
                      const float* dO, const float* lse, float* dq, float* dk, float* dv,
                      void* workspace, size_t workspace_bytes, int B, int H, int N, int d,
                      float scale, int causal, const fa_mask* mask, void* stream);

/* Layout of one [B, H, N, d] tensor as element strides: element (b, h, n, c)
 * is at base + b*batch + h*head + n*row + c (the d elements of a row are
 * contiguous).  Dense [B,H,N,d] is {H*N*d, N*d, d}; a [B,N,H,d] buffer (the
 * heads of a packed projection side by side in each row) read as [B,H,N,d]
 * is {N*H*d, d, H*d}.  Rules, checked on the host before any launch:
 *   - the stride of a dimension of size 1 is ignored;
 *   - every other stride is positive (FA_ERR_UNSUPPORTED otherwise), a
 *     multiple of 16 bytes (8 bf16 or 4 fp32 elements; FA_ERR_ALIGNMENT
 *     otherwise) and below 2^40 bytes (FA_ERR_UNSUPPORTED otherwise);
 *   - the row stride is at least d when N > 1 (FA_ERR_UNSUPPORTED).
 * An output must not overlap another tensor of the same call; this is not
 * checked. */
typedef struct {
  int64_t batch, head, row;
} fa_layout;

/* Layouts of the tensors of one call.  The forward reads q, k, v, o and
 * ignores the rest. */
typedef struct {
  fa_layout q, k, v, o, dO, dq, dk, dv;
} fa_layouts;

/* Dropout on the attention probabilities.  The summary page lists dropout
 * among the operations fused into the attention kernel and says that the
 * backward pass keeps the generator's state to regenerate the mask on chip
 * ("Key ideas: kernel fusion"; its question on the auxiliary memory of the
 * backward pass).  Reading: with Z_ij in {0, 1} kept with probability 1 - p,
 *     O = (P o Z) V / (1 - p),   lse of the undropped scores,
 * and the backward is the chain rule through it (dV = (P o Z)^T dO / (1-p),
 * dS = P o (Z o dO V^T / (1-p) - D), D = rowsum(dO o O) as without dropout).
 * Z is drawn from Philox4x32-10 (Salmon et al., "Parallel random numbers: as
 * easy as 1, 2, 3", SC 2011): element (i, j) of head (b, h) takes the call
 * with counter (j / 8, i, b*H + h, offset) and key (seed & 0xFFFFFFFF,
 * seed >> 32); of its four output words, key j takes the low (j even) or
 * high (j odd) 16 bits of word (j % 8) / 2 and is kept when they are >= t,
 * t = min(65535, floor(p * 65536 + 0.5)) -- so the keep probability is
 * exactly 1 - t/65536 and the kept entries are scaled by 65536 / (65536 - t).
 * The forward and backward of one step must use the same p, seed, offset. */
typedef struct {
  float p;          /* drop probability, 0 <= p < 1 (0: no dropout)          */
  uint64_t seed;    /* generator key                                         */
  uint32_t offset;  /* fourth counter word: a new value per step (e.g. the step number) */
} fa_dropout;

/* Additive score bias: the "+ mask" term of the scores as a tensor,
 *     S_ij = scale q_i . k_j + bias[b, h, i, j]
 * added before the causal / padding / block masks (summary page, "Problem
 * and motivation"; the masks of the glossary page "Flash Attention",
 * "Normalization and Masking").  fp32 in device memory; element (b, h, i, j)
 * at ptr + b*batch + h*head + i*row + j.  A stride of 0 broadcasts (one
 * [N, N] bias for every head: batch = head = 0).  -inf hides a key; +inf
 * and NaN are not allowed.  Rules: ptr 16-byte aligned; strides >= 0,
 * multiples of 4 elements, row >= N unless 0 (FA_ERR_ALIGNMENT /
 * FA_ERR_UNSUPPORTED otherwise).  The bias receives no gradient. */
typedef struct {
  const float* ptr;
  int64_t batch, head, row;
} fa_bias;

/* Options of the *_ex calls.  NULL options, or NULL members, mean dense
 * tensors, no dropout and no bias. */
typedef struct {
  const fa_layouts* layouts;
  const fa_dropout* dropout;  /* bf16 calls only: FA_ERR_UNSUPPORTED for fp32 */
  const fa_bias* bias;        /* bf16 calls only: FA_ERR_UNSUPPORTED for fp32 */
} fa_options;

/* fa_fwd / fa_bwd / fa_fwd_fp32 / fa_bwd_fp32 and the three backward steps
 * with options; every other argument as in the plain call.  With dense
 * layouts and no dropout the work and results are those of the plain call;
 * other layouts give the same results on the same values (the kernels read
 * and write through the strides -- the TMA descriptors of the bf16 kernels
 * carry them -- and nothing is copied).  Errors: a p outside [0, 1)
 * (or NaN) is FA_ERR_INVALID_ARG; dropout or a bias on an fp32 call,
 * FA_ERR_UNSUPPORTED. */
fa_status fa_fwd_ex(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                    int N, int d, float scale, int causal, const fa_mask* mask,
                    const fa_options* options, void* stream);
fa_status fa_bwd_ex(const void* q, const void* k, const void* v, const void* o, const void* dO,
                    const float* lse, void* dq, void* dk, void* dv, void* workspace,
                    size_t workspace_bytes, int B, int H, int N, int d, float scale, int causal,
                    const fa_mask* mask, const fa_options* options, void* stream);
fa_status fa_fwd_fp32_ex(const float* q, const float* k, const float* v, float* o, float* lse,
                         int B, int H, int N, int d, float scale, int causal, const fa_mask* mask,
                         const fa_options* options, void* stream);
fa_status fa_bwd_fp32_ex(const float* q, const float* k, const float* v, const float* o,
                         const float* dO, const float* lse, float* dq, float* dk, float* dv,
                         void* workspace, size_t workspace_bytes, int B, int H, int N, int d,
                         float scale, int causal, const fa_mask* mask, const fa_options* options,
                         void* stream);
/* The backward steps with options (layouts of o, dO for the preprocess;
 * dropout and bias for fa_bwd_dkdv_ex and fa_bwd_dq_ex). */
fa_status fa_bwd_preprocess_ex(const void* o, const void* dO, float* D, int B, int H, int N, int d,
                               const fa_options* options, void* stream);
fa_status fa_bwd_dkdv_ex(const void* q, const void* k, const void* v, const void* dO,
                         const float* lse, const float* D, void* dk, void* dv, int B, int H,
                         int N, int d, float scale, int causal, const fa_mask* mask,
                         const fa_options* options, void* stream);
fa_status fa_bwd_dq_ex(const void* q, const void* k, const void* v, const void* dO,
                       const float* lse, const float* D, void* dq, int B, int H, int N, int d,
                       float scale, int causal, const fa_mask* mask, const fa_options* options,
                       void* stream);

/* Size of the fixed scratch array fa_bwd_noalloc works in: 32 MiB. */
#define FA_NOALLOC_SCRATCH_BYTES (32u << 20)

/* fa_bwd for callers that cannot allocate device memory.  The pages have no
 * counterpart to this call.  fa_bwd needs a caller-allocated workspace; some
 * callers cannot provide one, for example a plugin inside a host framework
 * that has reserved all device memory for its own pool and does not let
 * extensions call cudaMalloc, or latency-critical code that must avoid
 * cudaMalloc/cudaFree because they can synchronize the whole device.  This
 * call takes the workspace from a fixed array of FA_NOALLOC_SCRATCH_BYTES
 * compiled into the library (every GPU that loads the library holds it until
 * the process exits) and calls no allocator at all.
 *   Arguments and results are those of fa_bwd without the workspace pair;
 *   argument errors come back with fa_bwd's codes, from host-only checks
 *   made before any CUDA runtime call.
 *   Sizes whose workspace (fa_bwd_workspace_size) exceeds
 *   FA_NOALLOC_SCRATCH_BYTES are rejected with FA_ERR_UNSUPPORTED.
 *   The first call on a device looks up the array's device address (a CUDA
 *   runtime query, done once per device with that device current); make that
 *   first call before any stream capture.
 *   Every call shares the one array, which keeps the previous call's
 *   contents; each call rewrites what it needs before reading it.  Calls that
 *   overlap on the GPU (other streams, other host threads) race on the array:
 *   serialize them. */
fa_status fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* o,
                         const void* dO, const float* lse, void* dq, void* dk, void* dv, int B,
                         int H, int N, int d, float scale, int causal, const fa_mask* mask,
                         void* stream);

/* ---------------------------------------------------------------------------
 * Decoding over a key/value cache: rotary positions, a paged cache in bf16 or
 * 8-bit floating point, and attention of a few new tokens over it.
 * ------------------------------------------------------------------------- */

/* Rotary positions.  The first `dim` elements of a row are dim / 2 pairs; pair
 * p of a row at position n turns by the angle a = n freq[p]:
 *     (x, y) -> factor (x cos a - y sin a, x sin a + y cos a)
 * and the elements from `dim` on are copied.  Pairs are (p, p + dim/2), or
 * (2p, 2p + 1) with interleaved = 1.  Scaling for long contexts is in the
 * caller's freq (and factor).  The angle is reduced in 64-bit fixed-point
 * turns, so it keeps fp32 accuracy at any int32 position.
 *   freq : device double [dim/2], radians per position, 8-byte aligned, finite.
 *   pos  : device int32, position of token n of batch element b at
 *          pos[b*pos_stride + n] (pos_stride 0: the same for every b; any
 *          other value >= the tokens per element), 4-byte aligned.  NULL: the
 *          row index n (fa_cache_write: the cache row).  Negative positions
 *          turn backwards.
 *   dim  : a multiple of 16, 16..d (FA_ERR_UNSUPPORTED otherwise).
 *   factor : finite, not 0. */
typedef struct {
  const double* freq;
  const int32_t* pos;
  int64_t pos_stride;
  int dim;
  int interleaved;
  float factor;
} fa_rotary;

typedef struct {
  fa_layout q, k, q_out, k_out;
} fa_rope_layouts;

/* Rotates q [B,Hq,N,d] and k [B,Hk,N,d] (bf16; *_fp32: fp32) into q_out and
 * k_out in one launch.  k = k_out = NULL with Hk = 0 rotates q alone.  d is 64
 * or 128.  In place (q_out == q with the same layout, k likewise) is allowed.
 * layouts NULL: dense.  fa_rope_bwd maps the gradients of q_out and k_out to
 * those of q and k: the rotation by -a with the same factor.  Rotations are
 * computed in fp32 and rounded once. */
fa_status fa_rope(const void* q, const void* k, void* q_out, void* k_out, int B, int Hq, int Hk,
                  int N, int d, const fa_rotary* rotary, const fa_rope_layouts* layouts,
                  void* stream);
fa_status fa_rope_bwd(const void* dq_out, const void* dk_out, void* dq, void* dk, int B, int Hq,
                      int Hk, int N, int d, const fa_rotary* rotary,
                      const fa_rope_layouts* layouts, void* stream);
fa_status fa_rope_fp32(const float* q, const float* k, float* q_out, float* k_out, int B, int Hq,
                       int Hk, int N, int d, const fa_rotary* rotary,
                       const fa_rope_layouts* layouts, void* stream);
fa_status fa_rope_bwd_fp32(const float* dq_out, const float* dk_out, float* dq, float* dk, int B,
                           int Hq, int Hk, int N, int d, const fa_rotary* rotary,
                           const fa_rope_layouts* layouts, void* stream);

typedef enum {
  FA_CACHE_BF16 = 0, /* rows of d bf16                                          */
  FA_CACHE_E4M3 = 1  /* rows of d e4m3 values and one fp32 scale: x = value scale */
} fa_cache_format;

/* A key/value cache of `pages` pages of `page_size` rows for `heads` heads.
 * Row r of sequence b is row r % page_size of page block_table[b*table_stride
 * + r / page_size]; a sequence holds up to table_width * page_size rows.
 * Without a block table (NULL) sequence b owns page b, so pages >= B and a
 * sequence holds up to page_size rows.
 *   k, v    : [pages, heads, page_size, d] device, 16-byte aligned, both with
 *             `layout` (batch: page stride; the rules of fa_layout, 16 bytes =
 *             16 e4m3 elements; NULL: dense).
 *   k_scale, v_scale : E4M3: fp32 [pages, heads, page_size], rows contiguous,
 *             16-byte aligned; page and head strides in scale_layout (positive
 *             multiples of 4 elements; NULL: dense).  BF16: NULL.
 *   page_size : with a block table a power of two >= 16; without one >= 1 (a
 *             multiple of 4 for E4M3).
 *   pages below 2^31, pages * page_size * heads * d below 2^40.
 * A block-table entry outside [0, pages) is never followed: a row that needs
 * it is not written, and reads as zeros; fa_get_device_status then reports
 * FA_ERR_PAGE.  Pages may be shared by sequences that only read them; rows
 * that two tokens of one fa_cache_write name end up unspecified. */
typedef struct {
  int format; /* an fa_cache_format */
  int pages, page_size, heads, d;
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  const fa_layout* layout;
  const fa_layout* scale_layout; /* row is ignored */
  const int32_t* block_table;    /* device, 4-byte aligned */
  int table_width;
  int64_t table_stride; /* >= table_width */
} fa_cache;

/* Layouts of the dense-side tensors of a cache call (NULL: dense). */
typedef struct {
  fa_layout k, v;
} fa_cache_layouts;

/* Writes new rows: token t < q_len[b] of sequence b (k, v: [B,heads,T,d] bf16)
 * to cache row start[b] + t.  Tokens t >= q_len[b] are not read, and no other
 * row of the cache changes.  With `rotary`, k is rotated first (fp32, not
 * rounded in between); rotary->pos NULL means the cache row.
 * E4M3: scale = max over the row's finite |x| / 448, at least 2^-64, and the
 * value is x / scale (both fp32 quotients) rounded to nearest (ties to even); infinities become
 * +-448, NaN stays NaN.
 *   start, q_len : device int32 [B]; q_len NULL: T for every sequence.  q_len
 *   is clamped to 0..T; a row outside the sequence's capacity is not written,
 *   and reported like a bad page. */
fa_status fa_cache_write(const void* k, const void* v, const fa_cache* cache,
                         const int32_t* start, const int32_t* q_len, int B, int T,
                         const fa_rotary* rotary, const fa_cache_layouts* layouts, void* stream);

/* Reads rows back as bf16: row start[b] + n of sequence b to row n of k and v
 * ([B,heads,N,d]) for n < len[b].  Rows n >= len[b] of k and v are left as they
 * were.  start NULL: 0; len NULL: N (clamped to 0..N).  Rows outside the
 * sequence's capacity read as zeros and are reported like a bad page. */
fa_status fa_cache_read(const fa_cache* cache, const int32_t* start, const int32_t* len, void* k,
                        void* v, int B, int N, const fa_cache_layouts* layouts, void* stream);

/* Bytes of workspace fa_cache_fwd needs.  0 on bad sizes. */
size_t fa_cache_fwd_workspace_size(int B, int Hq, int Hkv, int T, int d);

/* Attention of new tokens over the cache: one token (T = 1), a chain, or a
 * tree of drafted tokens.  Token t < q_len[b] of sequence b, whose own rows
 * have already been written to cache rows start[b] .. start[b] + q_len[b] - 1,
 * sees
 *   - every row below start[b], and
 *   - row start[b] + u for u < q_len[b] where bit u % 32 of word
 *     tree_mask[(b*T + t)*W + u/32] is set, W = ceil(T/32); without a
 *     tree_mask, where u <= t.
 * Query head h reads cache head h / (Hq / heads).  O = softmax(scale q K^T) V
 * over the rows seen and lse as in fa_fwd; a token that sees nothing gets O = 0
 * and lse = -inf.  Rows t >= q_len[b] of o and lse are left as they were.  What
 * rows that a token does not see hold (infinities and NaN too) never reaches
 * its output; an infinity among the values that it does see makes it infinite or
 * NaN.
 *   q, o : [B,Hq,T,d] bf16 (lq, lo NULL: dense).   lse : fp32 [B,Hq,T].
 *   start, q_len : as in fa_cache_write; start is clamped to the capacity, and
 *   rows past it do not exist.
 *   workspace : device, >= fa_cache_fwd_workspace_size bytes, 16-byte aligned;
 *   contents on entry are ignored.  Calls that may run at the same time (on two
 *   streams, or two graphs) need one each.
 *   E4M3: scales are finite and not negative; value scales below 2^-64 may count as
 *   2^-64 (fa_cache_write leaves none).  Elements of q below 2^-13 of their row's largest
 *   are off by up to 2^-21 of that, larger ones are exact.  With G = Hq / heads and T*G
 *   <= 16 a weight is rounded by 2^-8 of itself, or by 2^-30 of the row's largest weight
 *   times value scale; with more, by 2^-11, or 2^-24 of that product, and a value by
 *   2^-10.
 * Limits: T <= 1024; Hq a multiple of cache->heads; B*Hq <= 65535; with G = Hq /
 * heads, B * heads * ceil(T*G / 32) * ceil(capacity / 128) below 2^31; with T*G > 32
 * (E4M3: 16) scores, scale q k, below 2^24 in magnitude. */
fa_status fa_cache_fwd(const void* q, const fa_cache* cache, const int32_t* start,
                       const int32_t* q_len, const uint32_t* tree_mask, void* o, float* lse,
                       void* workspace, size_t workspace_bytes, int B, int Hq, int T, float scale,
                       const fa_layout* lq, const fa_layout* lo, void* stream);

/* Human-readable name of a status code (static string, never NULL). */
const char* fa_status_string(fa_status s);

/* Text of the CUDA error behind the last FA_ERR_CUDA that a launching call
 * of the calling thread returned ("no CUDA error" if none).  Static string. */
const char* fa_last_cuda_error(void);

/* Synchronizes `stream`, then reports and clears the device-side status that
 * the kernels raise when a wait inside them gives up (FA_ERR_TIMEOUT) or a
 * cache call met a bad page or row (FA_ERR_PAGE), or
 * FA_ERR_CUDA if the stream reports an error.  FA_OK otherwise.  If site is
 * not NULL it receives the id of the wait that gave up. */
fa_status fa_get_device_status(void* stream, int* site);

/* Diagnostic: launches one CTA that waits on an mbarrier no one arrives on,
 * with the given limit (1..1000000 microseconds), exactly as the attention
 * kernels bound their waits.  The kernel returns normally; a following
 * fa_get_device_status reports FA_ERR_TIMEOUT.  Lets the failure path be
 * checked without hanging or faulting a GPU. */
fa_status fa_debug_wait_timeout(unsigned int limit_us, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_H_ */
