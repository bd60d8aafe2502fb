/*
 * csa_compressor.h -- C ABI of the GB300 (sm_103a) CSA/HCA KV-compressor
 * gated-softmax pooling over THD-packed ragged sequences.
 *
 * The operation (pages "Megatron-LM PR #5984", commit "CSA: add fused Compressor
 * forward+backward CuTe-DSL kernels", and "cudnn-frontend PR #710"):
 *
 *   A pack holds S segments; segment s covers tokens [cu_seqlens[s], cu_seqlens[s+1]).
 *   A segment of length L has floor(L / ratio) blocks of ratio consecutive tokens,
 *   starting at the segment's first token; its last L mod ratio tokens belong to no
 *   block. Output rows are the blocks of all segments in order (total_comp rows).
 *   For block b of a segment and output column j < d, the window is:
 *     coff=1: the block's own ratio tokens at column j;
 *     coff=2: the previous block's ratio tokens at column j (absent for b = 0)
 *             followed by the block's own ratio tokens at column d + j.
 *   Each position adds ape[q, column read] to its score, q = the token's position in
 *   its own block. A float32 softmax over the window positions weights kv, and the
 *   weighted sum is rounded to bf16: out[row, j].
 *   The backward gives dKV = p * dout and dScore = p * dout * (kv - out) at every slot
 *   a window reads (out unrounded), +0 at every slot no window reads (the last
 *   block's first-half columns at coff=2, tails, segments shorter than ratio, rows
 *   outside [cu_seqlens[0], cu_seqlens[S])), and dAPE[q, col] = the sum of the
 *   unrounded dScore terms that used ape[q, col].
 *
 * Conventions common to every entry point
 *   - Every buffer belongs to the caller. The library allocates nothing, never
 *     synchronises, and never reads device memory from the host.
 *   - Work is enqueued on `stream` (NULL: the legacy default stream) of the current
 *     device; calls return as soon as it is enqueued. The kernels are launched as
 *     programmatic dependents of the stream's previous kernel: they may start while it
 *     finishes, but read and write nothing before it has completed, so stream order
 *     holds exactly as for ordinary launches (also inside CUDA graphs).
 *   - bf16 tensors are row-major and contiguous, fp32 tensors (ape, dape, workspace) too.
 *     Pointers need their natural alignment (2 bytes for bf16, 4 for fp32). The fast
 *     kernels run when d is a multiple of 8 and every pointer is 16-byte aligned; any
 *     other shape takes a scalar kernel, which accepts windows (coff * ratio) of up to
 *     CSA_MAX_GENERIC_WINDOW positions.
 *   - Host-side argument checks return a status and enqueue nothing. Problems that
 *     only the device can see (cu_seqlens decreasing, negative or past capacity;
 *     more blocks than out_rows) make the kernels write a code to *dev_error (when
 *     dev_error is not NULL), skip all output writes, and finish normally; outputs are
 *     then unspecified. The library never clears *dev_error.
 *   - Results are bitwise reproducible run to run (no atomics anywhere).
 */
#ifndef CSA_COMPRESSOR_H_
#define CSA_COMPRESSOR_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t. */
typedef struct CUstream_st* csa_stream_t;

typedef enum {
  CSA_OK = 0,
  CSA_ERR_INVALID_VALUE = 1, /* NULL pointer, negative size, misaligned pointer */
  CSA_ERR_UNSUPPORTED = 2,   /* coff not in {1,2}, size limits below */
  CSA_ERR_WORKSPACE = 3,     /* backward workspace NULL or smaller than the query's size */
  CSA_ERR_CUDA = 4           /* a CUDA runtime call or kernel launch failed */
} csa_status_t;

/* Codes the kernels write to *dev_error. */
#define CSA_DEVERR_CU_SEQLENS 1 /* cu_seqlens[0] < 0, decreasing, or cu_seqlens[S] > capacity */
#define CSA_DEVERR_OUT_ROWS 2   /* total_comp > out_rows */
#define CSA_DEVERR_TIMEOUT 3    /* a wait for an asynchronous copy gave up (about 2 s); the
                                   kernel stopped early, outputs (dAPE included) are
                                   incomplete */
#define CSA_DEVERR_LEAD 4       /* KPool: a negative lead */
#define CSA_DEVERR_SLOT 5       /* cache: a slot >= num_slots (that row alone is skipped) */
#define CSA_DEVERR_ENTRIES 6    /* cache attention: entries[s] < 0 or > max_pages * page_size */
#define CSA_DEVERR_PAGE 7       /* cache attention: a page number a sequence needs is outside
                                   [0, num_pages); its entries are not read */

/* Limits checked on the host (CSA_ERR_UNSUPPORTED beyond them). */
#define CSA_MAX_SEGMENTS 16384   /* S */
#define CSA_MAX_WINDOW 2048      /* coff * ratio */
#define CSA_MAX_GENERIC_WINDOW 256 /* coff * ratio when d % 8 != 0 or a pointer is not 16-byte aligned */
#define CSA_MAX_ELEMS 2147483647 /* capacity*coff*d and out_rows*d must stay below 2^31 */
#define CSA_KPOOL_MAX_POOL 1024  /* KPool pool size */
#define CSA_MAX_HEAD_DIM 1024    /* d of the head norm / rotation and of the cache attention */
#define CSA_CACHE_GROUP 32       /* columns that share a scale byte in the quantised cache formats */

/* Element types of csa_norm_rope_*, csa_cache_write and csa_cache_read. */
#define CSA_DTYPE_BF16 0
#define CSA_DTYPE_FP16 1
#define CSA_DTYPE_FP32 2

/* Frequency scaling of csa_rope_table. */
#define CSA_ROPE_PLAIN 0
#define CSA_ROPE_LINEAR 1
#define CSA_ROPE_YARN 2

/* Pairing of the rotated columns: column i with i + rot_dim/2, or 2i with 2i + 1. */
#define CSA_ROPE_HALF 0
#define CSA_ROPE_INTERLEAVED 1

/* Formats of the paged cache (see csa_cache_write). */
#define CSA_CACHE_BF16 0
#define CSA_CACHE_E4M3 1
#define CSA_CACHE_E2M1 2

/* Text for a status code (static storage). */
const char* csa_status_string(int status);

/* Text of the last CUDA runtime error a call of this library met on the calling host
 * thread (why a call returned CSA_ERR_CUDA); static storage. */
const char* csa_last_error_string(void);

/* total_comp = sum over s of floor((cu[s+1] - cu[s]) / ratio), from a HOST copy of
 * cu_seqlens [S+1]. Returns -1 when cu_seqlens is NULL, S < 0, ratio < 1 or the
 * offsets decrease. Definition: "Megatron-LM PR #5984", commit "fold dKV/dScore
 * zero-init into the backward kernel" (tails are seqlen mod ratio). */
int64_t csa_compressor_total_comp(const int32_t* cu_seqlens_host, int32_t S, int32_t ratio);

/* Forward pooling ("Megatron-LM PR #5984", commit "CSA: add fused Compressor
 * forward+backward CuTe-DSL kernels"; coff=1 per commit "widen the validated
 * envelope to coff in {1, 2}"; any ratio >= 1 per "cudnn-frontend PR #710").
 *   kv, score   bf16 [capacity, coff*d] (device)
 *   ape         fp32 [ratio, coff*d] (device)
 *   cu_seqlens  int32 [S+1] (device), non-decreasing, cu_seqlens[S] <= capacity
 *   out         bf16 [out_rows, d] (device); rows >= total_comp are not written
 *   dev_error   int32 (device) or NULL
 * S = 0 or out_rows = 0 with no block is a valid no-op. */
csa_status_t csa_compressor_fwd(const void* kv, const void* score, const float* ape,
                                const int32_t* cu_seqlens, int32_t S, int32_t ratio,
                                int32_t coff, int32_t d, int64_t capacity, void* out,
                                int64_t out_rows, int32_t* dev_error, csa_stream_t stream);

/* Bytes of device workspace csa_compressor_bwd needs for these sizes on the current
 * device: per-row-group dAPE partial sums (reduced in a fixed order) and a 16-byte status
 * block through which the pooling kernel tells the reduction whether the call's
 * cu_seqlens were valid. 0 on bad sizes. */
size_t csa_compressor_bwd_workspace_bytes(int32_t S, int32_t ratio, int32_t coff, int32_t d,
                                          int64_t capacity, int64_t out_rows);

/* Backward pooling ("Megatron-LM PR #5984", commits "CSA: add fused Compressor
 * forward+backward CuTe-DSL kernels" and "fold dKV/dScore zero-init into the
 * backward kernel"). Inputs as for the forward, plus
 *   dout        bf16 [out_rows, d] (device); rows >= total_comp are not read
 *   dkv, dscore bf16 [capacity, coff*d] (device): EVERY element is written
 *   dape        fp32 [ratio, coff*d] (device): accumulate_dape = 0 stores the sum,
 *               1 adds it to the current contents; left untouched when the device
 *               rejects cu_seqlens or out_rows
 *   workspace   device scratch of at least csa_compressor_bwd_workspace_bytes(...)
 *               bytes (CSA_ERR_WORKSPACE otherwise), 16-byte aligned for the vector
 *               kernels; contents on entry do not matter
 * Two kernels are enqueued: the pooling backward and a fixed-order dAPE reduction. */
csa_status_t csa_compressor_bwd(const void* kv, const void* score, const float* ape,
                                const int32_t* cu_seqlens, const void* dout, int32_t S,
                                int32_t ratio, int32_t coff, int32_t d, int64_t capacity,
                                int64_t out_rows, void* dkv, void* dscore, float* dape,
                                int32_t accumulate_dape, void* workspace, size_t workspace_bytes,
                                int32_t* dev_error, csa_stream_t stream);

/* Size of the device scratch array csa_compressor_bwd_noalloc uses (4 MiB per GPU). */
#define CSA_NOALLOC_SCRATCH_BYTES (4 << 20)

/* Backward pooling for callers that cannot allocate device memory when they run it --
 * for example code running inside an allocator or memory-pool callback (allocating there
 * would re-enter the allocator), or a plugin in a host that reserves all device memory up
 * front. The pages describe no such entry point; it is this library's addition. Same
 * arguments and results as csa_compressor_bwd, without the workspace: the dAPE partial
 * sums go to a file-scope device array of CSA_NOALLOC_SCRATCH_BYTES bytes that every GPU
 * loading the library holds until the process unloads it. Nothing is allocated.
 *   - Sizes whose workspace (csa_compressor_bwd_workspace_bytes) exceeds
 *     CSA_NOALLOC_SCRATCH_BYTES are rejected with CSA_ERR_UNSUPPORTED, enqueueing nothing.
 *   - The first call on a device (that device current) looks up the array's device
 *     address once; make that first call before any stream capture.
 *   - All calls on a device share the array, which keeps the last call's contents
 *     (nothing in it needs to start at zero). Calls whose GPU work overlaps -- on
 *     different streams or host threads of the same device -- race on it: order them. */
csa_status_t csa_compressor_bwd_noalloc(const void* kv, const void* score, const float* ape,
                                        const int32_t* cu_seqlens, const void* dout, int32_t S,
                                        int32_t ratio, int32_t coff, int32_t d, int64_t capacity,
                                        int64_t out_rows, void* dkv, void* dscore, float* dape,
                                        int32_t accumulate_dape, int32_t* dev_error,
                                        csa_stream_t stream);

/* Smallest non-zero wait bound csa_compressor_test_hooks accepts, in SM clock cycles. */
#define CSA_TEST_MIN_WAIT_CYCLES 1000000

/* Test hook for the bounded waits: lets a test make a pipeline wait run out without any
 * fault. The pages have no counterpart; it is this library's own.
 *   wait_cycles   bound of every later pooling or cache attention launch's pipeline waits,
 *                 in SM clock cycles (CSA_TEST_MIN_WAIT_CYCLES .. about 2 s); 0 restores the
 *                 default of about 2 s
 *   withhold_row  >= 0: in every later launch of a bulk-copy kernel (the block-streaming
 *                 and long-window kernels), the producer of CTA (0, 0) skips the copies
 *                 of row `withhold_row` of its row range, so the waits for that stage run
 *                 out, the kernel writes CSA_DEVERR_TIMEOUT to *dev_error, lets its own
 *                 copies land and returns; in every later launch of the cache attention's
 *                 tensor-core kernel, the first CTA never fills the place of tile
 *                 `withhold_row` (128 entries) of its first unit, with the same outcome; < 0:
 *                 off (the default)
 * Process-wide; applies to calls made after it returns, from any host thread.
 * CSA_ERR_INVALID_VALUE for a bound outside the range above. */
csa_status_t csa_compressor_test_hooks(int64_t wait_cycles, int32_t withhold_row);

/* Index map only (the THD segment/block mapping the pooling kernels use), for
 * checking it bit for bit: for every output row o < out_rows writes
 * seg_blk_base[3*o .. 3*o+2] = {segment, block inside the segment, first token of the
 * block}, or {-1, -1, -1} when o >= total_comp. seg_blk_base: int32 [out_rows, 3],
 * device. Reads cu_seqlens on the device like the pooling kernels. */
csa_status_t csa_compressor_map_blocks(const int32_t* cu_seqlens, int32_t S, int32_t ratio,
                                       int64_t capacity, int64_t out_rows, int32_t* seg_blk_base,
                                       int32_t* dev_error, csa_stream_t stream);

/* ------------------------------------------------------------------------------------
 * KPool: the DSA indexer's key pooling ("Megatron-LM PR #8835", the KPool commits: the
 * one adding dsa_indexer_kpool_key_dtype_compression and the explicit-mask pool origin,
 * and the one with the empty-query guard; KPool selection is NVIDIA#8287 there).
 *
 *   Segment s covers keys [cu_seqlens[s], cu_seqlens[s+1]); its first valid key is
 *   f = cu_seqlens[s] + lead[s] (lead NULL: 0). Its keys from f on are grouped into
 *   pools of `pool` consecutive keys, the grid restarting at every segment; the
 *   fewer-than-pool keys after its last complete pool form no pool (tail selection, which
 *   appends them individually, is part of the selection, not of this pooling). Output
 *   rows are the pools of all segments in order (csa_kpool_total rows).
 *   For a pool and column j < d: an FP32 softmax of gate[t, j] over the pool's keys t
 *   weights key[t, j]:
 *     compress = 0: out = bf16(sum_t p_t key[t, j]), the sum in fp32;
 *     compress = 1 (key-dtype compression): each weight is cast to bf16 before
 *       multiplying and reducing: out = bf16(sum_t bf16(bf16(p_t) * key[t, j])), the sum
 *       of the bf16 products in fp32.
 *   Forward only: the selection that consumes the pooled keys records no gradient.
 * ------------------------------------------------------------------------------------ */

/* Number of pools: sum over s of floor(max(0, cu[s+1] - cu[s] - lead[s]) / pool), from
 * HOST copies of cu_seqlens [S+1] and lead [S] (lead may be NULL). Returns -1 when
 * cu_seqlens is NULL, S < 0, pool < 1, the offsets decrease or a lead is negative. */
int64_t csa_kpool_total(const int32_t* cu_seqlens_host, const int32_t* lead_host, int32_t S,
                        int32_t pool);

/* KPool forward.
 *   key, gate   bf16 [capacity, d] (device)
 *   cu_seqlens  int32 [S+1] (device), non-decreasing, cu_seqlens[S] <= capacity
 *   lead        int32 [S] (device), >= 0, or NULL (every segment starts at cu_seqlens[s];
 *               a lead at or past the segment's end leaves it without pools)
 *   pool        1 .. CSA_KPOOL_MAX_POOL
 *   out         bf16 [out_rows, d] (device); rows >= the pool count are not written
 *   compress    0 or 1 (see above)
 *   dev_error   int32 (device) or NULL: CSA_DEVERR_CU_SEQLENS, CSA_DEVERR_LEAD or
 *               CSA_DEVERR_OUT_ROWS (more pools than out_rows); nothing is written then
 * The vector kernel runs when d is a multiple of 8, pool <= 8 and key, gate and out are
 * 16-byte aligned; anything else takes a scalar kernel. One kernel is enqueued (none when
 * S = 0). Status codes as for the compressor. */
csa_status_t csa_kpool_fwd(const void* key, const void* gate, const int32_t* cu_seqlens,
                           const int32_t* lead, int32_t S, int32_t pool, int32_t d,
                           int64_t capacity, void* out, int64_t out_rows, int32_t compress,
                           int32_t* dev_error, csa_stream_t stream);

/* ------------------------------------------------------------------------------------
 * Head norm and rotation: what queries and pooled entries go through before attention.
 *
 *   x is [rows, heads, d]; element (r, h, c) lies at x[r*x_row_stride + h*x_head_stride + c]
 *   (strides in elements, the columns contiguous). For every row and head:
 *     norm = 1:  n = x * rsqrt(mean over the d columns of x^2 + eps) * weight   (weight NULL: 1)
 *     norm = 0:  n = x
 *   then the rot_dim columns from rot_start on are turned in pairs (a, b), pair i by the
 *   angle t = 2 pi * (positions[r] * turns[i] mod 2^64) / 2^64:
 *     a' = amplitude * (a cos t - b sin t),   b' = amplitude * (a sin t + b cos t).
 *   The product is exact integer arithmetic, so a position near 2^31 turns as exactly as
 *   a small one. The columns outside the rotated part keep n. All arithmetic is in fp32
 *   (cos and sin within 1e-6 for 16-bit types, which round by 2^-12 or more), rounded once.
 *   A row whose position is negative is left out: its y (or dx) stays as it was, and it
 *   adds nothing to dweight. So a padded pack needs no row count on the host.
 * ------------------------------------------------------------------------------------ */

/* Frequencies of the rotation, on the host: turns_host[i], i < rot_dim/2, is
 * round(2^64 * f_i / (2 pi)), the part of a full turn that one position turns pair i by.
 *   CSA_ROPE_PLAIN   f_i = base^(-2i/rot_dim)
 *   CSA_ROPE_LINEAR  f_i / factor (position interpolation)
 *   CSA_ROPE_YARN    (f_i / factor) m_i + f_i (1 - m_i), m_i = clamp((i - lo)/(hi - lo), 0, 1),
 *                    lo = floor, hi = ceil of rot_dim ln(original_length / (2 pi b)) / (2 ln base)
 *                    at b = beta_fast and b = beta_slow, clamped to [0, rot_dim - 1]
 *                    (hi - lo at least 0.001); *amplitude = 0.1 ln(factor) + 1
 * *amplitude (may be NULL) is 1 for the other two. factor, original_length and the betas are
 * read only by the scalings that use them. CSA_ERR_INVALID_VALUE for an odd or negative
 * rot_dim, base <= 1, factor < 1, original_length < 1 or betas that are not positive;
 * CSA_ERR_UNSUPPORTED for rot_dim > CSA_MAX_HEAD_DIM or an unknown scaling. */
csa_status_t csa_rope_table(int32_t rot_dim, double base, int32_t scaling, double factor,
                            double original_length, double beta_fast, double beta_slow,
                            uint64_t* turns_host, float* amplitude);

/* Head norm and rotation, forward.
 *   x, y        dtype [rows, heads, d] with their strides (device); y may be x itself with
 *               the same strides, and overlaps it in no other way
 *   weight      fp32 [d] (device) or NULL; must be NULL when norm = 0
 *   positions   int32 [rows] (device); NULL: every row is taken, needs rot_dim = 0
 *   turns       uint64 [rot_dim/2] (device), from csa_rope_table; NULL when rot_dim = 0
 * rows = 0 is a valid no-op. CSA_ERR_INVALID_VALUE for NULL or misaligned pointers, odd
 * rot_dim, rot_start + rot_dim > d, negative strides, strides of y under which two elements
 * share a place (an input may repeat: a stride of 0), eps negative or not finite;
 * CSA_ERR_UNSUPPORTED for d > CSA_MAX_HEAD_DIM, rows * heads >= 2^31 or an unknown dtype or
 * layout. The vector kernel runs when d, the strides and rot_start are multiples of 8
 * and rot_dim of 16 (half) or 8 (interleaved), and x and y (weight too) are 16-byte
 * aligned; anything else takes a scalar kernel. */
csa_status_t csa_norm_rope_fwd(const void* x, int32_t dtype, int64_t rows, int32_t heads,
                               int32_t d, int64_t x_row_stride, int64_t x_head_stride,
                               const float* weight, int32_t norm, float eps,
                               const int32_t* positions, const uint64_t* turns, int32_t rot_dim,
                               int32_t rot_start, int32_t layout, float amplitude, void* y,
                               int64_t y_row_stride, int64_t y_head_stride, csa_stream_t stream);

/* Bytes of device workspace csa_norm_rope_bwd needs for these sizes on the current device
 * when dweight is asked for (per-block dweight sums, reduced in a fixed order); 0 on bad
 * sizes. */
size_t csa_norm_rope_bwd_workspace_bytes(int64_t rows, int32_t heads, int32_t d);

/* Gradients of csa_norm_rope_fwd from its input x (the statistics are recomputed).
 *   dy, dx      dtype [rows, heads, d] with their strides; dx may be dy or x itself with the
 *               same strides, and overlaps neither in another way
 *   x           not read (may be NULL) when norm = 0
 *   dweight     fp32 [d] or NULL (not wanted; must be NULL when norm = 0): the sum over rows
 *               and heads of dn * x * rsqrt(...), dn the gradient turned back;
 *               accumulate_dweight = 0 stores it, 1 adds it to the current contents. It may be
 *               asked for with weight NULL (the gradient at a weight of ones).
 *   workspace   csa_norm_rope_bwd_workspace_bytes(...) bytes, 16-byte aligned, when dweight
 *               is asked for (CSA_ERR_WORKSPACE otherwise); calls that may run at the same time
 *               need workspaces of their own
 * dweight is bitwise reproducible (no atomics). Other arguments as for the forward. */
csa_status_t csa_norm_rope_bwd(const void* x, const void* dy, int32_t dtype, int64_t rows,
                               int32_t heads, int32_t d, int64_t x_row_stride,
                               int64_t x_head_stride, int64_t dy_row_stride,
                               int64_t dy_head_stride, const float* weight, int32_t norm, float eps,
                               const int32_t* positions, const uint64_t* turns, int32_t rot_dim,
                               int32_t rot_start, int32_t layout, float amplitude, void* dx,
                               int64_t dx_row_stride, int64_t dx_head_stride, float* dweight,
                               int32_t accumulate_dweight, void* workspace, size_t workspace_bytes,
                               csa_stream_t stream);

/* ------------------------------------------------------------------------------------
 * Paged cache of entries. A pool of num_pages pages of page_size entries each; slot
 * page * page_size + offset holds one entry of `heads` heads of d columns:
 *   CSA_CACHE_BF16   data bf16 [slots, heads, d]; scales unused (NULL)
 *   CSA_CACHE_E4M3   data e4m3 [slots, heads, d], scales uint8 [slots, heads, d/32]
 *   CSA_CACHE_E2M1   data [slots, heads, d/2] bytes, column 2j in a byte's low four bits and
 *                    2j + 1 in its high ones, scales uint8 [slots, heads, d/32]
 * A scale byte k stands for 2^(k - 127) and belongs to 32 consecutive columns; a value is
 * code * scale. Writing picks the smallest scale (from 2^-127 on) at which the group's
 * largest magnitude does not exceed the format's largest value (448; 6), so nothing
 * saturates, and rounds value / scale to the nearest code, ties to the even one. A group
 * that holds an infinity or NaN gets scale byte 255 and reads back as NaN.
 * ------------------------------------------------------------------------------------ */

/* Writes rows into the cache.
 *   x           dtype [rows, heads, d] with row and head strides in elements (device)
 *   slots       int64 [rows] (device): where each row goes; a negative one leaves its row
 *               out; the others must differ from one another within a call (the contents of a
 *               slot that two rows name are unspecified). slots >= num_slots: the row is left
 *               out and CSA_DEVERR_SLOT reported
 *   data, scales   the pool as above; every other slot stays as it was
 * d must be a multiple of 32 for the quantised formats (CSA_ERR_UNSUPPORTED). The vector
 * kernel runs when x, data (and d and the strides in multiples of 8 elements) are 16-byte
 * aligned; anything else takes a scalar kernel. */
csa_status_t csa_cache_write(const void* x, int32_t dtype, int64_t rows, int32_t heads, int32_t d,
                             int64_t x_row_stride, int64_t x_head_stride, const int64_t* slots,
                             int64_t num_slots, int32_t format, void* data, uint8_t* scales,
                             int32_t* dev_error, csa_stream_t stream);

/* Reads rows of the cache back: out[r] = the entry in slots[r], in `dtype`, out [rows, heads,
 * d] with strides in elements that give every element a place of its own. A negative slot
 * leaves its row of out as it was, so does one >= num_slots, which reports CSA_DEVERR_SLOT. Any
 * slot may be read by several rows. */
csa_status_t csa_cache_read(const void* data, const uint8_t* scales, int32_t format,
                            const int64_t* slots, int64_t rows, int64_t num_slots, int32_t heads,
                            int32_t d, void* out, int32_t dtype, int64_t out_row_stride,
                            int64_t out_head_stride, int32_t* dev_error, csa_stream_t stream);

/* ------------------------------------------------------------------------------------
 * Attention of new tokens over the paged cache; an entry is key and value at once, as the
 * compressor's pooled kv is.
 *
 *   Sequence s has the new tokens [cu_seqlens[s], cu_seqlens[s+1]) and entries[s] entries;
 *   entry e lies in page page_table[s*max_pages + e / page_size] at offset e % page_size.
 *   Its token i stands at position p = first[s] + i (first NULL: 0) and sees the entries
 *   e < entries[s] with (e + 1) * ratio <= p + 1, those whose block of `ratio` tokens is
 *   complete by then (ratio 1: causal attention to single tokens); ratio 0: all of them.
 *   Query head h reads the entries' head h / (q_heads / kv_heads):
 *     out = sum_e w_e k_e,  w_e = exp(softmax_scale q.k_e) / (sum over seen entries + exp(sink[h]))
 *     lse = log(that denominator)
 *   (sink NULL: no such term, nor at a sink of -inf; one of +inf takes all the weight). A token that sees nothing gets out = 0 and lse = sink[h], or
 *   -inf without a sink. An entry that holds an infinity or NaN makes out and lse NaN for the tokens
 *   that see it (all columns of the heads that read it), and reaches no other token. A score of +inf
 *   or NaN does the same to its row; one of -inf (finite values past fp32) weighs nothing.
 *   Scores, maxima and sums are fp32; the weights are rounded to bf16 before the second
 *   product on the tensor cores (off by at most 2^-8 of each, as the outputs themselves are).
 * ------------------------------------------------------------------------------------ */

/* Bytes of device workspace csa_cache_attn needs on the current device; 0 on bad sizes.
 * max_entries = max_pages * page_size of the call. */
size_t csa_cache_attn_workspace_bytes(int32_t S, int64_t tokens, int32_t q_heads, int32_t kv_heads,
                                      int32_t d, int64_t max_entries);

/*   q           bf16 [tokens, q_heads, d], row and head strides in elements (device)
 *   cu_seqlens  int32 [S+1] (device), non-decreasing, cu_seqlens[S] <= tokens; rows of out and
 *               lse that belong to no sequence stay as they were
 *   data, scales, format   the cache of num_pages * page_size slots, kv_heads heads of d
 *   page_table  int32 [S, max_pages] (device); only the pages that entries[s] needs are read
 *   entries     int32 [S] (device), first int32 [S] (device) or NULL
 *   sink        fp32 [q_heads] (device) or NULL
 *   out         bf16 [tokens, q_heads, d], row and head strides in elements
 *   lse         fp32 [tokens, q_heads], contiguous, or NULL
 *   workspace   at least csa_cache_attn_workspace_bytes(...) bytes, 16-byte aligned
 *               (CSA_ERR_WORKSPACE otherwise); calls that may run at the same time need
 *               workspaces of their own
 * out and lse overlap no input. CSA_ERR_INVALID_VALUE: NULL or misaligned pointers, q_heads not a
 * multiple of kv_heads, negative sizes or strides, strides of out under which two elements share
 * a place, softmax_scale not finite. CSA_ERR_UNSUPPORTED: d >
 * CSA_MAX_HEAD_DIM, quantised formats with d not a multiple of 32, S > CSA_MAX_SEGMENTS,
 * tokens * q_heads >= 2^31 - 256, max_pages * page_size >= 2^31, an unknown format. A bad
 * cu_seqlens or entries (CSA_DEVERR_CU_SEQLENS, CSA_DEVERR_ENTRIES) skips all outputs; after
 * CSA_DEVERR_PAGE the outputs of that sequence are unspecified. Results are bitwise
 * reproducible for the same arguments on the same device. The tensor-core kernel runs when
 * d <= 512, d and the strides of q and out are multiples of 8, and q, out and data 16-byte
 * aligned; anything else takes a scalar kernel, many times slower (with many rows, slower than
 * ordinary matrix products would be). With many new tokens a sequence the workspace has room
 * for the sequences' entries as bf16 rows of 128, 256 or 512 columns (up to 4 GiB, of max_entries
 * each), whether the format and the pages come to use it or not. "Many" is the average of
 * `tokens` over S: where a few long chunks come with many single tokens, or `tokens` is far above
 * cu_seqlens[S], a call for each kind, or with the tokens there are, is faster. A wait that runs out reports CSA_DEVERR_TIMEOUT
 * and leaves the outputs unspecified. */
csa_status_t csa_cache_attn(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                            const int32_t* cu_seqlens, int32_t S, int64_t tokens, int32_t q_heads,
                            int32_t kv_heads, int32_t d, const void* data, const uint8_t* scales,
                            int32_t format, const int32_t* page_table, int32_t max_pages,
                            int64_t num_pages, int32_t page_size, const int32_t* entries,
                            const int32_t* first, int32_t ratio, float softmax_scale,
                            const float* sink, void* out, int64_t out_row_stride,
                            int64_t out_head_stride, float* lse, void* workspace,
                            size_t workspace_bytes, int32_t* dev_error, csa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CSA_COMPRESSOR_H_ */
