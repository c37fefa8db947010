/*
 * libmxqdq -- microscaling (MX) quantize / dequantize on AMD Instinct MI355X
 * (gfx950, CDNA4).  C ABI: plain pointers and sizes, no framework types.
 *
 * The operation (what each call computes):
 *   - A row-major [M x K] matrix is split along each row into contiguous
 *     groups of 32 elements; K must be a multiple of 32 ("use cute-dsl to
 *     speedup mxfp QDQ", Description: group size 32, K divisible by 32,
 *     contiguous input).
 *   - Each group gets one shared power-of-two scale from its abs-max
 *     ("[Transform] [Quantization] Add QuTLASS support to vLLM", Purpose:
 *     Abs-Max scheme), stored as an E8M0 byte b meaning 2^(b-127) (same page,
 *     review of vllm/_custom_ops.py: float8_e8m0fnu scale tensor).  Exponent
 *     rule (OCP MX v1.0; the pages do not print one): s = floor(log2 amax)
 *     - emax_elem, emax_elem = 2 for E2M1 and 8 for E4M3, clamped to
 *     [-127, 127]; an all-zero group gets s = -127 (byte 0).
 *   - Each element y becomes y * 2^-s rounded to nearest, ties to even, onto
 *     the FP4 E2M1 (MXFP4) or FP8 E4M3 (MXFP8) grid, saturating at 6 / 448.
 *     The sign of a result that rounds to zero is kept.
 *   - Optional rotation before the scale ("Add QuTLASS support to vLLM",
 *     Online rotations: transform + quantization + scale computation fused,
 *     matrix loaded at runtime, sizes 16/32/64/128): every r-element chunk x
 *     of a row (chunks start at column 0) is replaced by y = x . R, i.e.
 *     y[j] = sum_t x[t] * R[t][j], with R an r x r row-major matrix in the
 *     source dtype, accumulated in fp32.  bf16 sources multiply exactly (bf16
 *     matrix cores); fp32 sources run on the fp32 matrix cores, whose
 *     products are rounded once to fp32.  For a symmetric
 *     matrix such as the normalised Hadamard H * r^-0.5 the side does not
 *     matter.  QDQ then returns the dequantized rotated values (no inverse).
 *
 * Layouts:
 *   src, dst     [M x K] row-major, contiguous, 16-byte aligned.
 *   codes        E2M1: [M x K/2] bytes, column 2k in bits 3:0 and column
 *                2k+1 in bits 7:4; E4M3: [M x K] bytes.  16-byte aligned.
 *   scales       [M x K/32] bytes, row-major, unpadded (the non-swizzled
 *                [M, K/32] layout of the MXFP8 quantize on the FlashInfer
 *                cute-dsl digest page, key source excerpt).  4-byte aligned.
 *   rot          [r x r] row-major in the source dtype, 16-byte aligned.
 *
 * Ownership and execution: every pointer is device memory owned by the
 * caller.  The library allocates nothing, frees nothing and never
 * synchronizes; every call validates its arguments on the host, enqueues one
 * kernel (attention, verification and pages: up to three) on the calling thread's stream
 * (mx_set_stream) and returns.  Calls
 * are therefore safe to capture in a HIP graph.  dst == src (an exact alias)
 * is allowed for mx_qdq; any other overlap between inputs and outputs is
 * undefined.  Faults inside a kernel surface at the caller's next
 * synchronization, as for any HIP kernel.
 *
 * Errors: 0 on success, a negative MX_E* code otherwise; argument errors are
 * returned before anything is enqueued.  M == 0 or K == 0 is a successful
 * no-op.  There is no fallback path: unsupported arguments are errors.
 *
 * Non-finite input (outside every accuracy contract): a group holding NaN or
 * Inf gets scale byte 0xFF, E4M3 codes 0x7F (E2M1 codes 0x0), and
 * dequantized values NaN.  With a rotation the group is the rotated one, and
 * a NaN or Inf input reaches every output of the block the kernel rotates it
 * in (products with Inf and sums of opposite infinities give NaN, and so do
 * the zeros of a block-diagonal matrix): bf16 sources rotate blocks of
 * max(r, 64) elements when M*K is a multiple of 64 (for blocked scales:
 * when K is) and max(r, 32) otherwise, fp32 sources blocks of max(r, 32);
 * each group of such a block is non-finite.
 */
#ifndef LIBMXQDQ_H
#define LIBMXQDQ_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MX_API __attribute__((visibility("default")))

/* Element formats. */
#define MX_FMT_E2M1 0 /* MXFP4 */
#define MX_FMT_E4M3 1 /* MXFP8 */

/* Source / destination dtypes. */
#define MX_DTYPE_BF16 0
#define MX_DTYPE_F32 1

/* Status codes. */
#define MX_OK 0
#define MX_EFMT (-1)    /* fmt is not MX_FMT_E2M1 / MX_FMT_E4M3            */
#define MX_EDTYPE (-2)  /* dtype is not MX_DTYPE_BF16 / MX_DTYPE_F32        */
#define MX_ESHAPE (-3)  /* M < 0, K < 0, K % 32 != 0 (NVFP4: K % 16), or
                           M*K too large                                    */
#define MX_EROT (-4)    /* rot_size not in {0,16,32,64,128}, K % rot_size,
                           rot == NULL with rot_size > 0, or (NVFP4)
                           a rotation with K % 32 != 0                       */
#define MX_ENULL (-5)   /* a required pointer is NULL                       */
#define MX_EALIGN (-6)  /* a pointer breaks the alignment stated above      */
#define MX_ELAUNCH (-7) /* the kernel launch failed (hipGetLastError)       */
#define MX_ELAYOUT (-8) /* scale_layout is not one of MX_SCALES_*, or a
                           rotary layout not one of MX_ROTARY_*             */
#define MX_EARG (-9)    /* a rotary, cache, attention or verification argument
                           is outside the range stated at its call          */

/* Scale layouts. */
#define MX_SCALES_ROWMAJOR 0 /* [M x K/32] bytes, row-major, unpadded      */
#define MX_SCALES_BLOCKED 1  /* the blocked layout described below         */

/*
 * Fused quantize-dequantize ("use cute-dsl to speedup mxfp QDQ",
 * Description: mxfp4_qdq / mxfp8_qdq).
 *   fmt        MX_FMT_E2M1 or MX_FMT_E4M3.
 *   src        [M x K] in src_dtype (MX_DTYPE_BF16 or MX_DTYPE_F32).
 *   rot        NULL, or the r x r rotation in src_dtype; rot_size = r or 0.
 *   dst        [M x K] in src_dtype: code_value * 2^s, rounded to
 *              nearest-even into src_dtype (exact whenever representable).
 */
MX_API int mx_qdq(int fmt, const void *src, int src_dtype, int64_t M,
                  int64_t K, const void *rot, int rot_size, void *dst);

/*
 * Quantize a bf16 matrix to MX codes and E8M0 scales ("Add QuTLASS support
 * to vLLM", review of vllm/_custom_ops.py: fusedQuantizeMx returning the
 * E2M1 codes and E8M0 scales; FlashInfer cute-dsl digest page, key source
 * excerpt: MXFP8 quantize returning (x_q, x_scales)).
 *   src        [M x K] bf16.
 *   rot        NULL, or the r x r bf16 rotation; rot_size = r or 0.
 *   codes      [M x K/2] (E2M1, packed) or [M x K] (E4M3) bytes.
 *   scales     [M x K/32] E8M0 bytes.
 */
MX_API int mx_quantize(int fmt, const void *src, int64_t M, int64_t K,
                       const void *rot, int rot_size, uint8_t *codes,
                       uint8_t *scales);

/*
 * Dequantize codes + scales (the inverse used by the MXFP4 GEMM test on
 * "Add QuTLASS support to vLLM", review of the test file: a_dq / b_dq built
 * by a dequantize helper).  dst[i][k] = code_value * 2^(scale-127) rounded
 * to nearest-even into dst_dtype; a scale byte of 0xFF or an E4M3 NaN code
 * gives NaN.
 */
MX_API int mx_dequantize(int fmt, const uint8_t *codes, const uint8_t *scales,
                         int64_t M, int64_t K, int dst_dtype, void *dst);

/*
 * The rotation step alone: dst[M x K] (fp32) = per-chunk x . R with fp32
 * accumulation, exactly as the fused calls compute it before the scale.
 * Exposed so that the rotation's accuracy can be checked directly.
 */
MX_API int mx_rotate(const void *src, int src_dtype, int64_t M, int64_t K,
                     const void *rot, int rot_size, float *dst);

/*
 * Blocked scale layout: the E8M0 scales in the order the gfx950 scaled
 * matrix cores read them (32x32 tiles, 64-deep k-steps), so that a GEMM
 * fetches each lane's scales with one coalesced 32-bit load per 256-deep
 * k-span.  The pages pad and re-block the scale tensor for their GEMM
 * ("Add QuTLASS support to vLLM", review of vllm/_custom_ops.py and
 * vllm/qutlass_utils/utils.py: padded_rows x padded_cols, to_blocked;
 * FlashInfer cute-dsl digest page: is_sf_swizzled_layout) but define it
 * only for another GPU's matrix cores; this is the same idea for CDNA4.
 *   - Rows are padded to a multiple of 32 and the K/32 groups of a row to a
 *     multiple of 8.
 *   - The scales form 256-byte blocks of 32 rows x 8 groups, stored in
 *     row-major order over (row block, group block).
 *   - In a block, 32-bit word l (l = 0..63) holds row l%32 of the block
 *     and, in bytes 0..3, its groups h, 2+h, 4+h, 6+h (h = l/32).
 *   - Padding bytes are 127 (the scale 2^0).
 * mx_blocked_scales_bytes returns the size in bytes (MX_ESHAPE for a bad
 * shape); blocked buffers must be 4-byte aligned.
 */
MX_API int64_t mx_blocked_scales_bytes(int64_t M, int64_t K);

/* Re-blocks row-major [M x K/32] scales into the blocked layout (every byte
 * of the blocked buffer is written, padding included). */
MX_API int mx_scales_to_blocked(const uint8_t *scales, int64_t M, int64_t K,
                                uint8_t *blocked);

/* mx_quantize with the scales written directly in the blocked layout
 * (padding included); codes as for mx_quantize. */
MX_API int mx_quantize_blocked(int fmt, const void *src, int64_t M, int64_t K,
                               const void *rot, int rot_size, uint8_t *codes,
                               uint8_t *blocked_scales);

/*
 * MX GEMM: c[M x N] (row-major) = alpha * A_dq . B_dq^T, where A is [M x K]
 * and B is [N x K], both with codes in the layout mx_quantize writes
 * (K-contiguous: the "TN" operand order) and scales in scale_layout
 * (MX_SCALES_ROWMAJOR or MX_SCALES_BLOCKED, both operands alike), on the
 * CDNA4 scaled matrix cores.  Products of codes are exact, each product
 * carries the two scales of its groups, and accumulation is fp32; the
 * result is multiplied by alpha in fp32 and stored as out_dtype (bf16 by
 * nearest-even rounding, or fp32).  This is the consumer of the quantized
 * layout, with the call shape and check of the pages' MXFP4 GEMM ("Add
 * QuTLASS support to vLLM", Purpose: MXFP4 matmul kernel with alpha and
 * bf16 output; review of the MXFP4 test: compared with a_dq @ b_dq^T).
 *   codes      16-byte aligned; c 16-byte aligned; row-major scales any
 *              alignment, blocked scales 4-byte aligned.  Row-major
 *              scales load fastest when K/32 is a multiple of 16 and
 *              they are 16-byte aligned (MXFP4), next when K/32 is a
 *              multiple of 8 (MXFP4) or 4 (MXFP8) and they are 4-byte
 *              aligned; other shapes read them byte by byte (same
 *              results, slower).  Blocked scales are faster still: for a
 *              large product, re-blocking row-major scales first
 *              (mx_scales_to_blocked, or mx_quantize_blocked in place of
 *              mx_quantize) and passing MX_SCALES_BLOCKED costs less than
 *              the row-major read (on MI355X, 8192 x 8192 x 28672 MXFP4:
 *              about 6 us of re-blocking against 130 us saved).
 *   K == 0 stores zeros.  M <= 65535 * 128; K <= 2^24 (MXFP4) or 2^23
 *   (MXFP8), else MX_ESHAPE.
 *   A scale byte of 0xFF (NaN) or an E4M3 NaN code gives NaN in the
 *   affected outputs.
 */
MX_API int mx_matmul(int fmt, const uint8_t *a_codes, const uint8_t *a_scales,
                     const uint8_t *b_codes, const uint8_t *b_scales,
                     int scale_layout, int64_t M, int64_t N, int64_t K,
                     float alpha, int out_dtype, void *c);

/*
 * NVFP4: the second 4-bit format the pages name beside MXFP4, with the same
 * fused rotations ("Add QuTLASS support to vLLM", Purpose: NVFP4 and MXFP4;
 * review of benchmarks/kernels/bench_nvfp4_qutlass.py: fusedQuantizeNv(a,
 * rotation, global_scale), scales viewed as [-1, K/16]).  The pages give no
 * rule; the reading is the published two-level NVFP4 format: groups of 16
 * elements along K, one E4M3 block scale per group, E2M1 elements, and a
 * per-tensor fp32 multiplier g = *global_scale (positive and finite; e.g.
 * 448 * 6 / amax of the tensor).  The steps are fp32 operations, each
 * rounded to nearest-even, so that the codes are defined exactly:
 *   c6 = g / 6;  q = amax * c6 (amax: the group's abs-max);
 *   scale byte = E4M3(q), nearest-even, saturating at 448 (0x7E); q <= 2^-10
 *   gives 0;  m = g / value(scale), or 0 for a zero scale;
 *   code = E2M1(x * m), nearest-even, saturating at 6, sign kept;
 *   dequantized value = value(code) * (value(scale) / g), then nearest-even
 *   into the destination type.
 * With a rotation, x is the rotated value (fp32 accumulation), as for MX.
 *   src          [M x K] bf16, K % 16 == 0 (with a rotation also K % r == 0
 *                and K % 32 == 0), 16-byte aligned.
 *   codes        [M x K/2] bytes, column 2k in bits 3:0; 16-byte aligned.
 *   scales       [M x K/16] E4M3 bytes, row-major; 4-byte aligned.
 *   global_scale device pointer to one fp32, 4-byte aligned; read by the
 *                kernel (so it may be computed on the device).
 * Non-finite input, or g not positive and finite, is outside the contract.
 * mx_nvfp4_qdq writes dst [M x K] bf16 (16-byte aligned); dst == src (an
 * exact alias) is allowed there, as for mx_qdq.
 */
MX_API int mx_nvfp4_quantize(const void *src, int64_t M, int64_t K,
                             const void *rot, int rot_size,
                             const float *global_scale, uint8_t *codes,
                             uint8_t *scales);
MX_API int mx_nvfp4_qdq(const void *src, int64_t M, int64_t K,
                        const void *rot, int rot_size,
                        const float *global_scale, void *dst);
MX_API int mx_nvfp4_dequantize(const uint8_t *codes, const uint8_t *scales,
                               int64_t M, int64_t K,
                               const float *global_scale, int dst_dtype,
                               void *dst);

/*
 * Rotary positions.  On the first `rot` dimensions of every head, pair p of
 * rot/2 is turned by the angle positions[token] * inv_freq[p]:
 *   a' = a c - b s,  b' = b c + a s,  c, s = scale * cos, scale * sin;
 * the other dimensions are copied.  With inverse != 0 s is negated: the
 * transposed rotation, which takes the gradient of y to that of x.
 *   src, dst   [tokens x heads x dim] in dtype, dimensions contiguous; token
 *              and head strides in elements, so that a head range of a wider
 *              row can be passed.  dst == src is allowed with equal strides;
 *              any other overlap is undefined.  Any alignment; 16-byte
 *              pointers, strides and halves are fastest.
 *   positions  [tokens] int64; inv_freq [rot/2] fp64 (scaled for long contexts
 *              by the caller).  Angles are formed and reduced in fp64 (accurate
 *              below 2^50 rad) and rounded once to fp32.
 *   tokens     below 2^31, and with a rotation up to (2^24 - 1) times 4096 / rot
 *              (rounded down), what a launch holds (MX_ESHAPE); heads up to
 *              65535.
 *   rot        even, 0 <= rot <= dim <= 4096 (MX_EARG).
 *   layout     MX_ROTARY_HALF: pair p is dimensions p and p + rot/2;
 *              MX_ROTARY_INTERLEAVED: dimensions 2p and 2p + 1.
 */
#define MX_ROTARY_HALF 0
#define MX_ROTARY_INTERLEAVED 1

MX_API int mx_rope(const void *src, int64_t src_token_stride,
                   int64_t src_head_stride, int dtype, int64_t tokens,
                   int64_t heads, int64_t dim, const int64_t *positions,
                   const double *inv_freq, int64_t rot, int layout,
                   double scale, int inverse, void *dst,
                   int64_t dst_token_stride, int64_t dst_head_stride);

/*
 * mx_rope with several positions a token (time, height and width of an image
 * or video, say): pair p is turned by
 *   positions[axes[p] * axis_stride + token] * inv_freq[p].
 *   positions  [axis_count x tokens] int64, rows axis_stride elements apart.
 *   axis_count 1 or more (MX_EARG).
 *   axes       [rot/2] int32: the axis of each pair, in any order; the angle of
 *              a pair whose axis is outside 0 .. axis_count - 1 is zero.
 */
MX_API int mx_rope_axes(const void *src, int64_t src_token_stride,
                        int64_t src_head_stride, int dtype, int64_t tokens,
                        int64_t heads, int64_t dim, const int64_t *positions,
                        int64_t axis_stride, int64_t axis_count,
                        const int32_t *axes, const double *inv_freq,
                        int64_t rot, int layout, double scale, int inverse,
                        void *dst, int64_t dst_token_stride,
                        int64_t dst_head_stride);

/*
 * Paged MX cache of keys and values.  A plain description: the caller owns
 * the memory and may keep the struct where it likes (it is read during the
 * call only).
 *   page       tokens of a page: a power of two, 16 to 65536.
 *   dim        a multiple of 32, 32 to 256; pages * heads * page * dim <= 2^46.
 *   codes      [pages x heads x page x dim] bytes (E4M3) or
 *              [pages x heads x page x dim/2] (E2M1, the even dimension in
 *              bits 3:0); 16-byte aligned.
 *   scales     [pages x heads x dim/32 x page] E8M0 bytes, one for each 32
 *              dimensions of a token; 16-byte aligned.
 * Token slots are page number * page + row.
 */
typedef struct mx_cache {
  int32_t fmt, heads, page, dim;
  int64_t pages;
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
} mx_cache;

/*
 * Quantise new keys and values into their slots (the scale and element rules
 * of mx_quantize).  With rot > 0 the keys are rotated first (as by mx_rope, in
 * fp64) and rounded to bf16 (by way of fp32).
 *   k, v       [tokens x heads x dim] bf16, strides in elements as above.
 *   slots      [tokens] int64; a slot outside the cache (a negative one, say)
 *              is skipped.  Two tokens with one slot leave either's bytes.
 *   tokens     up to 2^27 - 8, what a launch holds (MX_ESHAPE).
 */
MX_API int mx_cache_write(const mx_cache *cache, const void *k,
                          int64_t k_token_stride, int64_t k_head_stride,
                          const void *v, int64_t v_token_stride,
                          int64_t v_head_stride, const int64_t *slots,
                          int64_t tokens, const int64_t *positions,
                          const double *inv_freq, int64_t rot, int layout,
                          double scale);

/* mx_cache_write with several positions a token, as for mx_rope_axes. */
MX_API int mx_cache_write_axes(const mx_cache *cache, const void *k,
                               int64_t k_token_stride, int64_t k_head_stride,
                               const void *v, int64_t v_token_stride,
                               int64_t v_head_stride, const int64_t *slots,
                               int64_t tokens, const int64_t *positions,
                               int64_t axis_stride, int64_t axis_count,
                               const int32_t *axes, const double *inv_freq,
                               int64_t rot, int layout, double scale);

/*
 * Read slots back: k, v [tokens x heads x dim] bf16, contiguous, 16-byte
 * aligned; values rounded to nearest-even.  A slot outside the cache gives
 * zeros.  tokens: up to 2^28 - 16 (MX_ESHAPE).
 */
MX_API int mx_cache_read(const mx_cache *cache, const int64_t *slots,
                         int64_t tokens, void *k, void *v);

/*
 * Attention over the cache: out[i] = softmax_j(scale * q[i] . k[j]) v[j].
 * Query head h reads key/value head h / (q_heads / cache->heads).
 * Sequence b has the queries q_starts[b] .. q_starts[b+1] - 1 and
 * kv_lens[b] tokens in the cache, of which its new ones (one for each query)
 * are the last; token t is in page block_table[b][t / page], row t % page.
 * A query sees every token before the new ones, and of these
 *   tree == NULL  the ones up to its own;
 *   otherwise     the ones whose bits are set in its row: new token j is bit
 *                 j % 64 of word j / 64 of tree[query * tree_words ..]
 *                 (64 * tree_words >= max_q, MX_EARG).
 * A query that sees nothing gives zeros; what it does not see has no part in
 * its result, NaN included.  Tokens of a page that is not in the cache count
 * as not seen.  A value above the range of bf16 (a large code with a scale of
 * 2^120 and more, which mx_cache_write does not produce) is an infinity of
 * its sign, in every row that sees it with a weight that is not too small for
 * fp32.
 *   q          [total_q x q_heads x dim] bf16, 16-byte aligned, strides (in
 *              elements) multiples of 8; out the same, contiguous.
 *   q_starts   [batch + 1] int32, ascending from 0; queries from q_starts[batch]
 *              on (padding) give zeros.  kv_lens [batch] int32;
 *              block_table [batch x table_stride] int32, of which the first
 *              table_pages of a row may be read; tree [total_q x tree_words].
 *   max_q, max_kv  at least the most queries and tokens of a sequence.  With
 *              less, a sequence's queries from max_q on are not computed (what
 *              their rows hold is undefined), and its tokens from max_kv on
 *              count as not seen; so do tokens behind the pages of table_pages.
 *              batch * q_heads * max_q is 2^32 at most (MX_ESHAPE).
 *   workspace  mx_cache_attention_workspace bytes, 16-byte aligned, contents
 *              free; it may be NULL where that is 0.
 * dim is 64, 96, 128, 192 or 256 and scale is positive, and finite also times
 * log2(e) (MX_EARG); scores, weights' sums and output sums are fp32, weights
 * are rounded to bf16 for their products with the values.  Weights are powers
 * of two of up to 2^8 before they are divided by their sum, so values times the
 * number of tokens should stay below 2^119.  Enqueues one kernel, or two where
 * the tokens are split over workgroups.  max_q chooses the kernel for the whole
 * batch: long chunks and many single tokens are quicker in two calls.
 */
MX_API int64_t mx_cache_attention_workspace(const mx_cache *cache,
                                            int64_t q_heads, int64_t batch,
                                            int64_t total_q, int64_t max_q,
                                            int64_t max_kv);
MX_API int mx_cache_attention(const mx_cache *cache, const void *q,
                              int64_t q_token_stride, int64_t q_head_stride,
                              int64_t q_heads, const int32_t *q_starts,
                              const int32_t *kv_lens, int64_t batch,
                              const int32_t *block_table, int64_t table_stride,
                              int64_t table_pages, int64_t total_q,
                              int64_t max_q, int64_t max_kv,
                              const int64_t *tree, int64_t tree_words,
                              float scale, void *out, void *workspace,
                              int64_t workspace_bytes);

/*
 * Attention to another sequence's tokens (an encoder's states, the tokens of
 * images): as mx_cache_attention, but every query of sequence b sees all of its
 * kv_lens[b] tokens, whatever the number of its queries.  It has a workspace size
 * of its own.
 */
MX_API int64_t mx_cache_cross_attention_workspace(const mx_cache *cache,
                                                  int64_t q_heads,
                                                  int64_t batch,
                                                  int64_t total_q,
                                                  int64_t max_q,
                                                  int64_t max_kv);
MX_API int mx_cache_cross_attention(const mx_cache *cache, const void *q,
                                    int64_t q_token_stride,
                                    int64_t q_head_stride, int64_t q_heads,
                                    const int32_t *q_starts,
                                    const int32_t *kv_lens, int64_t batch,
                                    const int32_t *block_table,
                                    int64_t table_stride, int64_t table_pages,
                                    int64_t total_q, int64_t max_q,
                                    int64_t max_kv, float scale, void *out,
                                    void *workspace, int64_t workspace_bytes);

/*
 * The cache's pages.  block_table is [rows x table_stride] int32, of which the
 * first table_pages of a row are used; an entry outside 0 .. pages - 1 is no
 * page.  refs [cache->pages] int32 counts the rows that hold each page; a page
 * is free where it is zero (one that is kept from being handed out starts with a
 * count of its own).  Free pages are handed out lowest first, in the order of rows
 * and columns, so that the same tables give the same pages.  The calls change
 * refs without a lock: those that share it follow one another on a stream.
 */

/*
 * Copy whole pages, keys and values: page src[i] to page dst[i], i < count
 * (int32; count up to 2^24 - 1, MX_ESHAPE).  Pairs with a page outside the cache,
 * or twice the same one, are skipped.  The pages of dst are distinct and no other
 * pair's source; the bytes of one that is are undefined.
 */
MX_API int mx_cache_copy(const mx_cache *cache, const int32_t *src,
                         const int32_t *dst, int64_t count);

/*
 * Row r of block_table holds the pages for kv_lens[r] tokens and no more:
 * pages behind them are released first, in all rows, and their entries become
 * -1; then entries without a page get free ones.  missing [rows] int32: the
 * pages that a row needs and did not get, because none was free or the row is
 * too short.  rows up to 2^24; 1024 of them (or all, if fewer) have less than
 * 2^31 entries (MX_ESHAPE).
 */
MX_API int mx_cache_resize(const mx_cache *cache, int32_t *refs,
                           int32_t *block_table, int64_t table_stride,
                           int64_t table_pages, const int32_t *kv_lens,
                           int64_t rows, int32_t *missing);

/*
 * Rows for sequences that go on from others: row c of child_table (columns and
 * meaning as block_table, no overlap with it) gets the full pages of row
 * parents[c], which both hold from then on, and, where the last page is not
 * full, a free page into which that page's tokens are copied (rows behind them
 * keep what they held, and so do all where the parent has no page there).  The
 * rest of the row is -1; so is all of it for a parent outside 0 .. rows - 1.
 * missing [children] int32: the pages that a child needs and does not hold.
 * children * cache->heads is below 2^23 (MX_ESHAPE).  Caches that share a table
 * and refs (the layers of a model) are forked in one call, with one of them; the
 * others copy the last pages with mx_cache_copy, from the parents' rows to the
 * children's.
 */
MX_API int mx_cache_fork(const mx_cache *cache, int32_t *refs,
                         const int32_t *block_table, int64_t table_stride,
                         int64_t table_pages, const int32_t *kv_lens,
                         int64_t rows, const int32_t *parents,
                         int64_t children, int32_t *child_table,
                         int64_t child_stride, int32_t *missing);

/*
 * Move the tokens that are kept of each sequence together, in place: place
 * kv_starts[b] + i gets what place kv_starts[b] + keep[b * keep_stride + i] held
 * before the call, for 0 <= i < min(counts[b], max_keep), where keep >= i (other
 * entries, and places without a page of the cache, are skipped).  A page that is
 * changed is held by one sequence of the batch.  kv_lens [batch] int32, not one
 * of the inputs, gets kv_starts + the count.  batch * cache->heads is below 2^20
 * (MX_ESHAPE).
 */
MX_API int mx_cache_compact(const mx_cache *cache, const int32_t *kv_starts,
                            const int32_t *keep, int64_t keep_stride,
                            int64_t max_keep, const int32_t *counts,
                            const int32_t *block_table, int64_t table_stride,
                            int64_t table_pages, int64_t batch,
                            int32_t *kv_lens);

/*
 * Verification of drafted tokens: what is kept of them, and the token sampled
 * after it, are distributed as the target's own.  Sequence b has the nodes
 * q_starts[b] .. q_starts[b+1] - 1 (int32 [batch + 1], ascending from 0): node 0
 * is its last settled token, the others are drafted, each a child of a node
 * before it.  From node c = 0 on, with w = target[c] and W = 1, the children of
 * c are asked in their order:
 *   child i with token x is kept if uniforms[i] * W * q(x) < w(x), then c = i;
 *   if not, w = max(w - W q, 0) and W = sum w, unless that would be zero
 * (q: draft[c], or 1 for x and 0 for all others if draft == NULL).  Behind the
 * last kept node a token is sampled from w: the first whose cumulative sum is
 * above uniforms[node 0] * sum w.  Computed in fp64; probabilities that are
 * negative or NaN count as zero, infinite ones as fp32's largest number; nodes
 * with tokens outside the vocabulary are passed over.
 *   target, draft  [total_q x vocab] in dtype, strides in elements: row c holds
 *              the probabilities after node c, and those that its children were
 *              drawn from, independently (siblings may have the same token).
 *              vocab 1 to 2^30 (MX_ESHAPE).
 *   tokens     [total_q] int64; uniforms [total_q] fp64 in [0, 1).
 *   batch      up to 2^22 - 1 (MX_ESHAPE).
 *   parents    [total_q] int32: a node's parent by its place in the sequence
 *              (nodes whose parent is not before them are passed over), or NULL:
 *              each node follows the one before.
 *   max_q      at least the most nodes of a sequence, 1024 at most (MX_ESHAPE);
 *              nodes from max_q on are passed over.
 *   counts     [batch] int32: nodes that stay, node 0 among them (0 for a
 *              sequence without nodes).
 *   path       [batch x max_q] int32: their places in the sequence, then -1.
 *   out        [batch x max_q] int64: the kept tokens and the sampled one, then
 *              -1; the sampled one is -1 if its row has no weight.
 *   workspace  mx_verify_workspace bytes, 16-byte aligned, contents free; it may
 *              be NULL where that is 0.
 */
MX_API int64_t mx_verify_workspace(int64_t batch, int64_t total_q,
                                   int64_t max_q, int64_t vocab);
MX_API int mx_verify(const void *target, int64_t target_stride,
                     const void *draft, int64_t draft_stride, int dtype,
                     int64_t vocab, const int64_t *tokens,
                     const double *uniforms, const int32_t *q_starts,
                     const int32_t *parents, int64_t batch, int64_t total_q,
                     int64_t max_q, int32_t *counts, int32_t *path,
                     int64_t *out, void *workspace, int64_t workspace_bytes);

/* Stream used by the calling thread's subsequent calls (a hipStream_t;
 * NULL = the default stream).  The setting is thread-local. */
MX_API void mx_set_stream(void *stream);
MX_API void *mx_get_stream(void);

/* Static, human-readable text for a status code. */
MX_API const char *mx_status_string(int status);

#ifdef __cplusplus
}
#endif
#endif
