/*
 * dsa.h: C ABI of libdsa.so, the GB300 (sm_103a) hot path of DeepSeek Sparse
 * Attention (DSA).
 *
 * The method (release summary "DeepSeek-V3.2-Exp: Boosting Long-Context
 * Efficiency with DeepSeek Sparse Attention", section "Method"; AMD article
 * "AMD Instinct MI355X GPUs Power DeepSeek-V3.2-Exp", section "DeepSeek Sparse
 * Attention (DSA)") has three stages, one entry point each, plus the paged
 * decode form of the attention stage:
 *   1. lightning indexer   I[t,s] = sum_j w[t,j] * ReLU(q[t,j] . k[s]), in FP8
 *   2. top-k selection     the k (= 2048) highest-scoring prior tokens per query
 *   3. sparse MLA          MQA-mode attention over only the selected latent rows
 *
 * Conventions shared by every entry point
 *   - Every pointer named as a tensor is a DEVICE pointer; shapes are row-major
 *     and contiguous unless a leading dimension is given.  The caller owns every
 *     buffer; the library allocates nothing, frees nothing and keeps no pointer
 *     after a call returns.
 *   - Work is enqueued asynchronously on `stream` (0 = legacy default stream).
 *     Nothing synchronises inside the library and nothing falls back to the
 *     host.
 *   - Arguments are checked on the host before any launch.  On error the call
 *     returns a non-zero dsa_status, launches nothing, leaves outputs untouched
 *     and records a message for dsa_last_error().
 *   - Data-dependent problems that only the device can see (a bad page id, a
 *     position past the buffer, a pipeline wait that ran out of time) never
 *     cause an out-of-bounds access: the kernel skips the offending element and
 *     sets a bit in a per-device status word, read with dsa_get_device_status().
 *   - "FP8" is E4M3 (OCP "fn" variant, max 448), passed as raw bytes.  "bf16" is
 *     IEEE binary32 truncated to its upper 16 bits, passed as raw uint16.
 */
#ifndef DSA_H
#define DSA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *dsa_stream_t; /* same type as cudaStream_t */

typedef enum {
    DSA_OK = 0,
    DSA_ERR_INVALID_ARG = 1, /* null pointer, negative size, inconsistent shapes   */
    DSA_ERR_UNSUPPORTED = 2, /* a size the library has no kernel for (see below)   */
    DSA_ERR_ALIGNMENT = 3,   /* a pointer or stride breaks a 16-byte TMA rule       */
    DSA_ERR_WORKSPACE = 4,   /* workspace missing or smaller than the query says    */
    DSA_ERR_CUDA = 5,        /* a CUDA runtime/driver call or a launch failed       */
    DSA_ERR_DEVICE = 6       /* dsa_get_device_status() found a device-side error   */
} dsa_status;

/* Bits of the device status word (dsa_get_device_status). */
#define DSA_DEV_TIMEOUT      0x1u /* a bounded pipeline wait gave up; outputs of that CTA are invalid */
#define DSA_DEV_BAD_POSITION 0x2u /* a query position / valid length exceeded the key range or ld     */
#define DSA_DEV_BAD_PAGE     0x4u /* a block-table entry outside [0, num_pages); those keys skipped    */

/* Message for the last failing call on this host thread ("" if none). */
const char *dsa_last_error(void);

/* Library version, major * 10000 + minor * 100 + patch. */
int dsa_version(void);

/*
 * dsa_get_device_status: copy the device status word of the current device to
 * *status_out (DSA_DEV_* bits, 0 = clean) and clear it.  Enqueued on `stream`
 * and then waits for that stream, so it sees every earlier kernel on it.
 * Returns DSA_ERR_CUDA if the copy fails.
 */
int dsa_get_device_status(dsa_stream_t stream, uint32_t *status_out);

/*
 * dsa_selftest_wait_timeout: exercises the failure detection that every
 * kernel's pipeline waits share (the pages have no counterpart).  Launches
 * one CTA that waits, through the same bounded mbarrier wait, on a barrier
 * nothing arrives on; after limit_us microseconds (1 .. 1000000) the wait
 * gives up, sets DSA_DEV_TIMEOUT in the device status word and the kernel
 * returns, leaving the context usable.  Read the bit with
 * dsa_get_device_status().  Nothing faults, traps or hangs.
 */
int dsa_selftest_wait_timeout(uint32_t limit_us, dsa_stream_t stream);

/*
 * dsa_indexer_logits: lightning-indexer scores (stage 1).
 *
 * Defines, for each query row r at absolute position p = q_pos[r] and each key
 * position s in [0, p]:
 *     logits[r*ld_logits + s] = sum_{j<H_I} w[r,j] * ReLU( sum_{d<d_I}
 *                               (q8[r,j,d]*q_scale[r]) * (k8[s,d]*k_scale[s]) )
 * ("DeepSeek-V3.2-Exp: Boosting Long-Context Efficiency with DeepSeek Sparse
 * Attention", section "Method": index score against all prior tokens, ReLU,
 * FP8, few heads).  The query's own position is included (causal s <= p).
 * Entries with s > p are unspecified (the kernel may write -inf there, but
 * never at or past ld_logits).
 *
 *   q8        [T, H_I, d_I]  FP8 codes of the indexer queries
 *   q_scale   [T]            fp32, > 0: one dequantisation scale per query token
 *   w         [T, H_I]       fp32 head weights (any sign)
 *   q_pos     [T]            int32 absolute position of each query row
 *   logits    [T, ld_logits] fp32 output, ld_logits >= 1 + max position used
 *
 * Keys, contiguous form (block_table == NULL):
 *   k8        [S, d_I]       FP8 codes;   k_scale [S] fp32 > 0
 *   A position q_pos[r] >= S is clamped to S-1 and flagged DSA_DEV_BAD_POSITION.
 * Keys, paged form (block_table != NULL; used by decode, "indexer-logit kernels
 * (incl. paged versions)", same page, "Key claims"):
 *   k8        [num_pages, page_size, d_I] pool of FP8 codes
 *   k_scale   [num_pages, page_size]      fp32 scales
 *   block_table [T, max_pages] int32: row r's logical page i lives in pool page
 *             block_table[r*max_pages + i]; a key at logical position s lives at
 *             slot s % page_size of page block_table[r*max_pages + s/page_size].
 *   S is ignored.  Each row is its own sequence.  An out-of-range page id is
 *   skipped (its logits are left unwritten) and flagged DSA_DEV_BAD_PAGE.
 *
 * Supported sizes: (H_I, d_I) = (64,128) or (32,128), contiguous or paged;
 * (4,32) contiguous only; any other pair returns DSA_ERR_UNSUPPORTED.
 * page_size in {32, 64, 128}; T >= 0 (T = 0 is a no-op).
 * Alignment: q8 and k8 16-byte aligned; ld_logits >= 1.
 */
int dsa_indexer_logits(const void *q8, const float *q_scale, const float *w,
                       int T, int H_I, int d_I,
                       const void *k8, const float *k_scale, int S,
                       const int32_t *block_table, int max_pages, int num_pages, int page_size,
                       const int32_t *q_pos,
                       float *logits, int64_t ld_logits, dsa_stream_t stream);

/*
 * dsa_quantize_fp8: per-token FP8 (E4M3) quantisation of the indexer inputs.
 *
 * The indexer runs in FP8 with one positive scale per token ("AMD Instinct
 * MI355X GPUs Power DeepSeek-V3.2-Exp", section "DeepSeek Sparse Attention
 * (DSA)", item 1; release summary "DeepSeek-V3.2-Exp: Boosting Long-Context
 * Efficiency with DeepSeek Sparse Attention", section "Method"); the gist
 * page's indexer test script casts to E4M3 with an option for power-of-two
 * (UE8M0) scales.  For each row r of cols values x[r*cols + c]:
 *   DSA_SCALE_AMAX  scale[r] = amax / 448 in fp32 (1 for an all-zero row)
 *   DSA_SCALE_POW2  scale[r] = the smallest power of two >= that ratio
 *                   (1 for an all-zero row)
 *   codes[r*cols + c] = E4M3 nearest to x / scale[r] (fp32 division), ties to
 *                   the even code, magnitudes above 448 saturated to 448.
 * The indexer's q rows are tokens over all H_I * d_I entries, its k rows
 * tokens over d_I; dequantised value = code * scale.
 *
 *   x      [rows, cols] fp32, contiguous;  codes [rows, cols] uint8 (E4M3);
 *   scale  [rows] fp32.  rows = 0 is a no-op.  Inputs must be finite.
 * Any alignment works; 16-byte aligned rows of x (and 4-byte aligned rows of
 * codes) take the vector path.
 */
#define DSA_SCALE_AMAX 0
#define DSA_SCALE_POW2 1
int dsa_quantize_fp8(const float *x, int64_t rows, int64_t cols, int scale_mode,
                     void *codes, float *scale, dsa_stream_t stream);

/*
 * dsa_rmsnorm: residual addition, root-mean-square norm and FP8 output, the
 * step in front of a layer's projections (the pages name the FP8 arithmetic it
 * feeds: "AMD Instinct MI355X GPUs Power DeepSeek-V3.2-Exp", section "DeepSeek
 * Sparse Attention (DSA)", item 1; the norm itself has no counterpart there).
 * For each row r, in fp32,
 *     h = x + residual (x when residual is NULL)
 *     y = h / sqrt(mean_c(h^2) + eps) * weight
 * residual_out = h and out = y, each rounded once to the tensors' type; codes
 * and scale are the FP8 form of the fp32 y: E4M3 nearest to y / scale (fp32
 * division, ties to even, saturated), with, per row (block = 0) or per 128
 * consecutive columns (block = 128; the last block may be short), scale =
 * amax / 448 or the power of two of dsa_quantize_fp8's scale_mode.
 *
 *   x, residual, residual_out, out: [rows, cols] of `dtype` (DSA_BF16 or
 *             DSA_FP32), rows ldx, ldr, ldh, ldo elements apart (>= cols);
 *   weight    [cols] of `weight_dtype`
 *   codes     [rows, cols] uint8, contiguous;  scale [rows, n] fp32 with n = 1
 *             (block = 0) or ceil(cols / 128)
 * residual, residual_out, out and codes (with scale) may each be NULL, the last
 * three not all.  residual_out may be residual or x itself, and out may be x; no
 * other overlap of an output with another tensor.
 * 1 <= cols <= 16384; rows = 0 is a no-op; eps >= 0 (a row of zeros with eps = 0
 * has no norm: NaN).  Inputs must be finite, and a row's squares add up within
 * fp32's range (below 3.4e38; where they do not, y is 0).  Any alignment of whole elements
 * works; 16-byte aligned rows, with cols a multiple of 8, take the vector path.
 * All sums are fp32 in an order fixed by sizes and alignment: results repeat bit
 * for bit on one kind of device.
 */
#define DSA_BF16 0
#define DSA_FP32 1
int dsa_rmsnorm(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight,
                int64_t rows, int cols, int dtype, int weight_dtype, float eps,
                void *residual_out, int64_t ldh, void *out, int64_t ldo,
                void *codes, float *scale, int block, int scale_mode, dsa_stream_t stream);

/*
 * dsa_rmsnorm_backward: gradients of dsa_rmsnorm (the FP8 output passes
 * gradients straight through, as in dsa_indexer_warmup; no counterpart on the
 * pages).  With h the saved residual_out (x where there was no residual),
 * xhat = h / sqrt(mean(h^2) + eps) and g = dy * weight, per row
 *     dx = (g - xhat mean_c(g xhat)) / sqrt(mean(h^2) + eps) + dres
 *     dweight[c] = sum over rows of dy xhat
 * dx is the gradient of x and of the residual alike; dres is the gradient that
 * reaches residual_out from elsewhere (NULL: none).
 *
 *   dy, h, dres, dx: [rows, cols] of `dtype`, contiguous;  weight [cols] of
 *   `weight_dtype`;  dweight [cols] fp32, overwritten (zeros when rows = 0)
 *   workspace: dsa_rmsnorm_backward_workspace_size(rows, cols) bytes, 16-byte
 *   aligned, owned by the caller, used only while the call's kernels run
 *   (calls sharing one must be ordered).
 * dx may be dy, dres or h itself.  1 <= cols <= 16384.  All sums are fp32 in an
 * order fixed by sizes and alignment: results repeat bit for bit on one kind of device.
 */
int dsa_rmsnorm_backward(const void *dy, const void *h, const void *weight, const void *dres,
                         int64_t rows, int cols, int dtype, int weight_dtype, float eps,
                         void *dx, float *dweight, void *workspace, size_t workspace_bytes, dsa_stream_t stream);

/* Bytes of workspace dsa_rmsnorm_backward needs on the current device (0 on bad input). */
size_t dsa_rmsnorm_backward_workspace_size(int64_t rows, int cols);

/*
 * dsa_quantize_fp8_blocks: FP8 operands for dsa_gemm_fp8, from activations,
 * gradients or weights ("AMD Instinct MI355X GPUs Power DeepSeek-V3.2-Exp",
 * section "DeepSeek Sparse Attention (DSA)", item 1, for the FP8 arithmetic;
 * scales per 128 values have no counterpart on the pages).  Writes x [rows,
 * cols] and/or its transpose as E4M3 codes:
 *   codes   [rows, cols], scale per 1 x 128 piece of a row (block_rows = 1:
 *           scale [rows, ceil(cols / 128)]) or per 128 x 128 block (block_rows =
 *           128: scale [ceil(rows / 128), ceil(cols / 128)])
 *   codes_t [cols, rows], the same of x transposed: scale_t [cols, ceil(rows /
 *           128)] or [ceil(cols / 128), ceil(rows / 128)]
 * with scale = amax / 448 over the piece or block (the last ones may be short),
 * or the power of two of dsa_quantize_fp8's scale_mode, 1 for zeros, and code =
 * E4M3 nearest to x / scale (fp32 division, ties to even, saturated).
 *
 *   x        bf16 or fp32 (`dtype`), rows ldx elements apart (>= cols)
 *   codes, codes_t  uint8, rows ld_codes (>= cols) and ld_codes_t (>= rows) apart;
 *            dsa_gemm_fp8 wants them multiples of 16; what lies between rows is
 *            left alone
 * codes (with scale) or codes_t (with scale_t) may be NULL.  rows >= 0 (0 is a
 * no-op), cols >= 1.  Inputs must be finite.  Any alignment of whole elements works; x
 * with rows at 16 bytes, codes at 8 and codes_t at 16 take the vector path.
 * The outputs overlap neither x nor one another.
 */
int dsa_quantize_fp8_blocks(const void *x, int64_t ldx, int64_t rows, int64_t cols, int dtype,
                            int block_rows, int scale_mode, void *codes, int64_t ld_codes, float *scale,
                            void *codes_t, int64_t ld_codes_t, float *scale_t, dsa_stream_t stream);

/*
 * dsa_gemm_fp8: product of FP8 operands with a scale for every 128 values along
 * the summed axis: a projection of tokens (a: dsa_rmsnorm's or dsa_layernorm's
 * codes with block = 128) by weights, or a product of its backward (operands from
 * dsa_quantize_fp8_blocks).  Same page, section and item as there.
 *     out[m, n] = sum_p a_scale[m, p] b_scale[n', p] sum_{k in [128 p, 128 p + 128)} a[m, k] b[n, k]
 * with n' = n / 128 (b_block_rows = 128: b scaled per 128 x 128 block, as weights
 * are) or n (b_block_rows = 1: per row, for a weight's gradient, where K runs
 * over the tokens).  Both operands lie along K: y = x W^T takes W [N, K] as stored,
 * dx = dy W takes the transpose's codes, dW = dy^T x both transposes'.
 *
 *   a [M, K], b [N, K]  E4M3 codes, rows lda and ldb bytes apart
 *   a_scale [M, ceil(K / 128)], b_scale [N or ceil(N / 128), ceil(K / 128)] fp32
 *   out [M, N] bf16 or fp32 (`out_dtype`), rows ldo elements apart
 * 0 <= M, N, K <= 2^30 (M or N = 0 is a no-op, K = 0 writes zeros); a and b
 * 16-byte aligned, lda >= K and ldb >= K multiples of 16 (that of a single or empty row is not
 * looked at); out overlaps no input.  Codes behind K in a row are never used.
 *
 * Precision: the products of a piece are summed in fp32 by the tensor cores; the
 * pieces' sums are scaled and added in fp32, in an order fixed by the sizes and
 * the device: results repeat bit for bit.  A NaN code (or scale) makes NaN of its row's or column's
 * outputs and no others.  A piece's two scales are multiplied first, in fp32: the product
 * has to be 0, or at least 2^-126 and finite (as of scales of 0 and 2^-63 to 2^63).
 * Beyond, it loses bits, is 0 or is infinite (NaN with a sum of 0), although the term
 * itself may fit fp32.
 */
int dsa_gemm_fp8(const void *a, int64_t lda, const float *a_scale, const void *b, int64_t ldb,
                 const float *b_scale, int b_block_rows, int M, int N, int K,
                 void *out, int64_t ldo, int out_dtype, dsa_stream_t stream);

/*
 * dsa_layernorm: residual addition, layer norm and FP8 output: the norm of the
 * indexer's keys in front of dsa_cache_append, or of hidden states (no
 * counterpart on the pages).  For each row r, in fp32,
 *     h = x + residual (x when residual is NULL)
 *     y = (h - mean_c(h)) / sqrt(mean_c((h - mean)^2) + eps) * weight + bias
 * Tensors, types, strides, outputs, limits, aliasing and the FP8 form of y are those of
 * dsa_rmsnorm; bias [cols] is of `weight_dtype`, or NULL for none.  The variance is
 * taken about the mean, so a large common offset costs no more than the mean's own
 * rounding: none for a row of equal values whose sum is exact in fp32 (bf16 values
 * without a residual), which gives the bias, and with eps = 0 has no norm (NaN); else
 * that of a sum in fp32, over sqrt(var + eps).
 */
int dsa_layernorm(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight, const void *bias,
                  int64_t rows, int cols, int dtype, int weight_dtype, float eps,
                  void *residual_out, int64_t ldh, void *out, int64_t ldo,
                  void *codes, float *scale, int block, int scale_mode, dsa_stream_t stream);

/*
 * dsa_layernorm_backward: gradients of dsa_layernorm (the FP8 output passes
 * gradients straight through).  With h the saved residual_out (x where there was
 * no residual), xhat the normed row before weight and bias, g = dy * weight:
 *     dx = (g - mean_c(g) - xhat mean_c(g xhat)) / sqrt(var + eps) + dres
 *     dweight[c] = sum over rows of dy xhat,  dbias[c] = sum over rows of dy
 * Arguments as for dsa_rmsnorm_backward; dbias [cols] fp32, overwritten, or NULL.
 *   workspace: dsa_layernorm_backward_workspace_size(rows, cols) bytes, 16-byte
 *   aligned, as there.
 */
int dsa_layernorm_backward(const void *dy, const void *h, const void *weight, const void *dres,
                           int64_t rows, int cols, int dtype, int weight_dtype, float eps,
                           void *dx, float *dweight, float *dbias, void *workspace, size_t workspace_bytes,
                           dsa_stream_t stream);

/* Bytes of workspace dsa_layernorm_backward needs on the current device (0 on bad input). */
size_t dsa_layernorm_backward_workspace_size(int64_t rows, int cols);

/*
 * dsa_cache_append: writes new tokens into the paged caches that the paged
 * entry points read, applying the position rotation on the way ("DeepSeek-
 * V3.2-Exp: Boosting Long-Context Efficiency with DeepSeek Sparse Attention",
 * section "Key claims": the indexer's RoPE is non-interleaved, the MLA's is
 * interleaved).  Token t goes to logical position p = pos[t] of the sequence
 * whose pages block_table row seq[t] lists (row t when seq is NULL), i.e. to
 * slot p % page_size of pool page block_table[seq[t]*max_pages + p/page_size]:
 *   kv_pool  columns [0, 512): kv[t, 0:512], or its RMS norm
 *            c / sqrt(mean(c^2) + eps) * kv_weight when kv_weight is given;
 *            columns [512, 576): kv[t, 512:576] with the pairs (2i, 2i + 1)
 *            rotated by p * inv_freq[i]; rounded once to bf16
 *   k8_pool, ks_pool: kI[t] with the pairs (i, i + 32) of its first 64 columns
 *            rotated by p * inv_freq[i], as E4M3 codes and one scale per token
 *            (scale_mode as in dsa_quantize_fp8, from the unrounded values)
 * A rotation takes (a, b) to (a cos - b sin, a sin + b cos).
 *
 *   pos [T] int32;  seq [T] int32 or NULL;  block_table [num_seqs, max_pages]
 *   inv_freq [32] fp64, radians per position
 *   kv  [T, 576] bf16, rows ld_kv elements apart;  kv_weight [512] bf16/fp32
 *       (`weight_dtype`) or NULL;  kv_pool [num_pages, page_size, 576] bf16
 *   kI  [T, 128] bf16/fp32 (`k_dtype`), rows ld_kI elements apart;
 *       k8_pool [num_pages, page_size, 128], ks_pool [num_pages, page_size]
 * kv (with kv_pool) or kI (with k8_pool and ks_pool) may be NULL: that cache is
 * left alone.  page_size in {32, 64, 128}.  T = 0 is a no-op.  kv, kv_weight,
 * kI, the pools' bases and the row strides in bytes are multiples of 16.
 * A token with pos < 0 is padding: nothing is written for it.  A position past
 * the table's last page or a seq outside [0, num_seqs) is skipped and flagged
 * DSA_DEV_BAD_POSITION, a page id outside [0, num_pages) skipped and flagged
 * DSA_DEV_BAD_PAGE.  Slots no token names keep their bytes.  Two tokens of one
 * call must not name the same slot (that slot's bytes are then unspecified).
 */
int dsa_cache_append(const int32_t *pos, const int32_t *seq, int T,
                     const int32_t *block_table, int num_seqs, int max_pages, int num_pages, int page_size,
                     const double *inv_freq,
                     const void *kv, int64_t ld_kv, const void *kv_weight, int weight_dtype, float eps, void *kv_pool,
                     const void *kI, int64_t ld_kI, int k_dtype, int scale_mode, void *k8_pool, float *ks_pool,
                     dsa_stream_t stream);

/*
 * dsa_rope_queries: the queries' side of dsa_cache_append (same rotations, same
 * page and section).  For each token t at position p = pos[t]:
 *   q[t, h, 512:576] = q_rope[t, h, :] with the pairs (2i, 2i + 1) rotated by
 *            p * inv_freq[i], rounded once to bf16 (the other 512 columns are
 *            left alone)
 *   q8, q_scale: the index queries qI[t] with the pairs (i, i + 32) of each
 *            head's first 64 columns rotated, as E4M3 codes with one scale per
 *            token over its H_I * 128 values (scale_mode as in dsa_quantize_fp8)
 *
 *   pos [T] int32;  inv_freq [32] fp64, radians per position
 *   q_rope [T, H, 64] bf16, strides st_t and st_h in elements;  q [T, H, 576] bf16
 *   qI [T, H_I, 128] bf16/fp32 (`i_dtype`);  q8 [T, H_I, 128];  q_scale [T] fp32
 * q_rope (with q) or qI (with q8 and q_scale) may be NULL.  1 <= H <= 128 and
 * 1 <= H_I <= 64 where used; T = 0 is a no-op.  q_rope, q, qI and q8 are 16-byte
 * aligned, st_t and st_h multiples of 8.  q_rope may be q[:, :, 512:576] itself (the
 * rotation is then in place) and must not overlap q otherwise.  A negative
 * position is padding: that token's outputs are left alone.
 */
int dsa_rope_queries(const int32_t *pos, const double *inv_freq, int T,
                     const void *q_rope, int64_t st_t, int64_t st_h, int H, void *q,
                     const void *qI, int H_I, int i_dtype, int scale_mode, void *q8, float *q_scale,
                     dsa_stream_t stream);

/*
 * dsa_index_rope_backward: gradient of the index rotation, for training the
 * indexer's projections from dsa_indexer_warmup's dq (H_I heads) and dk (H_I =
 * 1), which are gradients of the rotated vectors (same page and section as
 * dsa_cache_append; the FP8 quantiser passes gradients straight through):
 *     dx[t, j, :] = g[t, j, :] with the pairs (i, i + 32) of the first 64
 *                   columns rotated by -pos[t] * inv_freq[i]
 *   g [T, H_I, 128] fp32;  pos [T] int32;  inv_freq [32] fp64;
 *   dx [T, H_I, 128] bf16/fp32 (`dtype`); fp32 dx may be g itself.
 * g and dx 16-byte aligned; 1 <= H_I <= 64; T = 0 is a no-op.  For pos < 0, dx
 * is zero (such a token was never rotated or used).
 */
int dsa_index_rope_backward(const float *g, const int32_t *pos, const double *inv_freq, int T, int H_I,
                            void *dx, int dtype, dsa_stream_t stream);

/*
 * dsa_topk: fine-grained token selection (stage 2).
 *
 * For each row t with n = valid_len[t] candidates logits[t*ld + s], s in [0, n):
 * keeps the min(k, n) candidates ranked first by (score descending, index
 * ascending) and writes their indices to idx[t*k ...] in ASCENDING index
 * order, padded with -1 ("AMD Instinct MI355X GPUs Power DeepSeek-V3.2-Exp",
 * section "DeepSeek Sparse Attention (DSA)", item 2: top-2048 per query).
 * -0.0 and +0.0 compare equal.  Scores must be finite (a NaN makes that row's
 * result unspecified, never out of bounds).  n > ld is clamped to ld and
 * flagged DSA_DEV_BAD_POSITION; n < 0 counts as 0.
 *
 *   logits    [T, ld] fp32;  valid_len [T] int32;  idx [T, k] int32 output.
 * Supported: 1 <= k <= 4096, ld >= 1, ld <= 2^28.  Deterministic: the same
 * inputs give the same bytes.
 */
int dsa_topk(const float *logits, int64_t ld, int T, const int32_t *valid_len,
             int k, int32_t *idx, dsa_stream_t stream);

/*
 * dsa_indexer_topk: stages 1 and 2 in one call, without the index scores ever
 * reaching memory.
 *
 * Result: exactly what dsa_indexer_logits (contiguous keys) followed by
 * dsa_topk with valid_len[r] = min(q_pos[r] + 1, S) writes to idx, byte for
 * byte: for each query row r, the k keys s in [0, q_pos[r]] with the highest
 * index score (score descending, position ascending), in ascending order,
 * padded with -1 (release summary "DeepSeek-V3.2-Exp: Boosting Long-Context
 * Efficiency with DeepSeek Sparse Attention", section "Method"; "AMD Instinct
 * MI355X GPUs Power DeepSeek-V3.2-Exp", section "Computational Efficiency":
 * attention drops from O(L^2) to O(Lk), which leaves the indexer's L x L
 * scores as the long-context cost; here they are neither written nor read).
 *
 * How: a per-row threshold from the scores of keys sampled at a fixed stride
 * (2048 of them, or S/32 past 65536 keys), which about 1.25k + 256 of the
 * row's keys reach (rows of at most max(4096, 2k) keys take every key); the
 * indexer then appends only the keys at or above it to per-row lists, and an
 * exact top-k runs over each list.  A row whose list misses
 * [k, max(4096, 2k)] (a row unlike its samples) is redone from its full
 * scores, so the result never depends on the sample.
 *
 *   q8, q_scale, w, q_pos, k8, k_scale, S: as for dsa_indexer_logits with
 *             contiguous keys ([S, d_I] codes, [S] scales); (H_I, d_I) =
 *             (64, 128) or (32, 128); 1 <= S <= DSA_INDEXER_TOPK_MAX_KEYS.
 *   k         1 <= k <= 4096;   idx [T, k] int32 output.
 *   workspace a device buffer of dsa_indexer_topk_workspace_size(T, S, H_I,
 *             d_I, k) bytes, 256-byte aligned, owned by the caller, used only
 *             while the call's kernels run on `stream` (calls sharing one must
 *             be ordered).  It holds the sampled keys and scores, the per-row
 *             candidate lists (T x max(4096, 2k) entries of 8 bytes) and, for
 *             the rows redone from full scores, T x S fp32 scores: most of it
 *             stays untouched; callers with long rows pass rows in chunks.
 * A position q_pos[r] >= S is clamped to S-1 and flagged DSA_DEV_BAD_POSITION.
 */
#define DSA_INDEXER_TOPK_MAX_KEYS 262144
int dsa_indexer_topk(const void *q8, const float *q_scale, const float *w, int T, int H_I, int d_I,
                     const void *k8, const float *k_scale, int S, const int32_t *q_pos,
                     int k, int32_t *idx, void *workspace, size_t workspace_bytes, dsa_stream_t stream);

/* Bytes of workspace dsa_indexer_topk needs (0 on unsupported sizes). */
size_t dsa_indexer_topk_workspace_size(int T, int S, int H_I, int d_I, int k);

/*
 * dsa_indexer_warmup: the indexer's dense warm-up step, loss and gradients.
 *
 * Release summary "DeepSeek-V3.2-Exp: Boosting Long-Context Efficiency with
 * DeepSeek Sparse Attention", section "Method": before sparse training a dense
 * warm-up trains only the lightning indexer, against a KL-divergence-to-main-
 * attention target.  Readings (the pages give no formula): for query row t at
 * position q_pos[t] (clamped to S-1) over keys s <= q_pos[t]
 *   p[t,s]   = mean over the H heads of softmax_s(sm_scale * <q[t,h,:576], kv[s,:576]>)
 *              (the main attention's dense causal distribution, MQA mode)
 *   I[t,s]   = the index score of dsa_indexer_logits, a[t,j,s] = <q8[t,j]*q_scale[t], k8[s]*k_scale[s]>
 *   loss[t]  = sum_s p (ln p - ln softmax_s I[t,:])
 *   dw[t,j]  = d(sum loss)/dw = sum_s g ReLU(a),      g = softmax(I) - p
 *   dq[t,j,:] = sum_s g w[t,j] [a > 0] k[s,:] * k_scale[s]      (w.r.t. the dequantised q)
 *   dk[s,:]  = sum_t sum_j g w[t,j] [a > 0] q[t,j,:] * q_scale[t] (w.r.t. the dequantised k)
 * (the FP8 quantiser passes gradients straight through; ReLU'(0) = 0).
 *
 *   q [T, H, 576] bf16, kv [S, 576] bf16, 1 <= H <= 128, sm_scale > 0;
 *   q8, q_scale, w, q_pos, k8, k_scale: as for dsa_indexer_logits with
 *   contiguous keys, (H_I, d_I) = (64, 128) or (32, 128);
 *   outputs fp32: loss [T], dw [T, H_I], dq [T, H_I, d_I], dk [S, d_I].
 *   workspace: dsa_indexer_warmup_workspace_size(T, S, H_I, d_I) bytes, 256-byte
 *   aligned, owned by the caller (it holds p, I and then g, 8 T S bytes, and the
 *   FP8 codes as bf16 with per-row bounds, about 264 (T H_I + S) bytes).
 * Precision: the target's scores on BF16 tensor cores with fp32 accumulation,
 * the index scores as dsa_indexer_logits; the gradient contractions on BF16
 * tensor cores (the codes exact, the coefficients g w [a > 0] as bf16 hi + lo
 * pairs, fp32 accumulation); the ReLU decision [a > 0] exact (the sign of the
 * exact dot product of the codes).  dk is summed with atomics across chunks of
 * rows, so its last bits may differ from call to call.
 */
int dsa_indexer_warmup(const void *q, const void *kv, int H, float sm_scale,
                       const void *q8, const float *q_scale, const float *w, int H_I, int d_I,
                       const void *k8, const float *k_scale, const int32_t *q_pos, int T, int S,
                       float *loss, float *dw, float *dq, float *dk,
                       void *workspace, size_t workspace_bytes, dsa_stream_t stream);

/* Bytes of workspace dsa_indexer_warmup needs (0 on unsupported sizes). */
size_t dsa_indexer_warmup_workspace_size(int T, int S, int H_I, int d_I);

/*
 * dsa_sparse_mla_prefill: MQA-mode sparse MLA over the selected rows (stage 3).
 *
 * For query row t, head h and its valid selected rows s_i = idx[t*k + i]
 * (0 <= s_i < S; other entries are skipped wherever they stand):
 *     S_i      = sm_scale * sum_{d<576} q[t,h,d] * kv[s_i,d]
 *     out[t,h,v] = sum_i softmax(S)_i * kv[s_i,v]          (v < 512)
 *     lse[t,h] = ln sum_i exp(S_i)
 * ("DeepSeek-V3.2-Exp: Boosting Long-Context Efficiency with DeepSeek Sparse
 * Attention", section "Method": main attention reads only the top-k entries,
 * in MLA's MQA mode so one latent row is shared by all heads of a token; the
 * first 512 columns are V, the last 64 are the RoPE part used only in scores.)
 * A row with no valid entry gets out = 0 and lse = -inf.
 *
 * Precision: scores accumulate in fp32 (each token runs on two SMs that each
 * hold half of the 576 score columns and exchange their fp32 partial scores,
 * so a score is off by a few fp32 ulps of its magnitude, however large); P is
 * rounded to bf16 before the PV product and out to bf16 (nearest even) at the
 * end.
 *
 *   q    [T, H, 576] bf16;  kv [S, 576] bf16;  idx [T, k] int32
 *   out  [T, H, 512] bf16 (rounded to nearest even);  lse [T, H] fp32
 * Supported: 1 <= H <= 128 (fewer than 128 heads run as zero-padded rows
 * that are never stored); D = 576, Dv = 512 fixed; 1 <= k <= 4096.  q, kv, out
 * 16-byte aligned.
 */
int dsa_sparse_mla_prefill(const void *q, const void *kv, int S,
                           const int32_t *idx, int T, int H, int k, float sm_scale,
                           void *out, float *lse, dsa_stream_t stream);

/*
 * dsa_sparse_mla_decode_paged: the same attention over a paged latent cache
 * (decode form of stage 3; "DeepSeek-V3.2-Exp: Boosting Long-Context
 * Efficiency with DeepSeek Sparse Attention", section "Key claims": the
 * released kernels are indexer-logit kernels, paged versions included, and
 * sparse-attention kernels; the attention itself is that of section "Method").
 *
 * Row b is one query: its token sits at position ctx_len[b]-1 of the sequence
 * whose pages block_table row b lists.  Rows are independent, so a batch may
 * hold one new token per sequence (decode), several positions of the same
 * sequence (multi-token decode), or every token of sequences of different
 * lengths (ragged batched prefill), all in one pool.  idx[b*k + i] holds
 * LOGICAL positions, read from slot s % page_size of pool page
 * block_table[b*max_pages + s/page_size].  Entries outside [0, ctx_len[b]) are
 * skipped; a page id outside [0, num_pages) is skipped and flagged
 * DSA_DEV_BAD_PAGE.
 *
 * Work split.  Attention runs on two-CTA clusters, one per pair of SMs.  With
 * more rows than two thirds of the clusters, each cluster takes whole rows, as
 * in prefill.  With fewer, the flattened (row, 64-entry block of idx) space is
 * cut into one contiguous share per cluster, so every SM works; a share that
 * holds only part of a row writes that part's softmax-normalised output and
 * LSE (fp32) to the workspace, and a second kernel merges the parts of each
 * row by their LSEs (LSE = ln sum exp LSE_p, O = sum exp(LSE_p - LSE) O_p)
 * into out and lse.  The split changes only the fp32 summation order.
 *
 *   q       [B, H, 576] bf16;  kv_pool [num_pages, page_size, 576] bf16
 *   block_table [B, max_pages] int32;  ctx_len [B] int32;  idx [B, k] int32
 *   out     [B, H, 512] bf16;  lse [B, H] fp32
 *   workspace: a device buffer of at least
 *           dsa_sparse_mla_decode_workspace_size(B, H, k) bytes, 256-byte
 *           aligned, owned by the caller, used only while the call's kernels
 *           run on `stream`; NULL is accepted when that size is 0.  Calls that
 *           share one workspace must be ordered on the GPU (same stream).
 *           A missing or short workspace returns DSA_ERR_WORKSPACE.
 */
int dsa_sparse_mla_decode_paged(const void *q, const void *kv_pool, int num_pages, int page_size,
                                const int32_t *block_table, int max_pages, const int32_t *ctx_len,
                                const int32_t *idx, int B, int H, int k, float sm_scale,
                                void *out, float *lse, void *workspace, size_t workspace_bytes,
                                dsa_stream_t stream);

/*
 * dsa_prefill_host: the whole prefill path (dsa_indexer_logits -> dsa_topk ->
 * dsa_sparse_mla_prefill, contiguous keys) on inputs in HOST memory, with the
 * outputs written back to HOST memory.  Row r is the query at position
 * q_pos[r] over keys [0, q_pos[r]] (release summary "DeepSeek-V3.2-Exp:
 * Boosting Long-Context Efficiency with DeepSeek Sparse Attention", section
 * "Method"); rows and their arguments mean what they mean for the three
 * device entry points, whose results this call reproduces byte for byte.
 *
 *   host: q8 [T, H_I, d_I] FP8, q_scale [T], w [T, H_I], q_pos [T] int32,
 *         k8 [S, d_I] FP8, k_scale [S], q [T, H, 576] bf16, kv [S, 576] bf16
 *         -> out [T, H, 512] bf16, lse [T, H] fp32.  0 <= q_pos[r] < S.
 *   workspace: device buffer of dsa_prefill_host_workspace_size(...) bytes,
 *         256-byte aligned, owned by the caller.
 *
 * Query rows go in chunks of at most chunk_rows (C): C/4 and C/2 rows first,
 * then C, and a last chunk of C/4, processed from the last chunk to the first
 * (short chunks at both ends: the kernels start after a short copy and little
 * is left to copy out after the last kernels; the first chunk processed brings
 * in the keys of every row, and the long rows' chunks, whose kernels outlast
 * their copies, come first).  The inputs of a chunk
 * are copied in on a copy stream, its kernels run on `stream`, its outputs are copied out on
 * a second copy stream, and four buffer slots let the copies run up to three
 * chunks ahead of the kernels.  The keys stay on the device for the call and are
 * copied in as far as each chunk's positions need them.  Host buffers should be
 * page-locked (cudaHostAlloc or cudaHostRegister) for the copies to overlap;
 * pageable memory gives the same results more slowly.  The call returns once
 * everything is enqueued; all of it is complete when `stream` reaches this
 * point, and the host buffers must stay untouched until then.  The first call
 * on a device creates the two copy streams and a few events, kept until exit;
 * calls from several host threads enqueue one at a time.  Errors of the three
 * stages are reported as they would be by their entry points.
 */
int dsa_prefill_host(const void *q8, const float *q_scale, const float *w, const int32_t *q_pos,
                     const void *k8, const float *k_scale, const void *q, const void *kv,
                     int T, int S, int H_I, int d_I, int H, int k, float sm_scale,
                     void *out, float *lse, int chunk_rows,
                     void *workspace, size_t workspace_bytes, dsa_stream_t stream);

/* Device workspace bytes dsa_prefill_host needs (0 on bad input). */
size_t dsa_prefill_host_workspace_size(int T, int S, int H_I, int d_I, int H, int k, int chunk_rows);

/*
 * dsa_prefill_host_trace: a per-chunk timeline of dsa_prefill_host calls on
 * the current device, to see which stream a slow call spent its time on (a
 * debugging record with no counterpart on the pages; off unless turned on).
 * max_chunks > 0 creates 6 * max_chunks + 1 timing events and starts an empty
 * record; every later call then records, for each of its chunks while the
 * record has room, an event on the input-copy stream before and after the
 * chunk's input copies, on `stream` before and after its three stages, and on
 * the output-copy stream before and after its output copies.  Each "before"
 * event follows the chunk's waits, so it marks when that stream began the
 * chunk.  max_chunks = 0 ends the record and destroys its events.  Returns
 * DSA_ERR_INVALID_ARG for max_chunks outside [0, 2^20], DSA_ERR_CUDA if the
 * events cannot be created (recording is then off).
 */
int dsa_prefill_host_trace(int max_chunks);

/*
 * dsa_prefill_host_trace_read: the record of dsa_prefill_host_trace.  Waits
 * for the recorded events and writes, for the first min(recorded, max_chunks)
 * chunks in enqueue order (HOST arrays): ms[6 j + e] = milliseconds from the
 * start of the first recorded call to event e of chunk j (0/1 input copies
 * begin/end, 2/3 stages begin/end, 4/5 output copies begin/end; NaN for an
 * event a failed call never reached), call[j] = the call the chunk belongs to
 * (0 = first recorded call), rows[j] = its query rows; *n_out = the chunks
 * written.  The record stays as it is. Returns DSA_ERR_INVALID_ARG for a null
 * pointer or max_chunks < 0.
 */
int dsa_prefill_host_trace_read(float *ms, int32_t *call, int32_t *rows, int max_chunks, int *n_out);

/*
 * dsa_sparse_mla_decode_paged_noalloc: dsa_sparse_mla_decode_paged without a
 * caller-provided workspace.  The pages have no counterpart to this entry
 * point: it is for callers that cannot allocate device memory while they
 * run, such as a plugin inside a host program that owns every device
 * allocation, or a service held to a fixed device-memory budget that must not
 * grow or wait on an allocator mid-request.  It allocates nothing (no
 * cudaMalloc, no cudaFree, no allocating library call): its workspace is a
 * static device buffer of DSA_DECODE_STATIC_WS_BYTES (40 MiB) built into the
 * library, which every GPU that loads libdsa.so holds until the process exits.
 *
 * Arguments, results and errors are those of dsa_sparse_mla_decode_paged.  A
 * call whose workspace need (dsa_sparse_mla_decode_workspace_size) exceeds the
 * buffer returns DSA_ERR_WORKSPACE with a message naming both sizes; with
 * H <= 128 that takes a device of 160 SMs or more.  The first call on each
 * device looks up the buffer's device address (cudaGetSymbolAddress, with
 * that device current) and keeps it; make that first call before any stream
 * capture.  All calls share the one buffer, which keeps the contents of the
 * last call (nothing in it needs to start at zero: each call writes every
 * part it reads), so calls whose kernels may overlap on the GPU (different
 * streams, or different host threads, on one device) race on it and must be
 * ordered by the caller.
 */
#define DSA_DECODE_STATIC_WS_BYTES (40u << 20)
int dsa_sparse_mla_decode_paged_noalloc(const void *q, const void *kv_pool, int num_pages, int page_size,
                                        const int32_t *block_table, int max_pages, const int32_t *ctx_len,
                                        const int32_t *idx, int B, int H, int k, float sm_scale,
                                        void *out, float *lse, dsa_stream_t stream);

/* Bytes of workspace dsa_sparse_mla_decode_paged needs for (B, H, k) on the
 * current device: 0 when the rows stay whole (3 B > 2 clusters), else
 * 2 * clusters * H * 513 * 4, with clusters = min(SM pairs, B * ceil(k / 64)).
 * 0 on bad input. */
size_t dsa_sparse_mla_decode_workspace_size(int B, int H, int k);

/*
 * dsa_mla_decode_paged: dense MLA of single tokens over the paged latent cache,
 * for layers, steps and contexts that select nothing (the attention that DSA's
 * selection narrows and its warm-up trains against: "DeepSeek-V3.2-Exp:
 * Boosting Long-Context Efficiency with DeepSeek Sparse Attention", section
 * "Method").  Row b's query attends over every position s < ctx_len[b] of the
 * sequence whose pages block_table row b lists:
 *     S_s = sm_scale * sum_{d<576} q[b,h,d] * kv[s,d]
 *     out[b,h,v] = sum_s softmax(S)_s * kv[s,v]  (v < 512),  lse = ln sum_s exp(S_s)
 * Rows are independent (one new token per sequence, several positions of one
 * sequence, or a ragged batch, as in dsa_sparse_mla_decode_paged).  A row with
 * ctx_len <= 0, or no valid page, gets out = 0 and lse = -inf.  A ctx_len past
 * the block table's last page is clamped to it and flagged
 * DSA_DEV_BAD_POSITION; keys on a page id outside [0, num_pages) are skipped and flagged
 * DSA_DEV_BAD_PAGE.  Slots past ctx_len are never used, whatever they hold.
 *
 * A NaN in a used key or in a head's query makes out and lse of the rows or
 * heads that use it NaN, and no others.
 *
 * Precision: scores and softmax in fp32; the weights exp(S - m) are rounded to
 * bf16 for the product with the values (m is a running maximum, so they lie in
 * (0, 2^8]; their sum is that of the unrounded ones), which the products
 * accumulate in fp32; out rounded once to bf16.  The keys of a row are split
 * over the SMs and joined by their LSEs in a fixed order, so results repeat bit
 * for bit on one kind of device.
 *
 *   q [B, H, 576] bf16;  kv_pool [num_pages, page_size, 576] bf16
 *   block_table [B, max_pages] int32;  ctx_len [B] int32
 *   out [B, H, 512] bf16;  lse [B, H] fp32
 *   workspace: dsa_mla_decode_workspace_size(B, H) bytes, 256-byte aligned,
 *   owned by the caller, used only while the call's kernels run on `stream`
 *   (calls sharing one must be ordered).
 * 1 <= H <= 128; page_size in {32, 64, 128}; 0 <= B <= 65535 (0 is a no-op);
 * q, kv_pool and out 16-byte aligned.
 */
int dsa_mla_decode_paged(const void *q, const void *kv_pool, int num_pages, int page_size,
                         const int32_t *block_table, int max_pages, const int32_t *ctx_len,
                         int B, int H, float sm_scale, void *out, float *lse,
                         void *workspace, size_t workspace_bytes, dsa_stream_t stream);

/* Bytes of workspace dsa_mla_decode_paged needs on the current device (0 on bad input). */
size_t dsa_mla_decode_workspace_size(int B, int H);

#ifdef __cplusplus
}
#endif
#endif /* DSA_H */
