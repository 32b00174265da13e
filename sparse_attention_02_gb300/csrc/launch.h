// Host-side interfaces between the C ABI (api.cu) and the kernel files.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace dsa {

// Encodes a 2-D tiled tensor map (dims/box in elements, row stride in bytes).
// Returns false and fills `err` on failure.
bool encode_tmap_2d(CUtensorMap *map, CUtensorMapDataType dtype, const void *base, uint64_t inner,
                    uint64_t rows, uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_rows,
                    CUtensorMapSwizzle swizzle, char *err, size_t errlen);

// `groups` groups of `rows` rows, each row `blocks` column blocks of `inner`
// elements: a box is box_blocks blocks of box_rows rows of one group, laid out
// block by block; rows past a group's end arrive as zeros.  Coordinates: column
// in the block, row, block, group.
bool encode_tmap_blocks(CUtensorMap *map, CUtensorMapDataType dtype, const void *base, uint64_t inner, uint64_t rows,
                        uint64_t blocks, uint64_t groups, uint64_t row_stride_bytes, uint64_t block_stride_bytes,
                        uint32_t box_rows, uint32_t box_blocks, CUtensorMapSwizzle swizzle, char *err, size_t errlen);

int num_sms();

// Records a message for dsa_last_error() on this host thread and returns `code`.
int report_error(int code, const char *fmt, ...);

// Raises `kernel`'s dynamic shared-memory limit to `bytes` on the current
// device, once per device (`done` holds one flag per device; a device past the
// table's end sets it on every call).  Two host threads may both find the flag
// clear and both set the attribute: the call is idempotent and the flag atomic.
template <typename... KArgs>
cudaError_t raise_smem_limit_once(void (*kernel)(KArgs...), int bytes, std::atomic<bool> (&done)[64])
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 64 && done[dev].load(std::memory_order_acquire))
        return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64)
        done[dev].store(true, std::memory_order_release);
    if (e != cudaSuccess)
        cudaGetLastError(); // the failure is reported to the caller; leave no error behind for the next call
    return e;
}

// Launches `kernel` on `stream` with programmatic dependent launch allowed
// (the kernel must call grid_dep_wait() before touching global memory) and,
// when cluster_x > 1, thread-block clusters of cluster_x CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       unsigned cluster_x, Args &&...args)
{
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
    if (cluster_x > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster_x;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args &&>(args)...);
}
unsigned *device_status_ptr(); // address of this device's status word, or null

struct QuantizeArgs {
    const float *x;  // [rows, cols] fp32
    int64_t rows, cols;
    int mode;        // 0: amax / 448, 1: power-of-two scale
    uint8_t *codes;  // [rows, cols] E4M3
    float *scale;    // [rows]
};
int launch_quantize(const QuantizeArgs &a, cudaStream_t stream, char *err, size_t errlen);

struct QuantizeBlocksArgs {
    const void *x;   // [rows, cols], row stride ldx; bf16, or fp32 with x32
    int64_t ldx, rows, cols;
    bool x32;
    int block_rows;  // 1 or 128
    int scale_mode;
    uint8_t *codes;  // [rows, cols], row stride ldc, or null
    int64_t ldc;
    float *scale;    // [rows / block_rows, cols / 128], rounded up
    uint8_t *codes_t; // [cols, rows], row stride ldt, or null
    int64_t ldt;
    float *scale_t;  // [cols / block_rows, rows / 128], rounded up
};
int launch_quantize_blocks(const QuantizeBlocksArgs &a, cudaStream_t stream, char *err, size_t errlen);

struct GemmFp8Args {
    const void *a;        // [M, K] E4M3, row stride lda
    int64_t lda;
    const float *a_scale; // [M, ceil(K / 128)]
    const void *b;        // [N, K] E4M3, row stride ldb
    int64_t ldb;
    const float *b_scale; // [N, or ceil(N / 128) with b_block; ceil(K / 128)]
    bool b_block;
    int M, N, K;
    void *out;            // [M, N] bf16, or fp32 with o32, row stride ldo
    int64_t ldo;
    bool o32;
};
int launch_gemm_fp8(const GemmFp8Args &a, cudaStream_t stream, char *err, size_t errlen);

struct NormArgs {
    const void *x;        // [rows, cols], row stride ldx; bf16, or fp32 with x32
    const void *residual; // like x (stride ldr), or null
    const void *weight;   // [cols] bf16, or fp32 with w32
    int64_t rows;
    int cols;
    int64_t ldx, ldr, ldh, ldo;
    bool x32, w32;
    float eps;
    void *residual_out; // like x (stride ldh), or null
    void *out;          // like x (stride ldo), or null
    uint8_t *codes;     // [rows, cols], or null
    float *scale;       // [rows, 1 or ceil(cols / 128)]
    int block;          // 0: one scale a row, 128: one per 128 columns
    int scale_mode;
    const void *bias = nullptr; // layer norm: like weight, or null
};
int launch_rmsnorm(const NormArgs &a, cudaStream_t stream, char *err, size_t errlen);
int launch_layernorm(const NormArgs &a, cudaStream_t stream, char *err, size_t errlen);

struct NormBackwardArgs {
    const void *dy, *h, *weight, *dres; // [rows, cols] (dres or null); weight [cols]
    int64_t rows;
    int cols;
    bool x32, w32;
    float eps;
    void *dx;
    float *dweight;
    void *workspace;
    float *dbias = nullptr; // layer norm; or null
};
int launch_rmsnorm_backward(const NormBackwardArgs &a, cudaStream_t stream, char *err, size_t errlen);
size_t rmsnorm_backward_workspace_bytes(int64_t rows, int cols);
int launch_layernorm_backward(const NormBackwardArgs &a, cudaStream_t stream, char *err, size_t errlen);
size_t layernorm_backward_workspace_bytes(int64_t rows, int cols);

struct CacheAppendArgs {
    const int32_t *pos;       // [T]
    const int32_t *seq;       // [T] block-table row of each token, or null: its own index
    const int32_t *block_table;
    int T, num_seqs, max_pages, num_pages, page_size;
    const double *inv_freq;   // [32]
    const void *kv;           // [T, 576] bf16, row stride ld_kv, or null
    int64_t ld_kv;
    const void *kv_weight;    // [512], or null
    bool w32;
    float eps;
    void *kv_pool;
    const void *kI;           // [T, 128], row stride ld_kI, or null
    int64_t ld_kI;
    bool k32;
    int scale_mode;
    uint8_t *k8_pool;
    float *ks_pool;
};
int launch_cache_append(const CacheAppendArgs &a, cudaStream_t stream, char *err, size_t errlen);

struct RopeQueriesArgs {
    const int32_t *pos; // [T]
    const double *inv_freq;
    int T, H, HI;
    const void *q_rope; // [T, H, 64] bf16, strides st_t, st_h, or null
    int64_t st_t, st_h;
    void *q;            // [T, H, 576] bf16
    const void *qI;     // [T, HI, 128], or null
    bool i32;           // fp32 qI
    int scale_mode;
    uint8_t *q8;
    float *q_scale;
};
int launch_rope_queries(const RopeQueriesArgs &a, cudaStream_t stream, char *err, size_t errlen);

struct IndexRopeBackwardArgs {
    const float *g;     // [T, HI, 128]
    const int32_t *pos; // [T]
    const double *inv_freq;
    int T, HI;
    void *dx;           // [T, HI, 128] bf16, or fp32 with o32
    bool o32;
    bool wide = false;  // g starts at 32 bytes (set by the launch)
};
int launch_index_rope_backward(const IndexRopeBackwardArgs &a, cudaStream_t stream, char *err, size_t errlen);

struct IndexerArgs {
    const void *q8;
    const float *q_scale;
    const float *w;
    int T, HI, dI;
    const void *k8;
    const float *k_scale;
    int S;
    const int32_t *block_table;
    int max_pages, num_pages, page_size;
    const int32_t *q_pos;
    float *logits;
    int64_t ld;
    // Candidate mode (cand != nullptr; contiguous keys, H_I in {32, 64}): no
    // logits are written; a key whose score is >= thr[r] is appended to row
    // r's list as {raw fp32 score bits, position}, in no particular order.  The
    // list is 128 regions of cap entries, one per epilogue lane scoring the row.
    const float *thr = nullptr;        // [T]
    uint2 *cand = nullptr;             // [T, 128, cap]
    int32_t *cand_cnt = nullptr;       // [T, 128] candidates each region found (only cap are stored)
    int cap = 0;
    const int32_t *row_flag = nullptr; // score only rows with row_flag[r] != 0 (nullptr: all rows)
};
// Returns 0 on success, else a dsa_status with `err` filled.
int launch_indexer(const IndexerArgs &a, cudaStream_t stream, char *err, size_t errlen);

struct TopkArgs {
    const float *logits;
    int64_t ld;
    int T;
    const int32_t *valid_len;
    int k;
    int32_t *idx;
    const int32_t *row_flag = nullptr; // only rows with row_flag[r] != 0 (nullptr: all rows)
};
int launch_topk(const TopkArgs &a, cudaStream_t stream, char *err, size_t errlen);

// Fused indexer -> top-k pieces (topk.cu): the per-row threshold from sampled
// scores, and the exact top-k over each row's candidate list.
int launch_topk_threshold(const float *samp, int ld_s, int T, const int32_t *q_pos, const int32_t *qpos_s, int S,
                          int k, int cap, float *thr, cudaStream_t stream, char *err, size_t errlen);
int launch_topk_candidates(const uint2 *cand, const int32_t *cand_cnt, int cap, int T, const int32_t *q_pos, int S,
                           int k, int32_t *idx, int32_t *flag, cudaStream_t stream, char *err, size_t errlen);
size_t topk_candidates_smem(int S, int cap);

struct IndexerTopkArgs {
    const void *q8;
    const float *q_scale;
    const float *w;
    int T, HI, dI;
    const void *k8;
    const float *k_scale;
    int S;
    const int32_t *q_pos;
    int k;
    int32_t *idx;
    void *workspace;
    size_t workspace_bytes;
};
int launch_indexer_topk(const IndexerTopkArgs &a, cudaStream_t stream, char *err, size_t errlen);
size_t indexer_topk_workspace_bytes(int T, int S, int dI, int k);

struct WarmupArgs {
    const void *q;       // [T, H, 576] bf16: main-attention queries
    const void *kv;      // [S, 576] bf16
    int H;
    float sm_scale;
    const void *q8;      // indexer inputs as for dsa_indexer_logits (contiguous keys)
    const float *q_scale;
    const float *w;
    int HI, dI;
    const void *k8;
    const float *k_scale;
    const int32_t *q_pos;
    int T, S;
    float *loss;         // [T]
    float *dw;           // [T, HI]
    float *dq;           // [T, HI, dI]
    float *dk;           // [S, dI]
    void *workspace;
    size_t workspace_bytes;
};
int launch_warmup(const WarmupArgs &a, cudaStream_t stream, char *err, size_t errlen);
size_t warmup_workspace_bytes(int T, int S, int HI);

struct MlaArgs {
    const void *q;      // [T, H, 576] bf16
    const void *kv;     // [S, 576] bf16, or pool [num_pages, page_size, 576]
    int S;              // rows of kv (prefill) / num_pages * page_size (paged)
    const int32_t *idx; // [T, k]
    int T, H, k;
    float sm_scale;
    void *out;          // [T, H, 512] bf16
    float *lse;         // [T, H]
    // paged decode
    const int32_t *block_table;
    int max_pages, num_pages, page_size;
    const int32_t *ctx_len;
    void *workspace;
    size_t workspace_bytes;
};
int launch_mla_prefill(const MlaArgs &a, cudaStream_t stream, char *err, size_t errlen);
int launch_mla_decode(const MlaArgs &a, cudaStream_t stream, char *err, size_t errlen);
size_t mla_decode_workspace_bytes(int B, int H, int k);

struct DenseMlaArgs {
    const void *q;       // [B, H, 576] bf16
    const void *kv_pool; // [num_pages, page_size, 576] bf16
    int num_pages, page_size;
    const int32_t *block_table;
    int max_pages;
    const int32_t *ctx_len;
    int B, H;
    float sm_scale;
    void *out;           // [B, H, 512] bf16
    float *lse;          // [B, H]
    void *workspace;
};
int launch_dense_mla(const DenseMlaArgs &a, cudaStream_t stream, char *err, size_t errlen);
size_t dense_mla_workspace_bytes(int B, int H);

} // namespace dsa
