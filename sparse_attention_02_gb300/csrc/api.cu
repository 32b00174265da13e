// C ABI of libdsa.so: host-side argument checks, then launches on the caller's
// stream.  See include/dsa.h for the contract of every entry point.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <initializer_list>
#include <mutex>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include "../../include/dsa.h"
#include "common.cuh"
#include "launch.h"

namespace dsa {

// Per-device status word (DSA_DEV_* bits); kernels receive its address.
__device__ unsigned g_device_status = 0u;

namespace {

thread_local char t_err[512] = "";

int fail(int code, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(t_err, sizeof t_err, fmt, ap);
    va_end(ap);
    return code;
}

int ok()
{
    t_err[0] = '\0';
    return DSA_OK;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned_to(size_t n, std::initializer_list<const void *> ps)
{
    for (const void *p : ps)
        if (reinterpret_cast<uintptr_t>(p) % n)
            return false;
    return true;
}

constexpr int kMaxDevices = 64;
std::mutex g_mu;
std::atomic<unsigned *> g_status_ptr[kMaxDevices]; // looked up once a device, by whichever call comes first
std::atomic<int> g_sms[kMaxDevices];
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

int current_device()
{
    int d = 0;
    cudaGetDevice(&d);
    return d;
}

} // namespace

int report_error(int code, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(t_err, sizeof t_err, fmt, ap);
    va_end(ap);
    return code;
}

unsigned *device_status_ptr()
{
    const int d = current_device();
    if (d < 0 || d >= kMaxDevices)
        return nullptr;
    unsigned *known = g_status_ptr[d].load(std::memory_order_acquire);
    if (!known) {
        void *p = nullptr;
        if (cudaGetSymbolAddress(&p, g_device_status) != cudaSuccess)
            return nullptr;
        known = static_cast<unsigned *>(p);
        g_status_ptr[d].store(known, std::memory_order_release);
    }
    return known;
}

int num_sms()
{
    const int d = current_device();
    if (d < 0 || d >= kMaxDevices)
        return 148;
    int known = g_sms[d].load(std::memory_order_relaxed);
    if (!known) {
        int n = 0;
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d);
        known = n > 0 ? n : 148;
        g_sms[d].store(known, std::memory_order_relaxed);
    }
    return known;
}

namespace {

bool encode_tmap(CUtensorMap *map, CUtensorMapDataType dtype, const void *base, int rank, const cuuint64_t *dims,
                 const cuuint64_t *strides, const cuuint32_t *box, CUtensorMapSwizzle swizzle, char *err, size_t errlen)
{
    {
        std::lock_guard<std::mutex> lk(g_mu);
        if (!g_encode) {
            void *fn = nullptr;
            cudaDriverEntryPointQueryResult q;
            if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
                    cudaSuccess ||
                q != cudaDriverEntryPointSuccess || !fn) {
                snprintf(err, errlen, "cuTensorMapEncodeTiled entry point unavailable");
                return false;
            }
            g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
        }
    }
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = g_encode(map, dtype, rank, const_cast<void *>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        snprintf(err, errlen, "cuTensorMapEncodeTiled failed (%d): inner=%llu rows=%llu stride=%llu box=%ux%u", (int)r,
                 (unsigned long long)dims[0], (unsigned long long)dims[1], (unsigned long long)strides[0], box[0], box[1]);
        return false;
    }
    return true;
}

} // namespace

bool encode_tmap_2d(CUtensorMap *map, CUtensorMapDataType dtype, const void *base, uint64_t inner, uint64_t rows,
                    uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_rows, CUtensorMapSwizzle swizzle,
                    char *err, size_t errlen)
{
    const cuuint64_t dims[2] = {inner, rows > 0 ? rows : 1};
    const cuuint64_t strides[1] = {row_stride_bytes};
    const cuuint32_t box[2] = {box_inner, box_rows};
    return encode_tmap(map, dtype, base, 2, dims, strides, box, swizzle, err, errlen);
}

bool encode_tmap_blocks(CUtensorMap *map, CUtensorMapDataType dtype, const void *base, uint64_t inner, uint64_t rows,
                        uint64_t blocks, uint64_t groups, uint64_t row_stride_bytes, uint64_t block_stride_bytes,
                        uint32_t box_rows, uint32_t box_blocks, CUtensorMapSwizzle swizzle, char *err, size_t errlen)
{
    const cuuint64_t dims[4] = {inner, rows, blocks, groups};
    const cuuint64_t strides[3] = {row_stride_bytes, block_stride_bytes, rows * row_stride_bytes};
    const cuuint32_t box[4] = {(cuuint32_t)inner, box_rows, box_blocks, 1};
    return encode_tmap(map, dtype, base, 4, dims, strides, box, swizzle, err, errlen);
}

} // namespace dsa

using namespace dsa;

extern "C" {

const char *dsa_last_error(void) { return t_err; }

int dsa_version(void) { return 100; }

int dsa_get_device_status(dsa_stream_t stream, uint32_t *status_out)
{
    if (!status_out)
        return fail(DSA_ERR_INVALID_ARG, "status_out is null");
    unsigned *dev = device_status_ptr();
    if (!dev)
        return fail(DSA_ERR_CUDA, "device status word unavailable");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    unsigned host = 0;
    cudaError_t e = cudaMemcpyAsync(&host, dev, sizeof host, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess)
        e = cudaMemsetAsync(dev, 0, sizeof(unsigned), s);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(s);
    if (e != cudaSuccess)
        return fail(DSA_ERR_CUDA, "reading device status: %s", cudaGetErrorString(e));
    *status_out = host;
    return ok();
}

int dsa_indexer_logits(const void *q8, const float *q_scale, const float *w, int T, int H_I, int d_I, const void *k8,
                       const float *k_scale, int S, const int32_t *block_table, int max_pages, int num_pages,
                       int page_size, const int32_t *q_pos, float *logits, int64_t ld_logits, dsa_stream_t stream)
{
    if (T < 0)
        return fail(DSA_ERR_INVALID_ARG, "T < 0");
    if (T == 0)
        return ok();
    if (!q8 || !q_scale || !w || !k8 || !k_scale || !q_pos || !logits)
        return fail(DSA_ERR_INVALID_ARG, "null pointer argument");
    if (H_I <= 0 || d_I <= 0 || ld_logits < 1)
        return fail(DSA_ERR_INVALID_ARG, "H_I, d_I and ld_logits must be positive");
    if (!aligned16(q8) || !aligned16(k8))
        return fail(DSA_ERR_ALIGNMENT, "q8 and k8 must be 16-byte aligned");
    if ((int64_t)T * H_I > (int64_t)INT32_MAX)
        return fail(DSA_ERR_UNSUPPORTED, "T * H_I too large");
    if (block_table) {
        if (max_pages <= 0 || num_pages <= 0)
            return fail(DSA_ERR_INVALID_ARG, "paged: max_pages and num_pages must be positive");
        if (page_size != 32 && page_size != 64 && page_size != 128)
            return fail(DSA_ERR_UNSUPPORTED, "paged: page_size must be 32, 64 or 128");
    } else {
        if (S <= 0)
            return fail(DSA_ERR_INVALID_ARG, "S must be positive");
    }
    IndexerArgs a{q8, q_scale, w, T, H_I, d_I, k8, k_scale, S, block_table, max_pages, num_pages, page_size,
                  q_pos, logits, ld_logits};
    int rc = launch_indexer(a, reinterpret_cast<cudaStream_t>(stream), t_err, sizeof t_err);
    return rc == DSA_OK ? ok() : rc;
}

size_t dsa_indexer_topk_workspace_size(int T, int S, int H_I, int d_I, int k)
{
    if (T < 0 || S < 1 || S > DSA_INDEXER_TOPK_MAX_KEYS || k < 1 || k > 4096 || d_I != 128 ||
        (H_I != 64 && H_I != 32))
        return 0;
    return indexer_topk_workspace_bytes(T, S, d_I, k);
}

int dsa_indexer_topk(const void *q8, const float *q_scale, const float *w, int T, int H_I, int d_I, const void *k8,
                     const float *k_scale, int S, const int32_t *q_pos, int k, int32_t *idx, void *workspace,
                     size_t workspace_bytes, dsa_stream_t stream)
{
    if (T < 0)
        return fail(DSA_ERR_INVALID_ARG, "T < 0");
    if (T == 0)
        return ok();
    if (!q8 || !q_scale || !w || !k8 || !k_scale || !q_pos || !idx)
        return fail(DSA_ERR_INVALID_ARG, "null pointer argument");
    if (d_I != 128 || (H_I != 64 && H_I != 32))
        return fail(DSA_ERR_UNSUPPORTED, "fused indexer -> top-k: (H_I, d_I) must be (64, 128) or (32, 128)");
    if (S < 1 || S > DSA_INDEXER_TOPK_MAX_KEYS)
        return fail(DSA_ERR_UNSUPPORTED, "fused indexer -> top-k: S must be in [1, %d]", DSA_INDEXER_TOPK_MAX_KEYS);
    if (k < 1 || k > 4096)
        return fail(DSA_ERR_UNSUPPORTED, "k must be in [1, 4096]");
    if (!aligned16(q8) || !aligned16(k8))
        return fail(DSA_ERR_ALIGNMENT, "q8 and k8 must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return fail(DSA_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
    if (!workspace || workspace_bytes < indexer_topk_workspace_bytes(T, S, d_I, k))
        return fail(DSA_ERR_WORKSPACE, "workspace missing or smaller than dsa_indexer_topk_workspace_size");
    IndexerTopkArgs a{q8, q_scale, w, T, H_I, d_I, k8, k_scale, S, q_pos, k, idx, workspace, workspace_bytes};
    int rc = launch_indexer_topk(a, reinterpret_cast<cudaStream_t>(stream), t_err, sizeof t_err);
    return rc == DSA_OK ? ok() : rc;
}

size_t dsa_indexer_warmup_workspace_size(int T, int S, int H_I, int d_I)
{
    if (T < 0 || S < 1 || d_I != 128 || (H_I != 64 && H_I != 32))
        return 0;
    return warmup_workspace_bytes(T, S, H_I);
}

int dsa_indexer_warmup(const void *q, const void *kv, int H, float sm_scale, const void *q8, const float *q_scale,
                       const float *w, int H_I, int d_I, const void *k8, const float *k_scale, const int32_t *q_pos,
                       int T, int S, float *loss, float *dw, float *dq, float *dk, void *workspace,
                       size_t workspace_bytes, dsa_stream_t stream)
{
    if (T < 0 || S < 1)
        return fail(DSA_ERR_INVALID_ARG, "T < 0 or S < 1");
    if (T == 0)
        return ok();
    if (!q || !kv || !q8 || !q_scale || !w || !k8 || !k_scale || !q_pos || !loss || !dw || !dq || !dk)
        return fail(DSA_ERR_INVALID_ARG, "null pointer argument");
    if (H < 1 || H > 128)
        return fail(DSA_ERR_UNSUPPORTED, "H must be in [1, 128]");
    if (d_I != 128 || (H_I != 64 && H_I != 32))
        return fail(DSA_ERR_UNSUPPORTED, "warm-up: (H_I, d_I) must be (64, 128) or (32, 128)");
    if (!(sm_scale > 0.f) || sm_scale > 1e30f)
        return fail(DSA_ERR_INVALID_ARG, "sm_scale must be positive and finite");
    if (!aligned16(q) || !aligned16(kv) || !aligned16(q8) || !aligned16(k8) || !aligned16(dq))
        return fail(DSA_ERR_ALIGNMENT, "q, kv, q8, k8 and dq must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return fail(DSA_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
    if (!workspace || workspace_bytes < warmup_workspace_bytes(T, S, H_I))
        return fail(DSA_ERR_WORKSPACE, "workspace missing or smaller than dsa_indexer_warmup_workspace_size");
    WarmupArgs a{q, kv, H, sm_scale, q8, q_scale, w, H_I, d_I, k8, k_scale, q_pos, T, S, loss, dw, dq, dk,
                 workspace, workspace_bytes};
    int rc = launch_warmup(a, reinterpret_cast<cudaStream_t>(stream), t_err, sizeof t_err);
    return rc == DSA_OK ? ok() : rc;
}

int dsa_quantize_fp8(const float *x, int64_t rows, int64_t cols, int scale_mode, void *codes, float *scale,
                     dsa_stream_t stream)
{
    if (rows < 0 || cols < 1)
        return fail(DSA_ERR_INVALID_ARG, "rows must be >= 0 and cols >= 1");
    if (scale_mode != DSA_SCALE_AMAX && scale_mode != DSA_SCALE_POW2)
        return fail(DSA_ERR_INVALID_ARG, "scale_mode must be DSA_SCALE_AMAX or DSA_SCALE_POW2");
    if (rows == 0)
        return ok();
    if (!x || !codes || !scale)
        return fail(DSA_ERR_INVALID_ARG, "null pointer argument");
    if (rows > (int64_t(1) << 40) / cols)
        return fail(DSA_ERR_UNSUPPORTED, "rows * cols too large");
    QuantizeArgs a{x, rows, cols, scale_mode, static_cast<uint8_t *>(codes), scale};
    int rc = launch_quantize(a, reinterpret_cast<cudaStream_t>(stream), t_err, sizeof t_err);
    return rc == DSA_OK ? ok() : rc;
}

namespace {

constexpr int kNormMaxCols = 16384;

bool bad_dtype(int t) { return t != DSA_BF16 && t != DSA_FP32; }
bool bad_scale_mode(int m) { return m != DSA_SCALE_AMAX && m != DSA_SCALE_POW2; }
bool bad_page_size(int n) { return n != 32 && n != 64 && n != 128; }

// rows * cols values of a tensor whose rows are ld apart stay addressable
bool too_large(int64_t rows, int64_t ld) { return rows > (int64_t(1) << 40) / ld; }

} // namespace

namespace {

// The argument checks of both norms: DSA_OK with *none set where there is nothing to do.
int check_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight, const void *bias, int64_t rows, int cols,
               int dtype, int weight_dtype, float eps, const void *residual_out, int64_t ldh, const void *out, int64_t ldo,
               const void *codes, const float *scale, int block, int scale_mode, bool *none)
{
    *none = rows == 0;
    if (rows < 0 || cols < 1)
        return fail(DSA_ERR_INVALID_ARG, "rows must be >= 0 and cols >= 1");
    if (cols > kNormMaxCols)
        return fail(DSA_ERR_UNSUPPORTED, "cols must be at most %d", kNormMaxCols);
    if (bad_dtype(dtype) || bad_dtype(weight_dtype))
        return fail(DSA_ERR_INVALID_ARG, "dtype and weight_dtype must be DSA_BF16 or DSA_FP32");
    if (!(eps >= 0.f) || eps > 1e30f)
        return fail(DSA_ERR_INVALID_ARG, "eps must be finite and not negative");
    if (bad_scale_mode(scale_mode))
        return fail(DSA_ERR_INVALID_ARG, "scale_mode must be DSA_SCALE_AMAX or DSA_SCALE_POW2");
    if (block != 0 && block != 128)
        return fail(DSA_ERR_INVALID_ARG, "block must be 0 (one scale per row) or 128");
    if (rows == 0)
        return DSA_OK;
    if (!x || !weight)
        return fail(DSA_ERR_INVALID_ARG, "null pointer argument");
    if ((codes == nullptr) != (scale == nullptr))
        return fail(DSA_ERR_INVALID_ARG, "codes and scale go together");
    if (!residual_out && !out && !codes)
        return fail(DSA_ERR_INVALID_ARG, "no output given");
    if (ldx < cols || (residual && ldr < cols) || (residual_out && ldh < cols) || (out && ldo < cols))
        return fail(DSA_ERR_INVALID_ARG, "a row stride is below cols");
    if (rows > (int64_t)INT32_MAX || too_large(rows, ldx) || (residual && too_large(rows, ldr)) ||
        (residual_out && too_large(rows, ldh)) || (out && too_large(rows, ldo)))
        return fail(DSA_ERR_UNSUPPORTED, "rows too large");
    if (!aligned_to(dtype == DSA_FP32 ? 4 : 2, {x, residual, residual_out, out}) ||
        !aligned_to(weight_dtype == DSA_FP32 ? 4 : 2, {weight, bias}) || !aligned_to(4, {scale}))
        return fail(DSA_ERR_ALIGNMENT, "tensors must be aligned to their elements");
    return DSA_OK;
}

int check_norm_backward(const void *dy, const void *h, const void *weight, const void *dres, int64_t rows, int cols, int dtype,
                        int weight_dtype, float eps, const void *dx, const float *dweight, const float *dbias, size_t need,
                        const void *workspace, size_t workspace_bytes)
{
    if (rows < 0 || cols < 1)
        return fail(DSA_ERR_INVALID_ARG, "rows must be >= 0 and cols >= 1");
    if (cols > kNormMaxCols)
        return fail(DSA_ERR_UNSUPPORTED, "cols must be at most %d", kNormMaxCols);
    if (bad_dtype(dtype) || bad_dtype(weight_dtype))
        return fail(DSA_ERR_INVALID_ARG, "dtype and weight_dtype must be DSA_BF16 or DSA_FP32");
    if (!(eps >= 0.f) || eps > 1e30f)
        return fail(DSA_ERR_INVALID_ARG, "eps must be finite and not negative");
    if (!dweight || (rows > 0 && (!dy || !h || !weight || !dx)))
        return fail(DSA_ERR_INVALID_ARG, "null pointer argument");
    if (rows > (int64_t)INT32_MAX)
        return fail(DSA_ERR_UNSUPPORTED, "rows too large");
    if (!aligned_to(dtype == DSA_FP32 ? 4 : 2, {dy, h, dres, dx}) || !aligned_to(weight_dtype == DSA_FP32 ? 4 : 2, {weight}) ||
        !aligned_to(4, {dweight, dbias}))
        return fail(DSA_ERR_ALIGNMENT, "tensors must be aligned to their elements");
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(DSA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? workspace_bytes : 0);
    if (!aligned16(workspace))
        return fail(DSA_ERR_ALIGNMENT, "workspace must be 16-byte aligned");
    return DSA_OK;
}

} // namespace

int dsa_rmsnorm(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight, int64_t rows, int cols,
                int dtype, int weight_dtype, float eps, void *residual_out, int64_t ldh, void *out, int64_t ldo, void *codes,
                float *scale, int block, int scale_mode, dsa_stream_t stream)
{
    bool none;
    int rc = check_norm(x, ldx, residual, ldr, weight, nullptr, rows, cols, dtype, weight_dtype, eps, residual_out, ldh, out, ldo, codes,
                        scale, block, scale_mode, &none);
    if (rc != DSA_OK)
        return rc;
    if (none)
        return ok();
    NormArgs a{x, residual, weight, rows, cols, ldx, ldr, ldh, ldo, dtype == DSA_FP32, weight_dtype == DSA_FP32, eps,
               residual_out, out, static_cast<uint8_t *>(codes), scale, block, scale_mode};
    rc = launch_rmsnorm(a, reinterpret_cast<cudaStream_t>(stream), t_err, sizeof t_err);
    return rc == DSA_OK ? ok() : rc;
}

int dsa_layernorm(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight, const void *bias,
                  int64_t rows, int cols, int dtype, int weight_dtype, float eps, void *residual_out, int64_t ldh, void *out,
                  int64_t ldo, void *codes, float *scale, int block, int scale_mode, dsa_stream_t stream)
{
    bool none;
    int rc = check_norm(x, ldx, residual, ldr, weight, bias, rows, cols, dtype, weight_dtype, eps, residual_out, ldh, out, ldo, codes,
                        scale, block, scale_mode, &none);
    if (rc != DSA_OK)
        return rc;
    if (none)
        return ok();
    NormArgs a{x, residual, weight, rows, cols, ldx, ldr, ldh, ldo, dtype == DSA_FP32, weight_dtype == DSA_FP32, eps,
               residual_out, out, static_cast<uint8_t *>(codes), scale, block, scale_mode, bias};
    rc = launch_layernorm(a, reinterpret_cast<cudaStream_t>(stream), t_err, sizeof t_err);
    return rc == DSA_OK ? ok() : rc;
}

size_t dsa_rmsnorm_backward_workspace_size(int64_t rows, int cols)
{
    if (rows < 0 || rows > (int64_t)INT32_MAX || cols < 1 || cols > kNormMaxCols)
        return 0;
    return rmsnorm_backward_workspace_bytes(rows, cols);
}

int dsa_rmsnorm_backward(const void *dy, const void *h, const void *weight, const void *dres, int64_t rows, int cols,
                         int dtype, int weight_dtype, float eps, void *dx, float *dweight, void *workspace,
                         size_t workspace_bytes, dsa_stream_t stream)
{
    int rc = check_norm_backward(dy, h, weight, dres, rows, cols, dtype, weight_dtype, eps, dx, dweight, nullptr,
                                 dsa_rmsnorm_backward_workspace_size(rows, cols), workspace, workspace_bytes);
    if (rc != DSA_OK)
        return rc;
    NormBackwardArgs a{dy, h, weight, dres, rows, cols, dtype == DSA_FP32, weight_dtype == DSA_FP32, eps, dx, dweight,
                       workspace};
    rc = launch_rmsnorm_backward(a, reinterpret_cast<cudaStream_t>(stream), t_err, sizeof t_err);
    return rc == DSA_OK ? ok() : rc;
}

size_t dsa_layernorm_backward_workspace_size(int64_t rows, int cols)
{
    if (rows < 0 || rows > (int64_t)INT32_MAX || cols < 1 || cols > kNormMaxCols)
        return 0;
    return layernorm_backward_workspace_bytes(rows, cols);
}

int dsa_layernorm_backward(const void *dy, const void *h, const void *weight, const void *dres, int64_t rows, int cols,
                           int dtype, int weight_dtype, float eps, void *dx, float *dweight, float *dbias, void *workspace,
                           size_t workspace_bytes, dsa_stream_t stream)
{
    int rc = check_norm_backward(dy, h, weight, dres, rows, cols, dtype, weight_dtype, eps, dx, dweight, dbias,
                                 dsa_layernorm_backward_workspace_size(rows, cols), workspace, workspace_bytes);
    if (rc != DSA_OK)
        return rc;
    NormBackwardArgs a{dy, h, weight, dres, rows, cols, dtype == DSA_FP32, weight_dtype == DSA_FP32, eps, dx, dweight,
                       workspace, dbias};
    rc = launch_layernorm_backward(a, reinterpret_cast<cudaStream_t>(stream), t_err, sizeof t_err);
    return rc == DSA_OK ? ok() : rc;
}

int dsa_quantize_fp8_blocks(const void *x, int64_t ldx, int64_t rows, int64_t cols, int dtype, int block_rows, int scale_mode,
                            void *codes, int64_t ld_codes, float *scale, void *codes_t, int64_t ld_codes_t, float *scale_t,
                            dsa_stream_t stream)
{
    if (rows < 0 || cols < 1)
        return fail(DSA_ERR_INVALID_ARG, "rows must be >= 0 and cols >= 1");
    if (bad_dtype(dtype))
        return fail(DSA_ERR_INVALID_ARG, "dtype must be DSA_BF16 or DSA_FP32");
    if (block_rows != 1 && block_rows != 128)
        return fail(DSA_ERR_INVALID_ARG, "block_rows must be 1 or 128");
    if (bad_scale_mode(scale_mode))
        return fail(DSA_ERR_INVALID_ARG, "scale_mode must be DSA_SCALE_AMAX or DSA_SCALE_POW2");
    if (rows == 0)
        return ok();
    if (!x)
        return fail(DSA_ERR_INVALID_ARG, "null pointer argument");
    if ((codes == nullptr) != (scale == nullptr) || (codes_t == nullptr) != (scale_t == nullptr))
        return fail(DSA_ERR_INVALID_ARG, "codes and scale go together, and so do codes_t and scale_t");
    if (!codes && !codes_t)
        return fail(DSA_ERR_INVALID_ARG, "no output given");
    if (ldx < cols || (codes && ld_codes < cols) || (codes_t && ld_codes_t < rows))
        return fail(DSA_ERR_INVALID_ARG, "a row stride is below the row's width");
    if (too_large(rows, ldx) || (codes && too_large(rows, ld_codes)) || (codes_t && too_large(cols, ld_codes_t)) ||
        (rows + 127) / 128 > (int64_t)INT32_MAX / ((cols + 127) / 128))
        return fail(DSA_ERR_UNSUPPORTED, "rows * cols too large");
    if (!aligned_to(dtype == DSA_FP32 ? 4 : 2, {x}) || !aligned_to(4, {scale, scale_t}))
        return fail(DSA_ERR_ALIGNMENT, "tensors must be aligned to their elements");
    QuantizeBlocksArgs a{x, ldx, rows, cols, dtype == DSA_FP32, block_rows, scale_mode, static_cast<uint8_t *>(codes), ld_codes,
                         scale, static_cast<uint8_t *>(codes_t), ld_codes_t, scale_t};
    int rc = launch_quantize_blocks(a, reinterpret_cast<cudaStream_t>(stream), t_err, sizeof t_err);
    return rc == DSA_OK ? ok() : rc;
}

int dsa_gemm_fp8(const void *a, int64_t lda, const float *a_scale, const void *b, int64_t ldb, const float *b_scale,
                 int b_block_rows, int M, int N, int K, void *out, int64_t ldo, int out_dtype, dsa_stream_t stream)
{
    constexpr int kMost = 1 << 30;
    if (M < 0 || N < 0 || K < 0)
        return fail(DSA_ERR_INVALID_ARG, "M, N and K must not be negative");
    if (b_block_rows != 1 && b_block_rows != 128)
        return fail(DSA_ERR_INVALID_ARG, "b_block_rows must be 1 or 128");
    if (bad_dtype(out_dtype))
        return fail(DSA_ERR_INVALID_ARG, "out_dtype must be DSA_BF16 or DSA_FP32");
    if (M > kMost || N > kMost || K > kMost)
        return fail(DSA_ERR_UNSUPPORTED, "M, N and K must be at most 2^30");
    if (M == 0 || N == 0)
        return ok();
    if (!out || (K > 0 && (!a || !a_scale || !b || !b_scale)))
        return fail(DSA_ERR_INVALID_ARG, "null pointer argument");
    // a stride that no address depends on says nothing
    if (M == 1 || K == 0)
        lda = ((int64_t)K + 15) & ~int64_t(15);
    if (N == 1 || K == 0)
        ldb = ((int64_t)K + 15) & ~int64_t(15);
    if (lda < K || ldb < K || ldo < N)
        return fail(DSA_ERR_INVALID_ARG, "a row stride is below the row's width");
    // a tile of 128 x 16 outputs, by up to 8 CTAs
    if (too_large(M, lda + 1) || too_large(N, ldb + 1) || too_large(M, ldo) ||
        ((int64_t)M + 127) / 128 * (((int64_t)N + 127) / 128) > (int64_t)INT32_MAX / 16)
        return fail(DSA_ERR_UNSUPPORTED, "tensors too large");
    if (!aligned16(a) || !aligned16(b) || lda % 16 || ldb % 16)
        return fail(DSA_ERR_ALIGNMENT, "a, b and their row strides must be 16-byte aligned");
    if (!aligned_to(4, {a_scale, b_scale}) || !aligned_to(out_dtype == DSA_FP32 ? 4 : 2, {out}))
        return fail(DSA_ERR_ALIGNMENT, "tensors must be aligned to their elements");
    GemmFp8Args g{a, lda, a_scale, b, ldb, b_scale, b_block_rows == 128, M, N, K, out, ldo, out_dtype == DSA_FP32};
    int rc = launch_gemm_fp8(g, reinterpret_cast<cudaStream_t>(stream), t_err, sizeof t_err);
    return rc == DSA_OK ? ok() : rc;
}

int dsa_cache_append(const int32_t *pos, const int32_t *seq, int T, const int32_t *block_table, int num_seqs, int max_pages,
                     int num_pages, int page_size, const double *inv_freq, const void *kv, int64_t ld_kv,
                     const void *kv_weight, int weight_dtype, float eps, void *kv_pool, const void *kI, int64_t ld_kI,
                     int k_dtype, int scale_mode, void *k8_pool, float *ks_pool, dsa_stream_t stream)
{
    if (T < 0)
        return fail(DSA_ERR_INVALID_ARG, "T < 0");
    if (bad_page_size(page_size))
        return fail(DSA_ERR_UNSUPPORTED, "page_size must be 32, 64 or 128");
    if (bad_dtype(weight_dtype) || bad_dtype(k_dtype))
        return fail(DSA_ERR_INVALID_ARG, "weight_dtype and k_dtype must be DSA_BF16 or DSA_FP32");
    if (bad_scale_mode(scale_mode))
        return fail(DSA_ERR_INVALID_ARG, "scale_mode must be DSA_SCALE_AMAX or DSA_SCALE_POW2");
    if (!(eps >= 0.f) || eps > 1e30f)
        return fail(DSA_ERR_INVALID_ARG, "eps must be finite and not negative");
    if (T == 0)
        return ok();
    if (!pos || !block_table || !inv_freq)
        return fail(DSA_ERR_INVALID_ARG, "null pointer argument");
    if (!kv && !kI)
        return fail(DSA_ERR_INVALID_ARG, "neither kv nor kI given");
    if ((kv && !kv_pool) || (kI && (!k8_pool || !ks_pool)))
        return fail(DSA_ERR_INVALID_ARG, "kv needs kv_pool, kI needs k8_pool and ks_pool");
    if (num_seqs <= 0 || max_pages <= 0 || num_pages <= 0)
        return fail(DSA_ERR_INVALID_ARG, "num_seqs, max_pages and num_pages must be positive");
    if (!seq && T > num_seqs)
        return fail(DSA_ERR_INVALID_ARG, "without seq the block table needs a row per token");
    if ((kv && ld_kv < 576) || (kI && ld_kI < 128))
        return fail(DSA_ERR_INVALID_ARG, "a row stride is below the row's width");
    if (T > (1 << 30))
        return fail(DSA_ERR_UNSUPPORTED, "T must be at most 2^30");
    if ((kv && too_large(T, ld_kv)) || (kI && too_large(T, ld_kI)))
        return fail(DSA_ERR_UNSUPPORTED, "row stride too large");
    if (!aligned_to(4, {pos, seq, block_table, kI ? ks_pool : nullptr}) || !aligned_to(8, {inv_freq}))
        return fail(DSA_ERR_ALIGNMENT, "tensors must be aligned to their elements");
    if (kv && (!aligned16(kv) || !aligned16(kv_pool) || !aligned16(kv_weight) || ld_kv % 8))
        return fail(DSA_ERR_ALIGNMENT, "kv, its row stride, kv_weight and kv_pool must be 16-byte aligned");
    if (kI && (!aligned16(kI) || !aligned16(k8_pool) || ld_kI % (k_dtype == DSA_FP32 ? 4 : 8)))
        return fail(DSA_ERR_ALIGNMENT, "kI, its row stride and k8_pool must be 16-byte aligned");
    CacheAppendArgs a{pos, seq, block_table, T, num_seqs, max_pages, num_pages, page_size, inv_freq, kv, ld_kv, kv_weight,
                      weight_dtype == DSA_FP32, eps, kv_pool, kI, ld_kI, k_dtype == DSA_FP32, scale_mode,
                      static_cast<uint8_t *>(k8_pool), ks_pool};
    int rc = launch_cache_append(a, reinterpret_cast<cudaStream_t>(stream), t_err, sizeof t_err);
    return rc == DSA_OK ? ok() : rc;
}

int dsa_rope_queries(const int32_t *pos, const double *inv_freq, int T, const void *q_rope, int64_t st_t, int64_t st_h, int H,
                     void *q, const void *qI, int H_I, int i_dtype, int scale_mode, void *q8, float *q_scale,
                     dsa_stream_t stream)
{
    if (T < 0)
        return fail(DSA_ERR_INVALID_ARG, "T < 0");
    if (bad_dtype(i_dtype))
        return fail(DSA_ERR_INVALID_ARG, "i_dtype must be DSA_BF16 or DSA_FP32");
    if (bad_scale_mode(scale_mode))
        return fail(DSA_ERR_INVALID_ARG, "scale_mode must be DSA_SCALE_AMAX or DSA_SCALE_POW2");
    if (T == 0)
        return ok();
    if (!pos || !inv_freq)
        return fail(DSA_ERR_INVALID_ARG, "null pointer argument");
    if (!q_rope && !qI)
        return fail(DSA_ERR_INVALID_ARG, "neither q_rope nor qI given");
    if ((q_rope && !q) || (qI && (!q8 || !q_scale)))
        return fail(DSA_ERR_INVALID_ARG, "q_rope needs q, qI needs q8 and q_scale");
    if (T > (1 << 30))
        return fail(DSA_ERR_UNSUPPORTED, "T must be at most 2^30");
    if (q_rope && (H < 1 || H > 128))
        return fail(DSA_ERR_UNSUPPORTED, "H must be in [1, 128]");
    if (qI && (H_I < 1 || H_I > 64))
        return fail(DSA_ERR_UNSUPPORTED, "H_I must be in [1, 64]");
    if (q_rope && (st_t < 0 || st_h < 0 || too_large(T, st_t + 1) || too_large(H, st_h + 1)))
        return fail(DSA_ERR_INVALID_ARG, "q_rope strides out of range");
    if (q_rope && (!aligned16(q_rope) || !aligned16(q) || st_t % 8 || st_h % 8))
        return fail(DSA_ERR_ALIGNMENT, "q_rope, its strides and q must be 16-byte aligned");
    if (qI && (!aligned16(qI) || !aligned16(q8)))
        return fail(DSA_ERR_ALIGNMENT, "qI and q8 must be 16-byte aligned");
    if (!aligned_to(4, {pos, qI ? q_scale : nullptr}) || !aligned_to(8, {inv_freq}))
        return fail(DSA_ERR_ALIGNMENT, "tensors must be aligned to their elements");
    RopeQueriesArgs a{pos, inv_freq, T, H, H_I, q_rope, st_t, st_h, q, qI, i_dtype == DSA_FP32, scale_mode,
                      static_cast<uint8_t *>(q8), q_scale};
    int rc = launch_rope_queries(a, reinterpret_cast<cudaStream_t>(stream), t_err, sizeof t_err);
    return rc == DSA_OK ? ok() : rc;
}

int dsa_index_rope_backward(const float *g, const int32_t *pos, const double *inv_freq, int T, int H_I, void *dx, int dtype,
                            dsa_stream_t stream)
{
    if (T < 0)
        return fail(DSA_ERR_INVALID_ARG, "T < 0");
    if (bad_dtype(dtype))
        return fail(DSA_ERR_INVALID_ARG, "dtype must be DSA_BF16 or DSA_FP32");
    if (H_I < 1 || H_I > 64)
        return fail(DSA_ERR_UNSUPPORTED, "H_I must be in [1, 64]");
    if (T == 0)
        return ok();
    if (!g || !pos || !inv_freq || !dx)
        return fail(DSA_ERR_INVALID_ARG, "null pointer argument");
    if (T > (1 << 30))
        return fail(DSA_ERR_UNSUPPORTED, "T must be at most 2^30");
    if (!aligned16(g) || !aligned16(dx))
        return fail(DSA_ERR_ALIGNMENT, "g and dx must be 16-byte aligned");
    if (!aligned_to(4, {pos}) || !aligned_to(8, {inv_freq}))
        return fail(DSA_ERR_ALIGNMENT, "tensors must be aligned to their elements");
    IndexRopeBackwardArgs a{g, pos, inv_freq, T, H_I, dx, dtype == DSA_FP32};
    int rc = launch_index_rope_backward(a, reinterpret_cast<cudaStream_t>(stream), t_err, sizeof t_err);
    return rc == DSA_OK ? ok() : rc;
}

size_t dsa_mla_decode_workspace_size(int B, int H)
{
    if (B < 1 || B > 65535 || H < 1 || H > 128)
        return 0;
    return dense_mla_workspace_bytes(B, H);
}

int dsa_mla_decode_paged(const void *q, const void *kv_pool, int num_pages, int page_size, const int32_t *block_table,
                         int max_pages, const int32_t *ctx_len, int B, int H, float sm_scale, void *out, float *lse,
                         void *workspace, size_t workspace_bytes, dsa_stream_t stream)
{
    if (B < 0)
        return fail(DSA_ERR_INVALID_ARG, "B < 0");
    if (B > 65535)
        return fail(DSA_ERR_UNSUPPORTED, "B must be at most 65535");
    if (H < 1 || H > 128)
        return fail(DSA_ERR_UNSUPPORTED, "H must be in [1, 128]");
    if (B == 0)
        return ok();
    if (!q || !kv_pool || !block_table || !ctx_len || !out || !lse)
        return fail(DSA_ERR_INVALID_ARG, "null pointer argument");
    if (num_pages <= 0 || max_pages <= 0)
        return fail(DSA_ERR_INVALID_ARG, "num_pages and max_pages must be positive");
    if (bad_page_size(page_size))
        return fail(DSA_ERR_UNSUPPORTED, "page_size must be 32, 64 or 128");
    if ((int64_t)num_pages * page_size > (int64_t)INT32_MAX || (int64_t)max_pages * page_size > (int64_t)INT32_MAX)
        return fail(DSA_ERR_UNSUPPORTED, "pool or block table too large");
    if (!aligned16(q) || !aligned16(kv_pool) || !aligned16(out))
        return fail(DSA_ERR_ALIGNMENT, "q, kv_pool and out must be 16-byte aligned");
    if (!aligned_to(4, {block_table, ctx_len, lse}))
        return fail(DSA_ERR_ALIGNMENT, "tensors must be aligned to their elements");
    if (!(sm_scale > 0.f) || sm_scale > 1e30f)
        return fail(DSA_ERR_INVALID_ARG, "sm_scale must be positive and finite");
    const size_t need = dense_mla_workspace_bytes(B, H);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(DSA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? workspace_bytes : 0);
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return fail(DSA_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
    DenseMlaArgs a{q, kv_pool, num_pages, page_size, block_table, max_pages, ctx_len, B, H, sm_scale, out, lse, workspace};
    int rc = launch_dense_mla(a, reinterpret_cast<cudaStream_t>(stream), t_err, sizeof t_err);
    return rc == DSA_OK ? ok() : rc;
}

int dsa_topk(const float *logits, int64_t ld, int T, const int32_t *valid_len, int k, int32_t *idx,
             dsa_stream_t stream)
{
    if (T < 0)
        return fail(DSA_ERR_INVALID_ARG, "T < 0");
    if (T == 0)
        return ok();
    if (!logits || !valid_len || !idx)
        return fail(DSA_ERR_INVALID_ARG, "null pointer argument");
    if (k < 1 || k > 4096)
        return fail(DSA_ERR_UNSUPPORTED, "k must be in [1, 4096]");
    if (ld < 1 || ld > (int64_t(1) << 28))
        return fail(DSA_ERR_UNSUPPORTED, "ld must be in [1, 2^28]");
    TopkArgs a{logits, ld, T, valid_len, k, idx};
    int rc = launch_topk(a, reinterpret_cast<cudaStream_t>(stream), t_err, sizeof t_err);
    return rc == DSA_OK ? ok() : rc;
}

int dsa_sparse_mla_prefill(const void *q, const void *kv, int S, const int32_t *idx, int T, int H, int k,
                           float sm_scale, void *out, float *lse, dsa_stream_t stream)
{
    if (T < 0 || S < 0)
        return fail(DSA_ERR_INVALID_ARG, "T < 0 or S < 0");
    if (T == 0)
        return ok();
    if (!q || !kv || !idx || !out || !lse)
        return fail(DSA_ERR_INVALID_ARG, "null pointer argument");
    if (H < 1 || H > 128)
        return fail(DSA_ERR_UNSUPPORTED, "H must be in [1, 128]");
    if (k < 1 || k > 4096)
        return fail(DSA_ERR_UNSUPPORTED, "k must be in [1, 4096]");
    if (!aligned16(q) || !aligned16(kv) || !aligned16(out))
        return fail(DSA_ERR_ALIGNMENT, "q, kv and out must be 16-byte aligned");
    if (!(sm_scale > 0.f) || sm_scale > 1e30f)
        return fail(DSA_ERR_INVALID_ARG, "sm_scale must be positive and finite");
    MlaArgs a{};
    a.q = q;
    a.kv = kv;
    a.S = S;
    a.idx = idx;
    a.T = T;
    a.H = H;
    a.k = k;
    a.sm_scale = sm_scale;
    a.out = out;
    a.lse = lse;
    int rc = launch_mla_prefill(a, reinterpret_cast<cudaStream_t>(stream), t_err, sizeof t_err);
    return rc == DSA_OK ? ok() : rc;
}

size_t dsa_sparse_mla_decode_workspace_size(int B, int H, int k)
{
    if (B < 0 || H < 1 || H > 128 || k < 1 || k > 4096)
        return 0;
    return mla_decode_workspace_bytes(B, H, k);
}

int dsa_sparse_mla_decode_paged(const void *q, const void *kv_pool, int num_pages, int page_size,
                                const int32_t *block_table, int max_pages, const int32_t *ctx_len, const int32_t *idx,
                                int B, int H, int k, float sm_scale, void *out, float *lse, void *workspace,
                                size_t workspace_bytes, dsa_stream_t stream)
{
    if (B < 0)
        return fail(DSA_ERR_INVALID_ARG, "B < 0");
    if (B == 0)
        return ok();
    if (!q || !kv_pool || !block_table || !ctx_len || !idx || !out || !lse)
        return fail(DSA_ERR_INVALID_ARG, "null pointer argument");
    if (H < 1 || H > 128)
        return fail(DSA_ERR_UNSUPPORTED, "H must be in [1, 128]");
    if (k < 1 || k > 4096)
        return fail(DSA_ERR_UNSUPPORTED, "k must be in [1, 4096]");
    if (num_pages <= 0 || max_pages <= 0 || page_size <= 0)
        return fail(DSA_ERR_INVALID_ARG, "num_pages, max_pages and page_size must be positive");
    if ((int64_t)num_pages * page_size > (int64_t)INT32_MAX)
        return fail(DSA_ERR_UNSUPPORTED, "pool too large");
    if (!aligned16(q) || !aligned16(kv_pool) || !aligned16(out))
        return fail(DSA_ERR_ALIGNMENT, "q, kv_pool and out must be 16-byte aligned");
    if (!(sm_scale > 0.f) || sm_scale > 1e30f)
        return fail(DSA_ERR_INVALID_ARG, "sm_scale must be positive and finite");
    const size_t need = mla_decode_workspace_bytes(B, H, k);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(DSA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
    if (workspace && (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return fail(DSA_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
    MlaArgs a{};
    a.q = q;
    a.kv = kv_pool;
    a.S = num_pages * page_size;
    a.idx = idx;
    a.T = B;
    a.H = H;
    a.k = k;
    a.sm_scale = sm_scale;
    a.out = out;
    a.lse = lse;
    a.block_table = block_table;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.ctx_len = ctx_len;
    a.workspace = workspace;
    a.workspace_bytes = workspace_bytes;
    int rc = launch_mla_decode(a, reinterpret_cast<cudaStream_t>(stream), t_err, sizeof t_err);
    return rc == DSA_OK ? ok() : rc;
}

} // extern "C"

// ---------------------------------------------------------------------------
// Self-test of the failure detection: one CTA waits, through the same bounded
// mbarrier wait every pipeline uses, on a barrier that nothing arrives on.
namespace dsa {
namespace {

__global__ void wait_timeout_kernel(uint64_t limit_ns, unsigned *status)
{
    __shared__ __align__(8) uint64_t bar;
    __shared__ int abort_flag;
    grid_dep_wait();
    grid_dep_launch();
    const uint32_t b = smem_u32(&bar);
    if (threadIdx.x == 0) {
        mbar_init(b, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    // phase 0 never completes: the wait gives up after limit_ns, sets
    // DSA_DEV_TIMEOUT and the kernel returns
    mbar_wait_warp(b, 0, &abort_flag, status, limit_ns);
}

} // namespace
} // namespace dsa

extern "C" int dsa_selftest_wait_timeout(uint32_t limit_us, dsa_stream_t stream)
{
    if (limit_us == 0 || limit_us > 1000000u)
        return fail(DSA_ERR_INVALID_ARG, "limit_us must be in [1, 1000000]");
    unsigned *status = device_status_ptr();
    if (!status)
        return fail(DSA_ERR_CUDA, "device status word unavailable");
    cudaError_t e = launch_pdl(wait_timeout_kernel, dim3(1), dim3(32), 0, reinterpret_cast<cudaStream_t>(stream), 1,
                               (uint64_t)limit_us * 1000u, status);
    if (e != cudaSuccess)
        return fail(DSA_ERR_CUDA, "self-test launch: %s", cudaGetErrorString(e));
    return ok();
}

// ---------------------------------------------------------------------------
// Allocation-free decode attention.  The workspace lives in this file-scope
// device array, which every device that loads the library holds until the
// process exits.  In host code the array's name only stands for it: the
// device address comes from cudaGetSymbolAddress, looked up once per device
// (with that device current) on the first call and kept.
namespace dsa {
namespace {

static __device__ __align__(256) unsigned char g_decode_static_ws[DSA_DECODE_STATIC_WS_BYTES];
void *g_decode_static_ws_ptr[kMaxDevices] = {};

// Device address of this device's static decode workspace, or null (message in *why).
void *decode_static_workspace(cudaError_t *why)
{
    *why = cudaSuccess;
    const int d = current_device();
    if (d < 0 || d >= kMaxDevices)
        return nullptr;
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_decode_static_ws_ptr[d]) {
        void *p = nullptr;
        *why = cudaGetSymbolAddress(&p, g_decode_static_ws);
        if (*why != cudaSuccess || !p)
            return nullptr;
        g_decode_static_ws_ptr[d] = p;
    }
    return g_decode_static_ws_ptr[d];
}

} // namespace
} // namespace dsa

extern "C" int dsa_sparse_mla_decode_paged_noalloc(const void *q, const void *kv_pool, int num_pages, int page_size,
                                                   const int32_t *block_table, int max_pages, const int32_t *ctx_len,
                                                   const int32_t *idx, int B, int H, int k, float sm_scale, void *out,
                                                   float *lse, dsa_stream_t stream)
{
    // 0 for bad arguments too: those are then reported by the call below
    const size_t need = dsa_sparse_mla_decode_workspace_size(B, H, k);
    if (need > (size_t)DSA_DECODE_STATIC_WS_BYTES)
        return fail(DSA_ERR_WORKSPACE,
                    "decode with B=%d, H=%d, k=%d needs %zu bytes of workspace on this device, more than the "
                    "%zu-byte static buffer of the allocation-free entry point",
                    B, H, k, need, (size_t)DSA_DECODE_STATIC_WS_BYTES);
    cudaError_t why;
    void *ws = decode_static_workspace(&why);
    if (!ws)
        return fail(DSA_ERR_CUDA, "address of the static decode workspace: %s",
                    why == cudaSuccess ? "no current device" : cudaGetErrorString(why));
    return dsa_sparse_mla_decode_paged(q, kv_pool, num_pages, page_size, block_table, max_pages, ctx_len, idx, B, H, k,
                                       sm_scale, out, lse, ws, (size_t)DSA_DECODE_STATIC_WS_BYTES, stream);
}
