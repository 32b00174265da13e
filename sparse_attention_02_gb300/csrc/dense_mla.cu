// Dense MLA attention of single tokens over the paged latent cache on sm_103a.
//
// The attention of layers, steps and contexts that select nothing: MQA mode,
// one 576-wide latent row is the key of every head and its first 512 columns
// the value (release summary "DeepSeek-V3.2-Exp: Boosting Long-Context
// Efficiency with DeepSeek Sparse Attention", section "Method"), over all keys
// s < ctx_len[b]:
//     S[h,s] = sm_scale * <q[b,h,:576], kv[s,:576]>
//     out[b,h] = sum_s softmax_s(S[h,:]) kv[s,:512],  lse = ln sum_s exp S[h,s]
//
// This form: one warp per head, eight heads a CTA, keys staged in shared
// memory 32 at a time; a row's keys are split over up to 64 CTAs whose
// normalised parts a second kernel joins by their LSEs.  All in fp32.
#include "common.cuh"
#include "launch.h"

#include <stdio.h>

namespace dsa {
namespace {

constexpr int kD = 576, kDv = 512;
constexpr int kTile = 32;
constexpr int kThreads = 256;
constexpr int kHeads = 8;
constexpr int kMaxSplits = 64;

struct Parts {
    float *o;   // [splits, B, H, 512]
    float *lse; // [splits, B, H]
    int splits;
};

__device__ __forceinline__ float lo16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi16(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

__global__ void __launch_bounds__(kThreads) dense_mla_simple_kernel(DenseMlaArgs a, Parts p, unsigned *status)
{
    __shared__ uint32_t kv[kTile][kD / 2];
    __shared__ int ok[kTile];
    grid_dep_wait();
    grid_dep_launch();
    const int split = blockIdx.x, b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.z * kHeads + warp;
    int64_t ctx = a.ctx_len[b];
    const int64_t most = (int64_t)a.max_pages * a.page_size;
    if (ctx > most) {
        if (threadIdx.x == 0)
            atomicOr(status, DSA_DEV_BAD_POSITION);
        ctx = most;
    }
    const int64_t tiles = ctx > 0 ? (ctx + kTile - 1) / kTile : 0;
    const int64_t t0 = tiles * split / p.splits, t1 = tiles * (split + 1) / p.splits;
    float q[18], acc[16] = {}, m = -INFINITY, l = 0.f;
    if (h < a.H) {
        const uint32_t *src = reinterpret_cast<const uint32_t *>(a.q) + ((int64_t)b * a.H + h) * (kD / 2);
#pragma unroll
        for (int i = 0; i < 9; ++i) {
            const uint32_t w = src[lane + 32 * i];
            q[2 * i] = lo16(w) * a.sm_scale;
            q[2 * i + 1] = hi16(w) * a.sm_scale;
        }
    }
    for (int64_t t = t0; t < t1; ++t) {
        __syncthreads();
        for (int r = warp; r < kTile; r += kThreads / 32) {
            const int64_t s = t * kTile + r;
            int page = -1;
            if (s < ctx) {
                page = a.block_table[(int64_t)b * a.max_pages + s / a.page_size];
                if (page < 0 || page >= a.num_pages) {
                    page = -1;
                    if (lane == 0)
                        atomicOr(status, DSA_DEV_BAD_PAGE);
                }
            }
            const uint32_t *src = reinterpret_cast<const uint32_t *>(a.kv_pool) +
                                  (page < 0 ? 0 : ((int64_t)page * a.page_size + s % a.page_size) * (kD / 2));
#pragma unroll
            for (int i = 0; i < 9; ++i)
                kv[r][lane + 32 * i] = page < 0 ? 0u : src[lane + 32 * i];
            if (lane == 0)
                ok[r] = page >= 0;
        }
        __syncthreads();
        if (h >= a.H)
            continue;
        float sc = -INFINITY;
        for (int r = 0; r < kTile; ++r) {
            float d = 0.f;
#pragma unroll
            for (int i = 0; i < 9; ++i) {
                const uint32_t w = kv[r][lane + 32 * i];
                d = fmaf(q[2 * i], lo16(w), fmaf(q[2 * i + 1], hi16(w), d));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                d += __shfl_xor_sync(0xffffffffu, d, o);
            if (lane == r && ok[r])
                sc = d;
        }
        float top = sc;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = fmaxf(top, m);
        if (top == -INFINITY)
            continue;
        const float keep = expf(m - top), pr = expf(sc - top);
        float sum = pr;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l = l * keep + sum;
        m = top;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            acc[i] *= keep;
        for (int r = 0; r < kTile; ++r) {
            const float w = __shfl_sync(0xffffffffu, pr, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t v = kv[r][lane + 32 * i];
                acc[2 * i] = fmaf(w, lo16(v), acc[2 * i]);
                acc[2 * i + 1] = fmaf(w, hi16(v), acc[2 * i + 1]);
            }
        }
    }
    if (h >= a.H)
        return;
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const int64_t row = ((int64_t)split * a.B + b) * a.H + h;
    float2 *o = reinterpret_cast<float2 *>(p.o + row * kDv);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        o[lane + 32 * i] = make_float2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    if (lane == 0)
        p.lse[row] = m == -INFINITY ? -INFINITY : m + logf(l);
}

// One warp per (row, head): O = sum_i exp(LSE_i - LSE) O_i.
__global__ void __launch_bounds__(kThreads) dense_mla_join_kernel(DenseMlaArgs a, Parts p)
{
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    const int64_t rows = (int64_t)a.B * a.H, row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (row >= rows)
        return;
    float top = -INFINITY, sum = 0.f, acc[16] = {};
    for (int s = 0; s < p.splits; ++s)
        top = fmaxf(top, p.lse[s * rows + row]);
    if (top != -INFINITY)
        for (int s = 0; s < p.splits; ++s) {
            const float w = expf(p.lse[s * rows + row] - top);
            const float2 *o = reinterpret_cast<const float2 *>(p.o + (s * rows + row) * kDv);
            sum += w;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 v = o[lane + 32 * i];
                acc[2 * i] = fmaf(w, v.x, acc[2 * i]);
                acc[2 * i + 1] = fmaf(w, v.y, acc[2 * i + 1]);
            }
        }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    __nv_bfloat162 *out = reinterpret_cast<__nv_bfloat162 *>(a.out) + row * (kDv / 2);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        out[lane + 32 * i] = __floats2bfloat162_rn(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    if (lane == 0)
        a.lse[row] = top == -INFINITY ? -INFINITY : top + logf(sum);
}

int splits_of(int B, int H)
{
    const int64_t ctas = (int64_t)B * ((H + kHeads - 1) / kHeads);
    const int64_t want = (4LL * num_sms() + ctas - 1) / ctas;
    return (int)(want < kMaxSplits ? want : kMaxSplits);
}

} // namespace

size_t dense_mla_workspace_bytes(int B, int H) { return (size_t)splits_of(B, H) * B * H * (kDv + 1) * sizeof(float); }

int launch_dense_mla(const DenseMlaArgs &a, cudaStream_t stream, char *err, size_t errlen)
{
    unsigned *status = device_status_ptr();
    if (!status) {
        snprintf(err, errlen, "device status word unavailable");
        return DSA_ERR_CUDA;
    }
    Parts p;
    p.splits = splits_of(a.B, a.H);
    p.o = static_cast<float *>(a.workspace);
    p.lse = p.o + (size_t)p.splits * a.B * a.H * kDv;
    cudaError_t e = launch_pdl(dense_mla_simple_kernel, dim3(p.splits, a.B, (a.H + kHeads - 1) / kHeads), dim3(kThreads), 0,
                               stream, 1, a, p, status);
    if (e == cudaSuccess)
        e = launch_pdl(dense_mla_join_kernel, dim3((unsigned)(((int64_t)a.B * a.H + 7) / 8)), dim3(kThreads), 0, stream, 1, a,
                       p);
    if (e != cudaSuccess) {
        snprintf(err, errlen, "dense MLA launch: %s", cudaGetErrorString(e));
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

} // namespace dsa
