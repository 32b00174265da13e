// FP8 operands of the 128-block product on sm_103a: E4M3 codes of a matrix and of
// its transpose, each with a scale for every 128 values along its rows (or for
// every 128 x 128 block), from one read.
//
// The indexer and the projections run in FP8 ("AMD Instinct MI355X GPUs Power
// DeepSeek-V3.2-Exp", section "DeepSeek Sparse Attention (DSA)", item 1).  A
// product sums along rows of both operands, so a training step needs a gradient
// (and an activation) along its columns too: as rows of the transpose, with scales
// of their own.  scale = amax / 448 (or its power of two), code = E4M3(x / scale),
// as dsa_quantize_fp8.
//
// HBM-bound: 2 or 4 bytes in and 1 or 2 out per value.  A CTA takes a 128 x 128
// tile, a thread 8 x 8 of it in registers: a row's piece is 16 lanes of one warp, a
// column's a register row of 16 threads' maxima that meet in shared memory.
#include "rmsnorm.cuh"

namespace dsa {
namespace {

constexpr int kTile = 128;
constexpr int kThreads = 256;

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) quantize_blocks_kernel(QuantizeBlocksArgs a)
{
    __shared__ __align__(16) uint8_t turned[kTile * kTile];
    __shared__ float tops[8][kTile];
    __shared__ __align__(16) float col_scale[kTile];
    grid_dep_wait();
    grid_dep_launch();
    const int cblocks = (int)((a.cols + kTile - 1) / kTile), rblocks = (int)((a.rows + kTile - 1) / kTile);
    const int cb = blockIdx.x % cblocks, rb = blockIdx.x / cblocks;
    const int c = threadIdx.x & 15, rg = threadIdx.x >> 4, warp = threadIdx.x >> 5;
    const int64_t col = (int64_t)cb * kTile + 8 * c, row0 = (int64_t)rb * kTile + 8 * rg;
    const int ncol = a.cols - col >= 8 ? 8 : a.cols > col ? (int)(a.cols - col) : 0; // of this thread
    const int nrow = a.rows - row0 >= 8 ? 8 : a.rows > row0 ? (int)(a.rows - row0) : 0;
    const T *x = static_cast<const T *>(a.x) + row0 * a.ldx + col;
    Vec8<T> v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i].zero();
        if (i < nrow) {
            if (VEC && ncol == 8) {
                v[i].load(x + i * a.ldx);
            } else if (ncol > 0) {
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    f[j] = j < ncol ? (float)x[i * a.ldx + j] : 0.f;
                v[i].set(f);
            }
        }
    }
    float whole = 1.f; // scale of a 128 x 128 block
    if (a.block_rows == kTile) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float f[8];
            v[i].get(f);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                m = fmaxf(m, fabsf(f[j]));
        }
        m = warp_amax(m);
        if ((threadIdx.x & 31) == 0)
            tops[0][warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 8; ++w)
            m = fmaxf(m, tops[0][w]);
        whole = fp8_scale(m, a.scale_mode);
        if (threadIdx.x == 0) {
            if (a.codes)
                a.scale[(int64_t)rb * cblocks + cb] = whole;
            if (a.codes_t)
                a.scale_t[(int64_t)cb * rblocks + rb] = whole;
        }
    }
    if (a.codes) {
        uint8_t *codes = a.codes + row0 * a.ldc + col;
        const bool wide = ((reinterpret_cast<uintptr_t>(a.codes) | a.ldc) & 7) == 0 && ncol == 8;
        ScaleDivider div(whole);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float f[8];
            v[i].get(f);
            if (a.block_rows == 1) {
                float m = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    m = fmaxf(m, fabsf(f[j]));
#pragma unroll
                for (int o = 8; o > 0; o >>= 1)
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                div = ScaleDivider(fp8_scale(m, a.scale_mode));
                if (c == 0 && i < nrow)
                    a.scale[(row0 + i) * cblocks + cb] = div.s;
            }
            const uint32_t lo = e4m3x4(div, f[0], f[1], f[2], f[3]), hi = e4m3x4(div, f[4], f[5], f[6], f[7]);
            if (i < nrow) {
                if (wide) {
                    *reinterpret_cast<uint2 *>(codes + i * a.ldc) = make_uint2(lo, hi);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < ncol)
                            codes[i * a.ldc + j] = (uint8_t)((j < 4 ? lo : hi) >> (8 * (j & 3)));
                }
            }
        }
    }
    if (!a.codes_t)
        return;
    if (a.block_rows == 1) {
        float top[8] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float f[8];
            v[i].get(f);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                top[j] = fmaxf(top[j], fabsf(f[j]));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 16));
        if ((threadIdx.x & 16) == 0)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                tops[warp][8 * c + j] = top[j];
        __syncthreads();
        if (threadIdx.x < kTile) {
            float m = tops[0][threadIdx.x];
#pragma unroll
            for (int w = 1; w < 8; ++w)
                m = fmaxf(m, tops[w][threadIdx.x]);
            const float s = fp8_scale(m, a.scale_mode);
            col_scale[threadIdx.x] = s;
            const int64_t k = (int64_t)cb * kTile + threadIdx.x;
            if (k < a.cols)
                a.scale_t[k * rblocks + rb] = s;
        }
        __syncthreads();
    }
    // a column's eight codes of this thread go to shared memory as one word, at
    // place rg ^ c of the column's sixteen: the warp's words then fall into all banks
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const ScaleDivider div(a.block_rows == 1 ? col_scale[8 * c + j] : whole);
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float r[8];
            v[i].get(r);
            f[i] = r[j];
        }
        *reinterpret_cast<uint2 *>(turned + (8 * c + j) * kTile + ((rg ^ c) << 3)) =
            make_uint2(e4m3x4(div, f[0], f[1], f[2], f[3]), e4m3x4(div, f[4], f[5], f[6], f[7]));
    }
    __syncthreads();
    const bool wide = ((reinterpret_cast<uintptr_t>(a.codes_t) | a.ldt) & 15) == 0;
#pragma unroll
    for (int k = threadIdx.x; k < kTile * 8; k += kThreads) {
        const int64_t kc = (int64_t)cb * kTile + (k >> 3), r = (int64_t)rb * kTile + 16 * (k & 7);
        if (kc >= a.cols || r >= a.rows)
            continue;
        const int s = (k >> 6) & 15; // the c of this column
        uint4 w = *reinterpret_cast<const uint4 *>(turned + (k >> 3) * kTile + (((k & 7) ^ (s >> 1)) << 4));
        if (s & 1)
            w = make_uint4(w.z, w.w, w.x, w.y);
        uint8_t *dst = a.codes_t + kc * a.ldt + r;
        if (wide && r + 16 <= a.rows) {
            *reinterpret_cast<uint4 *>(dst) = w;
        } else {
            const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (r + j < a.rows)
                    dst[j] = (uint8_t)(words[j >> 2] >> (8 * (j & 3)));
        }
    }
}

} // namespace

int launch_quantize_blocks(const QuantizeBlocksArgs &a, cudaStream_t stream, char *err, size_t errlen)
{
    const int64_t tiles = ((a.rows + kTile - 1) / kTile) * ((a.cols + kTile - 1) / kTile);
    const bool vec = chunked(a.x, a.ldx * (a.x32 ? 4 : 2));
    auto go = [&](auto kernel) { return launch_pdl(kernel, dim3((unsigned)tiles), dim3(kThreads), 0, stream, 1, a); };
    cudaError_t e = a.x32 ? (vec ? go(quantize_blocks_kernel<float, true>) : go(quantize_blocks_kernel<float, false>))
                          : (vec ? go(quantize_blocks_kernel<__nv_bfloat16, true>) : go(quantize_blocks_kernel<__nv_bfloat16, false>));
    if (e != cudaSuccess) {
        snprintf(err, errlen, "quantize_blocks launch: %s", cudaGetErrorString(e));
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

} // namespace dsa
