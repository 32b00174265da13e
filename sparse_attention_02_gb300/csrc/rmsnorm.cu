// Residual addition, root-mean-square norm and FP8 output on sm_103a, and the
// norm's backward.
//
// The step in front of a layer's projections: the indexer's and the main
// attention's inputs are projections of the normalised hidden state, and the
// indexer runs in FP8 ("AMD Instinct MI355X GPUs Power DeepSeek-V3.2-Exp",
// section "DeepSeek Sparse Attention (DSA)", item 1).  For each row
//     h = x + residual (fp32),  r = 1 / sqrt(mean(h^2) + eps),  y = h r weight
// with h and y rounded once, to the tensors' type, and the FP8 codes taken from
// the fp32 y (scale = amax / 448 or its power of two, per row or per 128
// columns, as dsa_quantize_fp8).  Backward, with xhat = h r and g = dy weight:
//     dx = r (g - xhat mean(g xhat)) + dres,   dweight = sum over rows of dy xhat
//
// Both are HBM-bound: every value is read once and written once.  A group of G
// threads (a warp, or the CTA) owns a row; where rows are aligned thread g holds
// the 8-value chunks c G + g, so a warp's loads are 32 consecutive 16-byte words
// and 16 neighbouring lanes hold one 128-column FP8 block.  Where rows are long
// and many, persistent CTAs take them through a ring in shared memory that bulk
// copies fill while earlier rows are worked on: with the row's values and sums in
// registers, direct loads left an SM too few threads to keep HBM busy (8191 x 8192
// bf16 with residual and block codes: 141 us; backward: 166 us).  Sums are fp32,
// first within a thread, then by shuffles and shared memory, in an order that
// depends on sizes and alignment alone: results repeat bit for bit.
//
// Measured: 8191 x 8192 bf16, residual, both outputs, block codes 96 us (93 % of
// measured HBM); backward of 8192 x 8192 with dres 94 us (84 %: four streams, and
// 5 us of the dweight sum); one row of 4096 2.5 us, launch and one load's latency.
// At 8191 columns no row but every eighth starts at 16 bytes: 219 us for 9000 rows
// where 8192 columns take 107 (backward 147 and 80; fp32 240 and 214), bound by
// instructions: 2-byte loads and stores in every other row.
#include "rmsnorm.cuh"

namespace dsa {
namespace {

// One row: x and res (null: none) point at it, in global memory or a stage of the
// ring.
template <typename T, typename W, int NV, bool WARP, bool VEC>
__device__ __forceinline__ void rmsnorm_row(const RmsNormArgs &a, const T *x, const T *res, int64_t row, float *red)
{
    const int G = WARP ? 32 : blockDim.x;
    const int g = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int cols = a.cols;
    const W *weight = static_cast<const W *>(a.weight);
    Vec8<T> xv[NV], rv[NV];
#pragma unroll
    for (int c = 0; c < NV; ++c)
        load_chunk<VEC>(xv[c], x, chunk_base<VEC>(c, G, g), cols);
    if (res) {
#pragma unroll
        for (int c = 0; c < NV; ++c)
            load_chunk<VEC>(rv[c], res, chunk_base<VEC>(c, G, g), cols);
    }
    float h[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        xv[c].get(h[c]);
        if (res) {
            float r[8];
            rv[c].get(r);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[c][i] += r[i];
        }
        float s = 0.f; // 8 values at a time, so no long fp32 chain
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s = fmaf(h[c][i], h[c][i], s);
        ss += s;
    }
    // a tensor may be overwritten in place: each value is written by the
    // thread that read it
    if (a.residual_out) {
        T *ho = static_cast<T *>(a.residual_out) + row * a.ldh;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            Vec8<T> v;
            v.set(h[c]);
            store_chunk<VEC>(v, ho, chunk_base<VEC>(c, G, g), cols);
        }
    }
    ss = group_reduce<WARP, false>(ss, 0.f, red).x;
    const float r = 1.f / sqrtf(ss / (float)cols + a.eps);
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        float w[8];
        load_weights<T, VEC>(w, weight, chunk_base<VEC>(c, G, g), cols);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            h[c][i] = h[c][i] * r * w[i];
    }
    if (a.out) {
        T *out = static_cast<T *>(a.out) + row * a.ldo;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            Vec8<T> v;
            v.set(h[c]);
            store_chunk<VEC>(v, out, chunk_base<VEC>(c, G, g), cols);
        }
    }
    if (!a.codes)
        return;
    uint8_t *codes = a.codes + row * cols;
    const int nblk = a.block ? (cols + a.block - 1) / a.block : 1;
    float *scale = a.scale + row * nblk;
    float s = 1.f;
    if (!a.block) {
        float m = 0.f;
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                m = fmaxf(m, fabsf(h[c][i]));
        m = group_reduce<WARP, true>(m, 0.f, red).x;
        s = fp8_scale(m, a.scale_mode);
        if (g == 0)
            scale[0] = s;
    }
    ScaleDivider div(s);
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int cb = chunk_base<VEC>(c, G, g);
        ScaleDivider div2 = div; // of the chunk's second half
        if (a.block) {
            float m = 0.f, m2 = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                m = fmaxf(m, fabsf(h[c][i]));
                m2 = fmaxf(m2, fabsf(h[c][4 + i]));
            }
            if (VEC) { // 16 lanes x 8 values = one 128-column block
                m = fmaxf(m, m2);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1)
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                div = div2 = ScaleDivider(fp8_scale(m, a.scale_mode));
                if ((g & 15) == 0 && cb < cols)
                    scale[cb / 128] = div.s;
            } else { // the warp's 256 columns: two blocks, of four values a thread each
                div = ScaleDivider(fp8_scale(warp_amax(m), a.scale_mode));
                div2 = ScaleDivider(fp8_scale(warp_amax(m2), a.scale_mode));
                if ((g & 31) == 0 && cb < cols)
                    scale[cb / 128] = div.s;
                if ((g & 31) == 0 && cb + 128 < cols)
                    scale[cb / 128 + 1] = div2.s;
            }
        }
        const uint32_t lo = e4m3x4(div, h[c][0], h[c][1], h[c][2], h[c][3]);
        const uint32_t hi = e4m3x4(div2, h[c][4], h[c][5], h[c][6], h[c][7]);
        store_codes<T, VEC>(lo, hi, codes, cb, cols);
    }
}

template <typename T, typename W, int NV, bool WARP, bool VEC>
__global__ void __launch_bounds__(WARP ? kRowThreads : 1024) rmsnorm_kernel(RmsNormArgs a)
{
    __shared__ float red[64];
    grid_dep_wait();
    grid_dep_launch();
    const int64_t row0 = WARP ? (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t step = (int64_t)gridDim.x * (WARP ? kRowThreads / 32 : 1);
    for (int64_t row = row0; row < a.rows; row += step)
        rmsnorm_row<T, W, NV, WARP, VEC>(a, static_cast<const T *>(a.x) + row * a.ldx,
                                         a.residual ? static_cast<const T *>(a.residual) + row * a.ldr : nullptr, row, red);
}

// WARP: a stage is a row for each warp.
template <typename T, typename W, int NV, bool WARP, bool VEC>
__global__ void __launch_bounds__(WARP ? 256 : 512, WARP ? 2 : 1)
    rmsnorm_ring_kernel(RmsNormArgs a, int stages, unsigned *status)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[64];
    const int bytes = a.cols * (int)sizeof(T), group = WARP ? blockDim.x >> 5 : 1, w = WARP ? threadIdx.x >> 5 : 0;
    const Ring<VEC> ring{{static_cast<const uint8_t *>(a.x), static_cast<const uint8_t *>(a.residual), nullptr},
                         {a.ldx * (int64_t)sizeof(T), a.ldr * (int64_t)sizeof(T), 0},
                         a.residual ? 2 : 1, group, bytes, stages, a.rows};
    ring.walk(smem, status, [&](uint8_t *stage, int64_t row) {
        if (row + w < a.rows)
            rmsnorm_row<T, W, NV, WARP, VEC>(a, reinterpret_cast<const T *>(stage + ring.at(0, row, w)),
                                             a.residual ? reinterpret_cast<const T *>(stage + ring.at(1, row, w)) : nullptr,
                                             row + w, red);
    });
}

} // namespace

int launch_rmsnorm(const RmsNormArgs &a, cudaStream_t stream, char *err, size_t errlen)
{
    const int e = a.x32 ? 4 : 2;
    // a null tensor counts as aligned
    const bool vec = a.cols % 8 == 0 && chunked(a.x, a.ldx * e) && (!a.residual || chunked(a.residual, a.ldr * e)) &&
                     (!a.residual_out || chunked(a.residual_out, a.ldh * e)) && (!a.out || chunked(a.out, a.ldo * e)) &&
                     chunked(a.weight, 0) && (reinterpret_cast<uintptr_t>(a.codes) & 7) == 0;
    const Shape s = shape_of(a.rows, a.cols, a.residual ? 2 : 1, e, vec, vec);
    unsigned *status = device_status_ptr();
    if (!status) {
        snprintf(err, errlen, "device status word unavailable");
        return DSA_ERR_CUDA;
    }
    cudaError_t rc = dispatch(s, a.x32, a.w32, [&](auto t, auto w, auto nv, auto warp) {
        using T = std::remove_pointer_t<decltype(t)>;
        using W = std::remove_pointer_t<decltype(w)>;
        constexpr int NV = decltype(nv)::value;
        constexpr bool WARP = decltype(warp)::value;
        if constexpr (WARP || NV != 1)
            if (s.stages) {
                auto go = [&](auto kernel, std::atomic<bool>(&raised)[64]) {
                    cudaError_t r = raise_smem_limit_once(kernel, kRingSmemMost, raised);
                    return r != cudaSuccess ? r
                                            : launch_pdl(kernel, dim3((unsigned)rows_grid(a.rows, s, (int64_t)s.ctas * num_sms())),
                                                         dim3(s.threads), s.smem, stream, 1, a, s.stages, status);
                };
                static std::atomic<bool> raised[2][64];
                return vec ? go(rmsnorm_ring_kernel<T, W, NV, WARP, true>, raised[0])
                           : go(rmsnorm_ring_kernel<T, W, NV, WARP, false>, raised[1]);
            }
        auto go = [&](auto kernel) {
            return launch_pdl(kernel, dim3((unsigned)rows_grid(a.rows, s, 1 << 30)), dim3(s.threads), 0, stream, 1, a);
        };
        if constexpr (NV == 1 || (NV == 2 && !WARP))
            return vec ? go(rmsnorm_kernel<T, W, NV, WARP, true>) : go(rmsnorm_kernel<T, W, NV, WARP, false>);
        return cudaErrorInvalidValue; // the others: the ring alone
    });
    if (rc != cudaSuccess) {
        snprintf(err, errlen, "rmsnorm launch: %s", cudaGetErrorString(rc));
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

} // namespace dsa
