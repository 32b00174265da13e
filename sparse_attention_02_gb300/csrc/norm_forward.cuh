// The forward kernels of the RMS norm and of layer norm (LN), and the choice among
// them.  The norms' formulas and what they measured stand in their own files.
#pragma once

#include "rmsnorm.cuh"

namespace dsa {
namespace {

struct Meet {
    __device__ __forceinline__ bool operator()() const
    {
        __syncthreads();
        return true;
    }
};

// One row: x and res (null: none) point at it, in global memory or a stage of the
// ring.  A CTA's rows have a barrier between them (the RMS norm's ring), or there is but one.
// RING (layer norm): held, of the weight and of the bias; meet, the threads' one meeting, after which the stage is not read;
// there: whether this warp has a row, and its wait for the stage ended with it: nothing is written of a row that never came.
// moments: of this row, 64 floats.
template <typename T, typename W, int NV, bool WARP, bool VEC, bool LN, bool RING = false, typename M = Meet>
__device__ __forceinline__ void norm_row(const NormArgs &a, const T *x, const T *res, int64_t row, float *red,
                                         [[maybe_unused]] float *moments = nullptr, [[maybe_unused]] const Counts &n = Counts(),
                                         [[maybe_unused]] const Held<T, W, NV, VEC> *held = nullptr,
                                         [[maybe_unused]] bool there = true, M meet = M())
{
    const int G = WARP ? 32 : blockDim.x;
    const int g = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int cols = a.cols;
    const W *weight = static_cast<const W *>(a.weight);
    const int mine = !RING || !WARP || there ? cols : 0; // of the stage's columns
    Vec8<T> xv[NV], rv[NV];
#pragma unroll
    for (int c = 0; c < NV; ++c)
        load_chunk<VEC>(xv[c], x, chunk_base<VEC>(c, G, g), mine);
    if (res) {
#pragma unroll
        for (int c = 0; c < NV; ++c)
            load_chunk<VEC>(rv[c], res, chunk_base<VEC>(c, G, g), mine);
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
        if (LN) {
            F2 s(0.f);
#pragma unroll
            for (int i = 0; i < 8; i += 2)
                s = s + F2(h[c][i], h[c][i + 1]);
            ss += s.sum();
        } else {
            float s = 0.f; // 8 values at a time, so no long fp32 chain
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s = fmaf(h[c][i], h[c][i], s);
            ss += s;
        }
    }
    if (RING && WARP) { // as soon as the stage is read
        if (!meet() || !there)
            return;
    }
    // a tensor may be overwritten in place: each value is written by the
    // thread that read it
    if (a.residual_out && there) {
        T *ho = static_cast<T *>(a.residual_out) + row * a.ldh;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            Vec8<T> v;
            v.set(h[c]);
            store_chunk<VEC>(v, ho, chunk_base<VEC>(c, G, g), cols);
        }
    }
    if (LN) {
        // about the warp's own mean first, from the registers
        ss = warp_sum(ss);
        float mean = n.mine.mean_by_remainder(ss);
        F2 sq2(0.f);
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int cb = chunk_base<VEC>(c, G, g);
            const F2 back(!VEC || cb < cols ? -mean : 0.f); // past cols: no part of the sum of squares
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                F2 d = F2(h[c][i], h[c][i + 1]) + back;
                if (!VEC && column<T, VEC>(cb, i + 1) >= cols)
                    d = F2(column<T, VEC>(cb, i) < cols ? h[c][i] - mean : 0.f, 0.f);
                sq2 = fma2(d, d, sq2);
            }
        }
        float sq = warp_sum(sq2.sum());
        if (!WARP) {
            const int lane = threadIdx.x & 31;
            if (lane == 0) {
                moments[threadIdx.x >> 5] = ss;
                moments[32 + (threadIdx.x >> 5)] = sq;
            }
            if (!meet())
                return;
            const bool is = n.other.n > 0.f;
            ss = is ? moments[lane] : 0.f;
            mean = n.all.mean_by_remainder(warp_sum(ss));
            const float d = n.other.mean_by_remainder(ss) - mean;
            sq = warp_sum(is ? moments[32 + lane] + n.other.n * d * d : 0.f);
        }
        const F2 r2(inv_sqrt(sq * n.all.inv + a.eps)), back(-mean);
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            float w[8], b[8] = {};
            if (RING)
                held[0].get(w, weight, c, chunk_base<VEC>(c, G, g), cols);
            else
                load_weights<T, VEC>(w, weight, chunk_base<VEC>(c, G, g), cols);
            if (a.bias) {
                if (RING)
                    held[1].get(b, static_cast<const W *>(a.bias), c, chunk_base<VEC>(c, G, g), cols);
                else
                    load_weights<T, VEC>(b, static_cast<const W *>(a.bias), chunk_base<VEC>(c, G, g), cols);
            }
#pragma unroll
            for (int i = 0; i < 8; i += 2)
                fma2((F2(h[c][i], h[c][i + 1]) + back) * r2, F2(w[i], w[i + 1]), F2(b[i], b[i + 1])).get(h[c][i], h[c][i + 1]);
        }
    } else {
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

template <typename T, typename W, int NV, bool WARP, bool VEC, bool LN>
__global__ void __launch_bounds__(WARP ? kRowThreads : 1024) norm_kernel(NormArgs a)
{
    __shared__ float red[64], moments[LN ? 64 : 1];
    grid_dep_wait();
    grid_dep_launch();
    const int64_t row0 = WARP ? (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t step = (int64_t)gridDim.x * (WARP ? kRowThreads / 32 : 1);
    [[maybe_unused]] const Counts n = LN ? Counts::of<NV, WARP>(WARP ? 32 : blockDim.x, a.cols) : Counts();
    for (int64_t row = row0; row < a.rows; row += step)
        norm_row<T, W, NV, WARP, VEC, LN>(a, static_cast<const T *>(a.x) + row * a.ldx,
                                         a.residual ? static_cast<const T *>(a.residual) + row * a.ldr : nullptr, row, red, moments, n);
}

// WARP: a stage is a row for each warp.
template <typename T, typename W, int NV, bool WARP, bool VEC, bool LN>
__global__ void __launch_bounds__(WARP ? 256 : 512, WARP ? 2 : 1)
    norm_ring_kernel(NormArgs a, int stages, unsigned *status)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[64], moments[LN ? 128 : 1]; // of two rows: one meeting lies between them
    const int bytes = a.cols * (int)sizeof(T), group = WARP ? blockDim.x >> 5 : 1, w = WARP ? threadIdx.x >> 5 : 0;
    const Ring<VEC> ring{{static_cast<const uint8_t *>(a.x), static_cast<const uint8_t *>(a.residual), nullptr},
                         {a.ldx * (int64_t)sizeof(T), a.ldr * (int64_t)sizeof(T), 0},
                         a.residual ? 2 : 1, group, bytes, stages, a.rows};
    auto at = [&](int k, uint8_t *stage, int64_t row) { return reinterpret_cast<const T *>(stage + ring.at(k, row, w)); };
    if constexpr (LN) {
        Held<T, W, NV, VEC> held[2];
        const Counts n = Counts::of<NV, WARP>(WARP ? 32 : blockDim.x, a.cols);
        int turn = -1; // before the first row
        ring.template walk<true>(smem, status, [&](uint8_t *stage, int64_t row, bool came, auto meet) {
            if (turn < 0) { // not before the walk has waited for the kernel in front
                const int G = WARP ? 32 : blockDim.x, g = WARP ? threadIdx.x & 31 : threadIdx.x;
                held[0].load(static_cast<const W *>(a.weight), G, g, a.cols);
                if (a.bias)
                    held[1].load(static_cast<const W *>(a.bias), G, g, a.cols);
                turn = 0;
            }
            norm_row<T, W, NV, WARP, VEC, true, true>(a, at(0, stage, row), a.residual ? at(1, stage, row) : nullptr, row + w, red,
                                                      moments + 64 * turn, n, held, came && row + w < a.rows, meet);
            turn ^= 1;
        });
    } else {
        ring.walk(smem, status, [&](uint8_t *stage, int64_t row) {
            if (row + w < a.rows)
                norm_row<T, W, NV, WARP, VEC, false>(a, at(0, stage, row), a.residual ? at(1, stage, row) : nullptr, row + w, red);
        });
    }
}

template <bool LN> int launch_norm(const NormArgs &a, const char *name, cudaStream_t stream, char *err, size_t errlen)
{
    const int e = a.x32 ? 4 : 2;
    // a null tensor counts as aligned
    const bool vec = a.cols % 8 == 0 && chunked(a.x, a.ldx * e) && (!a.residual || chunked(a.residual, a.ldr * e)) &&
                     (!a.residual_out || chunked(a.residual_out, a.ldh * e)) && (!a.out || chunked(a.out, a.ldo * e)) &&
                     chunked(a.weight, 0) && chunked(a.bias, 0) && (reinterpret_cast<uintptr_t>(a.codes) & 7) == 0;
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
                return vec ? go(norm_ring_kernel<T, W, NV, WARP, true, LN>, raised[0])
                           : go(norm_ring_kernel<T, W, NV, WARP, false, LN>, raised[1]);
            }
        auto go = [&](auto kernel) {
            return launch_pdl(kernel, dim3((unsigned)rows_grid(a.rows, s, 1 << 30)), dim3(s.threads), 0, stream, 1, a);
        };
        if constexpr (NV == 1 || (NV == 2 && !WARP))
            return vec ? go(norm_kernel<T, W, NV, WARP, true, LN>) : go(norm_kernel<T, W, NV, WARP, false, LN>);
        return cudaErrorInvalidValue; // the others: the ring alone
    });
    if (rc != cudaSuccess) {
        snprintf(err, errlen, "%s launch: %s", name, cudaGetErrorString(rc));
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

} // namespace
} // namespace dsa
