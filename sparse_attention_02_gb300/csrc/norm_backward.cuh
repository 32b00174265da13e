// The backward kernels of the RMS norm and of layer norm (LN): dx and the sums of
// the weight's gradient (and the bias's) over the rows of a CTA, then the sum of
// the CTAs' sums.  The norms' formulas stand in their own files.
#pragma once

#include "rmsnorm.cuh"

namespace dsa {
namespace {

// One row of the backward; dw: this thread's dweight sums, and behind them its
// dbias sums.
template <typename T, typename W, int NV, bool WARP, bool VEC, bool LN>
__device__ __forceinline__ void norm_backward_row(const NormBackwardArgs &a, const T *hp, const T *dp, const T *ep,
                                                  int64_t row, float (&dw)[LN ? 2 * NV : NV][8], float *red)
{
    const int G = WARP ? 32 : blockDim.x;
    const int g = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int cols = a.cols;
    const W *weight = static_cast<const W *>(a.weight);
    T *dx = static_cast<T *>(a.dx) + row * cols;
    Vec8<T> hv[NV], dv[NV];
    float ss = 0.f, sg = 0.f;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        load_chunk<VEC>(hv[c], hp, chunk_base<VEC>(c, G, g), cols);
        load_chunk<VEC>(dv[c], dp, chunk_base<VEC>(c, G, g), cols);
    }
    float mean = 0.f, mean_g = 0.f;
    if (LN) {
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            float h[8], d[8], w[8], s = 0.f, t = 0.f;
            load_weights<T, VEC>(w, weight, chunk_base<VEC>(c, G, g), cols);
            hv[c].get(h);
            dv[c].get(d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s += h[i];
                t = fmaf(d[i], w[i], t);
            }
            ss += s;
            sg += t;
        }
        const float2 sums = group_reduce<WARP, false>(ss, sg, red);
        mean = sums.x / (float)cols;
        mean_g = sums.y / (float)cols;
        ss = sg = 0.f;
    }
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int cb = chunk_base<VEC>(c, G, g);
        float h[8], d[8], w[8], s = 0.f, t = 0.f;
        load_weights<T, VEC>(w, weight, cb, cols);
        hv[c].get(h);
        dv[c].get(d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (LN)
                h[i] = (VEC ? cb < cols : column<T, VEC>(cb, i) < cols) ? h[i] - mean : 0.f;
            s = fmaf(h[i], h[i], s);
            t = fmaf(d[i] * w[i], h[i], t);
        }
        ss += s;
        sg += t;
    }
    const float2 sums = group_reduce<WARP, false>(ss, sg, red);
    const float r = 1.f / sqrtf(sums.x / (float)cols + a.eps);
    const float k = sums.y * r * r / (float)cols; // mean(g xhat) r
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int cb = chunk_base<VEC>(c, G, g);
        float h[8], d[8], w[8], o[8];
        load_weights<T, VEC>(w, weight, cb, cols);
        hv[c].get(h);
        dv[c].get(d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (LN) { // past cols d is zero
                h[i] -= mean;
                o[i] = r * ((d[i] * w[i] - mean_g) - h[i] * k);
                dw[NV + c][i] += d[i];
            } else {
                o[i] = r * (d[i] * w[i] - h[i] * k);
            }
            dw[c][i] = fmaf(d[i], h[i] * r, dw[c][i]);
        }
        if (ep) {
            float e[8];
            Vec8<T> ev;
            load_chunk<VEC>(ev, ep, cb, cols);
            ev.get(e);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                o[i] += e[i];
        }
        Vec8<T> v;
        v.set(o);
        store_chunk<VEC>(v, dx, cb, cols);
    }
}

// A CTA's sums as one fp32 row of the workspace: dweight's, then (LN) dbias's.
template <typename T, bool VEC, int NV, int N>
__device__ __forceinline__ void store_part(float *part, const float (&dw)[N][8], int G, int g, int cols)
{
#pragma unroll
    for (int c = 0; c < N; ++c) {
        float *row = part + ((int64_t)blockIdx.x * (N / NV) + c / NV) * cols;
        const int cb = chunk_base<VEC>(c % NV, G, g);
        if (VEC) {
            Vec8<float> v;
            v.set(dw[c]);
            store_chunk<VEC>(v, row, cb, cols);
            continue;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (column<T, VEC>(cb, i) < cols)
                row[column<T, VEC>(cb, i)] = dw[c][i];
    }
}

// The CTA's warps add their sums up in turn, in 32 * 8 * NV floats of shared
// memory; true in the warp that has the total.
template <int NV> __device__ __forceinline__ bool join_warps(float (&dw)[NV][8], float *sums)
{
    const int lane = threadIdx.x & 31;
    for (int w = 0; w < (int)blockDim.x >> 5; ++w) {
        if ((int)threadIdx.x >> 5 == w) {
#pragma unroll
            for (int c = 0; c < NV; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float &d = sums[(c * 8 + i) * 32 + lane];
                    d = w == 0 ? dw[c][i] : d + dw[c][i];
                }
        }
        __syncthreads();
    }
    if (threadIdx.x >= 32)
        return false;
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            dw[c][i] = sums[(c * 8 + i) * 32 + lane];
    return true;
}

// Backward.  Each CTA walks rows b, b + grid, ... with its dweight sums in
// registers.
template <typename T, typename W, int NV, bool WARP, bool VEC, bool LN>
__global__ void __launch_bounds__(WARP ? kRowThreads : 1024)
    norm_backward_kernel(NormBackwardArgs a, float *part)
{
    __shared__ float red[64];
    constexpr int N = LN ? 2 * NV : NV;
    __shared__ float dws[WARP ? 32 * 8 * N : 1];
    grid_dep_wait();
    grid_dep_launch();
    const int G = WARP ? 32 : blockDim.x;
    const int g = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t row0 = WARP ? (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t step = (int64_t)gridDim.x * (WARP ? kRowThreads / 32 : 1);
    const int cols = a.cols;
    float dw[N][8] = {};
    for (int64_t row = row0; row < a.rows; row += step)
        norm_backward_row<T, W, NV, WARP, VEC, LN>(a, static_cast<const T *>(a.h) + row * cols,
                                                  static_cast<const T *>(a.dy) + row * cols,
                                                  a.dres ? static_cast<const T *>(a.dres) + row * cols : nullptr, row, dw, red);
    if (WARP && !join_warps<N>(dw, dws))
        return;
    store_part<T, VEC, NV>(part, dw, G, g, cols);
}

template <typename T, typename W, int NV, bool WARP, bool VEC, bool LN>
__global__ void __launch_bounds__(WARP ? 256 : 512, WARP ? 2 : 1)
    norm_backward_ring_kernel(NormBackwardArgs a, float *part, int stages, unsigned *status)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[64];
    const int bytes = a.cols * (int)sizeof(T), group = WARP ? blockDim.x >> 5 : 1, w = WARP ? threadIdx.x >> 5 : 0;
    const Ring<VEC> ring{{static_cast<const uint8_t *>(a.h), static_cast<const uint8_t *>(a.dy), static_cast<const uint8_t *>(a.dres)},
                         {bytes, bytes, bytes}, a.dres ? 3 : 2, group, bytes, stages, a.rows};
    constexpr int N = LN ? 2 * NV : NV;
    float dw[N][8] = {};
    ring.walk(smem, status, [&](uint8_t *stage, int64_t row) {
        auto at = [&](int k) { return reinterpret_cast<const T *>(stage + ring.at(k, row, w)); };
        if (row + w < a.rows)
            norm_backward_row<T, W, NV, WARP, VEC, LN>(a, at(0), at(1), a.dres ? at(2) : nullptr, row + w, dw, red);
    });
    if (WARP && !join_warps<N>(dw, reinterpret_cast<float *>(smem + kRingBars)))
        return;
    store_part<T, VEC, NV>(part, dw, WARP ? 32 : blockDim.x, WARP ? threadIdx.x & 31 : threadIdx.x, a.cols);
}

// dweight[c] = sum of the nparts partial rows, ld apart: 32 columns a CTA, the
// rows dealt to 32 warps, whose sums are added in order.  Grid row 1: dbias, from
// the rows' second half.
__global__ void __launch_bounds__(1024) dweight_kernel(const float *part, int nparts, int cols, int ld, float *dweight, float *dbias)
{
    __shared__ float s[32][33];
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    if (blockIdx.y) {
        part += cols;
        dweight = dbias;
    }
    constexpr int kAhead = 10; // rows of a warp whose loads are in flight: two CTAs an SM leave it ten
    float t = 0.f;
    if (c < cols)
        for (int p = w; p < nparts; p += 32 * kAhead) {
            float v[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                v[k] = p + 32 * k < nparts ? part[(int64_t)(p + 32 * k) * ld + c] : 0.f;
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                t += v[k];
        }
    s[w][lane] = t;
    __syncthreads();
    t = s[lane][w]; // warp w: the 32 sums of column w
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane == 0 && blockIdx.x * 32 + w < cols)
        dweight[blockIdx.x * 32 + w] = t;
}

// CTAs of a backward: a row of the workspace each.
int64_t backward_ctas(int64_t rows, const Shape &s)
{
    return rows_grid(rows, s, (int64_t)(s.stages ? s.ctas : s.warp ? 4 : 2) * num_sms());
}

// The most that any alignment, type and dres needs: which of them a call has is
// not known here.
template <bool LN> size_t norm_backward_workspace(int64_t rows, int cols)
{
    int64_t most = 0;
    for (int esize = 2; esize <= 4; esize += 2)
        for (int n = 2; n <= 3; ++n)
            for (int vec = 0; vec < 2; ++vec) {
                const int64_t c = backward_ctas(rows, shape_of(rows, cols, n, esize, vec != 0, true));
                most = c > most ? c : most;
            }
    return (size_t)most * cols * (LN ? 2 : 1) * sizeof(float);
}

template <bool LN>
int launch_norm_backward(const NormBackwardArgs &a, const char *name, cudaStream_t stream, char *err, size_t errlen)
{
    const int e = a.x32 ? 4 : 2;
    const int64_t ld = (int64_t)a.cols * e;
    const bool vec = a.cols % 8 == 0 && chunked(a.h, ld) && chunked(a.dy, ld) && chunked(a.dres, ld) && chunked(a.dx, ld) &&
                     chunked(a.weight, 0); // a null dres counts as aligned
    const Shape s = shape_of(a.rows, a.cols, a.dres ? 3 : 2, e, vec, true);
    const int grid = (int)backward_ctas(a.rows, s);
    float *part = static_cast<float *>(a.workspace);
    unsigned *status = device_status_ptr();
    if (!status) {
        snprintf(err, errlen, "device status word unavailable");
        return DSA_ERR_CUDA;
    }
    cudaError_t rc = cudaSuccess;
    if (grid > 0)
        rc = dispatch(s, a.x32, a.w32, [&](auto t, auto w, auto nv, auto warp) {
            using T = std::remove_pointer_t<decltype(t)>;
            using W = std::remove_pointer_t<decltype(w)>;
            constexpr int NV = decltype(nv)::value;
            constexpr bool WARP = decltype(warp)::value;
            if constexpr (WARP || NV != 1)
                if (s.stages) {
                    auto go = [&](auto kernel, std::atomic<bool>(&raised)[64]) {
                        cudaError_t r = raise_smem_limit_once(kernel, kRingSmemMost, raised);
                        return r != cudaSuccess ? r
                                                : launch_pdl(kernel, dim3((unsigned)grid), dim3(s.threads), s.smem, stream, 1, a, part,
                                                             s.stages, status);
                    };
                    static std::atomic<bool> raised[2][64];
                    return vec ? go(norm_backward_ring_kernel<T, W, NV, WARP, true, LN>, raised[0])
                               : go(norm_backward_ring_kernel<T, W, NV, WARP, false, LN>, raised[1]);
                }
            auto go = [&](auto kernel) {
                return launch_pdl(kernel, dim3((unsigned)grid), dim3(s.threads), 0, stream, 1, a, part);
            };
            if constexpr (NV == 1 || (NV == 2 && !WARP))
                return vec ? go(norm_backward_kernel<T, W, NV, WARP, true, LN>) : go(norm_backward_kernel<T, W, NV, WARP, false, LN>);
            return cudaErrorInvalidValue; // the others: the ring alone
        });
    if (rc == cudaSuccess) // no rows: the sum of nothing, zeros
        rc = launch_pdl(dweight_kernel, dim3((unsigned)((a.cols + 31) / 32), LN && a.dbias ? 2 : 1), dim3(1024), 0, stream, 1,
                        (const float *)part, grid, a.cols, LN ? 2 * a.cols : a.cols, a.dweight, a.dbias);
    if (rc != cudaSuccess) {
        snprintf(err, errlen, "%s launch: %s", name, cudaGetErrorString(rc));
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

} // namespace
} // namespace dsa
