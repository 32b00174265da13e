// The backward kernels of the RMS norm and of layer norm (LN): dx and the sums of
// the weight's gradient (and the bias's) over the rows of a CTA, then the sum of
// the CTAs' sums.  The norms' formulas stand in their own files.
#pragma once

#include "rmsnorm.cuh"

namespace dsa {
namespace {

constexpr int kLayerRowThreads = 512, kLayerRowCtas = 2; // of layer norm whose warps own rows, and CTAs an SM

// One row of the RMS norm's backward; dw: this thread's dweight sums.
template <typename T, typename W, int NV, bool WARP, bool VEC>
__device__ __forceinline__ void rmsnorm_backward_row(const NormBackwardArgs &a, const T *hp, const T *dp, const T *ep,
                                                     int64_t row, float (&dw)[NV][8], float *red)
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
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        float h[8], d[8], w[8], s = 0.f, t = 0.f;
        load_weights<T, VEC>(w, weight, chunk_base<VEC>(c, G, g), cols);
        hv[c].get(h);
        dv[c].get(d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
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
            o[i] = r * (d[i] * w[i] - h[i] * k);
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

template <int N> __device__ __forceinline__ void clear(F2 (&v)[N][4])
{
#pragma unroll
    for (int c = 0; c < N; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[c][i] = F2(0.f);
}

template <int N> __device__ __forceinline__ void unpack(const F2 (&v)[N][4], float (&f)[N][8])
{
#pragma unroll
    for (int c = 0; c < N; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[c][i].get(f[c][2 * i], f[c][2 * i + 1]);
}

// One row of layer norm's backward.  WARP: LANES lanes own it.  dw: this thread's dweight sums, and behind them its dbias
// sums.  red: kMoments floats.  Values are unpacked once and worked on in pairs: with a CTA's 512 threads on one row, its
// instructions and the meeting's latency add up.
template <typename T, typename W, int NV, bool WARP, bool VEC, int LANES>
__device__ __forceinline__ void layernorm_backward_row(const NormBackwardArgs &a, const T *hp, const T *dp, const T *ep, int64_t row,
                                                       bool there, const Held<T, W, NV, VEC> &held, const Counts &n,
                                                       F2 (&dw)[2 * NV][4], float *red)
{
    const int G = WARP ? LANES : blockDim.x;
    const int g = WARP ? (threadIdx.x & (LANES - 1)) : threadIdx.x;
    const int cols = a.cols;
    const W *weight = static_cast<const W *>(a.weight);
    F2 h[NV][4], d[NV][4], gw[NV][4]; // h, dy, dy weight
    F2 s2(0.f), t2(0.f);
    {
        Vec8<T> hv[NV], dv[NV];
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            load_chunk<VEC>(hv[c], hp, chunk_base<VEC>(c, G, g), there ? cols : 0);
            load_chunk<VEC>(dv[c], dp, chunk_base<VEC>(c, G, g), there ? cols : 0);
        }
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            float x[8], y[8], w[8];
            held.get(w, weight, c, chunk_base<VEC>(c, G, g), cols);
            hv[c].get(x);
            dv[c].get(y);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[c][i] = F2(x[2 * i], x[2 * i + 1]);
                d[c][i] = F2(y[2 * i], y[2 * i + 1]);
                gw[c][i] = d[c][i] * F2(w[2 * i], w[2 * i + 1]);
                s2 = s2 + h[c][i];
                t2 = t2 + gw[c][i];
            }
        }
    }
    float sum, sg, sums = 0.f;
    if constexpr (WARP) {
        sums = half_sums<LANES>(s2.sum(), t2.sum());
        sum = from_half<LANES, 0>(sums);
    } else { // four sums beside one another: what counts is how long a row's meeting takes
        sum = warp_sum(s2.sum());
        sg = warp_sum(t2.sum());
    }
    const float mean = n.mine.mean_by_parts(sum); // the warp's own
    s2 = t2 = F2(0.f);
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int cb = chunk_base<VEC>(c, G, g);
        const F2 back(!VEC || cb < cols ? -mean : 0.f); // past cols: no part of the sum of squares
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[c][i] = h[c][i] + back;
            if (!VEC && column<T, VEC>(cb, 2 * i + 1) >= cols) {
                float lo, hi;
                h[c][i].get(lo, hi);
                h[c][i] = F2(column<T, VEC>(cb, 2 * i) < cols ? lo : 0.f, 0.f);
            }
            s2 = fma2(h[c][i], h[c][i], s2);
            t2 = fma2(gw[c][i], h[c][i], t2);
        }
    }
    float off = 0.f, sq, gd; // off: of the row's mean from the warp's
    if constexpr (WARP) {
        const float squares = half_sums<LANES>(s2.sum(), t2.sum());
        sq = from_half<LANES, 0>(squares);
        gd = from_half<LANES, 1>(squares);
        sg = from_half<LANES, 1>(sums);
    } else {
        sq = warp_sum(s2.sum());
        gd = warp_sum(t2.sum());
        const int lane = threadIdx.x & 31;
        if (lane == 0) {
            float *to = red + (threadIdx.x >> 5);
            to[0] = sum, to[32] = sq, to[64] = sg, to[96] = gd;
        }
        __syncthreads();
        const bool is = n.other.n > 0.f;
        const float its = is ? red[lane] : 0.f, its_g = is ? red[64 + lane] : 0.f;
        const float all = n.all.mean_by_parts(warp_sum(its)), dm = is ? n.other.mean_by_parts(its) - all : 0.f;
        sg = warp_sum(its_g);
        sq = warp_sum(is ? red[32 + lane] + n.other.n * dm * dm : 0.f);
        gd = warp_sum(is ? fmaf(dm, its_g, red[96 + lane]) : 0.f);
        off = mean - all;
    }
    const float r = inv_sqrt(sq * n.all.inv + a.eps);
    const float k = gd * n.all.inv * r * r, mean_g = sg * n.all.inv; // k: mean(g xhat) r
    if (!there)
        return;
    const F2 off2(off * r), r2(r), k2(-k), mg2(-mean_g * r);
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int cb = chunk_base<VEC>(c, G, g);
        F2 o2[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) { // past cols d is zero
            const F2 xhat = fma2(h[c][i], r2, off2);
            o2[i] = fma2(xhat, k2, fma2(gw[c][i], r2, mg2));
            dw[c][i] = fma2(d[c][i], xhat, dw[c][i]);
            dw[NV + c][i] = dw[NV + c][i] + d[c][i];
        }
        if (ep) {
            float e[8];
            Vec8<T> ev;
            load_chunk<VEC>(ev, ep, cb, cols);
            ev.get(e);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o2[i] = o2[i] + F2(e[2 * i], e[2 * i + 1]);
        }
        float o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o2[i].get(o[2 * i], o[2 * i + 1]);
        Vec8<T> v;
        v.set(o);
        store_chunk<VEC>(v, static_cast<T *>(a.dx) + row * cols, cb, cols);
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

// Layer norm's form: every warp's sums side by side, [warps][32 * 8 * N] floats, added up column by column.
template <int N, int LANES> __device__ __forceinline__ bool join_warps_at_once(float (&dw)[N][8], float *sums)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int c = 0; c < N; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (LANES == 16) // both halves hold the same columns
                dw[c][i] += __shfl_xor_sync(0xffffffffu, dw[c][i], 16);
            sums[((threadIdx.x >> 5) * N + c) * 256 + i * 32 + lane] = dw[c][i];
        }
    __syncthreads();
    for (int x = threadIdx.x; x < 256 * N; x += blockDim.x) {
        float t = sums[x];
        for (int w = 1; w < (int)blockDim.x >> 5; ++w)
            t += sums[w * 256 * N + x];
        sums[x] = t;
    }
    __syncthreads();
    if (threadIdx.x >= LANES)
        return false;
#pragma unroll
    for (int c = 0; c < N; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            dw[c][i] = sums[c * 256 + i * 32 + lane];
    return true;
}

// Backward.  Each CTA walks rows b, b + grid, ... with its dweight sums in
// registers.
// LANES: 16 where layer norm's rows are that many chunks (two rows a warp: 32767 x 128 fp32 20 us with one).
template <typename T, typename W, int NV, bool WARP, bool VEC, bool LN, int LANES>
__global__ void __launch_bounds__(WARP ? (LN ? kLayerRowThreads : kRowThreads) : 1024, WARP && LN ? kLayerRowCtas : 1)
    norm_backward_kernel(NormBackwardArgs a, float *part)
{
    constexpr int N = LN ? 2 * NV : NV, kOwners = (LN ? kLayerRowThreads : kRowThreads) / LANES; // rows a CTA has at work
    __shared__ float red[LN ? 2 * kMoments : 64];
    __shared__ float dws[WARP ? 32 * 8 * N * (LN ? kLayerRowThreads / 32 : 1) : 1];
    grid_dep_wait();
    grid_dep_launch();
    const int G = WARP ? LANES : blockDim.x;
    const int g = WARP ? (threadIdx.x & (LANES - 1)) : threadIdx.x;
    const int64_t row0 = WARP ? (int64_t)blockIdx.x * kOwners + threadIdx.x / LANES : blockIdx.x;
    const int64_t step = (int64_t)gridDim.x * (WARP ? kOwners : 1);
    const int cols = a.cols;
    const T *h = static_cast<const T *>(a.h), *dy = static_cast<const T *>(a.dy), *dres = static_cast<const T *>(a.dres);
    [[maybe_unused]] F2 dw2[N][4];
    float dw[N][8] = {};
    if constexpr (LN) {
        Held<T, W, NV, VEC> held;
        const Counts n = Counts::of<NV, WARP>(G, cols);
        clear(dw2);
        held.load(static_cast<const W *>(a.weight), G, g, cols);
        int turn = 0;
        // a warp's two rows walk together: its lanes add up among themselves
        for (int64_t row = row0; row - (WARP ? threadIdx.x % 32 / LANES : 0) < a.rows; row += step, turn ^= 1)
            layernorm_backward_row<T, W, NV, WARP, VEC, LANES>(a, h + row * cols, dy + row * cols, dres ? dres + row * cols : nullptr,
                                                               row, LANES == 32 || row < a.rows, held, n, dw2, red + turn * kMoments);
        unpack(dw2, dw);
    } else {
        for (int64_t row = row0; row < a.rows; row += step)
            rmsnorm_backward_row<T, W, NV, WARP, VEC>(a, h + row * cols, dy + row * cols, dres ? dres + row * cols : nullptr, row, dw, red);
    }
    bool mine = true;
    if constexpr (WARP && LN)
        mine = join_warps_at_once<N, LANES>(dw, dws);
    else if constexpr (WARP)
        mine = join_warps<N>(dw, dws);
    if (mine)
        store_part<T, VEC, NV>(part, dw, G, g, cols);
}

template <typename T, typename W, int NV, bool WARP, bool VEC, bool LN>
__global__ void __launch_bounds__(WARP ? 256 : 512, WARP ? 2 : 1)
    norm_backward_ring_kernel(NormBackwardArgs a, float *part, int stages, unsigned *status)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[LN ? kMoments : 64]; // rows have a barrier between them
    const int bytes = a.cols * (int)sizeof(T), group = WARP ? blockDim.x >> 5 : 1, w = WARP ? threadIdx.x >> 5 : 0;
    const Ring<VEC> ring{{static_cast<const uint8_t *>(a.h), static_cast<const uint8_t *>(a.dy), static_cast<const uint8_t *>(a.dres)},
                         {bytes, bytes, bytes}, a.dres ? 3 : 2, group, bytes, stages, a.rows};
    constexpr int N = LN ? 2 * NV : NV;
    const int G = WARP ? 32 : blockDim.x, g = WARP ? threadIdx.x & 31 : threadIdx.x;
    [[maybe_unused]] F2 dw2[N][4];
    clear(dw2);
    float dw[N][8] = {};
    [[maybe_unused]] Held<T, W, NV, VEC> held;
    [[maybe_unused]] const Counts n = Counts::of<NV, WARP>(G, a.cols);
    [[maybe_unused]] bool first = true;
    ring.walk(smem, status, [&](uint8_t *stage, int64_t row) {
        auto at = [&](int k) { return reinterpret_cast<const T *>(stage + ring.at(k, row, w)); };
        if constexpr (LN) {
            if (first) // not before the walk has waited for the kernel in front
                held.load(static_cast<const W *>(a.weight), G, g, a.cols);
            first = false;
        }
        if (row + w < a.rows) {
            if constexpr (LN)
                layernorm_backward_row<T, W, NV, WARP, VEC, 32>(a, at(0), at(1), a.dres ? at(2) : nullptr, row + w, true, held, n, dw2, red);
            else
                rmsnorm_backward_row<T, W, NV, WARP, VEC>(a, at(0), at(1), a.dres ? at(2) : nullptr, row + w, dw, red);
        }
    });
    if constexpr (LN)
        unpack(dw2, dw);
    bool mine = true;
    if constexpr (WARP && LN)
        mine = join_warps_at_once<N, 32>(dw, reinterpret_cast<float *>(smem + kRingBars));
    else if constexpr (WARP)
        mine = join_warps<N>(dw, reinterpret_cast<float *>(smem + kRingBars));
    if (mine)
        store_part<T, VEC, NV>(part, dw, G, g, a.cols);
}

// dweight[c] = sum of the nparts partial rows: 32 columns a CTA, the rows dealt
// to 32 warps, whose sums are added in order.
__global__ void __launch_bounds__(1024) dweight_kernel(const float *part, int nparts, int cols, float *dweight)
{
    __shared__ float s[32][33];
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    constexpr int kAhead = 10; // rows of a warp whose loads are in flight: two CTAs an SM leave it ten
    float t = 0.f;
    if (c < cols)
        for (int p = w; p < nparts; p += 32 * kAhead) {
            float v[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                v[k] = p + 32 * k < nparts ? part[(int64_t)(p + 32 * k) * cols + c] : 0.f;
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

// Layer norm's: twice the columns, dweight's and dbias's.  WARPS: 32 for the shortest way through few columns, 16 where the
// CTAs of 32 would take turns (a whole backward of 8192 x 8192 97.6 us with 32, 95.8 so; of 4096 x 4096 30.6 and 31.8).
template <int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 64 / WARPS) norm_sums_kernel(const float *part, int nparts, int cols, float *dweight, float *dbias)
{
    __shared__ float s[WARPS][32];
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    constexpr int kAhead = 10; // rows of a warp whose loads are in flight
    float t = 0.f;
    if (c < 2 * cols)
        for (int p = w; p < nparts; p += WARPS * kAhead) {
            float v[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                v[k] = p + WARPS * k < nparts ? part[(int64_t)(p + WARPS * k) * 2 * cols + c] : 0.f;
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                t += v[k];
        }
    s[w][lane] = t;
    __syncthreads();
    if (w > 0 || c >= 2 * cols)
        return;
    t = s[0][lane];
#pragma unroll
    for (int k = 1; k < WARPS; ++k)
        t += s[k][lane];
    if (c < cols)
        dweight[c] = t;
    else if (dbias)
        dbias[c - cols] = t;
}

// CTAs of a backward: a row of the workspace each.
template <bool LN> int64_t backward_ctas(int64_t rows, const Shape &s)
{
    return rows_grid(rows, s, (int64_t)(s.stages ? s.ctas : s.warp ? (LN ? kLayerRowCtas : 4) : 2) * num_sms());
}

template <bool LN> Shape backward_shape(int64_t rows, int cols, int n, int esize, bool vec)
{
    Shape s = shape_of(rows, cols, n, esize, vec, true, !LN);
    if (LN && s.warp && !s.stages)
        s.threads = kLayerRowThreads;
    if (LN && s.warp && s.stages) { // room for the warps' sums
        const size_t join = kRingBars + (size_t)(s.threads / 32) * 2 * s.nv * 256 * sizeof(float);
        s.smem = s.smem < join ? join : s.smem;
    }
    return s;
}

// The most that any alignment, type and dres needs: which of them a call has is
// not known here.
template <bool LN> size_t norm_backward_workspace(int64_t rows, int cols)
{
    int64_t most = 0;
    for (int esize = 2; esize <= 4; esize += 2)
        for (int n = 2; n <= 3; ++n)
            for (int vec = 0; vec < 2; ++vec) {
                const int64_t c = backward_ctas<LN>(rows, backward_shape<LN>(rows, cols, n, esize, vec != 0));
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
    const Shape s = backward_shape<LN>(a.rows, a.cols, a.dres ? 3 : 2, e, vec);
    const int grid = (int)backward_ctas<LN>(a.rows, s);
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
            if constexpr ((WARP || NV != 1) && !(LN && WARP && NV == 4))
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
            if constexpr (NV == 1 && WARP && LN)
                if (vec && a.cols <= 128)
                    return go(norm_backward_kernel<T, W, NV, WARP, true, LN, 16>);
            if constexpr (NV == 1 || (NV == 2 && !WARP))
                return vec ? go(norm_backward_kernel<T, W, NV, WARP, true, LN, 32>) : go(norm_backward_kernel<T, W, NV, WARP, false, LN, 32>);
            return cudaErrorInvalidValue; // the others: the ring alone
        });
    if (rc == cudaSuccess) { // no rows: the sum of nothing, zeros
        if constexpr (LN) {
            const int ctas = ((a.dbias ? 2 : 1) * a.cols + 31) / 32;
            auto go = [&](auto kernel, int warps) {
                return launch_pdl(kernel, dim3((unsigned)ctas), dim3(32 * warps), 0, stream, 1, (const float *)part, grid, a.cols, a.dweight,
                                  a.dbias);
            };
            rc = ctas <= 2 * num_sms() ? go(norm_sums_kernel<32>, 32) : go(norm_sums_kernel<16>, 16);
        } else
            rc = launch_pdl(dweight_kernel, dim3((unsigned)((a.cols + 31) / 32)), dim3(1024), 0, stream, 1, (const float *)part, grid, a.cols,
                            a.dweight);
    }
    if (rc != cudaSuccess) {
        snprintf(err, errlen, "%s launch: %s", name, cudaGetErrorString(rc));
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

} // namespace
} // namespace dsa
