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
// threads (a warp, or the CTA) owns a row; thread g holds the 8-value chunks
// c G + g, so a warp's loads are 32 consecutive 16-byte words and 16
// neighbouring lanes hold one 128-column FP8 block.  Where rows are aligned,
// long and many, persistent CTAs (two an SM) take them through a ring in shared
// memory that bulk copies fill while earlier rows are worked on: with the row's
// values and sums in registers, direct loads left an SM too few threads to keep
// HBM busy (8191 x 8192 bf16 with residual and block codes: 141 us; backward:
// 166 us).  Sums are fp32, first within a thread, then by shuffles and shared
// memory, in an order that depends on sizes and alignment alone: results repeat
// bit for bit.
#include "common.cuh"
#include "fp8.cuh"
#include "launch.h"

#include <atomic>
#include <stdio.h>
#include <type_traits>

namespace dsa {
namespace {

constexpr int kRowThreads = 128; // threads of a CTA whose warps each own rows

template <typename T> struct Vec8; // eight values as loaded

template <> struct Vec8<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void load_n(const __nv_bfloat16 *p, int n)
    {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                w[i >> 1] |= (uint32_t)reinterpret_cast<const uint16_t *>(p)[i] << (16 * (i & 1));
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&f)[8])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void set_words(const uint32_t *w) { v = make_uint4(w[0], w[1], w[2], w[3]); }
    __device__ __forceinline__ void get_words(uint32_t *w) const { w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w; }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint4 *>(p) = v; }
    template <typename F> __device__ __forceinline__ void store_if(__nv_bfloat16 *p, int n, F &&f) const
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n && f(i))
                reinterpret_cast<uint16_t *>(p)[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
    __device__ __forceinline__ void store_n(__nv_bfloat16 *p, int n) const
    {
        store_if(p, n, [](int) { return true; });
    }
};

template <> struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void load(const float *p)
    {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void load_n(const float *p, int n)
    {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = i < n ? p[i] : 0.f;
        set(f);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
    __device__ __forceinline__ void set(const float (&f)[8])
    {
        a = make_float4(f[0], f[1], f[2], f[3]);
        b = make_float4(f[4], f[5], f[6], f[7]);
    }
    __device__ __forceinline__ void set_words(const uint32_t *w)
    {
        a = make_float4(__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2]), __uint_as_float(w[3]));
        b = make_float4(__uint_as_float(w[4]), __uint_as_float(w[5]), __uint_as_float(w[6]), __uint_as_float(w[7]));
    }
    __device__ __forceinline__ void get_words(uint32_t *w) const
    {
        float f[8];
        get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = __float_as_uint(f[i]);
    }
    template <typename F> __device__ __forceinline__ void store_if(float *p, int n, F &&fn) const
    {
        float f[8];
        get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n && fn(i))
                p[i] = f[i];
    }
    __device__ __forceinline__ void store(float *p) const
    {
        reinterpret_cast<float4 *>(p)[0] = a;
        reinterpret_cast<float4 *>(p)[1] = b;
    }
    __device__ __forceinline__ void store_n(float *p, int n) const
    {
        store_if(p, n, [](int) { return true; });
    }
};

// ---- rows at any address
//
// Where rows do not all start at 16 bytes, a chunk is put together from the
// aligned 16-byte words that it lies in (one more than it has, which the L1
// serves), and stored as such words by handing the bytes that belong to the
// next word to the next lane.  Value by value an 8000 x 4001 norm took 202 us,
// its backward 139.

// 32-bit words i .. i + N of the byte string w that starts `ph` bytes (0-15) in.
template <int N>
__device__ __forceinline__ void shift_down(uint32_t (&w)[N + 4], int ph)
{
    if (ph & 8) {
#pragma unroll
        for (int i = 0; i < N + 2; ++i)
            w[i] = w[i + 2];
    }
    if (ph & 4) {
#pragma unroll
        for (int i = 0; i < N + 1; ++i)
            w[i] = w[i + 1];
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        w[i] = __funnelshift_r(w[i], w[i + 1], 8 * (ph & 3));
}

// A tensor's rows: aligned words outside them are not touched.
struct Span {
    uintptr_t lo, hi;
    bool vec; // every row starts at 16 bytes (codes: 8) and is whole chunks
    __device__ __forceinline__ Span(const void *p, int64_t rows, int64_t ld, int cols, int esize, bool v)
        : lo(reinterpret_cast<uintptr_t>(p)), hi(lo + ((rows - 1) * ld + cols) * esize), vec(v)
    {
    }
};

// which tensors of a call are `vec` (the last two only in the backward)
enum : unsigned { kVecX = 1, kVecResidual = 2, kVecH = 4, kVecOut = 8, kVecWeight = 16, kVecCodes = 32, kVecDy = 64, kVecDx = 128 };

// Chunk of a row at column c0 (n valid columns of it; n <= 0: zeros).
template <typename T>
__device__ __forceinline__ void load_chunk(Vec8<T> &v, const T *row, int c0, int n, const Span &sp)
{
    constexpr int N = 2 * sizeof(T); // words of a chunk
    if (n <= 0) {
        v.zero();
        return;
    }
    if (sp.vec) {
        v.load(row + c0);
        return;
    }
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + c0), q = at & ~(uintptr_t)15;
    if (n < 8 || q < sp.lo || q + 4 * N + 16 > sp.hi) {
        v.load_n(row + c0, n < 8 ? n : 8);
        return;
    }
    uint32_t w[N + 4];
#pragma unroll
    for (int i = 0; i < N / 4 + 1; ++i) {
        const uint4 u = reinterpret_cast<const uint4 *>(q)[i];
        w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
    }
    shift_down<N>(w, (int)(at & 15));
    v.set_words(w);
}

// Stores a warp's 32 consecutive chunks (every lane calls; n <= 0: nothing of this lane's).  Aligned word k of a lane
// holds the last bytes of what stands before it and the first of what follows; its first word begins with the lane
// before's last bytes.
template <typename T>
__device__ __forceinline__ void store_chunk(const Vec8<T> &v, T *row, int c0, int n, const Span &sp)
{
    constexpr int N = 2 * sizeof(T);
    if (sp.vec) {
        if (n > 0)
            v.store(row + c0);
        return;
    }
    const int lane = threadIdx.x & 31;
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + c0);
    const int ph = (int)(at & 15);
    if (ph == 0 && n >= 8) // the same for the whole row, but for its short last chunk
        v.store(row + c0);
    const bool whole = n >= 8 && ph != 0;
    const uint32_t wholes = __ballot_sync(0xffffffffu, whole);
    if (ph == 0) {
        if (n > 0 && n < 8)
            v.store_n(row + c0, n);
        return;
    }
    uint32_t w[N + 4];
    v.get_words(w + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) // the lane before's last 16 bytes
        w[i] = __shfl_up_sync(0xffffffffu, w[N + i], 1);
    const bool joined = lane > 0 && whole && (wholes >> (lane - 1) & 1); // writes its first word whole
    const bool next = lane < 31 && (wholes >> lane & 3) == 3;            // its last bytes are the next lane's to write
    shift_down<N>(w, 16 - ph);                                           // w: the bytes from the first aligned word on
    uint4 *q = reinterpret_cast<uint4 *>(at - ph);
    if (joined)
        q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    if (N == 8 && whole)
        q[1] = make_uint4(w[4], w[5], w[6], w[7]);
    // what no aligned word took: a warp's first and last bytes, short chunks
    const int e = (int)sizeof(T), head = (16 - ph) / e, tail = N == 8 ? 8 - ph / e : head;
    if (n > 0)
        v.store_if(row + c0, n < 8 ? n : 8, [&](int i) { return !whole || (i < head && !joined) || (i >= tail && !next); });
}

// Codes of a warp's 32 consecutive chunks, 8 bytes a lane, in the same way.
__device__ __forceinline__ void store_codes(uint32_t lo, uint32_t hi, uint8_t *row, int c0, int n, bool vec)
{
    const uint64_t mine = (uint64_t)hi << 32 | lo;
    if (vec) {
        if (n > 0)
            *reinterpret_cast<uint64_t *>(row + c0) = mine;
        return;
    }
    const int lane = threadIdx.x & 31;
    uint8_t *at = row + c0;
    const int ph = (int)(reinterpret_cast<uintptr_t>(at) & 7);
    const uint64_t before = __shfl_up_sync(0xffffffffu, mine, 1);
    const uint32_t wholes = __ballot_sync(0xffffffffu, n >= 8);
    if (ph == 0 && n >= 8) {
        *reinterpret_cast<uint64_t *>(at) = mine;
        return;
    }
    const bool joined = ph && lane > 0 && (wholes >> (lane - 1) & 3) == 3;
    const bool next = ph && lane < 31 && (wholes >> lane & 3) == 3;
    if (joined)
        *reinterpret_cast<uint64_t *>(at - ph) = mine << (8 * ph) | before >> (64 - 8 * ph);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n && !(i < 8 - ph && joined) && !(i >= 8 - ph && next))
            at[i] = (uint8_t)(mine >> (8 * i));
}

// Two sums (or maxima) over the row's group; every thread gets the result.
// red: 2 x 32 floats of shared memory, only used when the group is the CTA.
template <bool WARP, bool MAX>
__device__ __forceinline__ float2 group_reduce(float a, float b, float *red)
{
    auto op = [](float x, float y) { return MAX ? fmaxf(x, y) : x + y; };
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a = op(a, __shfl_xor_sync(0xffffffffu, a, o));
        b = op(b, __shfl_xor_sync(0xffffffffu, b, o));
    }
    if (!WARP) {
        const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) {
            red[threadIdx.x >> 5] = a;
            red[32 + (threadIdx.x >> 5)] = b;
        }
        __syncthreads();
        a = lane < warps ? red[lane] : 0.f; // 0 leaves a maximum of magnitudes alone
        b = lane < warps ? red[32 + lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a = op(a, __shfl_xor_sync(0xffffffffu, a, o));
            b = op(b, __shfl_xor_sync(0xffffffffu, b, o));
        }
        __syncthreads(); // red is reused by the next reduction
    }
    return make_float2(a, b);
}

// One row: x and res (null: none) point at it, in global or shared memory.  VEC:
// every tensor of the call is vec.
template <typename T, typename W, int NV, bool WARP, bool VEC>
__device__ __forceinline__ void rmsnorm_row(const RmsNormArgs &a, const T *x, const T *res, int64_t row, float *red,
                                            unsigned vecs)
{
    const Span sx(a.x, a.rows, a.ldx, a.cols, sizeof(T), VEC || (vecs & kVecX));
    const Span sr(a.residual, a.rows, a.ldr, a.cols, sizeof(T), VEC || (vecs & kVecResidual));
    const Span sh(a.residual_out, a.rows, a.ldh, a.cols, sizeof(T), VEC || (vecs & kVecH));
    const Span so(a.out, a.rows, a.ldo, a.cols, sizeof(T), VEC || (vecs & kVecOut));
    const Span sw(a.weight, 1, 0, a.cols, sizeof(W), VEC || (vecs & kVecWeight));
    const int G = WARP ? 32 : blockDim.x;
    const int g = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int cols = a.cols;
    const W *weight = static_cast<const W *>(a.weight);
    Vec8<T> xv[NV], rv[NV];
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int c0 = (c * G + g) * 8;
        load_chunk(xv[c], x, c0, cols - c0, sx);
    }
    if (res) {
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int c0 = (c * G + g) * 8;
            load_chunk(rv[c], res, c0, cols - c0, sr);
        }
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
    // a tensor may be overwritten in place: each chunk is written by the
    // thread that read it
    if (a.residual_out) {
        T *ho = static_cast<T *>(a.residual_out) + row * a.ldh;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int c0 = (c * G + g) * 8;
            Vec8<T> v;
            v.set(h[c]);
            store_chunk(v, ho, c0, cols - c0, sh);
        }
    }
    ss = group_reduce<WARP, false>(ss, 0.f, red).x;
    const float r = 1.f / sqrtf(ss / (float)cols + a.eps);
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int c0 = (c * G + g) * 8;
        Vec8<W> wv;
        load_chunk(wv, weight, c0, cols - c0, sw);
        float w[8];
        wv.get(w);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            h[c][i] = h[c][i] * r * w[i];
    }
    if (a.out) {
        T *out = static_cast<T *>(a.out) + row * a.ldo;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int c0 = (c * G + g) * 8;
            Vec8<T> v;
            v.set(h[c]);
            store_chunk(v, out, c0, cols - c0, so);
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
        const int c0 = (c * G + g) * 8;
        if (a.block) { // 16 lanes x 8 values = one 128-column block
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                m = fmaxf(m, fabsf(h[c][i]));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            s = fp8_scale(m, a.scale_mode);
            if ((g & 15) == 0 && c0 < cols)
                scale[c0 / 128] = s;
            div = ScaleDivider(s);
        }
        const uint32_t lo = e4m3x4(div, h[c][0], h[c][1], h[c][2], h[c][3]);
        const uint32_t hi = e4m3x4(div, h[c][4], h[c][5], h[c][6], h[c][7]);
        store_codes(lo, hi, codes, c0, cols - c0, VEC || (vecs & kVecCodes));
    }
}

template <typename T, typename W, int NV, bool WARP, bool VEC>
__global__ void __launch_bounds__(WARP ? kRowThreads : 1024) rmsnorm_kernel(RmsNormArgs a, unsigned vecs)
{
    __shared__ float red[64];
    grid_dep_wait();
    grid_dep_launch();
    const int64_t row0 = WARP ? (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t step = (int64_t)gridDim.x * (WARP ? kRowThreads / 32 : 1);
    for (int64_t row = row0; row < a.rows; row += step)
        rmsnorm_row<T, W, NV, WARP, VEC>(a, static_cast<const T *>(a.x) + row * a.ldx,
                                    a.residual ? static_cast<const T *>(a.residual) + row * a.ldr : nullptr, row, red, vecs);
}

// ---- the ring of rows in shared memory
constexpr int kRingMost = 8;   // stages at most
constexpr int kRingBars = 128; // bytes in front of the stages: barriers and the abort flag
constexpr int kRingSmemMost = 222 << 10;

// Up to three tensors whose rows go through a ring, `group` rows a stage, each
// tensor's one after the other.
struct Ring {
    const uint8_t *src[3];
    int64_t ld[3]; // bytes
    int n, group, bytes, stages;
    int64_t rows;
    __device__ __forceinline__ int stage_bytes() const { return n * group * bytes; }
    __device__ __forceinline__ void load(int64_t row, uint32_t dst, uint32_t bar) const
    {
        const int g = rows - row < group ? (int)(rows - row) : group;
        mbar_arrive_expect_tx(bar, n * g * bytes);
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (k >= n)
                break;
            const bool one = ld[k] == bytes; // rows on end: one copy
            for (int i = 0; i < (one ? 1 : g); ++i)
                asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                 dst + (k * group + i) * bytes),
                             "l"(src[k] + (row + i) * ld[k]), "r"(one ? g * bytes : bytes), "r"(bar)
                             : "memory");
        }
    }
    // Walks the groups blockIdx.x, + gridDim.x, ...; row_fn(stage, first row) works on one with every thread of the CTA
    // and ends with its values in registers or written.  All threads meet before a stage is filled again.
    template <typename F> __device__ __forceinline__ void walk(uint8_t *smem, unsigned *status, F &&row_fn) const
    {
        const uint32_t bar0 = smem_u32(smem);
        volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + 8 * kRingMost);
        uint8_t *data = smem + kRingBars;
        if (threadIdx.x == 0) {
            for (int i = 0; i < stages; ++i)
                mbar_init(bar0 + 8 * i, 1);
            *abort_flag = 0;
            fence_mbar_init();
        }
        __syncthreads();
        grid_dep_wait();
        grid_dep_launch();
        const int64_t first = (int64_t)blockIdx.x * group, step = (int64_t)gridDim.x * group;
        if (threadIdx.x == 0)
            for (int i = 0; i < stages; ++i)
                if (first + i * step < rows)
                    load(first + i * step, smem_u32(data) + i * stage_bytes(), bar0 + 8 * i);
        int st = 0, phase = 0;
        for (int64_t row = first; row < rows; row += step) {
            const bool ok = mbar_wait(bar0 + 8 * st, phase, abort_flag, status);
            if (!__syncthreads_and(ok))
                break;
            row_fn(data + st * stage_bytes(), row);
            __syncthreads();
            if (threadIdx.x == 0 && row + stages * step < rows)
                load(row + stages * step, smem_u32(data) + st * stage_bytes(), bar0 + 8 * st);
            if (++st == stages) {
                st = 0;
                phase ^= 1;
            }
        }
        // after a wait that gave up: a millisecond is far longer than any copy in flight takes
        if (*abort_flag) {
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 1000000ull) {
            }
        }
    }
};

// WARP: a stage is a row for each warp.
template <typename T, typename W, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 512, WARP ? 2 : 1) rmsnorm_ring_kernel(RmsNormArgs a, int stages, unsigned *status)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[64];
    const int bytes = a.cols * (int)sizeof(T), group = WARP ? blockDim.x >> 5 : 1, w = WARP ? threadIdx.x >> 5 : 0;
    const Ring ring{{static_cast<const uint8_t *>(a.x), static_cast<const uint8_t *>(a.residual), nullptr},
                    {a.ldx * (int64_t)sizeof(T), a.ldr * (int64_t)sizeof(T), 0},
                    a.residual ? 2 : 1, group, bytes, stages, a.rows};
    ring.walk(smem, status, [&](uint8_t *stage, int64_t row) {
        if (row + w < a.rows)
            rmsnorm_row<T, W, NV, WARP, true>(a, reinterpret_cast<const T *>(stage + w * bytes),
                                              a.residual ? reinterpret_cast<const T *>(stage + (group + w) * bytes) : nullptr,
                                              row + w, red, 0);
    });
}

// One row of the backward; dw: this thread's dweight sums.
template <typename T, typename W, int NV, bool WARP, bool VEC>
__device__ __forceinline__ void rmsnorm_backward_row(const RmsNormBackwardArgs &a, const T *hp, const T *dp, const T *ep,
                                                     int64_t row, float (&dw)[NV][8], float *red, unsigned vecs)
{
    const Span sh(a.h, a.rows, a.cols, a.cols, sizeof(T), VEC || (vecs & kVecH)), sd(a.dy, a.rows, a.cols, a.cols, sizeof(T), VEC || (vecs & kVecDy));
    const Span se(a.dres, a.rows, a.cols, a.cols, sizeof(T), VEC || (vecs & kVecResidual));
    const Span sx(a.dx, a.rows, a.cols, a.cols, sizeof(T), VEC || (vecs & kVecDx));
    const Span sw(a.weight, 1, 0, a.cols, sizeof(W), VEC || (vecs & kVecWeight));
    const int G = WARP ? 32 : blockDim.x;
    const int g = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int cols = a.cols;
    Vec8<T> hv[NV], dv[NV];
    float ss = 0.f, sg = 0.f;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int c0 = (c * G + g) * 8;
        load_chunk(hv[c], hp, c0, cols - c0, sh);
        load_chunk(dv[c], dp, c0, cols - c0, sd);
    }
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int c0 = (c * G + g) * 8;
        float h[8], d[8], w[8], s = 0.f, t = 0.f;
        Vec8<W> wv;
        load_chunk(wv, static_cast<const W *>(a.weight), c0, cols - c0, sw);
        hv[c].get(h);
        dv[c].get(d);
        wv.get(w);
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
        const int c0 = (c * G + g) * 8;
        float h[8], d[8], w[8], o[8];
        Vec8<W> wv;
        load_chunk(wv, static_cast<const W *>(a.weight), c0, cols - c0, sw);
        hv[c].get(h);
        dv[c].get(d);
        wv.get(w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            o[i] = r * (d[i] * w[i] - h[i] * k);
            dw[c][i] = fmaf(d[i], h[i] * r, dw[c][i]);
        }
        if (ep) {
            float e[8];
            Vec8<T> ev;
            load_chunk(ev, ep, c0, cols - c0, se);
            ev.get(e);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                o[i] += e[i];
        }
        Vec8<T> v;
        v.set(o);
        store_chunk(v, static_cast<T *>(a.dx) + row * cols, c0, cols - c0, sx);
    }
}

// A CTA's dweight sums as one fp32 row of the workspace.
template <int NV>
__device__ __forceinline__ void store_part(float *part, const float (&dw)[NV][8], int G, int g, int cols)
{
    float *row = part + (int64_t)blockIdx.x * cols;
    const Span sp(row, 1, 0, cols, 4, cols % 8 == 0);
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int c0 = (c * G + g) * 8;
        Vec8<float> v;
        v.set(dw[c]);
        store_chunk(v, row, c0, cols - c0, sp);
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
template <typename T, typename W, int NV, bool WARP, bool VEC>
__global__ void __launch_bounds__(WARP ? kRowThreads : 1024)
    rmsnorm_backward_kernel(RmsNormBackwardArgs a, float *part, unsigned vecs)
{
    __shared__ float red[64];
    __shared__ float dws[WARP ? 32 * 8 * NV : 1];
    grid_dep_wait();
    grid_dep_launch();
    const int G = WARP ? 32 : blockDim.x;
    const int g = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t row0 = WARP ? (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t step = (int64_t)gridDim.x * (WARP ? kRowThreads / 32 : 1);
    const int cols = a.cols;
    float dw[NV][8] = {};
    for (int64_t row = row0; row < a.rows; row += step)
        rmsnorm_backward_row<T, W, NV, WARP, VEC>(a, static_cast<const T *>(a.h) + row * cols,
                                             static_cast<const T *>(a.dy) + row * cols,
                                             a.dres ? static_cast<const T *>(a.dres) + row * cols : nullptr, row, dw, red, vecs);
    if (WARP && !join_warps<NV>(dw, dws))
        return;
    store_part<NV>(part, dw, G, g, cols);
}

template <typename T, typename W, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 512, WARP ? 2 : 1)
    rmsnorm_backward_ring_kernel(RmsNormBackwardArgs a, float *part, int stages, unsigned *status)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[64];
    const int bytes = a.cols * (int)sizeof(T), group = WARP ? blockDim.x >> 5 : 1, w = WARP ? threadIdx.x >> 5 : 0;
    const Ring ring{{static_cast<const uint8_t *>(a.h), static_cast<const uint8_t *>(a.dy), static_cast<const uint8_t *>(a.dres)},
                    {bytes, bytes, bytes}, a.dres ? 3 : 2, group, bytes, stages, a.rows};
    float dw[NV][8] = {};
    ring.walk(smem, status, [&](uint8_t *stage, int64_t row) {
        const uint8_t *at = stage + w * bytes;
        if (row + w < a.rows)
            rmsnorm_backward_row<T, W, NV, WARP, true>(a, reinterpret_cast<const T *>(at),
                                                       reinterpret_cast<const T *>(at + group * bytes),
                                                       a.dres ? reinterpret_cast<const T *>(at + 2 * group * bytes) : nullptr,
                                                       row + w, dw, red, 0);
    });
    if (WARP && !join_warps<NV>(dw, reinterpret_cast<float *>(smem + kRingBars)))
        return;
    store_part<NV>(part, dw, WARP ? 32 : blockDim.x, WARP ? threadIdx.x & 31 : threadIdx.x, a.cols);
}

// dweight[c] = sum of the nparts partial rows: 32 columns a CTA, the rows
// dealt to 32 warps, whose sums are added in order.
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

bool chunked(const void *p, int64_t ld_bytes) { return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)ld_bytes) & 15) == 0; }

struct Shape {
    int nv;      // chunks per thread
    int threads; // per CTA
    bool warp;   // a warp per row
    int stages;  // > 0: the ring (nv = 4)
    int ctas;    // ring: CTAs per SM
    size_t smem; // ring
};

// Threads per row, and whether rows (of n tensors of esize-byte values) go
// through the ring: where they are aligned and at least four for each SM and
// row of threads.  Its CTAs per SM are as many as leave each two stages; more
// than 128 KB of stages an SM only slowed the writes among them (99.7 us with
// three stages, 95.8 with two, at 8191 x 8192).
Shape shape_of(int64_t rows, int cols, int n, int esize, bool vec)
{
    const bool warp = cols <= 1024; // rows of single warps: several a CTA, no barrier
    const int nv = cols <= 256 ? 1 : 4;
    const int ring_threads = warp ? 256 : cols > 8192 ? 512 : cols > 4096 ? 256 : 128;
    const int group = warp ? ring_threads / 32 : 1;
    if (vec && rows >= 4LL * num_sms() * group) {
        const size_t stage = (size_t)n * group * cols * esize;
        for (int ctas = 512 / ring_threads; ctas > 0; ctas /= 2) {
            size_t stages = ((size_t)kRingSmemMost / ctas - 1024 - kRingBars) / stage;
            if (stages < 2)
                continue;
            const size_t want = (size_t)(128 << 10) / ctas / stage;
            stages = stages < want ? stages : want < 2 ? 2 : want > kRingMost ? kRingMost : want;
            size_t smem = stages * stage;
            if (warp && smem < 32 * 8 * 4 * sizeof(float)) // the warps' sums of the backward
                smem = 32 * 8 * 4 * sizeof(float);
            return {nv, ring_threads, warp, (int)stages, ctas, kRingBars + smem};
        }
    }
    if (warp)
        return {nv, kRowThreads, true, 0, 0, 0};
    // a chunk a thread, the shortest way through a row, up to the 8192 values
    // that 1024 threads then hold (8000 unaligned rows of 4001: 151 us, 166 with
    // four chunks; backward 130 and 278)
    int threads = 64;
    while (threads < 1024 && threads * 8 < cols)
        threads *= 2;
    return {cols > 8192 ? 2 : 1, threads, false, 0, 0, 0};
}

template <typename F>
cudaError_t dispatch_types(bool x32, bool w32, F &&f)
{
    using bf16 = __nv_bfloat16;
    if (x32)
        return w32 ? f((float *)0, (float *)0) : f((float *)0, (bf16 *)0);
    return w32 ? f((bf16 *)0, (float *)0) : f((bf16 *)0, (bf16 *)0);
}

// f(t, w, chunks per thread, warp per row) for the shape's kernel.
template <typename F>
cudaError_t dispatch(const Shape &s, bool x32, bool w32, F &&f)
{
    using std::integral_constant;
    return dispatch_types(x32, w32, [&](auto t, auto w) {
        if (s.warp)
            return s.nv == 1 ? f(t, w, integral_constant<int, 1>(), std::true_type())
                             : f(t, w, integral_constant<int, 4>(), std::true_type());
        return s.nv == 1   ? f(t, w, integral_constant<int, 1>(), std::false_type())
               : s.nv == 2 ? f(t, w, integral_constant<int, 2>(), std::false_type())
                           : f(t, w, integral_constant<int, 4>(), std::false_type());
    });
}

int64_t rows_grid(int64_t rows, const Shape &s, int64_t most)
{
    const int64_t per = s.warp ? s.threads / 32 : 1;
    const int64_t n = (rows + per - 1) / per;
    return n < most ? n : most;
}

// CTAs of a backward: a row of the workspace each.
int64_t backward_ctas(int64_t rows, const Shape &s)
{
    return rows_grid(rows, s, (int64_t)(s.stages ? s.ctas : s.warp ? 4 : 2) * num_sms());
}

} // namespace

int launch_rmsnorm(const RmsNormArgs &a, cudaStream_t stream, char *err, size_t errlen)
{
    const int e = a.x32 ? 4 : 2;
    const bool whole = a.cols % 8 == 0;
    unsigned vecs = 0;
    vecs |= whole && chunked(a.x, a.ldx * e) ? kVecX : 0;
    vecs |= whole && chunked(a.residual, a.ldr * e) ? kVecResidual : 0;
    vecs |= whole && chunked(a.residual_out, a.ldh * e) ? kVecH : 0;
    vecs |= whole && chunked(a.out, a.ldo * e) ? kVecOut : 0;
    vecs |= whole && chunked(a.weight, 0) ? kVecWeight : 0;
    vecs |= whole && (reinterpret_cast<uintptr_t>(a.codes) & 7) == 0 ? kVecCodes : 0;
    const unsigned all = kVecX | kVecResidual | kVecH | kVecOut | kVecWeight | kVecCodes;
    const bool ring = (vecs & all) == all; // a null tensor counts as aligned
    const Shape s = shape_of(a.rows, a.cols, a.residual ? 2 : 1, e, ring);
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
        if constexpr (WARP || NV == 4)
            if (s.stages) {
                static std::atomic<bool> raised[64];
                cudaError_t r = raise_smem_limit_once(rmsnorm_ring_kernel<T, W, NV, WARP>, kRingSmemMost, raised);
                if (r != cudaSuccess)
                    return r;
                return launch_pdl(rmsnorm_ring_kernel<T, W, NV, WARP>,
                                  dim3((unsigned)rows_grid(a.rows, s, (int64_t)s.ctas * num_sms())), dim3(s.threads), s.smem,
                                  stream, 1, a, s.stages, status);
            }
        auto go = [&](auto kernel) {
            return launch_pdl(kernel, dim3((unsigned)rows_grid(a.rows, s, 1 << 30)), dim3(s.threads), 0, stream, 1, a, vecs);
        };
        if constexpr (NV == 2) // aligned rows too long for the ring
            if (ring)
                return go(rmsnorm_kernel<T, W, NV, WARP, true>);
        if constexpr (WARP || NV != 4)
            return go(rmsnorm_kernel<T, W, NV, WARP, false>);
        return cudaErrorInvalidValue; // four chunks a thread: the ring alone
    });
    if (rc != cudaSuccess) {
        snprintf(err, errlen, "rmsnorm launch: %s", cudaGetErrorString(rc));
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

// The most that any alignment, type and dres needs: which of them a call has is
// not known here.
size_t rmsnorm_backward_workspace_bytes(int64_t rows, int cols)
{
    int64_t most = 0;
    for (int esize = 2; esize <= 4; esize += 2)
        for (int n = 2; n <= 3; ++n)
            for (int vec = 0; vec < 2; ++vec) {
                const int64_t c = backward_ctas(rows, shape_of(rows, cols, n, esize, vec != 0));
                most = c > most ? c : most;
            }
    return (size_t)most * cols * sizeof(float);
}

int launch_rmsnorm_backward(const RmsNormBackwardArgs &a, cudaStream_t stream, char *err, size_t errlen)
{
    const int e = a.x32 ? 4 : 2;
    const int64_t ld = (int64_t)a.cols * e;
    const bool whole = a.cols % 8 == 0;
    unsigned vecs = 0;
    vecs |= whole && chunked(a.h, ld) ? kVecH : 0;
    vecs |= whole && chunked(a.dy, ld) ? kVecDy : 0;
    vecs |= whole && chunked(a.dres, ld) ? kVecResidual : 0;
    vecs |= whole && chunked(a.dx, ld) ? kVecDx : 0;
    vecs |= whole && chunked(a.weight, 0) ? kVecWeight : 0;
    const unsigned all = kVecH | kVecDy | kVecResidual | kVecDx | kVecWeight;
    const bool ring = (vecs & all) == all; // a null dres counts as aligned
    const Shape s = shape_of(a.rows, a.cols, a.dres ? 3 : 2, e, ring);
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
            if constexpr (WARP || NV == 4)
                if (s.stages) {
                    static std::atomic<bool> raised[64];
                    cudaError_t r = raise_smem_limit_once(rmsnorm_backward_ring_kernel<T, W, NV, WARP>, kRingSmemMost, raised);
                    if (r != cudaSuccess)
                        return r;
                    return launch_pdl(rmsnorm_backward_ring_kernel<T, W, NV, WARP>, dim3((unsigned)grid), dim3(s.threads), s.smem,
                                      stream, 1, a, part, s.stages, status);
                }
            auto go = [&](auto kernel) {
                return launch_pdl(kernel, dim3((unsigned)grid), dim3(s.threads), 0, stream, 1, a, part, vecs);
            };
            if constexpr (NV == 2) // aligned rows too long for the ring
                if (ring)
                    return go(rmsnorm_backward_kernel<T, W, NV, WARP, true>);
            if constexpr (WARP || NV != 4)
                return go(rmsnorm_backward_kernel<T, W, NV, WARP, false>);
            return cudaErrorInvalidValue; // four chunks a thread: the ring alone
        });
    if (rc == cudaSuccess) // no rows: the sum of nothing, zeros
        rc = launch_pdl(dweight_kernel, dim3((unsigned)((a.cols + 31) / 32)), dim3(1024), 0, stream, 1, (const float *)part,
                        grid, a.cols, a.dweight);
    if (rc != cudaSuccess) {
        snprintf(err, errlen, "rmsnorm backward launch: %s", cudaGetErrorString(rc));
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

} // namespace dsa
