// What the RMS norm and its backward share: eight values of a row as a thread
// holds them, rows at any address, sums over a row's threads, the ring of rows
// in shared memory, and which threads take which rows.
#pragma once

#include "common.cuh"
#include "f32x2.cuh"
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
};

template <> struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void load(const float *p)
    {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
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
    __device__ __forceinline__ void store(float *p) const
    {
        reinterpret_cast<float4 *>(p)[0] = a;
        reinterpret_cast<float4 *>(p)[1] = b;
    }
};

// ---- which columns a thread holds
//
// Chunk c of thread g of a row's G threads.  VEC (every row of every tensor of the
// call starts at 16 bytes and is whole chunks): the eight columns from
// (c G + g) 8 on, as 16-byte words.  Else the warp's 256 columns from
// (c G + its first thread) 8 on are dealt out value by value (fp32: 32 j + lane)
// or pair by pair (bf16: 64 j + 2 lane and the next), so that a warp's accesses
// are consecutive at any alignment and free of bank conflicts in shared memory.
// Eight columns a thread, put together from aligned words and handed to the next
// lane, took 9000 x 8191 rows with all outputs 330 us, laid out in shared memory
// and copied from there 226.
template <bool VEC> __device__ __forceinline__ int chunk_base(int c, int G, int g)
{
    return VEC ? (c * G + g) * 8 : (c * G + (g & ~31)) * 8;
}

// Column of value j of the chunk at cb.
template <typename T, bool VEC> __device__ __forceinline__ int column(int cb, int j)
{
    const int lane = threadIdx.x & 31;
    return VEC ? cb + j : sizeof(T) == 4 ? cb + 32 * j + lane : cb + 64 * (j >> 1) + 2 * lane + (j & 1);
}

template <bool VEC, typename T> __device__ __forceinline__ void load_chunk(Vec8<T> &v, const T *row, int cb, int cols)
{
    v.zero();
    if (cb >= cols)
        return;
    if (VEC) {
        v.load(row + cb);
        return;
    }
    constexpr int N = 2 * sizeof(T); // words
    const bool whole = cb + 256 <= cols;
    uint32_t w[N];
    if (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = column<T, VEC>(cb, j);
            w[j] = whole || c < cols ? reinterpret_cast<const uint32_t *>(row)[c] : 0;
        }
    } else {
        const uint16_t *r = reinterpret_cast<const uint16_t *>(row) + column<T, VEC>(cb, 0);
        const int left = cols - column<T, VEC>(cb, 0); // columns from this thread's first on
        if (!whole) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                w[j] = (64 * j < left ? r[64 * j] : 0u) | (64 * j + 1 < left ? (uint32_t)r[64 * j + 1] << 16 : 0u);
        } else if (reinterpret_cast<uintptr_t>(row) & 2) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                w[j] = __byte_perm(r[64 * j], r[64 * j + 1], 0x5410);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
                w[j] = *reinterpret_cast<const uint32_t *>(r + 64 * j);
        }
    }
    v.set_words(w);
}

template <bool VEC, typename T> __device__ __forceinline__ void store_chunk(const Vec8<T> &v, T *row, int cb, int cols)
{
    if (cb >= cols)
        return;
    if (VEC) {
        v.store(row + cb);
        return;
    }
    constexpr int N = 2 * sizeof(T);
    const bool whole = cb + 256 <= cols;
    uint32_t w[N];
    v.get_words(w);
    if (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = column<T, VEC>(cb, j);
            if (whole || c < cols)
                reinterpret_cast<uint32_t *>(row)[c] = w[j];
        }
    } else {
        uint16_t *r = reinterpret_cast<uint16_t *>(row) + column<T, VEC>(cb, 0);
        const int left = cols - column<T, VEC>(cb, 0);
        if (!whole) {
#pragma unroll
            for (int j = 0; j < 2 * N; ++j)
                if (64 * (j >> 1) + (j & 1) < left)
                    r[64 * (j >> 1) + (j & 1)] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
        } else if (reinterpret_cast<uintptr_t>(row) & 2) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                r[64 * j] = (uint16_t)w[j];
                r[64 * j + 1] = (uint16_t)(w[j] >> 16);
            }
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
                *reinterpret_cast<uint32_t *>(r + 64 * j) = w[j];
        }
    }
}

// Weights (or their like) of a chunk of T's columns.
template <typename T, bool VEC, typename W> __device__ __forceinline__ void load_weights(float (&f)[8], const W *row, int cb, int cols)
{
    if (VEC || sizeof(W) == sizeof(T)) {
        Vec8<W> v;
        load_chunk<VEC>(v, row, cb, cols);
        v.get(f);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = column<T, VEC>(cb, j);
        f[j] = c < cols ? (float)row[c] : 0.f;
    }
}

// Weights that a thread keeps for all its rows, as loaded: an SM's L1 beside a ring holds little else.
template <typename T, typename W, int NV, bool VEC> struct Held {
    static constexpr bool kHolds = (VEC || sizeof(W) == sizeof(T)) && sizeof(W) * NV <= 8;
    Vec8<W> v[kHolds ? NV : 1];
    __device__ __forceinline__ void load(const W *row, int G, int g, int cols)
    {
        if constexpr (kHolds)
#pragma unroll
            for (int c = 0; c < NV; ++c)
                load_chunk<VEC>(v[c], row, chunk_base<VEC>(c, G, g), cols);
    }
    __device__ __forceinline__ void get(float (&f)[8], const W *row, int c, int cb, int cols) const
    {
        if constexpr (kHolds)
            v[c].get(f);
        else
            load_weights<T, VEC>(f, row, cb, cols);
    }
};

// The codes of a chunk of T's columns.
template <typename T, bool VEC> __device__ __forceinline__ void store_codes(uint32_t lo, uint32_t hi, uint8_t *row, int cb, int cols)
{
    if (cb >= cols)
        return;
    if (VEC) {
        *reinterpret_cast<uint2 *>(row + cb) = make_uint2(lo, hi);
        return;
    }
    const bool whole = cb + 256 <= cols;
    if (sizeof(T) == 2 && whole && (reinterpret_cast<uintptr_t>(row) & 1) == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint16_t *>(row + column<T, VEC>(cb, 2 * j)) = (uint16_t)((j < 2 ? lo : hi) >> (16 * (j & 1)));
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (whole || column<T, VEC>(cb, j) < cols)
            row[column<T, VEC>(cb, j)] = (uint8_t)((j < 4 ? lo : hi) >> (8 * (j & 3)));
}

// Largest magnitude in the warp.
__device__ __forceinline__ float warp_amax(float m)
{
    float r;
    asm volatile("redux.sync.max.abs.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(m));
    return r;
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

// ---- sums about the mean (layer norm)
//
// A row's mean and sum of squares about it, from one meeting of its warps: each warp takes the sums about its own mean,
// and n (its mean - the row's)^2 is what that leaves out (T. Chan, G. Golub, R. LeVeque, "Algorithms for computing the
// sample variance", 1983).
template <int LANES = 32> __device__ __forceinline__ float warp_sum(float a)
{
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
        a += __shfl_xor_sync(0xffffffffu, a, o);
    return a;
}

// Sums of a and of b over the LANES lanes of a row together: where a lane ends with a's in the lower half, with b's in the
// upper one.
template <int LANES = 32> __device__ __forceinline__ float half_sums(float a, float b)
{
    const bool upper = threadIdx.x & (LANES / 2);
    const float give = upper ? a : b;
    a = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, give, LANES / 2);
    return warp_sum<LANES / 2>(a);
}

// What lane 0 (HALF = 0) or the upper half (1) of LANES lanes has.
template <int LANES, int HALF> __device__ __forceinline__ float from_half(float a)
{
    return __shfl_sync(0xffffffffu, a, HALF * (LANES / 2), LANES);
}

// Columns of a row that warp w of a row's G threads holds.
template <int NV> __device__ __forceinline__ int warp_columns(int G, int w, int cols)
{
    int n = 0;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int left = cols - (c * G + 32 * w) * 8;
        n += left < 0 ? 0 : left < 256 ? left : 256;
    }
    return n;
}

// A count of columns, its reciprocal, and what the reciprocal's rounding left out (48 bits together).
//
// A mean is the sum's quotient, correctly rounded: columns of one value whose sum is exact in fp32 (bf16 values, or as short
// ones) have that value as their mean, and nothing is left of them.  The product with the reciprocal alone is an ulp off for
// most counts: of 50432 in 1000 columns a deviation of 0.004 was left, 0.97 once normed.  By the remainder it is correctly rounded
// (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", 1990), by the parts but for
// quotients within 2^-47 of the middle between two fp32, an operation sooner: which of the two a kernel takes was measured (8192
// columns, us: forward with residual and codes 98.1 by the remainder, 99.1 by the parts; backward 96.7, 95.2).
struct Count {
    float n, inv, rest;
    __device__ __forceinline__ Count(int count = 0) : n((float)count), inv(count ? 1.f / n : 0.f), rest(fmaf(-inv, n, 1.f) * inv) {}
    __device__ __forceinline__ float mean_by_remainder(float s) const
    {
        const float q = s * inv;
        return fmaf(fmaf(-q, n, s), inv, q);
    }
    __device__ __forceinline__ float mean_by_parts(float s) const { return fmaf(s, inv, s * rest); }
};

// How many columns there are, before the first row: of a thread's warp, of warp `lane`, of the row.
struct Counts {
    Count mine, other, all;
    template <int NV, bool WARP> static __device__ __forceinline__ Counts of(int G, int cols)
    {
        const int lane = threadIdx.x & 31;
        return {Count(WARP ? cols : warp_columns<NV>(G, threadIdx.x >> 5, cols)),
                Count(WARP || 32 * lane >= G ? 0 : warp_columns<NV>(G, lane, cols)), Count(cols)};
    }
};

// 1 / sqrt(v), off by hardly more than its rounding: rsqrtf, up to 2 ulp off, and one of Newton's steps, r + r (1 - v r r) / 2
// with v r (which neither over- nor underflows) in two parts.  0, infinity and NaN, whose residual is NaN, keep rsqrtf's
// result.  1 / sqrtf(v) is further off, and took the backward of 8192 x 8192 from 95 to 108 us; this 96.
__device__ __forceinline__ float inv_sqrt(float v)
{
    const float r = rsqrtf(v), q = v * r;
    return fmaf(0.5f * r, fminf(fmaf(-fmaf(v, r, -q), r, fmaf(-q, r, 1.f)), 1.f), r); // fminf drops a NaN
}

constexpr int kMoments = 4 * 32; // floats that a meeting takes, at most; the next of the same CTA takes others

// ---- the ring of rows in shared memory
constexpr int kRingMost = 8;   // stages at most
constexpr int kRingBars = 128; // bytes in front of the stages: barriers and the abort flag
constexpr int kRingSmemMost = 222 << 10;

// Bytes that a row takes in a stage: rows that do not all start at 16 bytes come
// with the rest of their first and last aligned words.
__host__ __device__ __forceinline__ int ring_pitch(int bytes, bool vec) { return vec ? bytes : (bytes + 30) & ~15; }

// Up to three tensors whose rows go through a ring, `group` rows a stage, each
// tensor's one after the other.
template <bool VEC> struct Ring {
    const uint8_t *src[3];
    int64_t ld[3]; // bytes
    int n, group, bytes, stages;
    int64_t rows;
    __device__ __forceinline__ int pitch() const { return ring_pitch(bytes, VEC); }
    __device__ __forceinline__ int stage_bytes() const { return n * group * pitch(); }
    // Where row `row` + i of tensor k starts in a stage whose first row is `row`.
    __device__ __forceinline__ int at(int k, int64_t row, int i) const
    {
        if (VEC)
            return (k * group + i) * bytes;
        const bool one = ld[k] == bytes; // rows on end
        const int phase = (int)(reinterpret_cast<uintptr_t>(src[k] + (row + (one ? 0 : i)) * ld[k]) & 15);
        return k * group * pitch() + phase + i * (one ? bytes : pitch());
    }
    // `len` bytes of tensor k from row `row` on, as aligned words: those that reach past the tensor's own bytes are left to
    // plain copies of what they hold of it.
    __device__ __forceinline__ void words(int k, int64_t row, int len, uint8_t *dst, uint32_t bar) const
    {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(src[k]), hi = lo + (rows - 1) * ld[k] + bytes;
        const uintptr_t a = lo + row * ld[k], b = a + len, first = a & ~(uintptr_t)15, last = (b + 15) & ~(uintptr_t)15;
        uintptr_t s = first, e = last;
        if (first < lo || last > hi) { // the tensor's first or last row
            s += first < lo ? 16 : 0;
            e -= last > hi ? 16 : 0;
            e = e < s ? s : e;
            for (uintptr_t p = a; p < s && p < b; p += 2)
                *reinterpret_cast<uint16_t *>(dst + (p - first)) = *reinterpret_cast<const uint16_t *>(p);
            for (uintptr_t p = e > a ? e : a; p < b; p += 2)
                *reinterpret_cast<uint16_t *>(dst + (p - first)) = *reinterpret_cast<const uint16_t *>(p);
        }
        if (e > s) {
            asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"((uint32_t)(e - s)) : "memory");
            copy(smem_u32(dst) + (int)(s - first), reinterpret_cast<const uint8_t *>(s), (int)(e - s), bar);
        }
    }
    __device__ __forceinline__ static void copy(uint32_t dst, const uint8_t *p, int len, uint32_t bar)
    {
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(p),
                     "r"(len), "r"(bar)
                     : "memory");
    }
    __device__ __forceinline__ void load(int64_t row, uint8_t *dst, uint32_t bar) const
    {
        const int g = rows - row < group ? (int)(rows - row) : group;
        if (VEC) {
            mbar_arrive_expect_tx(bar, n * g * bytes);
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                if (k >= n)
                    break;
                const bool one = ld[k] == bytes;
                for (int i = 0; i < (one ? 1 : g); ++i)
                    copy(smem_u32(dst) + (k * group + i) * bytes, src[k] + (row + i) * ld[k], one ? g * bytes : bytes, bar);
            }
            return;
        }
        fence_proxy_async_smem(); // plain copies of this stage's last turn, before bulk ones
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (k >= n)
                break;
            const bool one = ld[k] == bytes;
            for (int i = 0; i < (one ? 1 : g); ++i)
                words(k, row + i, one ? g * bytes : bytes, dst + (k * group + i) * pitch(), bar);
        }
        mbar_arrive(bar); // after the plain copies, which it releases
    }
    // Walks the groups blockIdx.x, + gridDim.x, ...; row_fn(stage, first row) works on one with every thread of the CTA
    // and ends with its values in registers or written.  All threads meet before a stage is filled again.
    // MEETS: row_fn(stage, first row, came, meet) calls meet() once, when it has read the stage, as the threads' one meeting in a
    // row: the stage may be filled again, and what the threads wrote to shared memory before can be read.  Where that returns
    // false the stage never came for one of them, and the walk ends; came says so of this thread, before the meeting.
    template <bool MEETS = false, typename F> __device__ __forceinline__ void walk(uint8_t *smem, unsigned *status, F &&row_fn) const
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
                    load(first + i * step, data + i * stage_bytes(), bar0 + 8 * i);
        int st = 0, phase = 0;
        for (int64_t row = first; row < rows; row += step) {
            const bool ok = mbar_wait(bar0 + 8 * st, phase, abort_flag, status);
            auto fill = [&] {
                if (threadIdx.x == 0 && row + stages * step < rows)
                    load(row + stages * step, data + st * stage_bytes(), bar0 + 8 * st);
            };
            if constexpr (MEETS) {
                bool all = false;
                row_fn(data + st * stage_bytes(), row, ok, [&] {
                    all = __syncthreads_and(ok);
                    if (all)
                        fill();
                    return all;
                });
                if (!all)
                    break;
            } else {
                if (!__syncthreads_and(ok))
                    break;
                row_fn(data + st * stage_bytes(), row);
                __syncthreads();
                fill();
            }
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

bool chunked(const void *p, int64_t ld_bytes) { return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)ld_bytes) & 15) == 0; }

struct Shape {
    int nv;      // chunks per thread
    int threads; // per CTA
    bool warp;   // a warp per row
    int stages;  // > 0: the ring
    int ctas;    // ring: CTAs per SM
    size_t smem; // ring
};

// Threads per row, and whether rows (of n tensors of esize-byte values) go
// through the ring.  Its CTAs have 512 threads an SM together, with at most four
// chunks each, and are as many as leave each two stages: eight of 64 threads took
// 24000 x 2048 bf16 in 76 us, four of 128 in 96.  More than 128 KB of stages an SM
// only slowed the writes among them (99.7 us with three stages, 95.8 with two, at
// 8191 x 8192).  The ring pays where an SM has several turns of rows to keep loads
// ahead of; before that a chunk a thread is the shorter way, and with short rows it
// stays so longer, as twice the threads are at work (forward with residual and
// block codes, direct and ring, us: 400 x 8192 bf16 8.8, 8.0; 800 x 8192 16.1,
// 11.3; 800 x 4096 8.0, 7.8; 3200 x 1024 7.0, 14.5; 3200 x 2048 12.9, 14.7; 1600 x
// 4096 fp32 19.3, 25.6), up to 256 columns always (24000 x 256 10.5, 17.1; backward
// 11.8, 12.7).  So it does in the forward of rows of up to 2048 columns at any
// address, which instructions bound (wide = false: 24000 x 1111 84, 124; backward
// 163, 84).
//
// Layer norm's backward holds two sums a column, and so takes twice the threads for a row (light = false: 8192 x 8192
// with four chunks a thread, whose sums then spill, 157 us).
Shape shape_of(int64_t rows, int cols, int n, int esize, bool vec, bool wide, bool light = true)
{
    const size_t row = (size_t)n * ring_pitch(cols * esize, vec);
    const auto ring = [&](int threads, int ctas, int group, bool warp) {
        const size_t stage = row * group;
        const size_t fit = ((size_t)kRingSmemMost / ctas - 1024 - kRingBars) / stage, want = (size_t)(128 << 10) / ctas / stage;
        const int stages = (int)(fit < want ? fit : want < 2 ? 2 : want > kRingMost ? kRingMost : want);
        const int nv = (cols + 8 * threads / group - 1) / (8 * threads / group);
        size_t smem = stages * stage;
        if (warp && smem < 32 * 8 * 4 * sizeof(float)) // the warps' sums of the backward
            smem = 32 * 8 * 4 * sizeof(float);
        return Shape{nv <= 1 && warp ? 1 : nv <= 2 ? 2 : 4, threads, warp, fit < 2 ? 0 : stages, ctas, kRingBars + smem};
    };
    if (cols > 256 && cols <= (light ? 1024 : 512) && rows >= 32 * num_sms()) { // rows of single warps: no barrier among them
        const Shape s = ring(256, 2, 8, true);
        if (s.stages)
            return s;
    }
    const int direct = (cols + 255) / 256 * 32; // threads a row takes with a chunk each
    if (cols > (wide ? 256 : 2048) && rows * direct >= (cols > 4096 ? 2LL : 8LL) * 1024 * num_sms())
        for (int ctas = 8; ctas > 0; ctas /= 2)
            if (cols * ctas <= (light || ctas == 1 ? 32 : 16) * 512) { // four chunks a thread at most
                const Shape s = ring(512 / ctas, ctas, 1, false);
                if (s.stages)
                    return s;
            }
    if (cols <= 256)
        return {1, kRowThreads, true, 0, 0, 0};
    // a chunk a thread, the shortest way through a row, up to the 8192 values
    // that 1024 threads then hold
    const int nv = cols > 8192 ? 2 : 1;
    return {nv, (cols + 256 * nv - 1) / (256 * nv) * 32, false, 0, 0, 0};
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
            return s.nv == 1   ? f(t, w, integral_constant<int, 1>(), std::true_type())
                   : s.nv == 2 ? f(t, w, integral_constant<int, 2>(), std::true_type())
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

} // namespace
} // namespace dsa
