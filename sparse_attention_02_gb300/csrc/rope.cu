// Position rotation on the way into the caches and the attention, on sm_103a:
// appending tokens to the paged caches, preparing the queries, and the
// backward of the index rotation.
//
// The two rotations differ in which columns form a pair (release summary
// "DeepSeek-V3.2-Exp: Boosting Long-Context Efficiency with DeepSeek Sparse
// Attention", section "Key claims": the indexer's RoPE is non-interleaved, the
// MLA's interleaved).  With angle t_i = pos * inv_freq[i], i < 32:
//     main   (64 columns)         pairs (2i, 2i + 1)
//     index  (first 64 of 128)    pairs (i, i + 32)
//     (a, b) -> (a cos t - b sin t, a sin t + b cos t)
// The index vector then becomes E4M3 codes with one scale per token, as
// dsa_quantize_fp8, from the fp32 rotated values (no rounding in between).
//
// Angles.  pos * inv_freq in fp32 is off by up to pos * 2^-24 radians (0.008 at
// 131072).  Here inv_freq / (2 pi) becomes a 64-bit fixed-point fraction of a
// turn, once per lane; pos times it modulo 2^64 is then the angle's fraction of
// a turn with nothing rounded, and only that fraction is taken to fp32 for sine
// and cosine.  The same product in fp64 cost five fp64 operations an angle, on
// a GPU with 1/64 of its fp32 rate.
//
// All three kernels move each byte once.  The queries and the index rotation's
// backward are HBM-bound, the append by load latency and issue, and a decode step
// of any by launch and load latency.
#include "common.cuh"
#include "f32x2.cuh"
#include "fp8.cuh"
#include "launch.h"

#include <stdio.h>

namespace dsa {
namespace {

constexpr int kLatent = 576, kValue = 512, kIndex = 128;

// A frequency (radians per position) as a 2^-64 fraction of a turn per position.
__device__ __forceinline__ uint64_t turn_step(double freq)
{
    double f = freq * 0.15915494309189533577; // 1 / (2 pi)
    f -= floor(f);
    return (uint64_t)(f * 18446744073709551616.0);
}

// (cos, sin) at position pos >= 0.
__device__ __forceinline__ float2 rotation(int pos, uint64_t step)
{
    const uint64_t p = step * (uint32_t)pos + 0x80000000u;
    const float half_turns = (float)(int32_t)(p >> 32) * 4.656612873077393e-10f; // 2^-31
    float2 r;
    sincospif(half_turns, &r.y, &r.x);
    return r;
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
}

__device__ __forceinline__ void unpack_pairs(const uint4 &v, F2 (&f)[4])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = F2(bf16_lo(w[i]), bf16_hi(w[i]));
}

__device__ __forceinline__ uint4 pack_pairs(const F2 (&f)[4])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        f[i].get(lo, hi);
        w[i] = bf16_pair(lo, hi);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Largest magnitude in the warp.
__device__ __forceinline__ float warp_amax(float m)
{
    float r;
    asm volatile("redux.sync.max.abs.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(m));
    return r;
}

// ------------------------------------------------------------- cache append
// One warp per token.  Lane l holds latent chunks l and l + 32 (8 columns each),
// the rotated pair (2l, 2l + 1), the index pair (l, l + 32) and the index columns
// 64 + 2l and 65 + 2l: it computes the one angle that both its pairs turn by, and
// no lane needs another's.  One wave of warps, each with its next token's row in
// registers; the norm in pairs of fp32, the page size as a shift, quotients by
// reciprocals.  32768 tokens with norm and both caches: 17.2 us, its bytes at 76 % of
// measured HBM's rate, though they come out of L2 (DRAM at 33 %, 64 % of issue slots,
// loads the top stall); 65536 31.2, 131072 59.7, so a token more takes what its bytes
// would from HBM (93 %) and the rest is 3.5 us of filling and draining.  With rotated chunks of 8 columns
// and angles handed around, instructions bounded it: 22 us.  Pages looked up a
// token ahead, more or fewer warps: no faster.
constexpr int kAppendThreads = 128;

// What a token's warp reads of it: nothing depends on where it goes, so it is
// loaded while the position and page are looked up, and one token ahead.
template <typename K> struct TokenRow {
    uint4 v0, v1;
    uint32_t vr;
    float k[4];
    __device__ __forceinline__ void load(const CacheAppendArgs &a, int t, int lane)
    {
        if (a.kv) {
            const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.kv) + t * a.ld_kv;
            v0 = reinterpret_cast<const uint4 *>(src)[lane];
            v1 = reinterpret_cast<const uint4 *>(src)[lane + 32];
            vr = reinterpret_cast<const uint32_t *>(src + kValue)[lane];
        }
        if (a.kI) {
            const K *src = static_cast<const K *>(a.kI) + t * a.ld_kI;
            k[0] = (float)src[lane];
            k[1] = (float)src[lane + 32];
            if (sizeof(K) == 4) {
                const float2 f = reinterpret_cast<const float2 *>(src + 64)[lane];
                k[2] = f.x, k[3] = f.y;
            } else {
                const uint32_t f = reinterpret_cast<const uint32_t *>(src + 64)[lane];
                k[2] = bf16_lo(f), k[3] = bf16_hi(f);
            }
        }
    }
};

template <typename K, bool W32>
__global__ void __launch_bounds__(kAppendThreads, 8) cache_append_kernel(CacheAppendArgs a, int page_bits, unsigned *status)
{
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    const int step = gridDim.x * (kAppendThreads / 32);
    int t = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    if (t >= a.T)
        return;
    TokenRow<K> next;
    next.load(a, t, lane);
    int next_pos = a.pos[t], next_seq = a.seq ? a.seq[t] : t;
    const uint64_t freq = turn_step(a.inv_freq[lane]);
    for (; t < a.T; t += step) {
        const TokenRow<K> row = next;
        const int pos = next_pos, s = next_seq;
        if (t < a.T - step) {
            next.load(a, t + step, lane);
            next_pos = a.pos[t + step];
            next_seq = a.seq ? a.seq[t + step] : t + step;
        }
        if (pos < 0) // a padded row
            continue;
        const int lp = pos >> page_bits;
        if (s < 0 || s >= a.num_seqs || lp >= a.max_pages) {
            if (lane == 0)
                atomicOr(status, DSA_DEV_BAD_POSITION);
            continue;
        }
        const int page = a.block_table[(int64_t)s * a.max_pages + lp];
        const float2 turn = rotation(pos, freq);
        if (page < 0 || page >= a.num_pages) {
            if (lane == 0)
                atomicOr(status, DSA_DEV_BAD_PAGE);
            continue;
        }
        const int64_t slot = ((int64_t)page << page_bits) + (pos & ((1 << page_bits) - 1));
        if (a.kv) {
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.kv_pool) + slot * kLatent;
            uint4 *dst = reinterpret_cast<uint4 *>(out);
            uint4 v0 = row.v0, v1 = row.v1;
            if (a.kv_weight) {
                F2 f0[4], f1[4], w0[4], w1[4], sq(0.f);
                unpack_pairs(v0, f0);
                unpack_pairs(v1, f1);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sq = fma2(f0[i], f0[i], fma2(f1[i], f1[i], sq));
                float ss = sq.sum();
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float r = rsqrtf(ss * (1.f / kValue) + a.eps);
                if (W32) {
                    const float *w = static_cast<const float *>(a.kv_weight) + 8 * lane;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        w0[i] = F2(w[2 * i], w[2 * i + 1]);
                        w1[i] = F2(w[256 + 2 * i], w[256 + 2 * i + 1]);
                    }
                } else {
                    const uint4 *w = static_cast<const uint4 *>(a.kv_weight) + lane;
                    unpack_pairs(w[0], w0);
                    unpack_pairs(w[32], w1);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f0[i] = f0[i] * F2(r) * w0[i];
                    f1[i] = f1[i] * F2(r) * w1[i];
                }
                v0 = pack_pairs(f0);
                v1 = pack_pairs(f1);
            }
            dst[lane] = v0;
            dst[lane + 32] = v1;
            const float x = bf16_lo(row.vr), y = bf16_hi(row.vr);
            reinterpret_cast<uint32_t *>(out + kValue)[lane] =
                bf16_pair(x * turn.x - y * turn.y, x * turn.y + y * turn.x);
        }
        if (a.kI) {
            const float k0 = row.k[0] * turn.x - row.k[1] * turn.y, k1 = row.k[0] * turn.y + row.k[1] * turn.x;
            float m = fmaxf(fmaxf(fabsf(k0), fabsf(k1)), fmaxf(fabsf(row.k[2]), fabsf(row.k[3])));
            m = warp_amax(m);
            const float sc = fp8_scale(m, a.scale_mode);
            const uint32_t c = e4m3x4(ScaleDivider(sc), k0, k1, row.k[2], row.k[3]);
            uint8_t *codes = a.k8_pool + slot * kIndex;
            codes[lane] = (uint8_t)c;
            codes[lane + 32] = (uint8_t)(c >> 8);
            reinterpret_cast<uint16_t *>(codes + 64)[lane] = (uint16_t)(c >> 16);
            if (lane == 0)
                a.ks_pool[slot] = sc;
        }
    }
}

// ------------------------------------------------------------------ queries
// A CTA per token.  Everything a thread reads, of both parts, is in flight
// before the token's position and angles are there.  Main part: eight threads a
// head, 32 or 16 heads at a time.  Index part: four threads a head, thread r of them
// with the chunks (8 columns) r and r + 4, which turn into each other, r + 8 and
// r + 12; no value passes between threads but the token's amax.  HBM-bound: 37.2
// us for 4096 tokens of 128 and 64 heads, 93 % of measured bandwidth; CTAs of one
// part each 40.2 (the index part alone keeps too few bytes in flight), persistent
// ones with the next token in registers 40.5, pairs of chunks four lanes apart
// turned by shuffles 42.9.  Up to a token per SM each part has a CTA of its own:
// 2.5 us instead of 2.8 for 64 tokens, 2.8 and 2.9 for 152, 3.8 and 3.6 for 304.
// THREADS: 256, or 128 where that many do for the heads of either part (four chunks
// a thread at most): 4096 tokens of 64 and 32 heads 17.1 us, 23.5 with half of 256 idle.

// Turns chunks a and b (columns 8 r ... and 32 + 8 r ...) into each other by the angles 8 r ... of cs; sign -1: back.
__device__ __forceinline__ void turn_chunks(float (&a)[8], float (&b)[8], const float2 *cs, int r, float sign)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 t = cs[8 * r + i];
        const float sn = sign * t.y, x = a[i], y = b[i];
        a[i] = x * t.x - y * sn;
        b[i] = x * sn + y * t.x;
    }
}

template <typename K> struct IndexRow { // a thread's part of a token's index queries, as loaded
    static constexpr int kWords = sizeof(K) == 4 ? 8 : 4;
    uint4 v[kWords];
    __device__ __forceinline__ void load(const K *src) // the thread's first chunk
    {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < kWords / 4; ++k)
                v[kWords / 4 * j + k] = reinterpret_cast<const uint4 *>(src + 32 * j)[k];
    }
    __device__ __forceinline__ void get(int j, float (&f)[8]) const
    {
        if (sizeof(K) == 4) {
            const uint4 x = v[kWords / 4 * j], y = v[kWords / 4 * j + kWords / 4 - 1];
            const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = __uint_as_float(w[i]);
        } else {
            unpack8(v[j], f);
        }
    }
};

template <typename K, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) rope_queries_kernel(RopeQueriesArgs a, bool split)
{
    __shared__ __align__(16) float2 cs[32];
    __shared__ float red[THREADS / 32];
    grid_dep_wait();
    grid_dep_launch();
    const int t = split ? blockIdx.x >> 1 : blockIdx.x, tid = threadIdx.x;
    const bool main_part = a.q_rope && (!split || (blockIdx.x & 1)), index_part = a.qI && (!split || !(blockIdx.x & 1));
    const int pos = a.pos[t];
    const double freq = a.inv_freq[tid & 31];
    // main: eight threads a head, as many heads at a time as there are eights
    constexpr int kMost = 4, kHeads = THREADS / 8;
    const int h0 = tid >> 3, p = tid & 7;
    uint4 v[kMost];
    if (main_part) {
        const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.q_rope) + t * a.st_t + 8 * p;
#pragma unroll
        for (int j = 0; j < kMost; ++j)
            if (h0 + j * kHeads < a.H)
                v[j] = *reinterpret_cast<const uint4 *>(src + (h0 + j * kHeads) * a.st_h);
    }
    // index: four threads a head
    const int h = tid >> 2, r = tid & 3;
    const int64_t at = ((int64_t)t * a.HI + h) * kIndex + 8 * r;
    const bool mine = index_part && h < a.HI;
    IndexRow<K> row = {};
    if (mine)
        row.load(static_cast<const K *>(a.qI) + at);
    if (pos < 0) // a padded row
        return;
    if (tid < 32)
        cs[tid] = rotation(pos, turn_step(freq));
    __syncthreads();
    if (main_part) {
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.q) + (int64_t)t * a.H * kLatent + kValue + 8 * p;
        float2 turn[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            turn[i] = cs[4 * p + i];
#pragma unroll
        for (int j = 0; j < kMost; ++j) {
            if (h0 + j * kHeads >= a.H)
                continue;
            float x[8], o[8];
            unpack8(v[j], x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o[2 * i] = x[2 * i] * turn[i].x - x[2 * i + 1] * turn[i].y;
                o[2 * i + 1] = x[2 * i] * turn[i].y + x[2 * i + 1] * turn[i].x;
            }
            *reinterpret_cast<uint4 *>(dst + (int64_t)(h0 + j * kHeads) * kLatent) = pack8(o);
        }
    }
    if (!index_part)
        return;
    float f[4][8];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        row.get(j, f[j]);
    turn_chunks(f[0], f[1], cs, r, 1.f);
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = fmaxf(m, fabsf(f[j][i]));
    m = warp_amax(m);
    if ((tid & 31) == 0)
        red[tid >> 5] = m;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int w = 1; w < THREADS / 32; ++w)
        m = fmaxf(m, red[w]);
    const float sc = fp8_scale(m, a.scale_mode);
    const ScaleDivider div(sc);
    if (tid == 0)
        a.q_scale[t] = sc;
    if (!mine)
        return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t lo = e4m3x4(div, f[j][0], f[j][1], f[j][2], f[j][3]);
        const uint32_t hi = e4m3x4(div, f[j][4], f[j][5], f[j][6], f[j][7]);
        *reinterpret_cast<uint2 *>(a.q8 + at + 32 * j) = make_uint2(lo, hi);
    }
}

// ------------------------------------------------- backward of the rotation
// dx = R(pos)^T g per index vector, four threads each as above.  Each CTA takes
// kBackVecs consecutive vectors, of one token to kBackVecs (keys, one vector a
// token), and first computes the angles of the tokens it meets, 32 each.  HBM-bound:
// 30.2 us for 4096 tokens of 64 heads to bf16, 98 % of measured bandwidth (64 vectors
// a CTA the same, 128 32.6; 16-byte loads of pairs turned by shuffles 36.3).
constexpr int kBackVecs = 32, kBackThreads = 4 * kBackVecs;

// 8 values; wide: p is a multiple of 32 bytes.
__device__ __forceinline__ void load8(const float *p, float (&f)[8], bool wide)
{
    if (wide) {
        asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
                     : "l"(p));
    } else {
        const float4 u = reinterpret_cast<const float4 *>(p)[0], v = reinterpret_cast<const float4 *>(p)[1];
        f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w, f[4] = v.x, f[5] = v.y, f[6] = v.z, f[7] = v.w;
    }
}

template <typename O>
__global__ void __launch_bounds__(kBackThreads) index_rope_backward_kernel(IndexRopeBackwardArgs a)
{
    __shared__ __align__(16) float2 cs[kBackVecs][32];
    __shared__ bool padded[kBackVecs];
    grid_dep_wait();
    grid_dep_launch();
    const int64_t v0 = (int64_t)blockIdx.x * kBackVecs, vecs = (int64_t)a.T * a.HI;
    const int64_t vlast = (v0 + kBackVecs < vecs ? v0 + kBackVecs : vecs) - 1;
    const int t0 = (int)(v0 / a.HI), ntok = (int)(vlast / a.HI) - t0 + 1;
    const int64_t v = v0 + (threadIdx.x >> 2);
    const int r = threadIdx.x & 3;
    const bool mine = v < vecs;
    float f[4][8];
    if (mine) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            load8(a.g + v * kIndex + 32 * j + 8 * r, f[j], a.wide);
    }
    const uint64_t step = turn_step(a.inv_freq[threadIdx.x & 31]);
    for (int t = threadIdx.x >> 5; t < ntok; t += kBackThreads / 32) {
        const int pos = a.pos[t0 + t];
        cs[t][threadIdx.x & 31] = rotation(pos, step);
        if ((threadIdx.x & 31) == 0)
            padded[t] = pos < 0;
    }
    __syncthreads();
    if (!mine)
        return;
    const int t = (int)(v / a.HI) - t0;
    turn_chunks(f[0], f[1], cs[t], r, -1.f);
    const bool zero = padded[t];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (zero)
            for (int i = 0; i < 8; ++i)
                f[j][i] = 0.f;
        const int64_t c = v * kIndex + 32 * j + 8 * r;
        if (sizeof(O) == 4) {
            float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.dx) + c);
            o[0] = make_float4(f[j][0], f[j][1], f[j][2], f[j][3]);
            o[1] = make_float4(f[j][4], f[j][5], f[j][6], f[j][7]);
        } else {
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.dx) + c) = pack8(f[j]);
        }
    }
}

int finish(cudaError_t e, const char *what, char *err, size_t errlen)
{
    if (e == cudaSuccess)
        return DSA_OK;
    snprintf(err, errlen, "%s launch: %s", what, cudaGetErrorString(e));
    return DSA_ERR_CUDA;
}

} // namespace

int launch_cache_append(const CacheAppendArgs &a, cudaStream_t stream, char *err, size_t errlen)
{
    unsigned *status = device_status_ptr();
    if (!status) {
        snprintf(err, errlen, "device status word unavailable");
        return DSA_ERR_CUDA;
    }
    const int per = kAppendThreads / 32;
    const int want = (a.T + per - 1) / per, most = 8 * num_sms(); // one wave
    const int page_bits = a.page_size == 32 ? 5 : a.page_size == 64 ? 6 : 7;
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3((unsigned)(want < most ? want : most)), dim3(kAppendThreads), 0, stream, 1, a, page_bits, status);
    };
    cudaError_t e;
    if (a.k32)
        e = a.w32 ? go(cache_append_kernel<float, true>) : go(cache_append_kernel<float, false>);
    else
        e = a.w32 ? go(cache_append_kernel<__nv_bfloat16, true>) : go(cache_append_kernel<__nv_bfloat16, false>);
    return finish(e, "cache append", err, errlen);
}

int launch_rope_queries(const RopeQueriesArgs &a, cudaStream_t stream, char *err, size_t errlen)
{
    const bool split = a.q_rope && a.qI && a.T <= num_sms();
    const bool few = (!a.q_rope || a.H <= 64) && (!a.qI || a.HI <= 32);
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3((unsigned)a.T * (split ? 2 : 1)), dim3(few ? 128 : 256), 0, stream, 1, a, split);
    };
    cudaError_t e;
    if (a.i32)
        e = few ? go(rope_queries_kernel<float, 128>) : go(rope_queries_kernel<float, 256>);
    else
        e = few ? go(rope_queries_kernel<__nv_bfloat16, 128>) : go(rope_queries_kernel<__nv_bfloat16, 256>);
    return finish(e, "query rotation", err, errlen);
}

int launch_index_rope_backward(const IndexRopeBackwardArgs &a, cudaStream_t stream, char *err, size_t errlen)
{
    const unsigned grid = (unsigned)(((int64_t)a.T * a.HI + kBackVecs - 1) / kBackVecs);
    IndexRopeBackwardArgs b = a;
    b.wide = (reinterpret_cast<uintptr_t>(a.g) & 31) == 0;
    auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(grid), dim3(kBackThreads), 0, stream, 1, b); };
    return finish(a.o32 ? go(index_rope_backward_kernel<float>) : go(index_rope_backward_kernel<__nv_bfloat16>),
                  "index rotation backward", err, errlen);
}

} // namespace dsa
