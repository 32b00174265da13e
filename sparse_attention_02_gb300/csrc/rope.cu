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
// All three kernels move each byte once and are HBM-bound (or, for a decode
// step, bound by launch and load latency).
#include "common.cuh"
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

// ------------------------------------------------------------- cache append
// One warp per token.  Lane l holds latent chunks l and l + 32 (8 columns each),
// the rotated pair (2l, 2l + 1), the index pair (l, l + 32) and the index columns
// 64 + 2l and 65 + 2l: it computes the one angle that both its pairs turn by, and
// no lane needs another's.  Instructions bound this kernel more than bytes (70 %
// of issue slots with rotated chunks of 8 columns and angles handed around: 22 us
// for 32768 tokens, 18 so), so the page size comes as a shift and quotients by
// reciprocals.
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
                float f0[8], f1[8], ss = 0.f, w0[8], w1[8];
                unpack8(v0, f0);
                unpack8(v1, f1);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    ss = fmaf(f0[i], f0[i], fmaf(f1[i], f1[i], ss));
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float r = rsqrtf(ss * (1.f / kValue) + a.eps);
                if (W32) {
                    const float *w = static_cast<const float *>(a.kv_weight) + 8 * lane;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        w0[i] = w[i];
                        w1[i] = w[256 + i];
                    }
                } else {
                    const uint4 *w = static_cast<const uint4 *>(a.kv_weight) + lane;
                    unpack8(w[0], w0);
                    unpack8(w[32], w1);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    f0[i] = f0[i] * r * w0[i];
                    f1[i] = f1[i] * r * w1[i];
                }
                v0 = pack8(f0);
                v1 = pack8(f1);
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
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
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
// A CTA per token for each part that is asked for, the two side by side.
// Everything a thread reads is in flight before the token's position and angles
// are there.  Five CTAs an SM (51 registers a thread): 42.9 us for 4096 tokens of
// 128 and 64 heads, 81 % of measured HBM, 46.0 with four, 48 with all of one part
// first.  Index
// queries: thread t holds chunks t, t + 256, ... of the token's H_I x 128 values
// (8 columns each, 16 chunks a head), its pair's other half 4 lanes away; at
// most 64 heads, so four chunks a thread stay in registers while the token's
// amax is found.
constexpr int kQueryThreads = 256;
constexpr int kIndexChunks = 4;

// Rotates chunk c (0 .. 15) of a 128-wide index vector; other: the 8 values 4
// lanes away.  back turns by the negative angle.
__device__ __forceinline__ void rotate_index(float (&f)[8], int c, const float2 *cs, bool back)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float other = __shfl_xor_sync(0xffffffffu, f[i], 4);
        if (c < 8) {
            const float2 r = cs[8 * (c & 3) + i];
            const float sn = ((c < 4) != back) ? -r.y : r.y;
            f[i] = f[i] * r.x + other * sn;
        }
    }
}

template <typename K>
__device__ __forceinline__ void load8(const K *p, float (&f)[8])
{
    if (sizeof(K) == 4) {
        const float4 u = reinterpret_cast<const float4 *>(p)[0], v = reinterpret_cast<const float4 *>(p)[1];
        f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w, f[4] = v.x, f[5] = v.y, f[6] = v.z, f[7] = v.w;
    } else {
        unpack8(*reinterpret_cast<const uint4 *>(p), f);
    }
}

template <typename K>
__global__ void __launch_bounds__(kQueryThreads, 5) rope_queries_kernel(RopeQueriesArgs a)
{
    __shared__ float2 cs[32];
    __shared__ float red[kQueryThreads / 32];
    grid_dep_wait();
    grid_dep_launch();
    const bool both = a.q_rope && a.qI;
    const int t = both ? blockIdx.x >> 1 : blockIdx.x, tid = threadIdx.x;
    if (both ? blockIdx.x & 1 : a.q_rope != nullptr) {
        const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.q_rope) + t * a.st_t;
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.q) + (int64_t)t * a.H * kLatent + kValue;
        constexpr int kMost = 128 * 8 / kQueryThreads; // chunks of a thread
        const int h0 = tid >> 3, p = tid & 7;
        uint4 v[kMost];
#pragma unroll
        for (int j = 0; j < kMost; ++j)
            if (h0 + j * (kQueryThreads / 8) < a.H)
                v[j] = *reinterpret_cast<const uint4 *>(src + (h0 + j * (kQueryThreads / 8)) * a.st_h + 8 * p);
        const int pos = a.pos[t];
        if (pos < 0) // a padded row
            return;
        if (tid < 32)
            cs[tid] = rotation(pos, turn_step(a.inv_freq[tid]));
        __syncthreads();
        float2 r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = cs[4 * p + i];
#pragma unroll
        for (int j = 0; j < kMost; ++j) {
            const int h = h0 + j * (kQueryThreads / 8);
            if (h >= a.H)
                continue;
            float x[8], o[8];
            unpack8(v[j], x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o[2 * i] = x[2 * i] * r[i].x - x[2 * i + 1] * r[i].y;
                o[2 * i + 1] = x[2 * i] * r[i].y + x[2 * i + 1] * r[i].x;
            }
            *reinterpret_cast<uint4 *>(dst + (int64_t)h * kLatent + 8 * p) = pack8(o);
        }
        return;
    }
    float f[kIndexChunks][8];
    const int chunks = a.HI * 16;
#pragma unroll
    for (int j = 0; j < kIndexChunks; ++j) {
        const int c = j * kQueryThreads + tid;
        if (c < chunks)
            load8(static_cast<const K *>(a.qI) + ((int64_t)t * chunks + c) * 8, f[j]);
        else
            for (int i = 0; i < 8; ++i)
                f[j][i] = 0.f;
    }
    const int pos = a.pos[t];
    if (pos < 0)
        return;
    if (tid < 32)
        cs[tid] = rotation(pos, turn_step(a.inv_freq[tid]));
    __syncthreads();
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < kIndexChunks; ++j) {
        rotate_index(f[j], tid & 15, cs, false);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = fmaxf(m, fabsf(f[j][i]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((tid & 31) == 0)
        red[tid >> 5] = m;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int w = 1; w < kQueryThreads / 32; ++w)
        m = fmaxf(m, red[w]);
    const float sc = fp8_scale(m, a.scale_mode);
    const ScaleDivider div(sc);
    if (tid == 0)
        a.q_scale[t] = sc;
#pragma unroll
    for (int j = 0; j < kIndexChunks; ++j) {
        const int c = j * kQueryThreads + tid;
        if (c >= chunks)
            continue;
        const uint32_t lo = e4m3x4(div, f[j][0], f[j][1], f[j][2], f[j][3]);
        const uint32_t hi = e4m3x4(div, f[j][4], f[j][5], f[j][6], f[j][7]);
        reinterpret_cast<uint2 *>(a.q8)[(int64_t)t * chunks + c] = make_uint2(lo, hi);
    }
}

// ------------------------------------------------- backward of the rotation
// dx = R(pos)^T g per index vector.  Each CTA takes 64 consecutive vectors, of
// one token (64 heads) to 64 (keys, one vector a token), and first computes
// the angles of the tokens it meets, 32 each.
constexpr int kBackVecs = kQueryThreads * kIndexChunks / 16;

template <typename O>
__global__ void __launch_bounds__(kQueryThreads) index_rope_backward_kernel(IndexRopeBackwardArgs a)
{
    __shared__ float2 cs[kBackVecs][32];
    __shared__ bool padded[kBackVecs];
    grid_dep_wait();
    grid_dep_launch();
    const int64_t v0 = (int64_t)blockIdx.x * kBackVecs, vecs = (int64_t)a.T * a.HI;
    const int64_t vlast = (v0 + kBackVecs < vecs ? v0 + kBackVecs : vecs) - 1;
    const int t0 = (int)(v0 / a.HI), ntok = (int)(vlast / a.HI) - t0 + 1;
    float f[kIndexChunks][8];
#pragma unroll
    for (int j = 0; j < kIndexChunks; ++j) {
        const int64_t c = v0 * 16 + j * kQueryThreads + threadIdx.x;
        if (c < vecs * 16)
            load8(a.g + c * 8, f[j]);
        else
            for (int i = 0; i < 8; ++i)
                f[j][i] = 0.f;
    }
    const uint64_t step = turn_step(a.inv_freq[threadIdx.x & 31]);
    for (int t = threadIdx.x >> 5; t < ntok; t += kQueryThreads / 32) {
        const int pos = a.pos[t0 + t];
        cs[t][threadIdx.x & 31] = rotation(pos, step);
        if ((threadIdx.x & 31) == 0)
            padded[t] = pos < 0;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kIndexChunks; ++j) {
        const int64_t c = v0 * 16 + j * kQueryThreads + threadIdx.x;
        const int64_t v = c >> 4 < vecs ? c >> 4 : vecs - 1;
        const int t = (int)(v / a.HI) - t0;
        rotate_index(f[j], threadIdx.x & 15, cs[t], true);
        if (c >= vecs * 16)
            continue;
        if (padded[t])
            for (int i = 0; i < 8; ++i)
                f[j][i] = 0.f;
        if (sizeof(O) == 4) {
            float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.dx) + c * 8);
            o[0] = make_float4(f[j][0], f[j][1], f[j][2], f[j][3]);
            o[1] = make_float4(f[j][4], f[j][5], f[j][6], f[j][7]);
        } else {
            reinterpret_cast<uint4 *>(a.dx)[c] = pack8(f[j]);
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
    auto go = [&](auto kernel) { return launch_pdl(kernel, dim3((unsigned)a.T * (a.q_rope && a.qI ? 2 : 1)), dim3(kQueryThreads), 0, stream, 1, a); };
    return finish(a.i32 ? go(rope_queries_kernel<float>) : go(rope_queries_kernel<__nv_bfloat16>), "query rotation", err, errlen);
}

int launch_index_rope_backward(const IndexRopeBackwardArgs &a, cudaStream_t stream, char *err, size_t errlen)
{
    const unsigned grid = (unsigned)(((int64_t)a.T * a.HI + kBackVecs - 1) / kBackVecs);
    auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(grid), dim3(kQueryThreads), 0, stream, 1, a); };
    return finish(a.o32 ? go(index_rope_backward_kernel<float>) : go(index_rope_backward_kernel<__nv_bfloat16>),
                  "index rotation backward", err, errlen);
}

} // namespace dsa
