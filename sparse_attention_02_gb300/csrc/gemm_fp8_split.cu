// Product of FP8 operands with a scale for every 128 values along the summed axis,
// on sm_103a, for few rows of `a` (the tokens of a decode step).
//
//     out[m, n] = sum_p sa[m, p] sb[n, p] sum_{k in piece p} a[m, k] b[n, k]
//
// A piece's sum is a tensor-core product (kind::f8f6f4, E4M3 products summed in
// fp32); scaled by sa sb, in fp32, it is added to the running sum in registers, as
// the next piece's product runs.
//
// With few rows of `a` the bytes of `b` bound: rows of b (weights) are the MMA's 128
// rows and rows of a its BT columns, so that a tile of weights is read once and few
// tokens leave no part of it idle but the columns up to 16.  K is split over the
// CTAs of a cluster, each of which takes whole pieces; their sums meet through
// distributed shared memory, added in the CTAs' order: results repeat bit for bit.
//
// Measured: 1 x 704 x 4096 4.1 us (launch, a load's latency, four pieces and the meeting; 2.9 MB),
// 1 x 24576 x 1536 9.6 (58 % of measured HBM), 1 x 8192 x 8192 14.8 (67 %),
// 32 x 4096 x 7168 10.4 (44 %).
//
// Roles per CTA (8 warps): 0 loads, 1 MMAs, 2 column scales, 4-7 scaling and sums
// (a thread holds one row of b and all BT columns).
#include "gemm_fp8.cuh"

#include <atomic>
#include <stdio.h>

namespace dsa {
namespace {

constexpr int kRows = 128;              // rows of b per CTA
constexpr int kThreads = 256;
constexpr int kSumWarps = 4;
constexpr int kBatch = 8;               // pieces whose column scales are fetched at once
constexpr int kRowBytes = kRows * kGemmPiece;

template <int BT> struct Cfg {
    static constexpr int kStage = kRowBytes + BT * kGemmPiece;
    // two CTAs an SM
    static constexpr int kStages = BT <= 16 ? 6 : BT <= 32 ? 5 : 4;
    static constexpr int kScales = kStages * kStage;            // two batches of [kBatch][BT] fp32
    static constexpr int kBars = kScales + 2 * kBatch * BT * 4;
    static constexpr int kBuffers = 4;                           // of BT columns of TMEM
    static constexpr int kNumBars = 2 * kStages + 2 * kBuffers + 5;
    static constexpr int kMisc = kBars + 8 * kNumBars;
    static constexpr int kSmem = kMisc + 16;
    static constexpr int kTmemCols = kBuffers * BT;
    static_assert(BT * kRows * 4 <= kScales, "the split's sums take the stages' place");
};

struct Params {
    const float *a_scale, *b_scale;
    int M, N, pieces;
    bool b_block, o32;
    void *out;
    int64_t ldo;
    unsigned *status;
};

__device__ __forceinline__ void put(const Params &p, int64_t m, int64_t n, float v)
{
    if (p.o32)
        static_cast<float *>(p.out)[m * p.ldo + n] = v;
    else
        static_cast<__nv_bfloat16 *>(p.out)[m * p.ldo + n] = __float2bfloat16_rn(v);
}

// The sums of what the `split` (at most 8) CTAs of a cluster have in four words of their shared memory, in the CTAs' order,
// with all loads in flight at once (one word after the other, a tile's sums took 15 us).
__device__ __forceinline__ float4 sums_of_cluster(uint32_t addr, uint32_t split)
{
    float4 v[8];
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k)
        if (k < split)
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(v[k].x), "=f"(v[k].y), "=f"(v[k].z), "=f"(v[k].w)
                         : "r"(mapa_shared(addr, k))
                         : "memory");
#pragma unroll
    for (uint32_t k = 1; k < 8; ++k)
        if (k < split)
            v[0] = make_float4(v[0].x + v[k].x, v[0].y + v[k].y, v[0].z + v[k].z, v[0].w + v[k].w);
    return v[0];
}

template <int BT>
__global__ void __launch_bounds__(kThreads, 2)
    gemm_fp8_split_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, Params p)
{
    using C = Cfg<BT>;
    extern __shared__ __align__(1024) uint8_t smem[]; // the swizzle's period
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) { return sbase + C::kBars + 8u * i; };
    constexpr int B_FULL = 0, B_EMPTY = C::kStages, B_TF = 2 * C::kStages, B_TE = B_TF + C::kBuffers, B_SF = B_TE + C::kBuffers,
                  B_SE = B_SF + 2, B_DONE = B_SE + 2;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + C::kMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kMisc + 4);
    float *scales = reinterpret_cast<float *>(smem + C::kScales);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank(), split = cluster_nctarank();
    const int n0 = (int)(blockIdx.x / split) * kRows; // all rows of a: they are BT at most
    // this CTA's pieces
    const int k0 = (int)((int64_t)p.pieces * rank / split), k1 = (int)((int64_t)p.pieces * (rank + 1) / split);

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(bar(B_FULL + i), 1);
            mbar_init(bar(B_EMPTY + i), 1);
        }
        for (int i = 0; i < C::kBuffers; ++i) {
            mbar_init(bar(B_TF + i), 1);
            mbar_init(bar(B_TE + i), kSumWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_SF + i), 32);
            mbar_init(bar(B_SE + i), kSumWarps);
        }
        mbar_init(bar(B_DONE), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1)
        tmem_alloc(sbase + C::kMisc, C::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    grid_dep_wait(); // no global memory before this
    grid_dep_launch();

    float *part = reinterpret_cast<float *>(smem); // [BT][kRows]: a CTA's sums, over the stages once they are done with

    if (warp == 0) {
        // ------------------------------------------------------------ loads
        bool ok = true;
        for (int k = k0, i = 0; ok && k < k1; ++k, ++i) {
            const int st = i % C::kStages, use = i / C::kStages;
            if (use > 0 && !wait_warp(bar(B_EMPTY + st), (use - 1) & 1, abort_flag, p.status)) {
                ok = false;
                break;
            }
            if (elect_one()) {
                mbar_arrive_expect_tx(bar(B_FULL + st), C::kStage);
                tma_load_2d(sbase + st * C::kStage, &tm_b, bar(B_FULL + st), k * kGemmPiece, n0);
                tma_load_2d(sbase + st * C::kStage + kRowBytes, &tm_a, bar(B_FULL + st), k * kGemmPiece, 0);
            }
            __syncwarp();
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------- MMAs
        // one plain loop, nothing carried but its count: the MMAs' operands come from uniform registers
        if (elect_one()) {
            constexpr uint32_t idesc = idesc_f32acc(128, BT, 0u, false, false);
            const int total = k1 - k0;
            for (int i = 0; i < total; ++i) {
                const int st = i % C::kStages, t = i % C::kBuffers;
                if (!mbar_wait(bar(B_FULL + st), (i / C::kStages) & 1, abort_flag, p.status) ||
                    (i >= C::kBuffers && !mbar_wait(bar(B_TE + t), (i / C::kBuffers - 1) & 1, abort_flag, p.status)))
                    break;
                tc_fence_after();
                const uint64_t bd = sdesc(sbase + st * C::kStage, 16, 1024, 2), ad = sdesc(sbase + st * C::kStage + kRowBytes, 16, 1024, 2);
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    umma_f8f6f4(tmem + t * BT, bd + 2 * s, ad + 2 * s, idesc, s > 0);
                umma_commit(bar(B_TF + t));
                umma_commit(bar(B_EMPTY + st));
            }
            umma_commit(bar(B_DONE));
            mbar_drain(bar(B_DONE), 0);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ---------------------------------------------------- column scales
        // Eight lanes along the pieces, four columns at a time.  A block's one
        // scale of b goes in here, a scale for each row of b does not.
        const int kk = lane & 7;
        bool ok = true;
        for (int k = k0, i = 0; ok && k < k1; k += kBatch, ++i) {
            const int buf = i & 1;
            const bool in = k + kk < k1;
            const float sb = p.b_block && in ? p.b_scale[(int64_t)(n0 / kRows) * p.pieces + k + kk] : 1.f;
            float v[BT / 4];
#pragma unroll
            for (int j = 0; j < BT / 4; ++j) {
                const int m = 4 * j + (lane >> 3);
                v[j] = in && m < p.M ? p.a_scale[(int64_t)m * p.pieces + k + kk] * sb : 0.f;
            }
            if (i >= 2 && !wait_warp(bar(B_SE + buf), ((i >> 1) - 1) & 1, abort_flag, p.status)) {
                ok = false;
                break;
            }
#pragma unroll
            for (int j = 0; j < BT / 4; ++j)
                scales[(buf * kBatch + kk) * BT + 4 * j + (lane >> 3)] = v[j];
            mbar_arrive(bar(B_SF + buf));
        }
    } else if (warp >= 4) {
        // --------------------------------------------------- scaled sums
        const int quad = warp & 3, row = n0 + 32 * quad + lane;
        const uint32_t from = tmem + ((uint32_t)(32 * quad) << 16);
        const bool scaled = !p.b_block && row < p.N;
        const float *sb = p.b_scale + (int64_t)row * p.pieces;
        float next = scaled && k0 < k1 ? sb[k0] : 1.f;
        constexpr int W = BT < 32 ? BT : 32;
        F2 acc[BT / 2];
#pragma unroll
        for (int c = 0; c < BT / 2; ++c)
            acc[c] = F2(0.f);
        bool ok = true;
        for (int k = k0, i = 0; ok && k < k1; ++k, ++i) {
            const int t = i % C::kBuffers, batch = i / kBatch, buf = batch & 1;
            const F2 mine(next);
            next = scaled && k + 1 < k1 ? sb[k + 1] : 1.f;
            if ((i % kBatch == 0 && !wait_warp(bar(B_SF + buf), (batch >> 1) & 1, abort_flag, p.status)) ||
                !wait_warp(bar(B_TF + t), (i / C::kBuffers) & 1, abort_flag, p.status)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const float4 *cs = reinterpret_cast<const float4 *>(scales + (buf * kBatch + i % kBatch) * BT);
            auto add = [&](const uint32_t(&v)[W], int c) {
#pragma unroll
                for (int e = 0; e < W; e += 4) {
                    const float4 s = cs[(c + e) / 4];
                    const F2 v0(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), v1(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
                    F2 s0(s.x, s.y), s1(s.z, s.w);
                    if (!p.b_block) {
                        s0 = s0 * mine;
                        s1 = s1 * mine;
                    }
                    acc[(c + e) / 2] = fma2(v0, s0, acc[(c + e) / 2]);
                    acc[(c + e) / 2 + 1] = fma2(v1, s1, acc[(c + e) / 2 + 1]);
                }
            };
#pragma unroll
            for (int c = 0; c < BT; c += W) {
                uint32_t v[W];
                tmem_load(from + t * BT + c, v);
                tmem_ld_wait_for(v);
                if (c + W == BT) { // read: the buffer may take another product
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar(B_TE + t));
                }
                add(v, c);
            }
            __syncwarp();
            if (lane == 0 && i % kBatch == kBatch - 1)
                mbar_arrive(bar(B_SE + buf));
        }
        // every product is done, as the last one is.  Lanes hold consecutive columns of out.
#pragma unroll
        for (int c = 0; c < BT / 2; ++c) {
            float v[2];
            acc[c].get(v[0], v[1]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (split > 1)
                    part[(2 * c + e) * kRows + 32 * quad + lane] = v[e];
                else if (row < p.N && 2 * c + e < p.M)
                    put(p, 2 * c + e, row, v[e]);
            }
        }
    }
    __syncwarp();
    if (*abort_flag) { // copies may be in flight: a millisecond is far longer than any takes
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) {
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
    if (split == 1)
        return;
    cluster_sync_all();
    const int r = 4 * lane; // a warp takes a column of the sums, a lane four rows
    for (int t = (int)rank + (int)split * warp; t < p.M; t += split * (kThreads / 32)) {
        const float4 v = sums_of_cluster(sbase + (t * kRows + r) * 4, split);
        const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n0 + r + e < p.N)
                put(p, t, n0 + r + e, f[e]);
    }
    cluster_sync_all(); // no CTA leaves while its peers read its sums
}

template <int BT>
int launch(const GemmFp8Args &a, int split, cudaStream_t stream, char *err, size_t errlen)
{
    using C = Cfg<BT>;
    Params p{a.a_scale, a.b_scale, a.M, a.N, (a.K + kGemmPiece - 1) / kGemmPiece, a.b_block, a.o32, a.out,
             a.ldo, device_status_ptr()};
    if (!p.status) {
        snprintf(err, errlen, "device status word unavailable");
        return DSA_ERR_CUDA;
    }
    const int64_t grid = ((int64_t)a.N + kRows - 1) / kRows * split;
    CUtensorMap ta{}, tb{};
    if (a.K > 0 && (!gemm_fp8_map(&ta, a.a, a.lda, a.M, a.K, BT, err, errlen) ||
                    !gemm_fp8_map(&tb, a.b, a.ldb, a.N, a.K, kRows, err, errlen)))
        return DSA_ERR_CUDA;
    static std::atomic<bool> raised[64];
    cudaError_t e = raise_smem_limit_once(gemm_fp8_split_kernel<BT>, C::kSmem, raised);
    if (e == cudaSuccess)
        e = launch_pdl(gemm_fp8_split_kernel<BT>, dim3((unsigned)grid), dim3(kThreads), C::kSmem, stream, split, ta, tb, p);
    if (e != cudaSuccess) {
        snprintf(err, errlen, "gemm_fp8 launch: %s", cudaGetErrorString(e));
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

} // namespace

int launch_gemm_fp8_split(const GemmFp8Args &a, int cols, int split, cudaStream_t stream, char *err, size_t errlen)
{
    return cols <= 16   ? launch<16>(a, split, stream, err, errlen)
           : cols <= 32 ? launch<32>(a, split, stream, err, errlen)
                        : launch<64>(a, split, stream, err, errlen);
}

} // namespace dsa
