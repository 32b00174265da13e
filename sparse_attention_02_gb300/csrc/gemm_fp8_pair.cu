// The product of FP8 operands with a scale for every 128 values along the summed
// axis on sm_103a, where there are enough rows on both sides to fill the GPU with
// whole tiles (the formula stands in gemm_fp8_split.cu).
//
// Two CTAs (two SMs) share a tile of 256 x BN outputs through cta_group::2 MMAs of
// M = 256: CTA r holds rows [128 r, 128 r + 128) of a's tile and of the sums, and
// loads half of b's rows, which both SMs read: at BN = 256 a piece of 128 values
// takes 32 KB of shared memory per SM and 512 cycles of the tensor pipe.
// A piece's sums stay in TMEM (two buffers of BN columns) only until eight warps have
// read them, scaled them and added them to running sums in their registers: 128 fp32
// a thread, one multiply-add each, in pairs, or a product more where b has a scale
// for every row.  That is half of the FP32 pipe's rate (or all of it).
// Persistent: pair c takes tiles c, c + pairs, ..., ordered so that those under way at one
// time share rows of a and of b in L2.
//
// Roles per CTA (12 warps): 0 loads, 1 (of the leader CTA) MMAs, 2 and 3 b's scales where
// it has one for every row, 4-11 scaling, sums and output.
#include "gemm_fp8.cuh"

#include <atomic>
#include <stdio.h>

namespace dsa {
namespace {

constexpr int kThreads = 384;
constexpr int kSumWarp0 = 4, kSumWarps = 8;
constexpr int kBatch = 8;   // pieces whose scales of b's rows are fetched at once
constexpr int kGroup = 8;   // tiles along M that neighbouring tiles are taken from
constexpr int kAuxRegs = 40, kSumRegs = 232;
constexpr int kABytes = 128 * kGemmPiece;

template <int BN, bool ROWS> struct Cfg {
    static constexpr int kStage = kABytes + BN / 2 * kGemmPiece;
    static constexpr int kStages = BN == 256 ? 6 : 8;
    static constexpr int kScales = kStages * kStage; // two batches of [kBatch][BN] fp32
    static constexpr int kBars = kScales + (ROWS ? 2 * kBatch * BN * 4 : 0);
    static constexpr int kNumBars = 2 * kStages + 9;
    static constexpr int kMisc = kBars + 8 * kNumBars;
    static constexpr int kUnread = kMisc + 16; // where the other CTA's words go
    static constexpr int kSmem = kUnread + 4 * kSumWarps;
    static_assert(kSmem <= 232448, "dynamic shared memory above the 227 KB a CTA may hold");
};

struct Params {
    const float *a_scale, *b_scale;
    int M, N, pieces, tiles_m, tiles_n;
    bool o32;
    int wide; // bytes that every row of out starts at a multiple of: 32, 16 or less
    void *out;
    int64_t ldo;
    unsigned *status;
};

__device__ __forceinline__ void load_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t c0, int32_t c1)
{
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
                 "[%4];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void umma_fp8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}

__device__ __forceinline__ void tile_at(const Params &p, int tile, int &m, int &n)
{
    const int per = kGroup * p.tiles_n, g = tile / per, first = g * kGroup;
    const int rows = p.tiles_m - first < kGroup ? p.tiles_m - first : kGroup, r = tile - g * per;
    n = r / rows;
    m = first + r - n * rows;
}

// 32 sums of a row to out, from column n on.
__device__ __forceinline__ void store_sums(const Params &p, int64_t m, int n, const F2 *acc)
{
    const int left = p.N - n;
    float f[32];
#pragma unroll
    for (int i = 0; i < 16; ++i)
        acc[i].get(f[2 * i], f[2 * i + 1]);
    if (p.o32) {
        float *dst = static_cast<float *>(p.out) + m * p.ldo + n;
        if (left >= 32 && p.wide >= 16) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t w[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    w[k] = __float_as_uint(f[8 * e + k]);
                if (p.wide == 32) {
                    store32(dst + 8 * e, w);
                } else {
                    reinterpret_cast<uint4 *>(dst)[2 * e] = make_uint4(w[0], w[1], w[2], w[3]);
                    reinterpret_cast<uint4 *>(dst)[2 * e + 1] = make_uint4(w[4], w[5], w[6], w[7]);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i < left)
                    dst[i] = f[i];
        }
        return;
    }
    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + m * p.ldo + n;
    if (left >= 32 && p.wide >= 16) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                w[k] = pack2(f[16 * e + 2 * k], f[16 * e + 2 * k + 1]);
            if (p.wide == 32) {
                store32(dst + 16 * e, w);
            } else {
                reinterpret_cast<uint4 *>(dst)[2 * e] = make_uint4(w[0], w[1], w[2], w[3]);
                reinterpret_cast<uint4 *>(dst)[2 * e + 1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < left)
                dst[i] = __float2bfloat16_rn(f[i]);
    }
}

template <int BN, bool ROWS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gemm_fp8_pair_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, Params p)
{
    using C = Cfg<BN, ROWS>;
    extern __shared__ __align__(1024) uint8_t smem[]; // the swizzle's period
    const uint32_t sbase = smem_u32(smem), bar0 = sbase + C::kBars;
    auto bar = [&](int i) { return bar0 + 8u * i; };
    // FULL and TE are used in the leader CTA only; both CTAs' roles arrive there
    constexpr int B_FULL = 0, B_EMPTY = C::kStages, B_TF = 2 * C::kStages, B_TE = B_TF + 2, B_SF = B_TF + 4, B_SE = B_TF + 6,
                  B_DONE = B_TF + 8;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + C::kMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kMisc + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1, tiles = p.tiles_m * p.tiles_n;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(bar(B_FULL + i), 1);
            mbar_init(bar(B_EMPTY + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_TF + i), 1);
            mbar_init(bar(B_TE + i), kSumWarps);
            mbar_init(bar(B_SF + i), 64);
            mbar_init(bar(B_SE + i), kSumWarps);
        }
        mbar_init(bar(B_DONE), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1)
        tmem_alloc_pair(sbase + C::kMisc, 2 * BN);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all(); // the other CTA's barriers exist
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const uint32_t lead0 = mapa_shared(bar0, 0);
    auto lead = [&](int i) { return lead0 + 8u * i; };
    grid_dep_wait(); // no global memory before this
    grid_dep_launch();

    // each side takes its share of the registers in its own branch: what both run has to fit the smaller
    if (warp < kSumWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAuxRegs));
        if (warp == 0) {
            // ------------------------------------------------------------ loads
            int st = 0, phase = 0;
            bool ok = true, again = false; // again: every stage was filled once
            for (int tile = pair; ok && tile < tiles; tile += pairs) {
                int tm, tn;
                tile_at(p, tile, tm, tn);
                const int ra = tm * 256 + 128 * (int)rank, rb = tn * BN + BN / 2 * (int)rank;
                for (int k = 0; k < p.pieces; ++k) {
                    if (again && !mbar_wait_warp<true>(bar(B_EMPTY + st), phase ^ 1, abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        if (rank == 0)
                            mbar_arrive_expect_tx(bar(B_FULL + st), 2 * C::kStage);
                        load_pair(sbase + st * C::kStage, &tm_a, lead(B_FULL + st), k * kGemmPiece, ra);
                        load_pair(sbase + st * C::kStage + kABytes, &tm_b, lead(B_FULL + st), k * kGemmPiece, rb);
                    }
                    __syncwarp();
                    if (++st == C::kStages) {
                        st = 0;
                        phase ^= 1;
                        again = true;
                    }
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------------------- MMAs
            if (elect_one()) {
                if (rank == 0) {
                    constexpr uint32_t idesc = idesc_f32acc(256, BN, 0u, false, false);
                    const uint64_t ad = sdesc(sbase, 16, 1024, 2), bd = sdesc(sbase + kABytes, 16, 1024, 2);
                    uint32_t i = 0;
                    int st = 0, phase = 0;
                    bool ok = true;
                    for (int tile = pair; ok && tile < tiles; tile += pairs)
                        for (int k = 0; k < p.pieces; ++k, ++i) {
                            const uint32_t t = i & 1;
                            ok = (i < 2 || mbar_wait<true>(bar(B_TE + t), ((i >> 1) - 1) & 1, abort_flag, p.status)) &&
                                 mbar_wait<true>(bar(B_FULL + st), phase, abort_flag, p.status);
                            if (!ok)
                                break;
                            tc_fence_after();
                            const uint64_t so = (uint64_t)((st * C::kStage) >> 4);
#pragma unroll
                            for (int s = 0; s < 4; ++s)
                                umma_fp8_pair(tmem + t * BN, ad + so + 2 * s, bd + so + 2 * s, idesc, s > 0);
                            umma_commit_pair(bar(B_TF + t));
                            umma_commit_pair(bar(B_EMPTY + st));
                            if (++st == C::kStages) {
                                st = 0;
                                phase ^= 1;
                            }
                        }
                    // the last words from the other CTA are stores into this one, which must outlive them
                    for (uint32_t j = i < 2 ? 0 : i - 2; ok && j < i; ++j)
                        ok = mbar_wait<true>(bar(B_TE + (j & 1)), (j >> 1) & 1, abort_flag, p.status);
                    umma_commit_pair(bar(B_DONE));
                }
                mbar_drain(bar(B_DONE), 0);
            }
            __syncwarp();
        } else {
            // ------------------------------------------------- scales of b's rows
            // Eight lanes along the pieces, four rows at a time; the two warps take half of the rows each.
            if constexpr (ROWS) {
                float *scales = reinterpret_cast<float *>(smem + C::kScales);
                const int kk = lane & 7, c0 = (warp - 2) * (BN / 2) + (lane >> 3);
                uint32_t i = 0;
                bool ok = true;
                for (int tile = pair; ok && tile < tiles; tile += pairs) {
                    int tm, tn;
                    tile_at(p, tile, tm, tn);
                    for (int k = 0; k < p.pieces; k += kBatch, ++i) {
                        const uint32_t buf = i & 1;
                        if (i >= 2 && !mbar_wait_warp(bar(B_SE + buf), ((i >> 1) - 1) & 1, abort_flag, p.status)) {
                            ok = false;
                            break;
                        }
                        const bool in = k + kk < p.pieces;
#pragma unroll 1
                        for (int j = 0; j < BN / 2; j += 32) {
                            float v[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const int n = tn * BN + c0 + j + 4 * e;
                                v[e] = in && n < p.N ? p.b_scale[(int64_t)n * p.pieces + k + kk] : 0.f;
                            }
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                scales[(buf * kBatch + kk) * BN + c0 + j + 4 * e] = v[e];
                        }
                        mbar_arrive(bar(B_SF + buf));
                    }
                }
            }
        }
    } else {
        // --------------------------------------------------- scaled sums
        // Warp: 32 rows (its TMEM lanes) and half of the columns.
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
        constexpr int W = BN / 2;
        const int quad = warp & 3, half = (warp - kSumWarp0) >> 2;
        const uint32_t from = tmem + ((uint32_t)(32 * quad) << 16) + W * half;
        const uint32_t lead_unread = mapa_shared(sbase + C::kUnread + 4 * (warp - kSumWarp0), 0);
        uint32_t i = 0, batch = 0;
        bool ok = true;
        for (int tile = pair; ok && tile < tiles; tile += pairs) {
            int tm, tn;
            tile_at(p, tile, tm, tn);
            const int64_t row = (int64_t)tm * 256 + 128 * rank + 32 * quad + lane;
            const int col = tn * BN + W * half, block = col >> 7;
            const bool in = row < p.M;
            const float *sa = p.a_scale + row * p.pieces, *sb = p.b_scale + (int64_t)block * p.pieces;
            const bool has_b = !ROWS && col < p.N;
            float na = in && p.pieces > 0 ? sa[0] : 0.f, nb = has_b && p.pieces > 0 ? sb[0] : 1.f;
            F2 acc[W / 2];
#pragma unroll
            for (int c = 0; c < W / 2; ++c)
                acc[c] = F2(0.f);
            for (int k = 0; k < p.pieces; ++k, ++i) {
                const uint32_t t = i & 1;
                const F2 mine(na * nb);
                if (k + 1 < p.pieces) {
                    na = in ? sa[k + 1] : 0.f;
                    nb = has_b ? sb[k + 1] : 1.f;
                }
                if ((ROWS && k % kBatch == 0 && !mbar_wait_warp(bar(B_SF + (batch & 1)), (batch >> 1) & 1, abort_flag, p.status)) ||
                    !mbar_wait_warp<true>(bar(B_TF + t), (i >> 1) & 1, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float4 *cs = reinterpret_cast<const float4 *>(smem + C::kScales) +
                                   ((batch & 1) * kBatch + k % kBatch) * (BN / 4) + half * (W / 4);
                auto add = [&](const uint32_t(&v)[32], int c) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const F2 v0(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), v1(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
                        F2 s0 = mine, s1 = mine;
                        if (ROWS) {
                            const float4 s = cs[(c + e) / 4];
                            s0 = mine * F2(s.x, s.y);
                            s1 = mine * F2(s.z, s.w);
                        }
                        acc[(c + e) / 2] = fma2(v0, s0, acc[(c + e) / 2]);
                        acc[(c + e) / 2 + 1] = fma2(v1, s1, acc[(c + e) / 2 + 1]);
                    }
                };
                uint32_t v[2][32];
                tmem_ld32(from + t * BN, v[0]);
                tmem_ld_wait_for(v[0]);
#pragma unroll
                for (int c = 32; c <= W; c += 32) {
                    if (c < W) {
                        tmem_ld32(from + t * BN + c, v[(c / 32) & 1]);
                    } else { // read: the buffer may take the piece after the next
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            // A release at cluster scope from the CTA that does not lead: a four-byte store carries it.
                            if (rank)
                                st_async_b32(lead_unread, 0u, lead(B_TE + t));
                            else if (warp == kSumWarp0)
                                mbar_arrive_expect_tx(bar(B_TE + t), kSumWarps * 4);
                            else
                                mbar_arrive(bar(B_TE + t));
                        }
                    }
                    add(v[(c / 32 - 1) & 1], c - 32);
                    if (c < W)
                        tmem_ld_wait_for(v[(c / 32) & 1]);
                }
                if (ROWS && (k % kBatch == kBatch - 1 || k == p.pieces - 1)) {
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar(B_SE + (batch & 1)));
                    ++batch;
                }
            }
            if (ok && in)
#pragma unroll
                for (int c = 0; c < W; c += 32)
                    if (col + c < p.N)
                        store_sums(p, row, col + c, acc + c / 2);
        }
    }

    // After a wait that gave up in either CTA, copies may be in flight whose barrier is the other's: a millisecond is
    // far longer than any takes.
    __syncwarp();
    if (*abort_flag) {
        st_cluster_u32(mapa_shared(sbase + C::kMisc + 4, rank ^ 1), 1u);
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) {
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all(); // no CTA leaves while its peer may still touch its shared memory
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 2 * BN);
    }
}

template <int BN, bool ROWS>
int launch(const GemmFp8Args &a, cudaStream_t stream, char *err, size_t errlen)
{
    using C = Cfg<BN, ROWS>;
    const uintptr_t rows = reinterpret_cast<uintptr_t>(a.out) | (uintptr_t)(a.M > 1 ? a.ldo * (a.o32 ? 4 : 2) : 0);
    Params p{a.a_scale, a.b_scale, a.M, a.N, (a.K + kGemmPiece - 1) / kGemmPiece, (a.M + 255) / 256, (a.N + BN - 1) / BN, a.o32,
             (int)(rows & 15 ? 0 : rows & 31 ? 16 : 32), a.out, a.ldo, device_status_ptr()};
    if (!p.status) {
        snprintf(err, errlen, "device status word unavailable");
        return DSA_ERR_CUDA;
    }
    CUtensorMap ta{}, tb{};
    if (a.K > 0 && (!gemm_fp8_map(&ta, a.a, a.lda, a.M, a.K, 128, err, errlen) ||
                    !gemm_fp8_map(&tb, a.b, a.ldb, a.N, a.K, BN / 2, err, errlen)))
        return DSA_ERR_CUDA;
    static std::atomic<bool> raised[64], fits;
    cudaError_t e = raise_smem_limit_once(gemm_fp8_pair_kernel<BN, ROWS>, C::kSmem, raised);
    if (e == cudaSuccess && !fits.load(std::memory_order_acquire)) {
        // the roles' shares of registers are cut from what the block is launched with
        cudaFuncAttributes f;
        e = cudaFuncGetAttributes(&f, gemm_fp8_pair_kernel<BN, ROWS>);
        if (e == cudaSuccess && f.numRegs * kThreads < 32 * (kSumWarp0 * kAuxRegs + kSumWarps * kSumRegs)) {
            snprintf(err, errlen, "gemm_fp8: built with %d registers a thread, too few to share out", f.numRegs);
            return DSA_ERR_UNSUPPORTED;
        }
        fits.store(e == cudaSuccess, std::memory_order_release);
    }
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n, most = num_sms() / 2;
    if (e == cudaSuccess)
        e = launch_pdl(gemm_fp8_pair_kernel<BN, ROWS>, dim3(2 * (unsigned)(tiles < most ? tiles : most)), dim3(kThreads), C::kSmem,
                       stream, 1, ta, tb, p);
    if (e != cudaSuccess) {
        snprintf(err, errlen, "gemm_fp8 launch: %s", cudaGetErrorString(e));
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

} // namespace

int launch_gemm_fp8_pair(const GemmFp8Args &a, int cols, cudaStream_t stream, char *err, size_t errlen)
{
    if (cols <= 128)
        return a.b_block ? launch<128, false>(a, stream, err, errlen) : launch<128, true>(a, stream, err, errlen);
    return a.b_block ? launch<256, false>(a, stream, err, errlen) : launch<256, true>(a, stream, err, errlen);
}

} // namespace dsa
