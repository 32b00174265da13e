// The product of FP8 operands with a scale for every 128 values along the summed
// axis on sm_103a, where there are enough rows on both sides to fill the GPU with
// whole tiles (the formula stands in gemm_fp8_split.cu).
//
// A CTA's tile is 128 rows of a by BN of b.  A piece of 128 values along K is one stage of
// shared memory and four MMAs, whose sums stay in TMEM (2 buffers of 256 or 192 columns, 4 of 128)
// only until warps have read them, scaled them and added them to running sums in their registers:
// a thread holds 128 columns (BN = 256) or 64 of one row, one multiply-add each, in pairs, or
// a product more where b has a scale for every row.
//
// Bounds.  A piece of 128 x 256 takes the tensor pipe 512 cycles and the FP32 pipe 256.  What a step
// of the loop takes is longer: 840 cycles a piece.  A buffer's way round is MMAs (512 and 150 until the sums
// are seen), 128 columns read in two halves, as 64 are what a thread's registers hold beside its sums, and 200
// until the next MMAs go out, and two buffers (all of TMEM) share that.  A warp of sums in turn waits, reads,
// waits and adds, piece by piece: with BN = 128, whose four buffers hide the way round, a piece still takes 660
// cycles for 256 of the tensor pipe.  Which of the two holds BN = 256 is not measured apart.  BN = 192 has
// registers for all of a piece at once, but more pieces, and takes the product with a scale for every row of
// b.  Those scales
// are read by quads of lanes, each of which holds pairs of columns of four rows: 20 words a thread and piece
// instead of 64 (lanes of one row each, 4096 x 4096 over 8191: 198 us, 178 so; without the product of the two
// scales 144; with scales by blocks 129).
//
// Measured: 8191 x 8192 x 8192 bf16 461 to 474 us call after call, where power limits the
// clock (by what the codes are: evenly spread ones 440), 396 to 417 in bursts, 2.7 PFLOP/s
// (143 % of measured BF16).  Of 417, the same loop takes 375 without the additions and 390
// without the loads.  Not kept: pairs of CTAs on one
// tile (cta_group::2, 256 x 256: 468, words between CTAs in the way round; in halves of 128
// columns with four buffers 655: more meetings), 16 warps of 64 columns (500, registers
// spill), the first columns of the next piece asked for among the additions (486: the
// reading waits), scales fetched by each warp for itself (610, spills), 16 loads of a scale
// warp's lanes in flight for 8 (597, spills).
//
// Roles per CTA (12 or 16 warps): 0 loads, 1 MMAs, 2 and 3 scales, the others scaling, sums and output.
// Persistent where a tile is a CTA's own: CTA c takes tiles c, c + CTAs, ..., ordered so that those
// under way at one time share rows of a and of b in L2.  With few tiles the CTAs of a cluster
// share one, a part of K each, and add up their sums in the CTAs' order.
#include "gemm_fp8.cuh"

#include <atomic>
#include <stdio.h>

namespace dsa {
namespace {

constexpr int kSumWarp0 = 4;
constexpr int kGroup = 8;   // tiles along M that neighbouring tiles are taken from
constexpr int kPatch = 32 * 64; // 64 bytes of each of a warp's rows of out, on their way there
constexpr int kRows = 128;  // of a
constexpr int kABytes = kRows * kGemmPiece;

template <int BN, bool ROWS> struct Cfg {
    static constexpr int kCols = BN == 256 ? 128 : 64;   // that a warp of sums takes, of 32 rows
    static constexpr int kSumWarps = 4 * BN / kCols;
    static constexpr int kThreads = 32 * (kSumWarp0 + kSumWarps);
    static constexpr int kBuffers = BN == 128 ? 4 : 2; // of BN columns of TMEM
    // Where sums fill them, the threads' registers are not shared evenly: of 168 a thread at launch 72 and 216 (BN = 256),
    // of 128 56 and 152 (192).
    static constexpr bool kShares = BN > 128;
    static constexpr int kAuxRegs = BN == 256 ? 72 : 56, kSumRegs = BN == 256 ? 216 : 152;
    static constexpr int kStage = kABytes + BN * kGemmPiece;
    static constexpr int kStages = BN == 128 ? 5 : 4;
    static constexpr int kBatch = 8;                               // pieces whose scales are fetched at once
    static constexpr int kScaled = kRows + (ROWS ? BN : 4);        // scales of a piece: a's, then b's
    static constexpr int kPatches = kStages * kStage;
    static constexpr int kScales = kPatches + kSumWarps * kPatch;  // two batches
    static constexpr int kBars = (kScales + 2 * kBatch * kScaled * 4 + 7) / 8 * 8;
    static constexpr int kNumBars = 2 * kStages + 2 * kBuffers + 5;
    static constexpr int kMisc = kBars + 8 * kNumBars;
    static constexpr int kSmem = kMisc + 16;
    static_assert(BN == 256 || (BN + BN / 2 + 1) * kRows * 4 <= kBars, "a split's sums, and what the CTA adds up, take the stages' place");
    static_assert(kSmem <= 232448, "dynamic shared memory above the 227 KB a CTA may hold");
};

struct Params {
    const float *a_scale, *b_scale;
    int M, N, pieces, tiles_m, tiles_n;
    bool o32;
    bool wide; // rows of out start at 16 bytes
    void *out;
    int64_t ldo;
    unsigned *status;
};

__device__ __forceinline__ void tile_at(const Params &p, int tile, int &m, int &n)
{
    const int per = kGroup * p.tiles_n, g = tile / per, first = g * kGroup;
    const int rows = p.tiles_m - first < kGroup ? p.tiles_m - first : kGroup, r = tile - g * per;
    n = r / rows;
    m = first + r - n * rows;
}

// Sums of a warp's 32 rows to out, from row m (of the first) and column n on: 32 columns as bf16 or 16 as fp32, by way of
// shared memory, where a row's four 16-byte words stand at place ^ (row / 2) so that neither side meets bank conflicts.
// Eight rows then leave at a time; straight from the registers, where a lane holds a row, a tile took 5000 cycles.
// QUADS: lanes hold pairs of columns of four rows (tmem_ld_quads), else a row each.
template <bool O32, bool QUADS>
__device__ __forceinline__ void store_sums(const Params &p, int64_t m, int n, const F2 *acc, uint8_t *patch)
{
    const int lane = threadIdx.x & 31;
    constexpr int e = O32 ? 4 : 2, cols = 64 / e;
    __syncwarp();
    if constexpr (QUADS) {
#pragma unroll
        for (int j = 0; j < cols / 8; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = 8 * k + (lane >> 2), byte = (8 * j + 2 * (lane & 3)) * e;
                uint8_t *to = patch + r * 64 + ((byte >> 4 ^ (r >> 1 & 3)) << 4) + (byte & 15);
                float lo, hi;
                acc[4 * j + k].get(lo, hi);
                if (O32)
                    *reinterpret_cast<float2 *>(to) = make_float2(lo, hi);
                else
                    *reinterpret_cast<uint32_t *>(to) = pack2(lo, hi);
            }
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float lo, hi;
                acc[O32 ? 2 * c + (k >> 1) : 4 * c + k].get(lo, hi);
                w[k] = !O32 ? pack2(lo, hi) : __float_as_uint(k & 1 ? hi : lo);
            }
            *reinterpret_cast<uint4 *>(patch + lane * 64 + ((c ^ (lane >> 1 & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    __syncwarp();
    uint8_t *out = static_cast<uint8_t *>(p.out) + (m * p.ldo + n) * e;
    if (p.wide && p.N - n >= cols) {
#pragma unroll
        for (int r = lane >> 2; r < 32; r += 8)
            if (m + r < p.M)
                *reinterpret_cast<uint4 *>(out + r * p.ldo * e + 16 * (lane & 3)) =
                    *reinterpret_cast<const uint4 *>(patch + r * 64 + (((lane & 3) ^ (r >> 1 & 3)) << 4));
        return;
    }
    const int c = lane % cols;
    if (n + c >= p.N)
        return;
#pragma unroll 4
    for (int r = lane / cols; r < 32; r += 32 / cols)
        if (m + r < p.M) {
            const uint8_t *at = patch + r * 64 + ((c * e / 16 ^ (r >> 1 & 3)) << 4) + c * e % 16;
            if (O32)
                *reinterpret_cast<uint32_t *>(out + (r * p.ldo + c) * e) = *reinterpret_cast<const uint32_t *>(at);
            else
                *reinterpret_cast<uint16_t *>(out + (r * p.ldo + c) * e) = *reinterpret_cast<const uint16_t *>(at);
        }
}

// 64 columns of 16 rows from TMEM, as quads of lanes hold them: lane l gets columns 8 j + 2 (l % 4) and the next of rows l / 4
// (v[4 j], v[4 j + 1]) and l / 4 + 8 (v[4 j + 2], v[4 j + 3]).
__device__ __forceinline__ void tmem_ld_quads(uint32_t at, uint32_t (&v)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x8.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
                   "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
                   "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
                   "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
                 : "r"(at));
}

// What the SPLIT CTAs of a cluster have in four words of their shared memory, with all loads in flight at once, and
// its sum in the CTAs' order.
template <int SPLIT> __device__ __forceinline__ void words_of_cluster(uint32_t addr, float4 (&v)[SPLIT])
{
#pragma unroll
    for (uint32_t k = 0; k < SPLIT; ++k)
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v[k].x), "=f"(v[k].y), "=f"(v[k].z), "=f"(v[k].w)
                     : "r"(mapa_shared(addr, k))
                     : "memory");
}

template <int SPLIT> __device__ __forceinline__ float4 sum_of(const float4 (&v)[SPLIT])
{
    float4 t = v[0];
#pragma unroll
    for (int k = 1; k < SPLIT; ++k)
        t = make_float4(t.x + v[k].x, t.y + v[k].y, t.z + v[k].z, t.w + v[k].w);
    return t;
}

// The CTAs of a cluster add up the columns of their tile between them, each sum in the CTAs' order: lanes along rows, as the
// sums lie, turned in this CTA's own shared memory into lanes along columns, as they leave.  The warps of sums do it: the
// others have given their registers away.
template <int BN, int SPLIT, int THREADS>
__device__ __forceinline__ void join(const Params &p, uint8_t *smem, int tm, int tn, uint32_t rank)
{
    constexpr int cols = BN / SPLIT, pitch = cols + 1, words = cols * kRows, A = 8 / SPLIT; // A: words of a thread in flight
    const uint32_t mine = smem_u32(smem) + 4 * words * rank;
    const int thread = threadIdx.x - 32 * kSumWarp0;
    float *turned = reinterpret_cast<float *>(smem) + BN * kRows;
    for (int x0 = 4 * thread; x0 < words; x0 += 4 * THREADS * A) {
        float4 v[A][SPLIT];
#pragma unroll
        for (int i = 0; i < A; ++i)
            if (x0 + 4 * THREADS * i < words)
                words_of_cluster(mine + 4 * (x0 + 4 * THREADS * i), v[i]);
#pragma unroll
        for (int i = 0; i < A; ++i) {
            const int x = x0 + 4 * THREADS * i;
            if (x < words) {
                const float4 t = sum_of(v[i]);
                float *to = turned + x % kRows * pitch + x / kRows;
                to[0] = t.x, to[pitch] = t.y, to[2 * pitch] = t.z, to[3 * pitch] = t.w;
            }
        }
    }
    named_bar_sync(1, THREADS);
    for (int x = thread; x < words; x += THREADS) {
        const int64_t m = (int64_t)tm * kRows + x / cols, n = (int64_t)tn * BN + cols * (int)rank + x % cols;
        const float v = turned[x / cols * pitch + x % cols];
        if (m < p.M && n < p.N) {
            if (p.o32)
                static_cast<float *>(p.out)[m * p.ldo + n] = v;
            else
                static_cast<__nv_bfloat16 *>(p.out)[m * p.ldo + n] = __float2bfloat16_rn(v);
        }
    }
}

template <int BN, bool ROWS>
__global__ void __launch_bounds__(Cfg<BN, ROWS>::kThreads, 1)
    gemm_fp8_tile_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, Params p)
{
    using C = Cfg<BN, ROWS>;
    extern __shared__ __align__(1024) uint8_t smem[]; // the swizzle's period
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) { return sbase + C::kBars + 8u * i; };
    constexpr int B_FULL = 0, B_EMPTY = C::kStages, B_TF = 2 * C::kStages, B_TE = B_TF + C::kBuffers,
                  B_SF = B_TE + C::kBuffers, B_SE = B_SF + 2, B_DONE = B_SE + 2;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + C::kMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kMisc + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // The CTAs of a cluster share a tile and take a part of its pieces each.
    const uint32_t rank = cluster_ctarank(), split = cluster_nctarank();
    const int tiles = p.tiles_m * p.tiles_n, first = blockIdx.x / split, step = gridDim.x / split;
    const int k0 = (int)((int64_t)p.pieces * rank / split), pieces = (int)((int64_t)p.pieces * (rank + 1) / split) - k0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(bar(B_FULL + i), 1);
            mbar_init(bar(B_EMPTY + i), 1);
        }
        for (int i = 0; i < C::kBuffers; ++i) {
            mbar_init(bar(B_TF + i), 1);
            mbar_init(bar(B_TE + i), C::kSumWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_SF + i), 64);
            mbar_init(bar(B_SE + i), C::kSumWarps);
        }
        mbar_init(bar(B_DONE), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1)
        tmem_alloc(sbase + C::kMisc, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    grid_dep_wait(); // no global memory before this
    grid_dep_launch();

    // each side takes its share of the registers in its own branch: what both run has to fit the smaller
    if (warp < kSumWarp0) {
        if constexpr (C::kShares)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kAuxRegs));
        if (warp == 0) {
            // -------------------------------------------------------- loads
            int st = 0, phase = 0;
            bool ok = true, again = false; // again: every stage was filled once
            for (int tile = first; ok && tile < tiles; tile += step) {
                int tm, tn;
                tile_at(p, tile, tm, tn);
                for (int k = 0; k < pieces; ++k) {
                    if (again && !wait_warp(bar(B_EMPTY + st), phase ^ 1, abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        mbar_arrive_expect_tx(bar(B_FULL + st), C::kStage);
                        tma_load_2d(sbase + st * C::kStage, &tm_a, bar(B_FULL + st), (k0 + k) * kGemmPiece, tm * kRows);
                        tma_load_2d(sbase + st * C::kStage + kABytes, &tm_b, bar(B_FULL + st), (k0 + k) * kGemmPiece, tn * BN);
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
            // --------------------------------------------------------- MMAs
            // One thread, one loop, and nothing carried from turn to turn but its count: the MMAs' operands then come from
            // uniform registers.  With stage and phase carried, or waits by the whole warp, four MMAs and two commits took
            // 300 cycles to issue where this takes 50.
            if (elect_one()) {
                constexpr uint32_t idesc = idesc_f32acc(kRows, BN, 0u, false, false);
                const int total = first < tiles ? ((tiles - 1 - first) / step + 1) * pieces : 0;
                for (int i = 0; i < total; ++i) {
                    const int st = i % C::kStages, t = i % C::kBuffers;
                    if (!mbar_wait(bar(B_FULL + st), (i / C::kStages) & 1, abort_flag, p.status) ||
                        (i >= C::kBuffers && !mbar_wait(bar(B_TE + t), (i / C::kBuffers - 1) & 1, abort_flag, p.status)))
                        break;
                    tc_fence_after();
                    const uint64_t ad = sdesc(sbase + st * C::kStage, 16, 1024, 2), bd = sdesc(sbase + st * C::kStage + kABytes, 16, 1024, 2);
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        umma_f8f6f4(tmem + t * BN, ad + 2 * s, bd + 2 * s, idesc, s > 0);
                    umma_commit(bar(B_TF + t));
                    umma_commit(bar(B_EMPTY + st));
                }
                umma_commit(bar(B_DONE));
                mbar_drain(bar(B_DONE), 0);
            }
            __syncwarp();
        } else {
            // ------------------------------------------------------- scales
            // Batches of this CTA's pieces, counted through its tiles: kBatch lanes along the pieces, 32 / kBatch rows at
            // a time; the two warps take half of the rows each.
            constexpr int R = 32 / C::kBatch;
            const int kk = lane % C::kBatch, r0 = lane / C::kBatch, half = warp - 2;
            const int total = first < tiles ? ((tiles - 1 - first) / step + 1) * pieces : 0;
            for (int i = 0; i < total; i += C::kBatch) {
                const int n = i / C::kBatch, buf = n & 1, mine = i + kk < total ? i + kk : total - 1, nth = mine / pieces;
                const int k = k0 + mine - nth * pieces;
                int tm, tn;
                tile_at(p, first + nth * step, tm, tn);
                if (n >= 2 && !wait_warp(bar(B_SE + buf), ((n >> 1) - 1) & 1, abort_flag, p.status))
                    break;
                float *to = reinterpret_cast<float *>(smem + C::kScales) + (buf * C::kBatch + kk) * C::kScaled;
                auto fetch = [&](const float *from, int row, int rows, float *dst, int count) {
                    from += (int64_t)row * p.pieces + k;
                    const int left = rows - row < count ? rows - row : count;
#pragma unroll 1
                    for (int j = r0; j < count; j += 8 * R) {
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            v[e] = j + R * e < left ? from[(int64_t)(j + R * e) * p.pieces] : 0.f;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (j + R * e < count)
                                dst[j + R * e] = v[e];
                    }
                };
                fetch(p.a_scale, tm * kRows + kRows / 2 * half, p.M, to + kRows / 2 * half, kRows / 2);
                if (ROWS)
                    fetch(p.b_scale, tn * BN + BN / 2 * half, p.N, to + kRows + BN / 2 * half, BN / 2);
                else if (half == 0)
                    fetch(p.b_scale, tn * BN / 128, (p.N + 127) / 128, to + kRows, 2);
                mbar_arrive(bar(B_SF + buf));
            }
        }
    } else {
        // --------------------------------------------------- scaled sums
        // Warp: 32 rows (its TMEM lanes) and W columns, 64 of which are in flight from TMEM at a time.  The last are read
        // before they are added: the next product in their buffer does not wait for that.
        if constexpr (C::kShares)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSumRegs));
        constexpr int W = C::kCols;
        const int quad = warp & 3, part = (warp - kSumWarp0) >> 2;
        const uint32_t from = tmem + ((uint32_t)(32 * quad) << 16) + W * part;
        const float *sc = reinterpret_cast<const float *>(smem + C::kScales);
        uint8_t *patch = smem + C::kPatches + (warp - kSumWarp0) * kPatch;
        uint32_t i = 0;
        bool ok = true;
        for (int tile = first; ok && tile < tiles; tile += step) {
            int block = kRows + W * part / 128; // where in a piece's scales that of these columns of b is
            if constexpr (BN == 192 && !ROWS) {
                int tm, tn;
                tile_at(p, tile, tm, tn);
                block = kRows + ((tn * BN + W * part) >> 7) - (tn * BN >> 7);
            }
            F2 acc[W / 2];
#pragma unroll
            for (int c = 0; c < W / 2; ++c)
                acc[c] = F2(0.f);
            for (int k = 0; k < pieces; ++k, ++i) {
                const uint32_t t = i % C::kBuffers, n = i / C::kBatch;
                if (i % C::kBatch == 0 && !wait_warp(bar(B_SF + (n & 1)), (n >> 1) & 1, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                const float *slot = sc + i % (2 * C::kBatch) * C::kScaled;
                const F2 whole(ROWS ? 0.f : slot[32 * quad + lane] * slot[block]); // ahead of the wait (after it 433 us for 415)
                if (!wait_warp(bar(B_TF + t), (i / C::kBuffers) & 1, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                auto read = [&] { // the buffer may take another product
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar(B_TE + t));
                };
                uint32_t v0[32], v1[32];
                if constexpr (ROWS) {
                    tmem_ld_quads(from + t * BN, v0);
                    tmem_ld_quads(from + (16u << 16) + t * BN, v1);
                    F2 mine[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        mine[r] = F2(slot[32 * quad + 8 * r + (lane >> 2)]);
                    const float2 *cs = reinterpret_cast<const float2 *>(slot + kRows + W * part + 2 * (lane & 3));
                    tmem_ld_wait_for(v0);
                    tmem_ld_wait_for(v1);
                    read();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 s = cs[4 * j];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const uint32_t *v = (r < 2 ? v0 : v1) + 4 * j + 2 * (r & 1);
                            acc[4 * j + r] = fma2(F2(__uint_as_float(v[0]), __uint_as_float(v[1])), mine[r] * F2(s.x, s.y), acc[4 * j + r]);
                        }
                    }
                } else {
                    auto add = [&](const uint32_t(&v)[32], int c) {
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            acc[(c + e) / 2] = fma2(F2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), whole, acc[(c + e) / 2]);
                    };
                    tmem_ld32(from + t * BN, v0);
                    tmem_ld32(from + t * BN + 32, v1);
                    tmem_ld_wait_for(v0);
                    tmem_ld_wait_for(v1);
                    if constexpr (W == 128) {
                        add(v0, 0);
                        tmem_ld32(from + t * BN + 64, v0);
                        add(v1, 32);
                        tmem_ld32(from + t * BN + 96, v1);
                        tmem_ld_wait_for(v0);
                        tmem_ld_wait_for(v1);
                    }
                    read();
                    add(v0, W - 64);
                    add(v1, W - 32);
                }
                if (i % C::kBatch == C::kBatch - 1) {
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar(B_SE + (n & 1)));
                }
            }
            if (BN != 256 && split > 1) { // this CTA's sums, over the stages: the last product is done
#pragma unroll
                for (int c = 0; c < W / 2; ++c) {
                    const int col = ROWS ? 8 * (c / 4) + 2 * (lane & 3) : 2 * c, row = ROWS ? 8 * (c & 3) + (lane >> 2) : lane;
                    float v[2];
                    acc[c].get(v[0], v[1]);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        reinterpret_cast<float *>(smem)[(W * part + col + e) * kRows + 32 * quad + row] = v[e];
                }
            } else if (ok) {
                int tm, tn;
                tile_at(p, tile, tm, tn);
                const int64_t row = (int64_t)tm * kRows + 32 * quad;
                const int col = tn * BN + W * part;
                if (p.o32) {
#pragma unroll
                    for (int c = 0; c < W; c += 16)
                        if (col + c < p.N)
                            store_sums<true, ROWS>(p, row, col + c, acc + c / 2, patch);
                } else {
#pragma unroll
                    for (int c = 0; c < W; c += 32)
                        if (col + c < p.N)
                            store_sums<false, ROWS>(p, row, col + c, acc + c / 2, patch);
                }
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
        tmem_dealloc(tmem, 512);
    }
    if (BN == 256 || split == 1) // 256: never split (launch_gemm_fp8)
        return;
    cluster_sync_all();
    int tm, tn;
    tile_at(p, first, tm, tn);
    if (warp >= kSumWarp0) {
        if (split == 2)
            join<BN, 2, 32 * C::kSumWarps>(p, smem, tm, tn, rank);
        else if (split == 4)
            join<BN, 4, 32 * C::kSumWarps>(p, smem, tm, tn, rank);
        else
            join<BN, 8, 32 * C::kSumWarps>(p, smem, tm, tn, rank);
    }
    cluster_sync_all(); // no CTA leaves while its peers read its sums
}

template <int BN, bool ROWS>
int launch(const GemmFp8Args &a, int split, cudaStream_t stream, char *err, size_t errlen)
{
    using C = Cfg<BN, ROWS>;
    const uintptr_t rows = reinterpret_cast<uintptr_t>(a.out) | (uintptr_t)(a.M > 1 ? a.ldo * (a.o32 ? 4 : 2) : 0);
    Params p{a.a_scale, a.b_scale, a.M, a.N, (a.K + kGemmPiece - 1) / kGemmPiece, (a.M + kRows - 1) / kRows, (a.N + BN - 1) / BN, a.o32,
             (rows & 15) == 0, a.out, a.ldo, device_status_ptr()};
    if (!p.status) {
        snprintf(err, errlen, "device status word unavailable");
        return DSA_ERR_CUDA;
    }
    CUtensorMap ta{}, tb{};
    if (a.K > 0 && (!gemm_fp8_map(&ta, a.a, a.lda, a.M, a.K, kRows, err, errlen) ||
                    !gemm_fp8_map(&tb, a.b, a.ldb, a.N, a.K, BN, err, errlen)))
        return DSA_ERR_CUDA;
    static std::atomic<bool> raised[64], fits;
    cudaError_t e = raise_smem_limit_once(gemm_fp8_tile_kernel<BN, ROWS>, C::kSmem, raised);
    if (C::kShares && e == cudaSuccess && !fits.load(std::memory_order_acquire)) {
        // the roles' shares of registers are cut from what the block is launched with
        cudaFuncAttributes f;
        e = cudaFuncGetAttributes(&f, gemm_fp8_tile_kernel<BN, ROWS>);
        if (e == cudaSuccess && f.numRegs * C::kThreads < 32 * (kSumWarp0 * C::kAuxRegs + C::kSumWarps * C::kSumRegs)) {
            snprintf(err, errlen, "gemm_fp8: built with %d registers a thread, too few to share out", f.numRegs);
            return DSA_ERR_UNSUPPORTED;
        }
        fits.store(e == cudaSuccess, std::memory_order_release);
    }
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n, most = num_sms();
    if (e == cudaSuccess)
        e = launch_pdl(gemm_fp8_tile_kernel<BN, ROWS>, dim3((unsigned)(split > 1 ? tiles * split : tiles < most ? tiles : most)),
                       dim3(C::kThreads), C::kSmem, stream, split, ta, tb, p);
    if (e != cudaSuccess) {
        snprintf(err, errlen, "gemm_fp8 launch: %s", cudaGetErrorString(e));
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

} // namespace

int launch_gemm_fp8_tile(const GemmFp8Args &a, int cols, int split, cudaStream_t stream, char *err, size_t errlen)
{
    if (cols == 128)
        return a.b_block ? launch<128, false>(a, split, stream, err, errlen) : launch<128, true>(a, split, stream, err, errlen);
    if (!a.b_block)
        return launch<192, true>(a, split, stream, err, errlen);
    return cols == 192 ? launch<192, false>(a, split, stream, err, errlen) : launch<256, false>(a, split, stream, err, errlen);
}

} // namespace dsa
