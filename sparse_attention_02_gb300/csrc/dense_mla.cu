// Dense MLA attention of single tokens over the paged latent cache on sm_103a.
//
// The attention of layers, steps and contexts that select nothing: MQA mode,
// one 576-wide latent row is the key of every head and its first 512 columns
// the value (release summary "DeepSeek-V3.2-Exp: Boosting Long-Context
// Efficiency with DeepSeek Sparse Attention", section "Method"), over all keys
// s < ctx_len[b]:
//     S[h,s] = sm_scale * <q[b,h,:576], kv[s,:576]>
//     out[b,h] = sum_s softmax_s(S[h,:]) kv[s,:512],  lse = ln sum_s exp S[h,s]
//
// Bounds.  A key is 1152 bytes from HBM and 2 H (576 + 512) operations: with
// 128 heads 0.170 ns of measured HBM and 0.147 ns of measured BF16 peak, so
// neither tensor pipe nor loads may wait for the other, and with fewer heads
// HBM alone bounds.
//
// Two CTAs (two SMs) share each 128-key tile through cta_group::2 MMAs of M =
// 128: CTA r holds heads [64 r, 64 r + 64) as rows of Q, P, S and O, and
//   keys [64 r, 64 r + 64) of the tile as its half of the score MMA's N, so
//   every latent row is loaded by one SM only;
//   value columns [256 r, 256 r + 256) as its half of the PV MMA's N, for which
//   it needs those columns of the peer's 64 keys too.  Shared memory has no
//   room beside two 72 KB stages, but once the scores are done a CTA no longer
//   needs the other half of its own keys' columns: the peer's keys' columns are
//   loaded over them (32 KB a tile, out of L2), so both CTAs end with 128 keys
//   of 256 columns at the same addresses, as the MMA requires.
// Accumulators (2 x 2 data path of M = 128, cta_group::2): TMEM lanes 0-63 hold
// the 64 heads with the first half of N, lanes 64-127 the same heads with the
// second: S 2 x 64 columns (two buffers), O 2 x 128.
//
// Roles per CTA (8 warps):
//   load warp    Q once per row, each tile's own 64 keys (9 atoms of 64 columns,
//                in two groups with barriers of their own), L2 prefetches some
//                tiles ahead (one instruction: a page is contiguous)
//   swap warp    the peer's keys' value columns over this CTA's spent ones
//   MMA warp     (leader CTA only) scores of tile i + 1, then PV of tile i
//   4 softmax    thread = (head, half of the tile's keys): the two threads of a
//   warps        head swap their maxima through shared memory, the running
//                maximum moves only when exceeded by 2^8 (O is then rescaled in
//                TMEM), P goes to shared memory as bf16.  In a row's last tile
//                they also zero the value rows past the end, whose stale bytes
//                might be NaN (0 * NaN).
// P is the one intermediate rounded to 16 bits: kind::f16 wants P in V's type.
// The sum l is that of the unrounded values, in fp32.
//
// Work split.  The rows' tiles laid end to end are cut into one contiguous
// share per CTA pair, computed on the device from ctx_len (the host never sees
// the lengths).  A share that holds part of a row leaves that part, normalised,
// with its LSE in the workspace, and a second kernel joins the parts.
#include "common.cuh"
#include "launch.h"

#include <atomic>
#include <stdio.h>

namespace dsa {
namespace {

constexpr int kD = 576, kDv = 512;
constexpr int kTile = 128;                // keys per tile, 64 per CTA
constexpr int kAtom = 64 * 128;           // 64 rows x 64 bf16 columns, SW128
constexpr int kAtoms = 9;
constexpr int kStage = kAtoms * kAtom;
constexpr int kStages = 2;
constexpr int kThreads = 256;
constexpr int kSoftWarp0 = 4;
constexpr int kBatch = 16;                // tiles whose pages a warp looks up at once (two half-blocks a tile)
constexpr int kPrefetch = 6;              // tiles ahead of the loads that are pulled into L2
constexpr float kRescaleLog2 = 8.f;

// shared memory
constexpr int OFF_Q = 0;
constexpr int OFF_KV = OFF_Q + kStage;
constexpr int OFF_P1 = OFF_KV + kStages * kStage; // P of the tile's second 64 keys (the first's takes the spent RoPE atom)
constexpr int OFF_X = OFF_P1 + kAtom;             // per-thread maxima (two buffers of 128) and sums (128)
constexpr int OFF_BAR = OFF_X + 3 * 128 * 4;
constexpr int NBAR = 30;
constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
constexpr int kSmem = OFF_MISC + 64 + 1024; // with room to start at a multiple of 1024
static_assert(kSmem <= 232448, "dynamic shared memory above the 227 KB a CTA may hold");

// barriers (L: used in the leader CTA only; both CTAs' roles arrive there)
constexpr int B_KF = 0,  // L [stage][group]: both CTAs' atoms 0-3 / 4-8 landed
              B_E = 4,   // [stage][half]: PV of the tile's first / second 64 keys done
              B_SF = 8,  // [buffer]: scores done
              B_SE = 10, // L [buffer]: scores read
              B_QD = 12, // [stage]: the score MMAs over atoms 0-3 done
              B_VL = 14, // [stage]: this CTA's swapped-in columns landed
              B_P0 = 16, // L [buffer]: P of the first 64 keys written and O rescaled
              B_P1 = 18, // L [buffer]: P of the second 64 keys written
              B_OF = 20, // O of a unit complete
              B_OE = 21, // L: O read
              B_QF = 22, // L: Q landed
              B_DONE = 23,
              B_RB = 24, // [pair][parity]: the two warps of 32 heads swapped their maxima
              B_RL = 28; // [pair]: ... their sums

constexpr uint32_t TM_O = 0, TM_S = 256, kTmemCols = 512;

struct Params {
    const __nv_bfloat16 *q;
    const __nv_bfloat16 *pool;
    const int32_t *block_table, *ctx_len;
    int num_pages, page_size, max_pages, B, H, clusters;
    float scale_log2;
    __nv_bfloat16 *out;
    float *lse;
    float *ws_o, *ws_lse; // [2 clusters, H, 512], [2 clusters, H]
    int64_t *row_start;   // [B + 1] first tile of each row
    unsigned *status;
};

__device__ __forceinline__ int context(const Params &p, int row)
{
    const int n = p.ctx_len[row];
    const int most = p.max_pages * p.page_size;
    return n < 0 ? 0 : n < most ? n : most;
}

// Tiles of a row; an empty one counts as one, so that some pair writes it.
__device__ __forceinline__ int tiles_of(int ctx) { return ctx > 0 ? (ctx - 1) / kTile + 1 : 1; }

struct Share {
    int64_t tiles;      // of this cluster
    int row, tile;      // where it starts
};

struct Unit {
    int row, ctx, jb, je; // tiles [jb, je) of the row
    int slot;             // -1: the whole row
};

struct Walk {
    int64_t left;
    int row, tile, first;
    __device__ explicit Walk(const volatile Share &s) : left(s.tiles), row(s.row), tile(s.tile), first(s.row) {}
    __device__ bool next(const Params &p, int cid, Unit &u)
    {
        if (left <= 0)
            return false;
        u.row = row;
        u.ctx = context(p, row);
        const int n = tiles_of(u.ctx);
        u.jb = tile;
        u.je = left < n - tile ? tile + (int)left : n;
        u.slot = u.jb == 0 && u.je == n ? -1 : 2 * cid + (row != first);
        left -= u.je - u.jb;
        ++row;
        tile = 0;
        return true;
    }
};

// Pool row of half-block `half` (32 keys) of key block kb of a tile, or -1 past
// the context, -2 on a bad page.  Pages of 64 keys and more: half 0 stands for
// all 64 keys.
__device__ __forceinline__ int pool_row(const Params &p, const Unit &u, int tile, int kb, int half)
{
    const int64_t key = (int64_t)tile * kTile + 64 * kb + 32 * half;
    if (key >= u.ctx)
        return -1;
    const int page = p.block_table[(int64_t)u.row * p.max_pages + key / p.page_size];
    if (page < 0 || page >= p.num_pages)
        return -2;
    return page * p.page_size + (int)(key % p.page_size);
}

// A warp's look-ahead over a unit's pages: lane 2 i + half holds tile base + i.
struct Pages {
    int cur, nxt, base, kb;
    __device__ void fetch(const Params &p, const Unit &u, int from, int &v) const
    {
        const int lane = threadIdx.x & 31, tile = from + (lane >> 1);
        v = tile < u.je ? pool_row(p, u, tile, kb, p.page_size == 32 ? lane & 1 : 0) : -1;
    }
    __device__ void start(const Params &p, const Unit &u, int block)
    {
        kb = block;
        base = u.jb;
        fetch(p, u, base, cur);
        fetch(p, u, base + kBatch, nxt);
    }
    __device__ void advance(const Params &p, const Unit &u, int tile) // before using tile: moves on when it leaves cur
    {
        if (tile - base >= kBatch) {
            base += kBatch;
            cur = nxt;
            fetch(p, u, base + kBatch, nxt);
        }
    }
    __device__ int get(int tile, int half) const // tile in [base, base + 2 kBatch)
    {
        const int i = tile - base;
        const int a = __shfl_sync(0xffffffffu, cur, (2 * i + half) & 31), b = __shfl_sync(0xffffffffu, nxt, (2 * i + half) & 31);
        return i < kBatch ? a : b;
    }
};

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 2-D tiled load into this CTA's shared memory, completion counted on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t c0, int32_t c1)
{
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
                 "[%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void *p, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

__device__ __forceinline__ void umma_f16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// Arrives on the barrier at this offset in both CTAs once the MMAs issued so far are done.
__device__ __forceinline__ void umma_commit_pair(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     bar),
                 "h"((uint16_t)3)
                 : "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    dense_mla_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv, Params p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + OFF_BAR;
    auto bar = [&](int i) { return bar0 + 8u * i; };
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + OFF_MISC + 4);
    volatile Share *share = reinterpret_cast<volatile Share *>(smem + OFF_MISC + 8);
    float *xs = reinterpret_cast<float *>(smem + OFF_X);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int cid = blockIdx.x >> 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(B_KF + i), 1);
            mbar_init(bar(B_E + i), 1);
            mbar_init(bar(B_RB + i), 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_SF + i), 1);
            mbar_init(bar(B_SE + i), 8);
            mbar_init(bar(B_QD + i), 1);
            mbar_init(bar(B_VL + i), 1);
            mbar_init(bar(B_P0 + i), 8);
            mbar_init(bar(B_P1 + i), 4);
            mbar_init(bar(B_RL + i), 2);
        }
        mbar_init(bar(B_OF), 1);
        mbar_init(bar(B_OE), 8);
        mbar_init(bar(B_QF), 1);
        mbar_init(bar(B_DONE), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1)
        tmem_alloc_pair(sbase + OFF_MISC, kTmemCols);
    grid_dep_wait(); // no global memory before this
    grid_dep_launch();

    // ---- this pair's share of the tiles
    {
        const int per = (p.B + kThreads - 1) / kThreads, r0 = threadIdx.x * per, r1 = r0 + per < p.B ? r0 + per : p.B;
        int64_t mine = 0;
        bool over = false;
        for (int r = r0; r < r1; ++r) {
            over |= p.ctx_len[r] > p.max_pages * p.page_size;
            mine += tiles_of(context(p, r));
        }
        if (over && blockIdx.x == 0)
            atomicOr(p.status, DSA_DEV_BAD_POSITION);
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += v;
        }
        int64_t *sums = reinterpret_cast<int64_t *>(xs);
        if (lane == 31)
            sums[warp] = incl;
        __syncthreads();
        int64_t before = incl - mine, total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp)
                before += sums[w];
            total += sums[w];
        }
        const int64_t g0 = total * cid / p.clusters, g1 = total * (cid + 1) / p.clusters;
        if (threadIdx.x == 0)
            share->tiles = g1 - g0;
        if (g0 >= before && g0 < before + mine) {
            int64_t at = before;
            int r = r0;
            for (;; ++r) {
                const int n = tiles_of(context(p, r));
                if (g0 < at + n)
                    break;
                at += n;
            }
            share->row = r;
            share->tile = (int)(g0 - at);
        }
        if (blockIdx.x == 0) { // for the joining kernel
            int64_t at = before;
            for (int r = r0; r < r1; ++r) {
                p.row_start[r] = at;
                at += tiles_of(context(p, r));
            }
            if (threadIdx.x == 0)
                p.row_start[p.B] = total;
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all(); // both CTAs' barriers exist before any remote operation
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const uint32_t lead0 = mapa_shared(bar0, 0);
    auto lead = [&](int i) { return lead0 + 8u * i; };
    const int oob = p.num_pages * p.page_size; // rows from here on arrive as zeros
    const int boxes = p.page_size == 32 ? 2 : 1, box_bytes = kAtom / boxes;

    if (warp == 0) {
        // ------------------------------------------------------------ loads
        uint32_t i = 0;
        int u = 0;
        bool ok = true;
        Walk it(*share);
        Unit un;
        Pages pg;
        while (ok && it.next(p, cid, un)) {
            if (un.ctx == 0)
                continue;
            pg.start(p, un, rank);
            // Q is free once the previous unit's last score MMAs are done
            if (u > 0 && !mbar_wait_warp(bar(B_SF + ((i - 1) & 1)), ((i - 1) >> 1) & 1, abort_flag, p.status)) {
                ok = false;
                break;
            }
            if (lane == 0) {
                if (rank == 0)
                    mbar_arrive_expect_tx(bar(B_QF), 2 * kStage);
                for (int a = 0; a < kAtoms; ++a)
                    tma_load_2d_pair(sbase + OFF_Q + a * kAtom, &tm_q, lead(B_QF), 64 * a, un.row * p.H + 64 * (int)rank);
            }
            ++u;
            for (int j = un.jb; j < un.je; ++j, ++i) {
                const int st = i & 1;
                pg.advance(p, un, j);
                int r[2] = {pg.get(j, 0), pg.get(j, 1)};
                // prefetch: the unit's first tiles at once, then one a tile
                for (int f = j == un.jb ? j + 1 : j + kPrefetch; f <= j + kPrefetch && f < un.je; ++f) {
                    const int r0 = pg.get(f, 0), r1 = pg.get(f, 1);
                    if (lane == 0 && r0 >= 0)
                        prefetch_l2(p.pool + (int64_t)r0 * kD, kStage / boxes);
                    if (lane == 0 && boxes == 2 && r1 >= 0)
                        prefetch_l2(p.pool + (int64_t)r1 * kD, kStage / 2);
                }
                if (lane == 0 && (r[0] == -2 || (boxes == 2 && r[1] == -2)))
                    atomicOr(p.status, DSA_DEV_BAD_PAGE);
                for (int g = 0; g < 2 && ok; ++g) {
                    if (i >= 2 && !mbar_wait_warp(bar(B_E + 2 * st + g), ((i >> 1) - 1) & 1, abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        const int a0 = g ? 4 : 0, a1 = g ? kAtoms : 4;
                        if (rank == 0)
                            mbar_arrive_expect_tx(bar(B_KF + 2 * st + g), 2 * (a1 - a0) * kAtom);
                        for (int a = a0; a < a1; ++a)
                            for (int b = 0; b < boxes; ++b)
                                tma_load_2d_pair(sbase + OFF_KV + st * kStage + a * kAtom + b * box_bytes, &tm_kv,
                                                 lead(B_KF + 2 * st + g), 64 * a, r[b] >= 0 ? r[b] : oob);
                    }
                    __syncwarp();
                }
                if (!ok)
                    break;
            }
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ swaps
        uint32_t i = 0;
        bool ok = true;
        Walk it(*share);
        Unit un;
        Pages pg;
        const int a0 = rank ? 4 : 0, y0 = rank ? 0 : 4; // columns wanted, atoms spent
        while (ok && it.next(p, cid, un)) {
            if (un.ctx == 0)
                continue;
            pg.start(p, un, rank ^ 1);
            for (int j = un.jb; j < un.je; ++j, ++i) {
                const int st = i & 1;
                pg.advance(p, un, j);
                const int r[2] = {pg.get(j, 0), pg.get(j, 1)};
                // CTA 1 gives up atoms 0-3, done with after the first group of score MMAs; CTA 0 atoms 4-7
                if (!mbar_wait_warp(bar((rank ? B_QD : B_SF) + st), (i >> 1) & 1, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar(B_VL + st), 4 * kAtom);
                    for (int a = 0; a < 4; ++a)
                        for (int b = 0; b < boxes; ++b)
                            tma_load_2d(sbase + OFF_KV + st * kStage + (y0 + a) * kAtom + b * box_bytes, &tm_kv, bar(B_VL + st),
                                        64 * (a0 + a), r[b] >= 0 ? r[b] : oob);
                }
                __syncwarp();
            }
        }
        if (i > 0 && lane == 0)
            mbar_drain(bar(B_VL + ((i - 1) & 1)), ((i - 1) >> 1) & 1);
        __syncwarp();
    } else if (warp == 1 && rank == 0) {
        // ------------------------------------------------------------- MMAs
        constexpr uint32_t idesc_qk = idesc_f32acc(128, 128, 1u, false, false);
        constexpr uint32_t idesc_pv = idesc_f32acc(128, 256, 1u, false, true);
        const uint64_t qd = sdesc(sbase + OFF_Q, 16, 1024, 2), kd = sdesc(sbase + OFF_KV, 16, 1024, 2);
        const uint64_t vd = sdesc(sbase + OFF_KV, kAtom, 1024, 2);
        const uint64_t pd0 = sdesc(sbase + OFF_KV + 8 * kAtom, 16, 1024, 2), pd1 = sdesc(sbase + OFF_P1, 16, 1024, 2);
        uint32_t i = 0;
        int u = 0;
        bool ok = true;
        auto scores = [&](bool first) { // of tile i
            const int st = i & 1;
            const uint64_t so = (uint64_t)((st * kStage) >> 4);
            if ((first && !mbar_wait_warp(bar(B_QF), u & 1, abort_flag, p.status)) ||
                (i >= 2 && !mbar_wait_warp<true>(bar(B_SE + st), ((i >> 1) - 1) & 1, abort_flag, p.status)) ||
                !mbar_wait_warp(bar(B_KF + 2 * st), (i >> 1) & 1, abort_flag, p.status))
                return false;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int s = 0; s < 16; ++s)
                    umma_f16_pair(tmem + TM_S + 64 * st, qd + (((s >> 2) * kAtom + (s & 3) * 32) >> 4),
                                  kd + so + (((s >> 2) * kAtom + (s & 3) * 32) >> 4), idesc_qk, s > 0);
                umma_commit_pair(bar(B_QD + st));
            }
            __syncwarp();
            if (!mbar_wait_warp(bar(B_KF + 2 * st + 1), (i >> 1) & 1, abort_flag, p.status))
                return false;
            if (lane == 0) {
#pragma unroll
                for (int s = 16; s < 36; ++s)
                    umma_f16_pair(tmem + TM_S + 64 * st, qd + (((s >> 2) * kAtom + (s & 3) * 32) >> 4),
                                  kd + so + (((s >> 2) * kAtom + (s & 3) * 32) >> 4), idesc_qk, 1u);
                umma_commit_pair(bar(B_SF + st));
            }
            __syncwarp();
            return true;
        };
        auto values = [&](uint32_t t, bool first, bool last) { // of tile t
            const int st = t & 1;
            const uint64_t so = (uint64_t)((st * kStage) >> 4);
            // a unit's first PV overwrites O: the previous unit's must have been read
            if (first && u > 0 && !mbar_wait_warp<true>(bar(B_OE), (u - 1) & 1, abort_flag, p.status))
                return false;
            for (int kb = 0; kb < 2; ++kb) {
                if (!mbar_wait_warp<true>(bar((kb ? B_P1 : B_P0) + st), (t >> 1) & 1, abort_flag, p.status))
                    return false;
                tc_fence_after();
                if (lane == 0) {
                    const uint64_t pd = kb ? pd1 : pd0 + so;
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            umma_f16_pair(tmem + TM_O + 128 * n, pd + 2 * k,
                                          vd + so + (((4 * kb + 2 * n) * kAtom + 16 * 128 * k) >> 4), idesc_pv,
                                          !(first && kb == 0 && k == 0));
                    umma_commit_pair(bar(B_E + 2 * st + kb));
                    if (kb == 1 && last)
                        umma_commit_pair(bar(B_OF));
                }
                __syncwarp();
            }
            return true;
        };
        Walk it(*share);
        Unit un;
        while (ok && it.next(p, cid, un)) {
            if (un.ctx == 0)
                continue;
            const int n = un.je - un.jb;
            for (int j = 0; j <= n && ok; ++j) {
                if (j < n)
                    ok = scores(j == 0);
                if (ok && j > 0)
                    ok = values(i - 1, j == 1, j == n);
                if (j < n)
                    ++i;
            }
            ++u;
        }
        if (lane == 0) {
            umma_commit_pair(bar(B_DONE));
            mbar_drain(bar(B_DONE), 0);
        }
        __syncwarp();
    } else if (warp >= kSoftWarp0) {
        // ---------------------------------------------------------- softmax
        const int quad = warp & 3, kb = quad >> 1, pair = quad & 1;
        const int t128 = 32 * quad + lane, hl = t128 & 63, h = 64 * (int)rank + hl;
        const uint32_t lane_off = (uint32_t)(32 * quad) << 16;
        const bool swapped = kb != (int)rank; // this CTA's value columns of key block kb are swapped in
        uint32_t i = 0;
        int u = 0;
        bool ok = true;
        Walk it(*share);
        Unit un;
        Pages pg;
        while (ok && it.next(p, cid, un)) {
            float m = -INFINITY, l = 0.f;
            const int64_t orow = (int64_t)un.row * p.H + h, prow = (int64_t)un.slot * p.H + h;
            if (un.ctx == 0) {
                if (h < p.H) {
                    uint4 *dst = reinterpret_cast<uint4 *>(p.out + orow * kDv + 256 * kb);
                    for (int c = 0; c < 32; ++c)
                        dst[c] = make_uint4(0, 0, 0, 0);
                    if (kb == 0)
                        p.lse[orow] = -INFINITY;
                }
                continue;
            }
            pg.start(p, un, kb);
            for (int j = un.jb; j < un.je; ++j, ++i) {
                const int st = i & 1;
                pg.advance(p, un, j);
                const bool bad0 = pg.get(j, 0) < 0, bad1 = boxes == 2 ? pg.get(j, 1) < 0 : bad0;
                const int64_t left = (int64_t)un.ctx - (int64_t)j * kTile - 64 * kb;
                const int valid = left < 0 ? 0 : left < 64 ? (int)left : 64;
                if (!mbar_wait_warp(bar(B_SF + st), (i >> 1) & 1, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t s[2][32];
                tmem_ld32(tmem + lane_off + TM_S + 64 * st, s[0]);
                tmem_ld32(tmem + lane_off + TM_S + 64 * st + 32, s[1]);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_remote(lead(B_SE + st));
                float mx = -INFINITY;
                if (valid < 64 || bad0 || bad1) {
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        if (c >= valid || (c < 32 ? bad0 : bad1))
                            s[c >> 5][c & 31] = 0xFF800000u;
                }
#pragma unroll
                for (int c = 0; c < 64; ++c)
                    mx = fmaxf(mx, __uint_as_float(s[c >> 5][c & 31]));
                mx *= p.scale_log2; // scale > 0; -inf stays
                // the head's other thread
                xs[128 * (i & 1) + t128] = mx;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(B_RB + 2 * pair + (i & 1)));
                if (!mbar_wait_warp(bar(B_RB + 2 * pair + (i & 1)), (i >> 1) & 1, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                mx = fmaxf(mx, xs[128 * (i & 1) + (t128 ^ 64)]);
                const bool first = j == un.jb;
                const bool move = mx > m + kRescaleLog2 || (m == -INFINITY && mx > m);
                const bool rescale = !first && __any_sync(0xffffffffu, move);
                // PV of the previous tile: before O is touched, and before P's second buffer is
                if ((rescale || (kb == 1 && i > 0)) &&
                    !mbar_wait_warp(bar(B_E + 2 * (st ^ 1) + 1), ((i - 1) >> 1) & 1, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                if (rescale) {
                    tc_fence_after();
                    const float f = move ? exp2_fast(m - mx) : 1.f;
                    l *= f;
#pragma unroll 1
                    for (int c = 0; c < 256; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(tmem + lane_off + TM_O + c, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st32(tmem + lane_off + TM_O + c, o);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                }
                if (move)
                    m = mx;
                if (kb == 1) { // O is as the first PV of this tile wants it
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_remote(lead(B_P0 + st));
                }
                const float ms = m == -INFINITY ? 0.f : m;
                uint8_t *prow_s = smem + (kb ? OFF_P1 : OFF_KV + st * kStage + 8 * kAtom) + hl * 128;
                float sum = 0.f;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    float e[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int x = 8 * c + k;
                        e[k] = exp2_fast(fmaf(__uint_as_float(s[x >> 5][x & 31]), p.scale_log2, -ms));
                    }
                    sum += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
                    *reinterpret_cast<uint4 *>(prow_s + ((c ^ (hl & 7)) << 4)) =
                        make_uint4(pack2(e[0], e[1]), pack2(e[2], e[3]), pack2(e[4], e[5]), pack2(e[6], e[7]));
                }
                l += sum;
                if (swapped && !mbar_wait_warp(bar(B_VL + st), (i >> 1) & 1, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                if (valid < 64) { // value rows past the end
                    for (int x = valid * 8 + 32 * pair + lane; x < 64 * 8; x += 64)
#pragma unroll
                        for (int a = 0; a < 4; ++a)
                            *reinterpret_cast<uint4 *>(smem + OFF_KV + st * kStage + (4 * kb + a) * kAtom + x * 16) =
                                make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_remote(lead((kb ? B_P1 : B_P0) + st));
            }
            if (!ok)
                break;
            // ---- the unit's output
            xs[256 + t128] = l;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(B_RL + pair));
            if (!mbar_wait_warp(bar(B_RL + pair), u & 1, abort_flag, p.status) ||
                !mbar_wait_warp(bar(B_OF), u & 1, abort_flag, p.status)) {
                ok = false;
                break;
            }
            ++u;
            l += xs[256 + (t128 ^ 64)];
            const float inv = l > 0.f ? 1.f / l : 0.f;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 256; c += 32) {
                uint32_t o[32];
                tmem_ld32(tmem + lane_off + TM_O + c, o);
                tmem_ld_wait();
                if (h >= p.H)
                    continue;
                // lanes 0-63: columns [0, 256); lanes 64-127: [256, 512)
                if (un.slot < 0) {
                    uint4 *dst = reinterpret_cast<uint4 *>(p.out + orow * kDv + 256 * kb + c);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            w[k] = pack2(__uint_as_float(o[8 * e + 2 * k]) * inv, __uint_as_float(o[8 * e + 2 * k + 1]) * inv);
                        dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(p.ws_o + prow * kDv + 256 * kb + c);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dst[e] = make_float4(__uint_as_float(o[4 * e]) * inv, __uint_as_float(o[4 * e + 1]) * inv,
                                             __uint_as_float(o[4 * e + 2]) * inv, __uint_as_float(o[4 * e + 3]) * inv);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_remote(lead(B_OE));
            if (h < p.H && kb == 0) {
                const float v = l > 0.f ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
                if (un.slot < 0)
                    p.lse[orow] = v;
                else
                    p.ws_lse[prow] = v;
            }
        }
    }

    // After a wait that gave up, copies may be in flight whose barrier is the other CTA's: a millisecond is far longer
    // than any takes.
    __syncwarp();
    if (*abort_flag) {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) {
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all(); // no CTA leaves while its peer may still touch its shared memory
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

// Joins the parts of each split row: a CTA per (row, head), its 8 warps taking
// parts w, w + 8, ... and adding up in order.  O = sum exp(LSE_i - LSE) O_i.
__global__ void __launch_bounds__(256) dense_mla_join_kernel(Params p)
{
    __shared__ float acc_s[8][kDv];
    __shared__ float sum_s[8];
    grid_dep_wait();
    grid_dep_launch();
    const int row = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t total = p.row_start[p.B], a = p.row_start[row], b = p.row_start[row + 1];
    // cluster c holds tiles [floor(total c / C), floor(total (c + 1) / C))
    auto cluster_of = [&](int64_t g) { return (int)(((g + 1) * p.clusters + total - 1) / total - 1); };
    const int c0 = cluster_of(a), c1 = cluster_of(b - 1);
    if (c0 == c1)
        return;
    // the row is its cluster's first unless the cluster began with an earlier one; with fewer tiles than clusters some
    // have none
    auto slot = [&](int c) {
        const int64_t g0 = total * c / p.clusters, g1 = total * (c + 1) / p.clusters;
        return g0 == g1 ? -1 : 2 * c + (g0 < a);
    };
    float top = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32)
        if (slot(c) >= 0)
            top = fmaxf(top, p.ws_lse[(int64_t)slot(c) * p.H + h]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float acc[16] = {}, sum = 0.f;
    if (top != -INFINITY)
        for (int c = c0 + warp; c <= c1; c += 8) {
            if (slot(c) < 0)
                continue;
            const int64_t r = (int64_t)slot(c) * p.H + h;
            const float w = expf(p.ws_lse[r] - top);
            const float4 *src = reinterpret_cast<const float4 *>(p.ws_o + r * kDv) + lane;
            sum += w;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 v = src[32 * e];
                acc[4 * e] = fmaf(w, v.x, acc[4 * e]);
                acc[4 * e + 1] = fmaf(w, v.y, acc[4 * e + 1]);
                acc[4 * e + 2] = fmaf(w, v.z, acc[4 * e + 2]);
                acc[4 * e + 3] = fmaf(w, v.w, acc[4 * e + 3]);
            }
        }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        reinterpret_cast<float4 *>(acc_s[warp])[lane + 32 * e] =
            make_float4(acc[4 * e], acc[4 * e + 1], acc[4 * e + 2], acc[4 * e + 3]);
    if (lane == 0)
        sum_s[warp] = sum;
    __syncthreads();
    float l = 0.f, x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        l += sum_s[w];
        const float2 v = reinterpret_cast<const float2 *>(acc_s[w])[threadIdx.x];
        x += v.x;
        y += v.y;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const int64_t orow = (int64_t)row * p.H + h;
    reinterpret_cast<uint32_t *>(p.out)[orow * (kDv / 2) + threadIdx.x] = pack2(x * inv, y * inv);
    if (threadIdx.x == 0)
        p.lse[orow] = top == -INFINITY ? -INFINITY : top + logf(l);
}

int clusters() { return num_sms() / 2 > 0 ? num_sms() / 2 : 1; }

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

} // namespace

size_t dense_mla_workspace_bytes(int B, int H)
{
    const size_t parts = 2 * (size_t)clusters() * H;
    return align256(parts * kDv * sizeof(float)) + align256(parts * sizeof(float)) + ((size_t)B + 1) * sizeof(int64_t);
}

int launch_dense_mla(const DenseMlaArgs &a, cudaStream_t stream, char *err, size_t errlen)
{
    Params p{};
    p.status = device_status_ptr();
    if (!p.status) {
        snprintf(err, errlen, "device status word unavailable");
        return DSA_ERR_CUDA;
    }
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.pool = static_cast<const __nv_bfloat16 *>(a.kv_pool);
    p.block_table = a.block_table;
    p.ctx_len = a.ctx_len;
    p.num_pages = a.num_pages;
    p.page_size = a.page_size;
    p.max_pages = a.max_pages;
    p.B = a.B;
    p.H = a.H;
    p.clusters = clusters();
    p.scale_log2 = a.sm_scale * 1.4426950408889634f;
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.lse = a.lse;
    const size_t parts = 2 * (size_t)p.clusters * a.H;
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    p.ws_o = reinterpret_cast<float *>(ws);
    p.ws_lse = reinterpret_cast<float *>(ws + align256(parts * kDv * sizeof(float)));
    p.row_start = reinterpret_cast<int64_t *>(ws + align256(parts * kDv * sizeof(float)) + align256(parts * sizeof(float)));
    CUtensorMap tq, tkv;
    if (!encode_tmap_2d(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, kD, (uint64_t)a.B * a.H, kD * 2, 64, 64,
                        CU_TENSOR_MAP_SWIZZLE_128B, err, errlen) ||
        !encode_tmap_2d(&tkv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.kv_pool, kD, (uint64_t)a.num_pages * a.page_size, kD * 2, 64,
                        a.page_size < 64 ? a.page_size : 64, CU_TENSOR_MAP_SWIZZLE_128B, err, errlen))
        return DSA_ERR_CUDA;
    static std::atomic<bool> raised[64];
    cudaError_t e = raise_smem_limit_once(dense_mla_kernel, kSmem, raised);
    if (e == cudaSuccess)
        e = launch_pdl(dense_mla_kernel, dim3(2 * p.clusters), dim3(kThreads), kSmem, stream, 1, tq, tkv, p);
    if (e == cudaSuccess)
        e = launch_pdl(dense_mla_join_kernel, dim3(a.B, a.H), dim3(256), 0, stream, 1, p);
    if (e != cudaSuccess) {
        snprintf(err, errlen, "dense MLA launch: %s", cudaGetErrorString(e));
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

} // namespace dsa
