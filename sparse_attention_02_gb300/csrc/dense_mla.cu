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
// Roles per CTA (12 warps; a wait is polled by all lanes, which answers sooner
// than one lane polling and a broadcast: 535 us against 607 when it came in):
//   warp 0       loads: Q once per row, each tile's own 64 keys (9 atoms of 64
//                columns, as four copies, 0-1, 2-3, 4-5 and 6-8, with barriers of
//                their own, the halves into what each half of the PV freed), and
//                behind them an L2 prefetch of the next tile (one instruction: a
//                page is contiguous; the copy engine takes requests in order)
//   warp 1       (leader CTA) scores of a tile, group by group as the atoms land;
//                all lanes of the CTA pair's two warps 1 allocate TMEM
//   warp 2       swaps: the peer's keys' value columns over this CTA's spent ones
//   warp 3       (leader CTA) PV.  A thread of its own: a thread that issues both
//                waits for P with the next scores unissued
//   warps 4-11   softmax: four threads a head, 32 of the tile's 128 keys each,
//                which swap their maxima through shared memory; the running maximum
//                moves only when exceeded by 2^8 (O is then rescaled in TMEM); P
//                goes to shared memory as bf16, the first 64 keys' over the spent
//                RoPE atom.  In a row's last tile they also zero the value rows past
//                the end, whose stale bytes might be NaN (0 * NaN).
// P is the one intermediate rounded to 16 bits: kind::f16 wants P in V's type.
// The sum l is that of the unrounded values, in fp32.
//
// Work split.  The rows' tiles (and their fixed cost, below) laid end to end are
// cut into one contiguous share per CTA pair, computed on the device from ctx_len
// (the host never sees the lengths).  A share that holds part of a row leaves that
// part, normalised, with its LSE in the workspace, and a second kernel joins the
// parts.
//
// Measured.  64 rows of 128 heads, 8192 to 65536 keys (2.73 GB): 457-486 us a call
// in bursts (83-88 % of measured HBM, 72-76 % of measured BF16; the join 10 of
// them), 542-551 when calls follow one another for long, the power limit then holding
// the SM clock near 1.5 GHz.  Without its loads the kernel takes 338 us, with every
// byte in L2 412: what is left is the chain of a tile (loads, scores, softmax, PV)
// over the two stages that fit.  9 rows of 16 heads, 1 to 131072 keys, pages of 32:
// 125 us (80 % of HBM).  One row of 1000 keys, 16 heads: 11.8 us.  Many short rows,
// 200 of 1 to 500 keys, 16 heads: 30.2 us.  Not kept: 64-key tiles over four stages
// (480 and 555 us where this took 473 and 530; 123 for the ragged rows; the MMAs of
// N = 64 run at 78 % of the rate), no prefetch (528 where one tile ahead took 496),
// two, three and four tiles ahead (504, 518, 557), prefetches by a warp's own loads
// or of the next row's queries (27.7 for 26.4 at 200 rows of one tile), a stage's
// pieces freed one by one.
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
constexpr int kGroups = 4;                // groups a stage's atoms arrive in: 0-1, 2-3, 4-5, 6-8
constexpr int kSoftWarp0 = 4, kSoftWarps = 8;
constexpr int kThreads = 32 * (kSoftWarp0 + kSoftWarps);
constexpr int kBatch = 16;                // tiles whose pages a warp looks up at once (two half-blocks a tile)
constexpr int kPrefetch = 1;              // tiles ahead of the loads that are pulled into L2
constexpr float kRescaleLog2 = 8.f;

// shared memory
constexpr int OFF_Q = 0;
constexpr int OFF_KV = OFF_Q + kStage;
constexpr int OFF_P1 = OFF_KV + kStages * kStage; // P of the tile's second 64 keys (the first's takes the spent RoPE atom)
constexpr int OFF_X = OFF_P1 + kAtom;             // per-thread maxima (two buffers); the first also takes the sums
constexpr int OFF_BAR = OFF_X + 2 * 256 * 4;
constexpr int NBAR = 36;
constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
constexpr int OFF_UNREAD = OFF_MISC + 64;         // where st.async leaves its words
constexpr int kSmem = OFF_UNREAD + 4 * kSoftWarps;
static_assert(kSmem <= 232448, "dynamic shared memory above the 227 KB a CTA may hold");

// barriers (L: used in the leader CTA only; both CTAs' roles arrive there).  What the other CTA's threads, loads or MMAs
// signal is waited for with an acquire at cluster scope (all but VL, RB, RL and DONE: 0.3 % of a call).
constexpr int B_KF = 0,  // L [stage][group]: both CTAs' atoms landed
              B_E = 8,   // [stage][half]: PV of the tile's first / second 64 keys done
              B_SF = 12, // [buffer]: scores done
              B_QD = 16, // [stage]: the score MMAs over atoms 0-3 done
              B_VL = 18, // [stage]: this CTA's swapped-in columns landed
              B_P = 20,  // L [buffer]: scores read, P written, O rescaled, value columns in place
              B_OF = 24, // O of a unit complete
              B_OE = 25, // L: O read
              B_QF = 26, // L: Q landed
              B_DONE = 27,
              B_RB = 28, // [pair][parity]: the four warps of 32 heads swapped their maxima
              B_RL = 32; // [pair][0/1]: ... their sums / read them

constexpr uint32_t TM_O = 0, TM_S = 256, kTmemCols = 512;

// A row in parts: the slot of its first, the cluster of its last.  Rows that are
// whole, and clusters that do not begin a row which others finish, have row = -1.
struct Split {
    int row, slot, last, pad;
};

struct Params {
    const __nv_bfloat16 *q;
    const __nv_bfloat16 *pool;
    const int32_t *block_table, *ctx_len;
    int num_pages, page_size, max_pages, B, H, clusters;
    float scale_log2;
    bool wide; // out starts at 32 bytes
    __nv_bfloat16 *out;
    float *lse;
    float *ws_o, *ws_lse; // [2 clusters, H, 512], [2 clusters, H]
    Split *splits;        // [min(B, clusters)], of rows where they are fewer than clusters, else of clusters
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

// Shares are cut from the rows' costs laid end to end: a row costs its tiles and,
// where there are more tiles than clusters, one more, about what its queries,
// lookups and output take (200 rows of 1 to 500 keys, 16 heads: 30.2 us, 32.8 cut
// from the tiles alone, as pairs with many short rows ended last).  The extra
// comes first: cost x of a row stands for tile x - extra.
struct Share {
    int64_t begin, end, total; // cost in front of its first row, of its end, of all rows
    int row, tile;             // where it starts
    int clusters;              // that have shares
    int extra;
};

struct Unit {
    int row, ctx, jb, je; // tiles [jb, je) of the row
    int64_t begin;        // cost in front of the row
    int slot;             // -1: the whole row
};

struct Walk {
    int64_t at, end;
    int row, tile, first, extra;
    __device__ explicit Walk(const volatile Share &s)
        : at(s.begin), end(s.end), row(s.row), tile(s.tile), first(s.row), extra(s.extra)
    {
    }
    __device__ bool next(const Params &p, int cid, Unit &u)
    {
        if (at + extra + tile >= end) // nothing of this row's is the share's
            return false;
        u.row = row;
        u.ctx = context(p, row);
        u.begin = at;
        const int n = tiles_of(u.ctx);
        u.jb = tile;
        u.je = end - at - extra < n ? (int)(end - at - extra) : n;
        u.slot = u.jb == 0 && u.je == n ? -1 : 2 * cid + (row != first);
        at += n + extra;
        ++row;
        tile = 0;
        return true;
    }
    __device__ bool next_filled(const Params &p, int cid, Unit &u) // skips empty rows
    {
        while (next(p, cid, u))
            if (u.ctx > 0)
                return true;
        u.jb = u.je = 0;
        return false;
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

// One softmax warp's arrival on a barrier of the leader CTA, which counts kSoftWarps arrivals of its own warps, one of
// them expecting kSoftWarps * 4 bytes (`arms`), and those bytes from CTA 1's.  What CTA 1 announces (P, value rows, O in its
// shared and tensor memory) the leader's MMA threads act on, so it takes a release at cluster scope: a four-byte
// st.async carries one without keeping the warp, where a plain arrival with it took most of a tile's time.
__device__ __forceinline__ void arrive_leader(uint32_t rank, uint32_t bar, uint32_t lead_bar, uint32_t lead_unread, bool arms)
{
    if (rank)
        st_async_b32(lead_unread, 0u, lead_bar);
    else if (arms)
        mbar_arrive_expect_tx(bar, kSoftWarps * 4);
    else
        mbar_arrive(bar);
}

// Atoms of 64 columns (block, block + 1, ... as the map's box has) of consecutive rows into this CTA's shared memory.
// The barrier may be either CTA's of the pair.
__device__ __forceinline__ void load_atoms(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t block, int32_t row,
                                           int32_t group = 0)
{
    asm volatile("cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
                 "[%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(block), "r"(group), "r"(bar)
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

// Whether a barrier's phase is over, without waiting for it.
__device__ __forceinline__ bool mbar_done(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return done != 0;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    dense_mla_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv2,
                     const __grid_constant__ CUtensorMap tm_kv3, Params p)
{
    extern __shared__ __align__(1024) uint8_t smem[]; // the swizzle's period; no other shared memory in this kernel
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
        for (int i = 0; i < kStages * kGroups; ++i)
            mbar_init(bar(B_KF + i), 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(B_E + i), 1);
            mbar_init(bar(B_RB + i), kSoftWarps / 2);
            mbar_init(bar(B_RL + i), kSoftWarps / 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_SF + i), 1);
            mbar_init(bar(B_QD + i), 1);
            mbar_init(bar(B_VL + i), 1);
            mbar_init(bar(B_P + i), kSoftWarps);
        }
        mbar_init(bar(B_OF), 1);
        mbar_init(bar(B_OE), kSoftWarps);
        mbar_init(bar(B_QF), 1);
        mbar_init(bar(B_DONE), 2);
        *abort_flag = 0;
        fence_mbar_init();
    }
    // this CTA's barriers exist (thread 0 is past its fence when it arrives); the peer's are waited for below
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
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
        const int extra = total > p.clusters;
        if (extra) {
            before += r0;
            mine += r1 > r0 ? r1 - r0 : 0;
            total += p.B;
        }
        const int n = total < p.clusters ? (int)total : p.clusters;
        auto start = [&](int c) {
            return total < (1 << 24) ? (int64_t)((uint32_t)total * (uint32_t)c / (uint32_t)n) : total * c / n;
        };
        const int64_t g0 = cid < n ? start(cid) : total, g1 = cid < n ? start(cid + 1) : total;
        if (threadIdx.x == 0) {
            share->end = g1;
            share->total = total;
            share->clusters = n;
            share->extra = extra;
            if (g0 == g1) { // no share
                share->begin = g1;
                share->row = share->tile = 0;
            }
        }
        if (g0 < g1 && g0 >= before && g0 < before + mine) {
            int64_t at = before;
            int r = r0;
            for (;; ++r) {
                const int t = tiles_of(context(p, r)) + extra;
                if (g0 < at + t)
                    break;
                at += t;
            }
            share->begin = at;
            share->row = r;
            share->tile = g0 - at > extra ? (int)(g0 - at) - extra : 0;
        }
    }
    tc_fence_before();
    __syncthreads();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); // before any remote operation
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
            // Q is free once the previous unit's last score MMAs are done.  Until then the unit's first tile goes ahead
            // of it: a row of one tile would otherwise wait for the row before it to load anything.
            const uint32_t last = i - 1;
            bool q_due = true;
            auto load_q = [&] {
                if (elect_one()) {
                    if (rank == 0)
                        mbar_arrive_expect_tx(bar(B_QF), 2 * kStage);
                    load_atoms(sbase + OFF_Q, &tm_q, lead(B_QF), 0, 64 * (int)rank, un.row); // heads past H: zeros
                }
                __syncwarp();
                q_due = false;
            };
            if (u == 0 || __all_sync(0xffffffffu, mbar_done(bar(B_SF + (last & 1)), (last >> 1) & 1)))
                load_q();
            for (int j = un.jb; j < un.je; ++j, ++i) {
                const int st = i & 1;
                pg.advance(p, un, j);
                int r[2] = {pg.get(j, 0), pg.get(j, 1)};
                if (lane == 0 && (r[0] == -2 || (boxes == 2 && r[1] == -2)))
                    atomicOr(p.status, DSA_DEV_BAD_PAGE);
                for (int g = 0; g < kGroups; ++g) {
                    // atoms 0-3 hold the value columns of the first 64 keys, 4-7 of the second
                    if ((g & 1) == 0 && i >= 2 &&
                        !mbar_wait_warp<true>(bar(B_E + 2 * st + (g >> 1)), ((i >> 1) - 1) & 1, abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        const int n = g == kGroups - 1 ? 3 : 2, per = boxes == 2 ? 1 : n;
                        if (rank == 0)
                            mbar_arrive_expect_tx(bar(B_KF + kGroups * st + g), 2 * n * kAtom);
                        for (int a = 0; a < n; a += per)
                            for (int b = 0; b < boxes; ++b)
                                load_atoms(sbase + OFF_KV + st * kStage + (2 * g + a) * kAtom + b * box_bytes,
                                           n == 3 ? &tm_kv3 : &tm_kv2, lead(B_KF + kGroups * st + g), 2 * g + a,
                                           r[b] >= 0 ? r[b] : oob);
                    }
                    __syncwarp();
                }
                if (!ok)
                    break;
                if (q_due) {
                    if (!mbar_wait_warp<true>(bar(B_SF + (last & 1)), (last >> 1) & 1, abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    load_q();
                }
                // behind this tile's loads, the one after the next: the copy engine takes requests in order
                if (j + kPrefetch < un.je) {
                    const int r0 = pg.get(j + kPrefetch, 0), r1 = pg.get(j + kPrefetch, 1);
                    if (elect_one()) {
                        if (r0 >= 0)
                            prefetch_l2(p.pool + (int64_t)r0 * kD, kStage / boxes);
                        if (boxes == 2 && r1 >= 0)
                            prefetch_l2(p.pool + (int64_t)r1 * kD, kStage / 2);
                    }
                    __syncwarp();
                }
            }
            ++u;
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
                if (!mbar_wait_warp<true>(bar((rank ? B_QD : B_SF) + st), (i >> 1) & 1, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    mbar_arrive_expect_tx(bar(B_VL + st), 4 * kAtom);
                    for (int a = 0; a < 4; a += boxes == 2 ? 1 : 2)
                        for (int b = 0; b < boxes; ++b)
                            load_atoms(sbase + OFF_KV + st * kStage + (y0 + a) * kAtom + b * box_bytes, &tm_kv2, bar(B_VL + st),
                                       a0 + a, r[b] >= 0 ? r[b] : oob);
                }
                __syncwarp();
            }
        }
        if (i > 0 && lane == 0)
            mbar_drain(bar(B_VL + ((i - 1) & 1)), ((i - 1) >> 1) & 1);
        __syncwarp();
    } else if (warp == 1 && rank == 0) {
        // ----------------------------------------------------- score MMAs
        // KF of a tile implies that its stage's last P, and with it the scores
        // that this buffer held, have been consumed.
        if (elect_one()) {
            constexpr uint32_t idesc = idesc_f32acc(128, 128, 1u, false, false);
            const uint64_t qd = sdesc(sbase + OFF_Q, 16, 1024, 2), kd = sdesc(sbase + OFF_KV, 16, 1024, 2);
            Walk it(*share);
            Unit un;
            uint32_t t = 0;
            bool ok = true;
            for (int u = 0; ok && it.next_filled(p, cid, un); ++u) {
                ok = mbar_wait<true>(bar(B_QF), u & 1, abort_flag, p.status);
                for (int j = un.jb; ok && j < un.je; ++j, ++t) {
                    const int st = t & 1;
                    const uint64_t so = (uint64_t)((st * kStage) >> 4);
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        if (!mbar_wait<true>(bar(B_KF + kGroups * st + g), (t >> 1) & 1, abort_flag, p.status)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll
                        for (int s = 8 * g; s < (g == kGroups - 1 ? 36 : 8 * g + 8); ++s)
                            umma_f16_pair(tmem + TM_S + 64 * st, qd + (((s >> 2) * kAtom + (s & 3) * 32) >> 4),
                                          kd + so + (((s >> 2) * kAtom + (s & 3) * 32) >> 4), idesc, s > 0);
                        if (g == 1)
                            umma_commit_pair(bar(B_QD + st));
                        if (g == kGroups - 1)
                            umma_commit_pair(bar(B_SF + st));
                    }
                }
            }
            umma_commit_pair(bar(B_DONE));
            mbar_drain(bar(B_DONE), 0);
        }
        __syncwarp();
    } else if (warp == 3 && rank == 0) {
        // -------------------------------------------------------- PV MMAs
        // A thread of its own: neither its waits nor the score MMAs' hold the
        // other up, and a PV frees the stage that the loads wait for.
        if (elect_one()) {
            constexpr uint32_t idesc = idesc_f32acc(128, 256, 1u, false, true);
            const uint64_t vd = sdesc(sbase + OFF_KV, kAtom, 1024, 2);
            const uint64_t pd0 = sdesc(sbase + OFF_KV + 8 * kAtom, 16, 1024, 2), pd1 = sdesc(sbase + OFF_P1, 16, 1024, 2);
            Walk it(*share);
            Unit un;
            uint32_t t = 0;
            bool ok = true;
            int u = 0;
            for (; ok && it.next_filled(p, cid, un); ++u) {
                // a unit's first PV overwrites O: the previous unit's must have been read
                ok = u == 0 || mbar_wait<true>(bar(B_OE), (u - 1) & 1, abort_flag, p.status);
                for (int j = un.jb; ok && j < un.je; ++j, ++t) {
                    const int st = t & 1;
                    const uint64_t so = (uint64_t)((st * kStage) >> 4);
                    if (!mbar_wait<true>(bar(B_P + st), (t >> 1) & 1, abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const int64_t valid = (int64_t)un.ctx - (int64_t)j * kTile; // past these P is zero
#pragma unroll
                    for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (64 * kb + 16 * k < valid)
                                    umma_f16_pair(tmem + TM_O + 128 * n, (kb ? pd1 : pd0 + so) + 2 * k,
                                              vd + so + (((4 * kb + 2 * n) * kAtom + 16 * 128 * k) >> 4), idesc,
                                              kb || k || j > un.jb);
                        umma_commit_pair(bar(B_E + 2 * st + kb));
                    }
                    if (j == un.je - 1)
                        umma_commit_pair(bar(B_OF));
                }
            }
            if (ok && u > 0) // the last words from CTA 1 are stores into this CTA, which must outlive them
                mbar_wait<true>(bar(B_OE), (u - 1) & 1, abort_flag, p.status);
            umma_commit_pair(bar(B_DONE));
            mbar_drain(bar(B_DONE), 0);
        }
        __syncwarp();
    } else if (warp >= kSoftWarp0) {
        // ---------------------------------------------------------- softmax
        // Warp: TMEM lane quadrant, and 32 of its 64 score columns.  Thread:
        // head hl of this CTA, keys [64 kb + 32 part, + 32) of the tile.
        const int quad = warp & 3, part = (warp - kSoftWarp0) >> 2, kb = quad >> 1, pair = quad & 1;
        const int hl = 32 * pair + lane, h = 64 * (int)rank + hl;
        const uint32_t lane_off = (uint32_t)(32 * quad) << 16;
        const bool swapped = kb != (int)rank; // this CTA's value columns of key block kb are swapped in
        float *xrow = xs + hl * 4, *xmine = xrow + 2 * kb + part;
        const uint32_t lead_unread = mapa_shared(sbase + OFF_UNREAD + 4 * (warp - kSoftWarp0), 0);
        uint32_t i = 0;
        int u = 0;
        bool ok = true;
        Walk it(*share);
        Unit un;
        Pages pg;
        // for the joining kernel: cost g of all lies in cluster ((g + 1) clusters - 1) / total
        const bool records = rank == 0 && threadIdx.x == 32 * kSoftWarp0, by_row = p.B < p.clusters;
        if (records && !by_row)
            p.splits[cid] = {-1, 0, 0, 0};
        bool have = it.next(p, cid, un);
        if (have)
            pg.start(p, un, kb);
        Unit ahead; // the unit after this one, looked up while this one's last PV runs
        Pages pg_ahead;
        bool more = false;
        auto look_ahead = [&] {
            more = it.next(p, cid, ahead);
            if (more)
                pg_ahead.start(p, ahead, kb);
        };
        for (; ok && have; have = more, un = ahead, pg = pg_ahead) {
            float m = -INFINITY, l = 0.f;
            if (records && un.jb == 0) {
                const int64_t end = un.begin + tiles_of(un.ctx) + share->extra; // of the row
                if (un.slot >= 0)
                    p.splits[by_row ? un.row : cid] = {un.row, un.slot, (int)((end * share->clusters - 1) / share->total), 0};
                else if (by_row)
                    p.splits[un.row].row = -1;
            }
            const int64_t orow = (int64_t)un.row * p.H + h, prow = (int64_t)un.slot * p.H + h;
            const int col0 = 256 * kb + 128 * part; // of O: lanes 0-63 hold columns [0, 256), lanes 64-127 the others
            if (un.ctx == 0) {
                if (h < p.H) {
                    uint4 *dst = reinterpret_cast<uint4 *>(p.out + orow * kDv + col0);
                    for (int c = 0; c < 16; ++c)
                        dst[c] = make_uint4(0, 0, 0, 0);
                    if (col0 == 0)
                        p.lse[orow] = -INFINITY;
                }
                look_ahead();
                continue;
            }
            for (int j = un.jb; j < un.je; ++j, ++i) {
                const int st = i & 1;
                pg.advance(p, un, j);
                const bool bad = pg.get(j, boxes == 2 ? part : 0) < 0;
                const int64_t left = (int64_t)un.ctx - (int64_t)j * kTile - 64 * kb - 32 * part;
                // heads past H have Q = 0; P = 0 too costs the MMAs the least power
                const int valid = bad || left < 0 || h >= p.H ? 0 : left < 32 ? (int)left : 32;
                if (!mbar_wait_warp<true>(bar(B_SF + st), (i >> 1) & 1, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t s[32];
                tmem_ld32(tmem + lane_off + TM_S + 64 * st + 32 * part, s);
                tmem_ld_wait();
                if (valid < 32) {
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (c >= valid)
                            s[c] = 0xFF800000u;
                }
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    mx4[c & 3] = fmaxf(mx4[c & 3], __uint_as_float(s[c]));
                // the head's four threads; scale > 0, and -inf stays
                xmine[256 * (i & 1)] = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * p.scale_log2;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(B_RB + 2 * pair + (i & 1)));
                if (!mbar_wait_warp(bar(B_RB + 2 * pair + (i & 1)), (i >> 1) & 1, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                const float4 x4 = *reinterpret_cast<const float4 *>(xrow + 256 * (i & 1));
                const float mx = fmaxf(fmaxf(x4.x, x4.y), fmaxf(x4.z, x4.w));
                const bool first = j == un.jb;
                const bool move = mx > m + kRescaleLog2 || (m == -INFINITY && mx > m);
                const bool rescale = !first && __any_sync(0xffffffffu, move);
                // PV of the previous tile: before O is touched, and before P's second buffer is
                if ((rescale || (kb == 1 && i > 0)) &&
                    !mbar_wait_warp<true>(bar(B_E + 2 * (st ^ 1) + 1), ((i - 1) >> 1) & 1, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                if (rescale) {
                    tc_fence_after();
                    const float f = move ? exp2_fast(m - mx) : 1.f;
                    l *= f;
#pragma unroll 1
                    for (int c = 0; c < 128; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(tmem + lane_off + TM_O + 128 * part + c, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st32(tmem + lane_off + TM_O + 128 * part + c, o);
                    }
                    tmem_st_wait();
                }
                if (move)
                    m = mx;
                const float ms = m == -INFINITY ? 0.f : m;
                uint8_t *prow_s = smem + (kb ? OFF_P1 : OFF_KV + st * kStage + 8 * kAtom) + hl * 128;
                float sum = 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float e[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        e[k] = exp2_fast(fmaf(__uint_as_float(s[8 * c + k]), p.scale_log2, -ms));
                    sum += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
                    *reinterpret_cast<uint4 *>(prow_s + (((4 * part + c) ^ (hl & 7)) << 4)) =
                        make_uint4(pack2(e[0], e[1]), pack2(e[2], e[3]), pack2(e[4], e[5]), pack2(e[6], e[7]));
                }
                l += sum;
                if (swapped && !mbar_wait_warp(bar(B_VL + st), (i >> 1) & 1, abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                if (left < 32) { // value rows past the end, of this warp's 32 keys
                    const int from = 32 * part + (left < 0 ? 0 : (int)left);
                    for (int x = from * 8 + 32 * pair + lane; x < (32 * part + 32) * 8; x += 64)
#pragma unroll
                        for (int a = 0; a < 4; ++a)
                            *reinterpret_cast<uint4 *>(smem + OFF_KV + st * kStage + (4 * kb + a) * kAtom + x * 16) =
                                make_uint4(0, 0, 0, 0);
                }
                tc_fence_before();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    arrive_leader(rank, bar(B_P + st), lead(B_P + st), lead_unread, warp == kSoftWarp0);
            }
            if (!ok)
                break;
            look_ahead();
            // ---- the unit's output
            // the sums go where the next tile's maxima do: all four threads have read the ones before
            xmine[256 * (i & 1)] = l;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(B_RL + 2 * pair));
            if (!mbar_wait_warp(bar(B_RL + 2 * pair), u & 1, abort_flag, p.status)) {
                ok = false;
                break;
            }
            const float4 l4 = *reinterpret_cast<const float4 *>(xrow + 256 * (i & 1));
            l = (l4.x + l4.y) + (l4.z + l4.w);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(B_RL + 2 * pair + 1)); // read
            if (!mbar_wait_warp(bar(B_RL + 2 * pair + 1), u & 1, abort_flag, p.status) ||
                !mbar_wait_warp<true>(bar(B_OF), u & 1, abort_flag, p.status)) {
                ok = false;
                break;
            }
            ++u;
            const float inv = l == 0.f ? 0.f : 1.f / l; // a NaN key's l is NaN, and so its row
            tc_fence_after();
            uint32_t o0[32], o1[32];
#pragma unroll
            for (int c = 0; c < 128; c += 32) {
                uint32_t(&o)[32] = c & 32 ? o1 : o0;
                if (!(c & 32)) {
                    tmem_ld32(tmem + lane_off + TM_O + 128 * part + c, o0);
                    tmem_ld32(tmem + lane_off + TM_O + 128 * part + c + 32, o1);
                    tmem_ld_wait();
                }
                if (h >= p.H)
                    continue;
                // a lane's columns are its own row's: 32 bytes a store fill whole sectors
                if (un.slot < 0) {
                    __nv_bfloat16 *dst = p.out + orow * kDv + col0 + c;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t w[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            w[k] = pack2(__uint_as_float(o[16 * e + 2 * k]) * inv, __uint_as_float(o[16 * e + 2 * k + 1]) * inv);
                        if (p.wide) {
                            store32(dst + 16 * e, w);
                        } else {
                            reinterpret_cast<uint4 *>(dst)[2 * e] = make_uint4(w[0], w[1], w[2], w[3]);
                            reinterpret_cast<uint4 *>(dst)[2 * e + 1] = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                    }
                } else {
                    float *dst = p.ws_o + prow * kDv + col0 + c;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t w[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            w[k] = __float_as_uint(__uint_as_float(o[8 * e + k]) * inv);
                        store32(dst + 8 * e, w);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                arrive_leader(rank, bar(B_OE), lead(B_OE), lead_unread, warp == kSoftWarp0);
            if (h < p.H && col0 == 0) {
                const float v = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
                if (un.slot < 0)
                    p.lse[orow] = v;
                else
                    p.ws_lse[prow] = v;
            }
        }
    }

    // After a wait that gave up in either CTA, copies may be in flight whose barrier is the other's: a millisecond is
    // far longer than any takes.
    __syncwarp();
    if (*abort_flag) {
        st_cluster_u32(mapa_shared(sbase + OFF_MISC + 4, rank ^ 1), 1u);
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

// Joins the parts of each split row, O = sum exp(LSE_i - LSE) O_i, in the order
// of the parts.  A CTA takes HEADS heads of a row: with eight and few parts a
// warp each, else its warps take parts w, w + 8, ... of one head after the
// other and add up.  A row's parts lie in consecutive clusters; in all but the
// first the row is the share's first, so its slot is 2 cluster.  At most one row
// a cluster begins there and ends elsewhere, so the grid has no more rows than
// clusters: looking at all 200 of a batch took 4 us of 33.
template <int HEADS>
__global__ void __launch_bounds__(256) dense_mla_join_kernel(Params p)
{
    __shared__ __align__(16) float acc_s[8][kDv];
    __shared__ float sum_s[8];
    grid_dep_wait();
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Split sp = p.splits[blockIdx.x];
    const int row = sp.row, c0 = sp.slot >> 1, np = sp.last - c0 + 1;
    // after a wait that gave up, records may be missing: nothing is read or written outside the buffers for it
    if (row < 0 || row >= p.B || sp.slot < 0 || np < 1 || sp.last >= p.clusters)
        return;
    auto slot = [&](int i) { return i == 0 ? sp.slot : 2 * (c0 + i); };
    const bool alone = HEADS > 1 && np <= 8; // a warp joins a head by itself
    for (int k = alone ? warp : 0; k < HEADS; k += alone ? 8 : 1) {
        const int h = blockIdx.y * HEADS + k;
        if (h >= p.H)
            break;
        float top = -INFINITY;
        for (int i = lane; i < np; i += 32)
            top = fmaxf(top, p.ws_lse[(int64_t)slot(i) * p.H + h]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float4 acc[4] = {};
        float sum = 0.f;
        const int step = alone ? 1 : 8;
#pragma unroll 4
        for (int i = alone ? 0 : warp; i < np; i += step) {
            const int64_t r = (int64_t)slot(i) * p.H + h;
            const float4 *src = reinterpret_cast<const float4 *>(p.ws_o + r * kDv) + lane;
            const float part = p.ws_lse[r], w = part == -INFINITY ? 0.f : expf(part - top);
            sum += w;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 v = src[32 * e];
                acc[e].x = fmaf(w, v.x, acc[e].x);
                acc[e].y = fmaf(w, v.y, acc[e].y);
                acc[e].z = fmaf(w, v.z, acc[e].z);
                acc[e].w = fmaf(w, v.w, acc[e].w);
            }
        }
        const int64_t orow = (int64_t)row * p.H + h;
        if (alone) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                reinterpret_cast<uint2 *>(p.out)[orow * (kDv / 4) + lane + 32 * e] =
                    make_uint2(pack2(acc[e].x * inv, acc[e].y * inv), pack2(acc[e].z * inv, acc[e].w * inv));
            if (lane == 0)
                p.lse[orow] = sum == 0.f ? -INFINITY : top + logf(sum);
            continue;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            reinterpret_cast<float4 *>(acc_s[warp])[lane + 32 * e] = acc[e];
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
        const float inv = l == 0.f ? 0.f : 1.f / l;
        reinterpret_cast<uint32_t *>(p.out)[orow * (kDv / 2) + threadIdx.x] = pack2(x * inv, y * inv);
        if (threadIdx.x == 0)
            p.lse[orow] = l == 0.f ? -INFINITY : top + logf(l);
        __syncthreads(); // the sums are used again for the next head
    }
}

int clusters() { return num_sms() / 2 > 0 ? num_sms() / 2 : 1; }

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

} // namespace

size_t dense_mla_workspace_bytes(int B, int H)
{
    const size_t parts = 2 * (size_t)clusters() * H;
    const size_t splits = B < clusters() ? B : clusters();
    return align256(parts * kDv * sizeof(float)) + align256(parts * sizeof(float)) + splits * sizeof(Split);
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
    p.wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
    p.lse = a.lse;
    const size_t parts = 2 * (size_t)p.clusters * a.H;
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    p.ws_o = reinterpret_cast<float *>(ws);
    p.ws_lse = reinterpret_cast<float *>(ws + align256(parts * kDv * sizeof(float)));
    p.splits = reinterpret_cast<Split *>(ws + align256(parts * kDv * sizeof(float)) + align256(parts * sizeof(float)));
    CUtensorMap tq, tkv2, tkv3;
    const uint64_t rows = (uint64_t)a.num_pages * a.page_size;
    const uint32_t box = a.page_size < 64 ? a.page_size : 64;
    auto map = [&](CUtensorMap *m, const void *base, uint64_t n, uint64_t groups, uint32_t box_rows, uint32_t atoms) {
        return encode_tmap_blocks(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, 64, n, kAtoms, groups, kD * 2, 128, box_rows,
                                  atoms, CU_TENSOR_MAP_SWIZZLE_128B, err, errlen);
    };
    // pages of 32: an atom takes two boxes, so a box holds one atom
    if (!map(&tq, a.q, a.H, a.B, 64, kAtoms) || !map(&tkv2, a.kv_pool, rows, 1, box, box < 64 ? 1 : 2) ||
        !map(&tkv3, a.kv_pool, rows, 1, box, box < 64 ? 1 : 3))
        return DSA_ERR_CUDA;
    static std::atomic<bool> raised[64];
    cudaError_t e = raise_smem_limit_once(dense_mla_kernel, kSmem, raised);
    if (e == cudaSuccess)
        e = launch_pdl(dense_mla_kernel, dim3(2 * p.clusters), dim3(kThreads), kSmem, stream, 1, tq, tkv2, tkv3, p);
    const int joins = a.B < p.clusters ? a.B : p.clusters; // rows that may be in parts
    if (e == cudaSuccess)
        e = joins * a.H <= 8 * num_sms()
                ? launch_pdl(dense_mla_join_kernel<1>, dim3(joins, a.H), dim3(256), 0, stream, 1, p)
                : launch_pdl(dense_mla_join_kernel<8>, dim3(joins, (a.H + 7) / 8), dim3(256), 0, stream, 1, p);
    if (e != cudaSuccess) {
        snprintf(err, errlen, "dense MLA launch: %s", cudaGetErrorString(e));
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

} // namespace dsa
