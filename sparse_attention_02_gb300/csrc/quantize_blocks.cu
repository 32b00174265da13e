// FP8 operands of the 128-block product on sm_103a: E4M3 codes of a matrix and of
// its transpose, each with a scale for every 128 values along its rows (or for
// every 128 x 128 block), from one read.
//
// The indexer and the projections run in FP8 ("AMD Instinct MI355X GPUs Power
// DeepSeek-V3.2-Exp", section "DeepSeek Sparse Attention (DSA)", item 1).  A
// product sums along rows of both operands, so a training step needs a gradient
// (and an activation) along its columns too: as rows of the transpose, with scales
// of their own.  scale = amax / 448 (or its power of two), code = E4M3(x / scale),
// as dsa_quantize_fp8.
//
// HBM-bound: 2 or 4 bytes in and 1 or 2 out per value, if the instructions stay few:
// what a tile's threads do besides loads and stores is counted below.  A CTA takes a
// 128 x 128 tile, a thread 8 columns of 8 rows (bf16) or 4 (fp32) in registers.
//   A row's piece is 16 lanes of one warp.  Its maximum comes from a butterfly in which
//   lanes hand over half of their rows in each step, so that a lane ends with one row,
//   whose scale and its reciprocal it alone computes and the others fetch.
//   A column's maximum is a thread's rows, then the warps' by shared memory.
//   bf16 maxima are taken of pairs as they are: sign bits masked, the order of the bit
//   patterns is that of the magnitudes.
//   Quotients are correctly rounded, three operations a pair (fp8.cuh); a tile with a
//   scale so small that its reciprocal overflows divides.
// Few pieces without the transpose go to half-warps by themselves, with no barrier and no
// tile to fill.
//
// Measured: 8191 x 8192 bf16 with its transpose 56 us (70 % of measured HBM; 84 with
// every lane working out its rows' scales and shared words unpacked once a use), four
// CTAs an SM, whose 64 registers a thread hold all but the division path, which spills
// (three CTAs 65, five 73), 4096 x 7168 fp32 by blocks both ways 32 us
// (80 %; three CTAs of 512 threads 71), 8192 x 8192 without the transpose bf16 39 us (77 %)
// and fp32 55 (90 %), the transpose alone 42 (72 %) and 63 (79 %), 64 x 4096 1.6: 17 instructions a value both ways in bf16, 60 % of an
// SM's slots, are what bytes wait for there.
#include "rmsnorm.cuh"

namespace dsa {
namespace {

constexpr int kTile = 128;

template <typename T> constexpr int rows_a_thread() { return sizeof(T) == 2 ? 8 : 4; } // of a tile

// A scale and its reciprocal; quick: quotients by the reciprocal are exact enough (ScaleDivider).
struct Scale {
    float s, inv;
    __device__ __forceinline__ Scale() {}
    __device__ __forceinline__ Scale(float amax, int mode) : s(fp8_scale(amax, mode)), inv(1.f / s) {}
    __device__ __forceinline__ bool quick() const { return s > 1e-30f; }
};

template <bool QUICK> __device__ __forceinline__ uint32_t codes4(float s, float inv, float a, float b, float c, float d)
{
    if (!QUICK)
        return e4m3x2(a / s, b / s) | (uint32_t)e4m3x2(c / s, d / s) << 16;
    const F2 x(a, b), y(c, d), i2(inv), ns(-s);
    const F2 p = x * i2, q = y * i2;
    fma2(fma2(p, ns, x), i2, p).get(a, b);
    fma2(fma2(q, ns, y), i2, q).get(c, d);
    return e4m3x2(a, b) | (uint32_t)e4m3x2(c, d) << 16;
}

// Eight values and their magnitudes' maxima: of all, and value by value with others.
template <typename T> struct Chunk;

template <> struct Chunk<__nv_bfloat16> {
    Vec8<__nv_bfloat16> v;
    using Tops = uint4; // eight magnitudes, as bf16 bits
    __device__ __forceinline__ static uint32_t max2(uint32_t a, uint32_t b)
    {
        uint32_t r;
        asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    __device__ __forceinline__ Tops tops() const
    {
        constexpr uint32_t m = 0x7FFF7FFFu;
        return make_uint4(v.v.x & m, v.v.y & m, v.v.z & m, v.v.w & m);
    }
    __device__ __forceinline__ static Tops join(Tops a, Tops b)
    {
        return make_uint4(max2(a.x, b.x), max2(a.y, b.y), max2(a.z, b.z), max2(a.w, b.w));
    }
    __device__ __forceinline__ static float all(Tops t)
    {
        const uint32_t m = max2(max2(t.x, t.y), max2(t.z, t.w));
        return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    }
    __device__ __forceinline__ static void each(Tops t, float (&f)[8])
    {
        Vec8<__nv_bfloat16> w;
        w.v = t;
        w.get(f);
    }
    __device__ __forceinline__ static Tops none() { return make_uint4(0, 0, 0, 0); }
};

template <> struct Chunk<float> {
    Vec8<float> v;
    struct Tops {
        float f[8];
    };
    __device__ __forceinline__ Tops tops() const
    {
        Tops t;
        v.get(t.f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            t.f[i] = fabsf(t.f[i]);
        return t;
    }
    __device__ __forceinline__ static Tops join(const Tops &a, const Tops &b)
    {
        Tops t;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            t.f[i] = fmaxf(a.f[i], b.f[i]);
        return t;
    }
    __device__ __forceinline__ static float all(const Tops &t)
    {
        return fmaxf(fmaxf(fmaxf(t.f[0], t.f[1]), fmaxf(t.f[2], t.f[3])), fmaxf(fmaxf(t.f[4], t.f[5]), fmaxf(t.f[6], t.f[7])));
    }
    __device__ __forceinline__ static void each(const Tops &t, float (&f)[8])
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = t.f[i];
    }
    __device__ __forceinline__ static Tops none() { return Tops{}; }
};

// Eight values from p on, zeros from the ncol-th on.  !VEC: p is aligned to its elements only, and eight values are cut
// from the aligned 16-byte words around them, where those lie within the tensor's own bytes [lo, hi); one by one else
// (4096 x 4099 bf16 all one by one 28 us).
template <typename T, bool VEC>
__device__ __forceinline__ void load8(Vec8<T> &v, const T *p, int ncol, [[maybe_unused]] const uint8_t *lo, [[maybe_unused]] const uint8_t *hi)
{
    v.zero();
    if (ncol <= 0)
        return;
    if constexpr (VEC) {
        if (ncol == 8) {
            v.load(p);
            return;
        }
    } else {
        constexpr int N = sizeof(T) == 2 ? 2 : 3; // 16-byte words
        const uintptr_t at = reinterpret_cast<uintptr_t>(p), first = at & ~(uintptr_t)15;
        if (ncol == 8 && first >= reinterpret_cast<uintptr_t>(lo) && first + 16 * N <= reinterpret_cast<uintptr_t>(hi)) {
            uint32_t w[4 * N], u[4 * N - 2];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const uint4 x = reinterpret_cast<const uint4 *>(first)[k];
                w[4 * k] = x.x, w[4 * k + 1] = x.y, w[4 * k + 2] = x.z, w[4 * k + 3] = x.w;
            }
            const int off = (int)(at & 15);
#pragma unroll
            for (int k = 0; k < 4 * N - 2; ++k)
                u[k] = off & 8 ? w[k + 2] : w[k];
#pragma unroll
            for (int k = 0; k < 4 * N - 3; ++k)
                u[k] = off & 4 ? u[k + 1] : u[k];
            if (sizeof(T) == 2 && (off & 2))
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    u[k] = __funnelshift_r(u[k], u[k + 1], 16);
            v.set_words(u);
            return;
        }
    }
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        f[j] = j < ncol ? (float)p[j] : 0.f;
    v.set(f);
}

// The bytes of x, from the first row's first value to the last row's last.
template <typename T> __device__ __forceinline__ const uint8_t *end_of(const QuantizeBlocksArgs &a)
{
    return reinterpret_cast<const uint8_t *>(static_cast<const T *>(a.x) + (a.rows - 1) * a.ldx + a.cols);
}

__device__ __forceinline__ void store8(uint8_t *p, uint32_t lo, uint32_t hi, bool wide, int ncol)
{
    if (wide) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(lo, hi);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < ncol)
            p[j] = (uint8_t)((j < 4 ? lo : hi) >> (8 * (j & 3)));
}

// N maxima over the 16 lanes of a half-warp: lane c gets number c / (16 / N).
template <int N> __device__ __forceinline__ float own_top(float (&m)[N], int c)
{
    int have = N;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        if (have > 1) { // hands over half of what it has
            const bool upper = c & o;
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                if (i < have / 2) {
                    const float give = upper ? m[i] : m[i + have / 2], keep = upper ? m[i + have / 2] : m[i];
                    m[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, o));
                }
            have /= 2;
        } else {
            m[0] = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
        }
    }
    return m[0];
}

// BLOCK: a scale for the whole tile, else for every 128 values of a row (of the matrix, of the transpose).
template <typename T, bool VEC, bool BLOCK>
__global__ void __launch_bounds__(16 * kTile / rows_a_thread<T>(), sizeof(T) == 2 ? 4 : 2) quantize_blocks_kernel(QuantizeBlocksArgs a)
{
    constexpr int RPT = rows_a_thread<T>(), kThreads = kTile / RPT * 16, kWarps = kThreads / 32; // rows a thread
    using C = Chunk<T>;
    __shared__ __align__(16) uint8_t turned[kTile * kTile];
    __shared__ __align__(16) float tops[BLOCK ? 1 : kWarps][BLOCK ? kWarps : kTile + 4];
    __shared__ __align__(16) float col_scale[kTile], col_inv[kTile];
    grid_dep_wait();
    grid_dep_launch();
    const int cblocks = (int)((a.cols + kTile - 1) / kTile), rblocks = (int)((a.rows + kTile - 1) / kTile);
    const int cb = blockIdx.x % cblocks, rb = blockIdx.x / cblocks;
    const int c = threadIdx.x & 15, rg = threadIdx.x >> 4, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t col = (int64_t)cb * kTile + 8 * c, row0 = (int64_t)rb * kTile + RPT * rg;
    const int ncol = a.cols - col >= 8 ? 8 : a.cols > col ? (int)(a.cols - col) : 0; // of this thread
    const int nrow = a.rows - row0 >= RPT ? RPT : a.rows > row0 ? (int)(a.rows - row0) : 0;
    const T *x = static_cast<const T *>(a.x) + row0 * a.ldx + col;
    const uint8_t *lo = static_cast<const uint8_t *>(a.x), *hi = end_of<T>(a);
    C v[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i)
        load8<T, VEC>(v[i].v, x + i * a.ldx, i < nrow ? ncol : 0, lo, hi);
    // ---- scales
    Scale whole, mine; // of the tile; of the row that this lane looks after
    typename C::Tops down = C::none(); // the columns' maxima over this thread's rows
    float m[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const typename C::Tops t = v[i].tops();
        down = C::join(down, t);
        m[i] = C::all(t);
    }
    bool quick;
    if constexpr (BLOCK) {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < RPT; ++i)
            top = fmaxf(top, m[i]);
        top = warp_amax(top);
        if (lane == 0)
            tops[0][warp] = top;
        __syncthreads();
        top = warp_amax(lane < kWarps ? tops[0][lane] : 0.f);
        whole = Scale(top, a.scale_mode);
        quick = whole.quick();
        if (threadIdx.x == 0) {
            if (a.codes)
                a.scale[(int64_t)rb * cblocks + cb] = whole.s;
            if (a.codes_t)
                a.scale_t[(int64_t)cb * rblocks + rb] = whole.s;
        }
    } else {
        mine = Scale(own_top<RPT>(m, c), a.scale_mode);
        const int r = c / (16 / RPT);
        if (a.codes && c % (16 / RPT) == 0 && r < nrow)
            a.scale[(row0 + r) * cblocks + cb] = mine.s;
        quick = mine.quick();
        if (a.codes_t) {
            float top[8];
            C::each(down, top);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 16));
            if (lane < 16) {
                reinterpret_cast<float4 *>(&tops[warp][8 * c])[0] = make_float4(top[0], top[1], top[2], top[3]);
                reinterpret_cast<float4 *>(&tops[warp][8 * c])[1] = make_float4(top[4], top[5], top[6], top[7]);
            }
            __syncthreads();
            if (threadIdx.x < kTile) {
                float t = tops[0][threadIdx.x];
#pragma unroll
                for (int w = 1; w < kWarps; ++w)
                    t = fmaxf(t, tops[w][threadIdx.x]);
                const Scale s(t, a.scale_mode);
                quick = quick && s.quick();
                col_scale[threadIdx.x] = s.s;
                col_inv[threadIdx.x] = s.inv;
                const int64_t k = (int64_t)cb * kTile + threadIdx.x;
                if (k < a.cols)
                    a.scale_t[k * rblocks + rb] = s.s;
            }
        }
        quick = __syncthreads_and(quick);
    }
    // ---- codes
    auto go = [&](auto q) {
        constexpr bool QUICK = decltype(q)::value;
        if (a.codes) {
            uint8_t *codes = a.codes + row0 * a.ldc + col;
            const bool wide = ((reinterpret_cast<uintptr_t>(a.codes) | a.ldc) & 7) == 0 && ncol == 8;
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                float f[8];
                v[i].v.get(f);
                float s = whole.s, inv = whole.inv;
                if (!BLOCK) {
                    const int from = (lane & 16) + i * (16 / RPT);
                    s = __shfl_sync(0xffffffffu, mine.s, from);
                    inv = __shfl_sync(0xffffffffu, mine.inv, from);
                }
                const uint32_t lo = codes4<QUICK>(s, inv, f[0], f[1], f[2], f[3]), hi = codes4<QUICK>(s, inv, f[4], f[5], f[6], f[7]);
                if (i < nrow)
                    store8(codes + i * a.ldc, lo, hi, wide, ncol);
            }
        }
        if (a.codes_t) {
            // a column's codes of this thread go to shared memory as one or two words, at place ^ 2 c of the column's 32: the
            // warp's words then fall into all banks
            float s[8], inv[8];
            if (BLOCK) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    s[j] = whole.s, inv[j] = whole.inv;
            } else {
                Vec8<float> t;
                t.load(col_scale + 8 * c);
                t.get(s);
                t.load(col_inv + 8 * c);
                t.get(inv);
            }
            float f[RPT][8];
#pragma unroll
            for (int i = 0; i < RPT; ++i)
                v[i].v.get(f[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t w[RPT / 4];
#pragma unroll
                for (int i = 0; i < RPT; i += 4)
                    w[i / 4] = codes4<QUICK>(s[j], inv[j], f[i][j], f[i + 1][j], f[i + 2][j], f[i + 3][j]);
                uint32_t *to = reinterpret_cast<uint32_t *>(turned + (8 * c + j) * kTile) + ((rg * (RPT / 4)) ^ (2 * c));
                if constexpr (RPT == 8)
                    *reinterpret_cast<uint2 *>(to) = make_uint2(w[0], w[RPT / 4 - 1]);
                else
                    *to = w[0];
            }
        }
    };
    if (quick)
        go(std::true_type());
    else
        go(std::false_type());
    if (!a.codes_t)
        return;
    __syncthreads();
    const bool wide = ((reinterpret_cast<uintptr_t>(a.codes_t) | a.ldt) & 15) == 0;
#pragma unroll
    for (int k = threadIdx.x; k < kTile * 8; k += kThreads) {
        const int64_t kc = (int64_t)cb * kTile + (k >> 3), r = (int64_t)rb * kTile + 16 * (k & 7);
        if (kc >= a.cols || r >= a.rows)
            continue;
        const int s = (k >> 6) & 15; // the c of this column
        uint4 w = *reinterpret_cast<const uint4 *>(turned + (k >> 3) * kTile + (((k & 7) ^ (s >> 1)) << 4));
        if (s & 1)
            w = make_uint4(w.z, w.w, w.x, w.y);
        uint8_t *dst = a.codes_t + kc * a.ldt + r;
        if (wide && r + 16 <= a.rows) {
            *reinterpret_cast<uint4 *>(dst) = w;
        } else {
            const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (r + j < a.rows)
                    dst[j] = (uint8_t)(words[j >> 2] >> (8 * (j & 3)));
        }
    }
}

// Pieces of 128 values of a row, by half-warps: N on end each, then the next N that are its.
template <typename T, bool VEC, int N> __global__ void __launch_bounds__(256, 4) quantize_pieces_kernel(QuantizeBlocksArgs a)
{
    using C = Chunk<T>;
    grid_dep_wait();
    grid_dep_launch();
    const int cblocks = (int)((a.cols + kTile - 1) / kTile);
    const int pieces = (int)a.rows * cblocks, step = gridDim.x * 16 * N; // few (launch_quantize_blocks)
    const int c = threadIdx.x & 15, half = threadIdx.x >> 4 & 1;
    const bool aligned = ((reinterpret_cast<uintptr_t>(a.codes) | a.ldc) & 7) == 0;
    const uint8_t *lo = static_cast<const uint8_t *>(a.x), *hi = end_of<T>(a);
    for (int p0 = (blockIdx.x * 16 + (threadIdx.x >> 4)) * N; p0 - N * half < pieces; p0 += step) { // whole warps
        int64_t row = p0 / cblocks;
        int at = p0 - (int)row * cblocks;
        C v[N];
        int64_t rows[N];
        int ats[N], ncol[N]; // columns of this lane; -1: no such piece
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int64_t col = (int64_t)at * kTile + 8 * c;
            rows[k] = row, ats[k] = at;
            ncol[k] = row >= a.rows ? -1 : a.cols - col >= 8 ? 8 : a.cols > col ? (int)(a.cols - col) : 0;
            load8<T, VEC>(v[k].v, static_cast<const T *>(a.x) + row * a.ldx + col, ncol[k], lo, hi);
            if (++at == cblocks)
                at = 0, ++row;
        }
        float m[N];
#pragma unroll
        for (int k = 0; k < N; ++k)
            m[k] = C::all(v[k].tops());
        const Scale mine(own_top<N>(m, c), a.scale_mode);
        auto go = [&](auto q) {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int from = (threadIdx.x & 16) + k * (16 / N);
                const float s = __shfl_sync(0xffffffffu, mine.s, from), inv = __shfl_sync(0xffffffffu, mine.inv, from);
                if (ncol[k] < 0)
                    continue;
                if (c == 0)
                    a.scale[rows[k] * cblocks + ats[k]] = s;
                float f[8];
                v[k].v.get(f);
                store8(a.codes + rows[k] * a.ldc + (int64_t)ats[k] * kTile + 8 * c, codes4<decltype(q)::value>(s, inv, f[0], f[1], f[2], f[3]),
                       codes4<decltype(q)::value>(s, inv, f[4], f[5], f[6], f[7]), aligned && ncol[k] == 8, ncol[k]);
            }
        };
        if (__all_sync(0xffffffffu, mine.quick()))
            go(std::true_type());
        else
            go(std::false_type());
    }
}

} // namespace

int launch_quantize_blocks(const QuantizeBlocksArgs &a, cudaStream_t stream, char *err, size_t errlen)
{
    const int64_t rblocks = (a.rows + kTile - 1) / kTile, cblocks = (a.cols + kTile - 1) / kTile;
    const bool vec = chunked(a.x, a.ldx * (a.x32 ? 4 : 2)), pieces = !a.codes_t && a.block_rows == 1 && rblocks * cblocks < 2 * num_sms();
    auto go = [&](auto t, auto v) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr bool VEC = decltype(v)::value;
        if (pieces) {
            // a piece a half-warp where that is a CTA an SM at most, the shortest way; else two, which share what finding a
            // scale takes, until tiles fill the GPU (bf16, us, one, two, tiles: 64 x 4096 1.6, 2.0, 2.7; 256 x 4096 2.6,
            // 2.1, 3.1; 512 x 8192 6.9, 5.3, 5.3; 2048 x 8192 21, 15, 13; 8192 x 8192 79, 51, 39)
            auto by = [&](auto n) {
                constexpr int N = decltype(n)::value;
                const int64_t all = (a.rows * cblocks + 16 * N - 1) / (16 * N), most = (int64_t)num_sms() * 4;
                return launch_pdl(quantize_pieces_kernel<T, VEC, N>, dim3((unsigned)(all < most ? all : most)), dim3(256), 0, stream, 1, a);
            };
            return a.rows * cblocks <= 16 * num_sms() ? by(std::integral_constant<int, 1>()) : by(std::integral_constant<int, 2>());
        }
        const dim3 tiles((unsigned)(rblocks * cblocks)), threads(16 * kTile / rows_a_thread<T>());
        return a.block_rows == 1 ? launch_pdl(quantize_blocks_kernel<T, VEC, false>, tiles, threads, 0, stream, 1, a)
                                 : launch_pdl(quantize_blocks_kernel<T, VEC, true>, tiles, threads, 0, stream, 1, a);
    };
    auto with = [&](auto t) { return vec ? go(t, std::true_type()) : go(t, std::false_type()); };
    const cudaError_t e = a.x32 ? with((float *)0) : with((__nv_bfloat16 *)0);
    if (e != cudaSuccess) {
        snprintf(err, errlen, "quantize_blocks launch: %s", cudaGetErrorString(e));
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

} // namespace dsa
