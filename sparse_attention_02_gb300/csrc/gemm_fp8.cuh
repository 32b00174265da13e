// What the kernels of the FP8 product share.
#pragma once

#include "common.cuh"
#include "f32x2.cuh"
#include "launch.h"

namespace dsa {

constexpr int kGemmPiece = 128; // values along K that share a scale; one row of a 128-byte swizzled tile

// The product for few rows of `a`, of which a CTA takes `cols` and 128 rows of `b`
// (gemm_fp8_split.cu), and for many, by tiles of 128 rows of `a` and `cols` rows of
// `b` (gemm_fp8_tile.cu).  Clusters of `split` CTAs divide K between them.
int launch_gemm_fp8_split(const GemmFp8Args &a, int cols, int split, cudaStream_t stream, char *err, size_t errlen);
int launch_gemm_fp8_tile(const GemmFp8Args &a, int cols, int split, cudaStream_t stream, char *err, size_t errlen);

// mbar_wait_warp with every branch decided by the whole warp: a wait for what is over costs it one poll and one vote.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int *abort_flag, unsigned *status)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
        return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t n = 1;; ++n) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
            return true;
        if ((n & 15) == 0) {
            const bool late = global_timer_ns() - t0 > DSA_WAIT_LIMIT_NS;
            if (__any_sync(0xffffffffu, late)) {
                atomicOr(status, DSA_DEV_TIMEOUT);
                *abort_flag = 1;
                return false;
            }
            if (__any_sync(0xffffffffu, *abort_flag != 0))
                return false;
        }
    }
}

inline bool gemm_fp8_map(CUtensorMap *map, const void *base, int64_t ld, int rows, int K, int box, char *err, size_t errlen)
{
    return encode_tmap_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, (uint64_t)K, (uint64_t)rows, (uint64_t)ld, kGemmPiece, box,
                          CU_TENSOR_MAP_SWIZZLE_128B, err, errlen);
}

// Waits for this warp's TMEM loads; the values depend on it, so nothing uses them earlier.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                   "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                   "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28])
                 :
                 : "memory");
    asm volatile("" : "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}

__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[32]) { tmem_ld32(at, r); }
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[16]) { tmem_ld16(at, r); }

} // namespace dsa
