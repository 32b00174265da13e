// Which kernel a product of FP8 operands goes to.
#include "gemm_fp8.cuh"

namespace dsa {

int launch_gemm_fp8(const GemmFp8Args &a, cudaStream_t stream, char *err, size_t errlen)
{
    if (a.M >= 256 && a.N >= 128)
        return launch_gemm_fp8_tile(a, 256, stream, err, errlen);
    const int cols = a.M <= 16 ? 16 : a.M <= 32 ? 32 : a.M <= 64 ? 64 : 128;
    const int pieces = (a.K + kGemmPiece - 1) / kGemmPiece;
    const int64_t tiles = (int64_t)((a.M + cols - 1) / cols) * ((a.N + 127) / 128);
    int split = 1;
    while (split < 8 && tiles * split * 2 <= 2 * num_sms() && pieces >= 4 * split)
        split *= 2;
    return launch_gemm_fp8_split(a, cols, split, stream, err, errlen);
}

} // namespace dsa
