// Which kernel a product of FP8 operands goes to.
#include "gemm_fp8.cuh"

namespace dsa {

int launch_gemm_fp8(const GemmFp8Args &a, cudaStream_t stream, char *err, size_t errlen)
{
    const int pieces = (a.K + kGemmPiece - 1) / kGemmPiece, sms = num_sms();
    if (a.M <= 32 || (a.M <= 64 && ((int64_t)a.N + 127) / 128 <= sms * 4 / 5)) {
        // b's bytes bound: as many CTAs as the GPU holds (two an SM), with two pieces each at least.  At 33 to 64 rows a
        // CTA's sums take as long as its loads, and tiles are the shorter way once they fill the GPU (64 x 24576 x 1536
        // 15.9 us here, 12.3 by tiles; 64 x 8192 x 8192 19.4 and 21.6).
        const int cols = a.M <= 16 ? 16 : a.M <= 32 ? 32 : 64;
        const int64_t tiles = ((int64_t)a.N + 127) / 128;
        int split = 1;
        while (split < 8 && tiles * split <= sms && pieces >= 4 * split)
            split *= 2;
        return launch_gemm_fp8_split(a, cols, split, stream, err, errlen);
    }
    // Time of a tile kernel's call, us, from what a piece, an output and a cluster's sum were measured at: 128 x 704 x 4096 of
    // 128 columns takes 13.5 whole, 10.2 split in 4 and 8.8 in 8; 1024 x 4096 x 1024 10.7 with 128 columns and 9.1 with
    // 256; 8192 x 8192 x 8192 537 and 436.  Clusters of eight find room for two thirds of the SMs.
    int best_cols = 256, best_split = 1;
    float best = 1e30f;
    for (int cols = 128; cols <= 256; cols *= 2)
        for (int split = 1; split <= 8; split *= 2) {
            const int64_t ctas = (((int64_t)a.M + 127) / 128) * (((int64_t)a.N + cols - 1) / cols) * split;
            if (split > 1 && (ctas > (split == 8 ? sms * 2 / 3 : sms) || pieces < 2 * split))
                break;
            const float piece = cols == 128 ? (a.b_block ? 0.34f : 0.48f) : (a.b_block ? 0.48f : 0.87f);
            const float turn = piece * (float)((pieces + split - 1) / split) + (cols == 128 ? 0.7f : 1.2f);
            const float t = (float)((ctas + sms - 1) / sms) * turn + (split > 1 ? (cols == 128 ? 4.5f : 7.5f) : 0.f);
            if (t < best)
                best = t, best_cols = cols, best_split = split;
        }
    return launch_gemm_fp8_tile(a, best_cols, best_split, stream, err, errlen);
}

} // namespace dsa
