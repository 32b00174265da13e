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
        // Clusters of four or eight leave some of that room: 304 CTAs in clusters of eight take two turns (1 x 4864 x 4096 10.8
        // us, in fours 7.1), 288 do not.
        int split = 1;
        while (split < 8 && 2 * tiles * split <= (split == 1 ? 2 * sms : sms * 9 / 5) && pieces >= 4 * split)
            split *= 2;
        return launch_gemm_fp8_split(a, cols, split, stream, err, errlen);
    }
    // By tiles: the widths of a tile and the splits of K by the time that they take, in us, from what a piece, a tile's
    // output and a cluster's sum were measured at (128 x 704 x 4096 bf16: 13.1 by tiles of 128, 14.9 of 192, 7.9 with K split
    // in 8; 4096 x 704 x 4096 25.0, 16.7 and, of 256, 19.5; 2048 x 2048 x 2048 15.1, 17.6, 12.3; 8191 x 8192 x 8192 534,
    // 458, 422).  Clusters of eight found room for 120 CTAs at once, of four for 144: a margin below, as another turn costs
    // twice the time (128 x 4632 x 1689 in 148 CTAs 20.9 us, without the split 12.4).  What is worth a split is too small for
    // tiles of 256.
    struct Width {
        int cols;
        float piece, rows_piece, out, join; // rows_piece: with a scale for every row of b; join: of a split
    };
    constexpr Width widths[] = {{128, 0.32f, 0.44f, 1.0f, 4.0f}, {192, 0.38f, 0.505f, 1.6f, 4.6f}, {256, 0.455f, 0.f, 2.4f, 0.f}};
    int best_cols = 0, best_split = 1;
    float best = 0.f;
    for (const Width &w : widths) {
        if (!a.b_block && w.cols == 256) // a multiply more a sum: more registers than its threads have
            continue;
        for (int split = 1; split <= 8; split *= 2) {
            const int64_t ctas = (((int64_t)a.M + 127) / 128) * (((int64_t)a.N + w.cols - 1) / w.cols) * split;
            const int room = split == 8 ? sms * 3 / 4 : split == 4 ? sms * 9 / 10 : sms;
            if (split > 1 && (w.cols == 256 || ctas > room || pieces < 2 * split))
                break;
            const float turn = (a.b_block ? w.piece : w.rows_piece) * (float)((pieces + split - 1) / split) + w.out * (a.o32 ? 2.f : 1.f);
            const float t = (float)((ctas + sms - 1) / sms) * turn + (split > 1 ? w.join : 0.f);
            if (!best_cols || t < best)
                best = t, best_cols = w.cols, best_split = split;
        }
    }
    return launch_gemm_fp8_tile(a, best_cols, best_split, stream, err, errlen);
}

} // namespace dsa
