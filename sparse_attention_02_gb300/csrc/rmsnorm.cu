// Residual addition, root-mean-square norm and FP8 output on sm_103a, and the
// norm's backward.
//
// The step in front of a layer's projections: the indexer's and the main
// attention's inputs are projections of the normalised hidden state, and the
// indexer runs in FP8 ("AMD Instinct MI355X GPUs Power DeepSeek-V3.2-Exp",
// section "DeepSeek Sparse Attention (DSA)", item 1).  For each row
//     h = x + residual (fp32),  r = 1 / sqrt(mean(h^2) + eps),  y = h r weight
// with h and y rounded once, to the tensors' type, and the FP8 codes taken from
// the fp32 y (scale = amax / 448 or its power of two, per row or per 128
// columns, as dsa_quantize_fp8).  Backward, with xhat = h r and g = dy weight:
//     dx = r (g - xhat mean(g xhat)) + dres,   dweight = sum over rows of dy xhat
//
// Both are HBM-bound: every value is read once and written once.  A group of G
// threads (a warp, or the CTA) owns a row; where rows are aligned thread g holds
// the 8-value chunks c G + g, so a warp's loads are 32 consecutive 16-byte words
// and 16 neighbouring lanes hold one 128-column FP8 block.  Where rows are long
// and many, persistent CTAs take them through a ring in shared memory that bulk
// copies fill while earlier rows are worked on: with the row's values and sums in
// registers, direct loads left an SM too few threads to keep HBM busy (8191 x 8192
// bf16 with residual and block codes: 141 us; backward: 166 us).  Sums are fp32,
// first within a thread, then by shuffles and shared memory, in an order that
// depends on sizes and alignment alone: results repeat bit for bit.
//
// Measured: 8191 x 8192 bf16, residual, both outputs, block codes 96 us (93 % of
// measured HBM); backward of 8192 x 8192 with dres 94 us (84 %: four streams, and
// 5 us of the dweight sum); one row of 4096 2.5 us, launch and one load's latency.
// At 8191 columns no row but every eighth starts at 16 bytes: 219 us for 9000 rows
// where 8192 columns take 107 (backward 147 and 80; fp32 240 and 214), bound by
// instructions: 2-byte loads and stores in every other row.
#include "norm_forward.cuh"

namespace dsa {

int launch_rmsnorm(const NormArgs &a, cudaStream_t stream, char *err, size_t errlen)
{
    return launch_norm<false>(a, "rmsnorm", stream, err, errlen);
}

} // namespace dsa
