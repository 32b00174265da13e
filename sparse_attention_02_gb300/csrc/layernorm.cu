// Layer norm with residual addition and FP8 output on sm_103a.
//
// The norm of the indexer's keys, between their projection and the rotation and
// FP8 codes of the cache append ("AMD Instinct MI355X GPUs Power DeepSeek-V3.2-
// Exp", section "DeepSeek Sparse Attention (DSA)", item 1), and of any hidden
// state.  For each row
//     h = x + residual,  mean = mean_c(h),  var = mean_c((h - mean)^2),
//     xhat = (h - mean) / sqrt(var + eps),  y = xhat weight + bias
// and backward, with g = dy weight and r = 1 / sqrt(var + eps),
//     dx = r (g - mean_c(g) - xhat mean_c(g xhat)) + dres
//     dweight = sum over rows of dy xhat,   dbias = sum over rows of dy
// The rows' layout and ring are the RMS norm's: every value is read and written once,
// so both are HBM-bound.  The variance is taken about the mean, from values that are
// in registers by then (the difference of the mean square and the squared mean would
// lose it where the mean is large); a row's warps meet once, each with sums about its
// own mean (rmsnorm.cuh).  Weight and bias stay in registers in the ring's kernels:
// beside a ring an SM's L1 does not hold both (8191 x 8192 with residual, both outputs
// and block codes 127 us when each row read them again, 111 so).
//
// An SM has a row of 8192 columns at work at a time, so that a row's instructions are
// what bytes wait for: arithmetic goes in pairs, counts are divided by once a call
// (Count), the root costs a Newton step (inv_sqrt), what lies past the columns is kept out
// by a chunk's offset instead of a choice a value, and the ring's threads meet once a row
// instead of three times (all of that 111 -> 99 us, and backward 116 -> 96).
//
// Measured: 8191 x 8192 bf16, residual, both outputs, block codes 99 us (90 % of
// measured HBM; the RMS norm 96); without residual and codes 46 (86 %).  64 x 128 3.1 us.
// Rows off 16 bytes are bound by 2-byte accesses: 9000 x 8191 100 us without and 145 with
// residual (43 and 60 %), 253 with block codes too (39 %).
// Backward of 8192 x 8192 with dres 96 us (82 %): its two sums a column leave room for
// one CTA of 512 threads an SM, and what a row's meeting takes is not hidden by another's.
// Beyond 8192 columns four chunks a thread and their sums do not fit its 128 registers, and
// spill: 2048 x 16384 102 us bf16 (39 %), 184 fp32 (43 %).
// Not kept there: two rows at once (146, spills), more stages (118 of 116 then), dres read before
// the meeting for the ring's single one (115, but 16384 x 2048 56 -> 60: registers).
// 32767 x 128 fp32 backward 13.5 us (4 to 5 of them the sums' own launch), two rows a
// warp, whose half-warps add up two quantities at once; 24.5 with one row a warp and as many
// CTAs as the RMS norm.
#include "norm_forward.cuh"

namespace dsa {

int launch_layernorm(const NormArgs &a, cudaStream_t stream, char *err, size_t errlen)
{
    return launch_norm<true>(a, "layernorm", stream, err, errlen);
}

} // namespace dsa
