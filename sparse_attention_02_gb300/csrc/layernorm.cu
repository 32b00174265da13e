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
// Measured: 8191 x 8192 bf16, residual, both outputs, block codes 111 us (81 % of
// measured HBM; the RMS norm 96).  64 x 128 3.2 us.  Backward of 8192 x 8192 with dres
// 117 us (68 %): its two sums a column leave room for one CTA of 512 threads an SM, and
// what a row's instructions (2200 cycles' issue) and its meeting take is not hidden by
// another's.  Not kept: two rows at once there (146, spills), more stages (118).
// 32767 x 128 fp32 backward 14.5 us (7 of them the dweight sum's own launch), two rows a
// warp; 24.5 with one row a warp and as many CTAs as the RMS norm.
#include "norm_forward.cuh"

namespace dsa {

int launch_layernorm(const NormArgs &a, cudaStream_t stream, char *err, size_t errlen)
{
    return launch_norm<true>(a, "layernorm", stream, err, errlen);
}

} // namespace dsa
