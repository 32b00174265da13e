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
// The rows' layout, ring and sums are the RMS norm's: every value is read and
// written once, so both are HBM-bound.  The variance is taken about the mean in a
// second pass over the values, which are in registers by then (the difference of
// the mean square and the squared mean would lose it where the mean is large);
// what the fp32 mean is off by is the mean of the differences, which the same pass
// sums and takes out (T. Chan, G. Golub, R. LeVeque, "Algorithms for computing the
// sample variance", 1983).
#include "norm_forward.cuh"

namespace dsa {

int launch_layernorm(const NormArgs &a, cudaStream_t stream, char *err, size_t errlen)
{
    return launch_norm<true>(a, "layernorm", stream, err, errlen);
}

} // namespace dsa
