// Backward of the RMS norm (the formulas stand in front of the norm).
#include "norm_backward.cuh"

namespace dsa {

size_t rmsnorm_backward_workspace_bytes(int64_t rows, int cols) { return norm_backward_workspace<false>(rows, cols); }

int launch_rmsnorm_backward(const NormBackwardArgs &a, cudaStream_t stream, char *err, size_t errlen)
{
    return launch_norm_backward<false>(a, "rmsnorm backward", stream, err, errlen);
}

} // namespace dsa
