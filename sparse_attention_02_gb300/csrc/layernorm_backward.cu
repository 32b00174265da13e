// Backward of layer norm (the formulas stand in front of the norm).
#include "norm_backward.cuh"

namespace dsa {

size_t layernorm_backward_workspace_bytes(int64_t rows, int cols) { return norm_backward_workspace<true>(rows, cols); }

int launch_layernorm_backward(const NormBackwardArgs &a, cudaStream_t stream, char *err, size_t errlen)
{
    return launch_norm_backward<true>(a, "layernorm backward", stream, err, errlen);
}

} // namespace dsa
