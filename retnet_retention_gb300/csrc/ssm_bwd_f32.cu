// The selective scan's gradients over fp32 tensors.
#include "ssm_bwd.cuh"

namespace la::ssm {

template <>
cudaError_t launch_gradients<float>(const SsmBwdParams& p, unsigned grid, cudaStream_t s) {
    return launch_gradients_here<float>(p, grid, s);
}

}  // namespace la::ssm
