// The selective scan's gradients over bf16 tensors.
#include "ssm_bwd.cuh"

namespace la::ssm {

template <>
cudaError_t launch_gradients<__nv_bfloat16>(const SsmBwdParams& p, unsigned grid, cudaStream_t s) {
    return launch_gradients_here<__nv_bfloat16>(p, grid, s);
}

}  // namespace la::ssm
