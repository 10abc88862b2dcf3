// The selective scan's walks over bf16 tensors.
#include "ssm.cuh"

namespace la::ssm {

template <>
cudaError_t launch_scan<__nv_bfloat16, kForward>(const SsmParams& p, Split split, unsigned grid, cudaStream_t s) {
    return launch_scan_here<__nv_bfloat16, kForward>(p, split, grid, s);
}
template <>
cudaError_t launch_scan<__nv_bfloat16, kState>(const SsmParams& p, Split split, unsigned grid, cudaStream_t s) {
    return launch_scan_here<__nv_bfloat16, kState>(p, split, grid, s);
}
template <>
cudaError_t launch_scan<__nv_bfloat16, kSummary>(const SsmParams& p, Split split, unsigned grid, cudaStream_t s) {
    return launch_scan_here<__nv_bfloat16, kSummary>(p, split, grid, s);
}

}  // namespace la::ssm
