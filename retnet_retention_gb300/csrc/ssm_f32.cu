// The selective scan's walks over fp32 tensors.
#include "ssm.cuh"

namespace la::ssm {

template <>
cudaError_t launch_scan<float, kForward>(const SsmParams& p, Split split, unsigned grid, cudaStream_t s) {
    return launch_scan_here<float, kForward>(p, split, grid, s);
}
template <>
cudaError_t launch_scan<float, kState>(const SsmParams& p, Split split, unsigned grid, cudaStream_t s) {
    return launch_scan_here<float, kState>(p, split, grid, s);
}
template <>
cudaError_t launch_scan<float, kSummary>(const SsmParams& p, Split split, unsigned grid, cudaStream_t s) {
    return launch_scan_here<float, kSummary>(p, split, grid, s);
}

}  // namespace la::ssm
