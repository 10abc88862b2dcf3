// Sums of per-CTA partial rows: the second step of the weight gradients of
// qk_rotate, head_gate, short_conv, ssm and block_norm.  Each CTA of the first kernel
// leaves one fp32 row; the order of the additions is fixed by the launch shape, so
// results repeat bit for bit (no atomics).
#include "rows.cuh"
#include "tc_ptx.cuh"
#include "trace.h"

namespace la {

namespace {

constexpr int kSumWarps = 32;

struct Sums {
    PartialSum of[kPartialSums];
};

// One CTA per 32 columns; warp w adds rows w, w + 32, ... of its lane's column.
__global__ void __launch_bounds__(kSumWarps * 32) partial_sum_kernel(const __grid_constant__ Sums s) {
    __shared__ float red[kSumWarps][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, which = blockIdx.y;
    const int c = blockIdx.x * 32 + lane;
    const float* part = s.of[which].part;
    float* out = s.of[which].out;
    const int rows = s.of[which].rows, cols = s.of[which].cols;
    if (!out || (int)blockIdx.x * 32 >= cols) return;
    tc::griddep_wait();  // the rows come from the previous kernel in the stream
    float acc = 0.f;
    if (c < cols) {
        constexpr int kBatch = 24;  // loads in flight together
        for (int r0 = w; r0 < rows; r0 += kBatch * kSumWarps) {
            float v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int r = r0 + i * kSumWarps;
                v[i] = r < rows ? part[(size_t)r * cols + c] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) acc += v[i];
        }
    }
    red[w][lane] = acc;
    __syncthreads();
    if (w == 0 && c < cols) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kSumWarps; ++i) sum += red[i][lane];
        out[c] = sum;
    }
}

}  // namespace

cudaError_t launch_partial_sums(const PartialSum* sums, int n, cudaStream_t s) {
    Sums all = {};
    int cols = 0, used = 0;
    for (int i = 0; i < n; ++i) {
        if (!sums[i].out) continue;
        all.of[used++] = sums[i];
        cols = sums[i].cols > cols ? sums[i].cols : cols;
    }
    if (used == 0) return cudaSuccess;
    TraceScope trace("partial_sum_kernel", s);
    cudaLaunchAttribute attr[1];  // scheduled while the kernel before it finishes
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((cols + 31) / 32, used);
    cfg.blockDim = dim3(kSumWarps * 32);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, partial_sum_kernel, all);
}

cudaError_t launch_partial_sum(const float* part0, int rows0, float* out0, const float* part1, int rows1,
                               float* out1, int cols, cudaStream_t s) {
    const PartialSum sums[2] = {{part0, out0, rows0, cols}, {part1, out1, rows1, cols}};
    return launch_partial_sums(sums, 2, s);
}

int sm_count() {
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms > 0 ? sms : 1;
}

}  // namespace la
