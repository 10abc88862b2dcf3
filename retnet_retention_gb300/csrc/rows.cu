// Sums of per-CTA partial rows: the second step of the weight gradients of
// qk_rotate and head_gate.  Each CTA of the first kernel leaves one fp32 row; the
// order of the additions is fixed by the launch shape, so results repeat bit for
// bit (no atomics).
#include "rows.cuh"
#include "trace.h"

namespace la {

namespace {

constexpr int kSumWarps = 16;

// One CTA per 32 columns; warp w adds rows w, w + 16, ... of its lane's column.
__global__ void __launch_bounds__(kSumWarps * 32) partial_sum_kernel(const float* __restrict__ part,
                                                                     int rows, float* out0,
                                                                     int cols0, float* out1,
                                                                     int cols) {
    __shared__ float red[kSumWarps][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float acc = 0.f;
    if (c < cols) {
#pragma unroll 8
        for (int r = w; r < rows; r += kSumWarps) acc += part[(size_t)r * cols + c];
    }
    red[w][lane] = acc;
    __syncthreads();
    if (w == 0 && c < cols) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kSumWarps; ++i) sum += red[i][lane];
        if (c < cols0) {
            if (out0) out0[c] = sum;
        } else if (out1) {
            out1[c - cols0] = sum;
        }
    }
}

}  // namespace

cudaError_t launch_partial_sum(const float* part, int rows, float* out0, int cols0, float* out1,
                               int cols1, cudaStream_t s) {
    const int cols = cols0 + cols1;
    TraceScope trace("partial_sum_kernel", s);
    partial_sum_kernel<<<(cols + 31) / 32, kSumWarps * 32, 0, s>>>(part, rows, out0, cols0, out1,
                                                                   cols);
    return cudaGetLastError();
}

int sm_count() {
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms > 0 ? sms : 1;
}

}  // namespace la
