// Sums of per-CTA partial rows: the second step of the weight gradients of
// qk_rotate, head_gate, short_conv, ssm and block_norm.  Each CTA of the first kernel
// leaves one fp32 row; the order of the additions is fixed by the launch shape, so
// results repeat bit for bit (no atomics).
#include "rows.cuh"
#include "tc_ptx.cuh"
#include "trace.h"

namespace la {

namespace {

// From kQuadColumns columns on a lane adds four: a quarter of the CTAs, of 1024 threads each (the scan's
// gradients, 64 to 256 rows: 65536 columns 15 us, one a lane 27; 32768 12 and 17; 16384 11 and 12: there and
// below the sums stay with one).
constexpr int kSumWarps = 32, kQuadColumns = 32768;

struct Sums {
    PartialSum of[kPartialSums];
};

__device__ __forceinline__ float plus(float a, float b) { return a + b; }
__device__ __forceinline__ float4 plus(float4 a, float4 b) {
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// One CTA per 32 columns (or 32 quads of them: V a float4, the same sums in the same order);
// warp w adds rows w, w + 32, ... of its lane's column.
template <typename V, int kBatch>
__global__ void __launch_bounds__(kSumWarps * 32) partial_sum_kernel(const __grid_constant__ Sums s) {
    __shared__ V red[kSumWarps][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, which = blockIdx.y;
    const int c = blockIdx.x * 32 + lane;
    const V* part = reinterpret_cast<const V*>(s.of[which].part);
    V* out = reinterpret_cast<V*>(s.of[which].out);
    const int rows = s.of[which].rows, cols = s.of[which].cols / (int)(sizeof(V) / sizeof(float));
    if (!out || (int)blockIdx.x * 32 >= cols) return;
    tc::griddep_wait();  // the rows come from the previous kernel in the stream
    V acc = {};
    if (c < cols) {
        for (int r0 = w; r0 < rows; r0 += kBatch * kSumWarps) {
            V v[kBatch];  // loads in flight together
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int r = r0 + i * kSumWarps;
                v[i] = V{};
                if (r < rows) v[i] = part[(size_t)r * cols + c];
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) acc = plus(acc, v[i]);
        }
    }
    red[w][lane] = acc;
    __syncthreads();
    if (w == 0 && c < cols) {
        V sum = {};
#pragma unroll
        for (int i = 0; i < kSumWarps; ++i) sum = plus(sum, red[i][lane]);
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
    // many columns: four a lane, a quarter of the CTAs
    const bool quads = cols >= kQuadColumns;
    cfg.gridDim = dim3(quads ? (cols / 4 + 31) / 32 : (cols + 31) / 32, used);
    cfg.blockDim = dim3(kSumWarps * 32);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return quads ? cudaLaunchKernelEx(&cfg, partial_sum_kernel<float4, 4>, all)
                 : cudaLaunchKernelEx(&cfg, partial_sum_kernel<float, 24>, all);
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
