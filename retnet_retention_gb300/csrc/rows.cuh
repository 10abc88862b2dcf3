// Helpers of the kernels that work on rows of one head (csrc/qk_rotate.cu,
// csrc/head_gate.cu): a row of d entries (a multiple of 16 up to 256) is held by
// a group of G lanes of one warp, eight entries a lane (G the power of two from
// d / 8 up; lanes past d / 8 hold zeros), so that its sums are log2 G shuffles.
#pragma once

#include "launch.h"

namespace la {

// Eight entries of a row as they lie in memory: two pieces of four at element
// offsets e1 and e2 (e2 = e1 + 4 where the lane's entries are one run).
template <typename T>
struct Raw8;

template <>
struct Raw8<__nv_bfloat16> {
    uint2 a, b;
};

template <>
struct Raw8<float> {
    float4 a, b;
};

template <bool RUN>
__device__ __forceinline__ Raw8<__nv_bfloat16> load_raw8(const __nv_bfloat16* row, int e1, int e2) {
    Raw8<__nv_bfloat16> r;
    if (RUN) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + e1));
        r.a = make_uint2(v.x, v.y);
        r.b = make_uint2(v.z, v.w);
    } else {
        r.a = __ldg(reinterpret_cast<const uint2*>(row + e1));
        r.b = __ldg(reinterpret_cast<const uint2*>(row + e2));
    }
    return r;
}

template <bool RUN>
__device__ __forceinline__ Raw8<float> load_raw8(const float* row, int e1, int e2) {
    Raw8<float> r;
    r.a = __ldg(reinterpret_cast<const float4*>(row + e1));
    r.b = __ldg(reinterpret_cast<const float4*>(row + e2));
    return r;
}

template <typename T>
__device__ __forceinline__ Raw8<T> zero_raw8() {
    Raw8<T> r;
    r.a = {};
    r.b = {};
    return r;
}

__device__ __forceinline__ void bf16x2_floats(uint32_t v, float* x) {
    x[0] = __uint_as_float(v << 16);
    x[1] = __uint_as_float(v & 0xffff0000u);
}

__device__ __forceinline__ void floats8(const Raw8<__nv_bfloat16>& r, float (&x)[8]) {
    bf16x2_floats(r.a.x, x);
    bf16x2_floats(r.a.y, x + 2);
    bf16x2_floats(r.b.x, x + 4);
    bf16x2_floats(r.b.y, x + 6);
}

__device__ __forceinline__ void floats8(const Raw8<float>& r, float (&x)[8]) {
    x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w;
    x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
}

// One rounding to bf16, to nearest even, where the fp32 result is stored.
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <bool RUN>
__device__ __forceinline__ void store8(__nv_bfloat16* row, int e1, int e2, const float (&x)[8]) {
    const uint2 a = make_uint2(bf16x2_bits(x[0], x[1]), bf16x2_bits(x[2], x[3]));
    const uint2 b = make_uint2(bf16x2_bits(x[4], x[5]), bf16x2_bits(x[6], x[7]));
    if (RUN) {
        *reinterpret_cast<uint4*>(row + e1) = make_uint4(a.x, a.y, b.x, b.y);
    } else {
        *reinterpret_cast<uint2*>(row + e1) = a;
        *reinterpret_cast<uint2*>(row + e2) = b;
    }
}

template <bool RUN>
__device__ __forceinline__ void store8(float* row, int e1, int e2, const float (&x)[8]) {
    *reinterpret_cast<float4*>(row + e1) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(row + e2) = make_float4(x[4], x[5], x[6], x[7]);
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

inline int group_lanes(int d) {  // the smallest power of two >= d / 8
    int g = 2;
    while (g * 8 < d) g *= 2;
    return g;
}

// rows.cu: the sums over the rows of part[rows][cols0 + cols1], in a fixed order; the
// first cols0 go to out0, the rest to out1 (a null output is left out).
cudaError_t launch_partial_sum(const float* part, int rows, float* out0, int cols0, float* out1,
                               int cols1, cudaStream_t s);

// rows.cu: multiprocessors of the current device
int sm_count();

}  // namespace la
