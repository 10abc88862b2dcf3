// Helpers of the kernels that work on rows of one head (csrc/qk_rotate.cu,
// csrc/head_gate.cu): a row of d entries (a multiple of 16 up to 256) is held by
// a group of G lanes of one warp, eight entries a lane (G the power of two from
// d / 8 up; lanes past d / 8 hold zeros), so that its sums are log2 G shuffles.
// Rows come through a ring of slots in shared memory, filled in the background a few
// rows ahead by the group that reads them, so that the loads in flight cost no
// registers and the ring needs no barrier beyond the warp's own.
#pragma once

#include "launch.h"

namespace la {

// 16 bytes from global to shared memory in the background, or 16 zero bytes.
__device__ __forceinline__ void copy16(void* to, const void* from, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(to)),
                 "l"(from), "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A group copies a row into its slot of 8 G entries; what lies past d, and a row that is
// not there, arrives as zeros.
template <typename T, int G>
__device__ __forceinline__ void copy_row(T* slot, const T* row, int lane, int d, bool there) {
    constexpr int kElems = 16 / (int)sizeof(T);
#pragma unroll
    for (int j = 0; j < 8 / kElems; ++j) {
        const int e = (j * G + lane) * kElems;
        const bool valid = there && e < d;
        copy16(slot + e, valid ? row + e : row, valid);
    }
}

// Eight entries of a row: two pieces of four at offsets e1 and e2 (RUN: e2 = e1 + 4).
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
__device__ __forceinline__ Raw8<__nv_bfloat16> raw8(const __nv_bfloat16* row, int e1, int e2) {
    Raw8<__nv_bfloat16> r;
    if (RUN) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + e1);
        r.a = make_uint2(v.x, v.y);
        r.b = make_uint2(v.z, v.w);
    } else {
        r.a = *reinterpret_cast<const uint2*>(row + e1);
        r.b = *reinterpret_cast<const uint2*>(row + e2);
    }
    return r;
}

template <bool RUN>
__device__ __forceinline__ Raw8<float> raw8(const float* row, int e1, int e2) {
    Raw8<float> r;
    r.a = *reinterpret_cast<const float4*>(row + e1);
    r.b = *reinterpret_cast<const float4*>(row + e2);
    return r;
}

// The eight entries as fp32 pairs for the packed arithmetic (__ffma2_rn and the like:
// two operations an instruction): in memory order, or with PAIRS, for rotations of
// neighbours, the even entries first (x[0], x[1]), then the odd ones.
template <bool PAIRS>
__device__ __forceinline__ void floats8(const Raw8<__nv_bfloat16>& r, float2 (&x)[4]) {
    const uint32_t w[4] = {r.a.x, r.a.y, r.b.x, r.b.y};
    float lo[4], hi[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        lo[j] = __uint_as_float(w[j] << 16);
        hi[j] = __uint_as_float(w[j] & 0xffff0000u);
    }
    if (PAIRS) {
        x[0] = make_float2(lo[0], lo[1]);
        x[1] = make_float2(lo[2], lo[3]);
        x[2] = make_float2(hi[0], hi[1]);
        x[3] = make_float2(hi[2], hi[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = make_float2(lo[j], hi[j]);
    }
}

template <bool PAIRS>
__device__ __forceinline__ void floats8(const Raw8<float>& r, float2 (&x)[4]) {
    if (PAIRS) {
        x[0] = make_float2(r.a.x, r.a.z);
        x[1] = make_float2(r.b.x, r.b.z);
        x[2] = make_float2(r.a.y, r.a.w);
        x[3] = make_float2(r.b.y, r.b.w);
    } else {
        x[0] = make_float2(r.a.x, r.a.y);
        x[1] = make_float2(r.a.z, r.a.w);
        x[2] = make_float2(r.b.x, r.b.y);
        x[3] = make_float2(r.b.z, r.b.w);
    }
}

// One rounding to bf16, to nearest even, where the fp32 result is stored.
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <bool RUN, bool PAIRS>
__device__ __forceinline__ void store8(__nv_bfloat16* row, int e1, int e2, const float2 (&x)[4]) {
    uint32_t w[4];
    if (PAIRS) {
        w[0] = bf16x2_bits(x[0].x, x[2].x);
        w[1] = bf16x2_bits(x[0].y, x[2].y);
        w[2] = bf16x2_bits(x[1].x, x[3].x);
        w[3] = bf16x2_bits(x[1].y, x[3].y);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = bf16x2_bits(x[j].x, x[j].y);
    }
    if (RUN) {
        *reinterpret_cast<uint4*>(row + e1) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        *reinterpret_cast<uint2*>(row + e1) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(row + e2) = make_uint2(w[2], w[3]);
    }
}

template <bool RUN, bool PAIRS>
__device__ __forceinline__ void store8(float* row, int e1, int e2, const float2 (&x)[4]) {
    if (PAIRS) {
        *reinterpret_cast<float4*>(row + e1) = make_float4(x[0].x, x[2].x, x[0].y, x[2].y);
        *reinterpret_cast<float4*>(row + e2) = make_float4(x[1].x, x[3].x, x[1].y, x[3].y);
    } else {
        *reinterpret_cast<float4*>(row + e1) = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
        *reinterpret_cast<float4*>(row + e2) = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
    }
}

// Entry (0 .. 7, as stored: e1 .. e1 + 3, e2 .. e2 + 3) that x[j].x / x[j].y stands for.
template <bool PAIRS>
__device__ __forceinline__ int entry8(int j, int half) {
    return PAIRS ? (j & 1) * 4 + half * 2 + (j >> 1) : j * 2 + half;
}

// The lane's eight entries of an fp32 row (weights), ones for a null row.
template <bool PAIRS>
__device__ __forceinline__ void row_weights(const float* w, bool on, int e1, int e2, float2 (&x)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = make_float2(1.f, 1.f);
    if (w && on) {
        Raw8<float> r;
        r.a = __ldg(reinterpret_cast<const float4*>(w + e1));
        r.b = __ldg(reinterpret_cast<const float4*>(w + e2));
        floats8<PAIRS>(r, x);
    }
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// sum over the lane's eight entries of x y
__device__ __forceinline__ float dot8(const float2 (&x)[4], const float2 (&y)[4]) {
    float2 s = __fmul2_rn(x[0], y[0]);
#pragma unroll
    for (int j = 1; j < 4; ++j) s = __ffma2_rn(x[j], y[j], s);
    return s.x + s.y;
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// m / T by a multiplication, exact for m < 2^31.
struct Divide {
    unsigned T, magic, shift;  // magic = ceil(2^shift / T), shift = 31 + ceil(log2 T)

    static Divide by(int T) {
        unsigned log2T = 0;
        while ((1ull << log2T) < (unsigned long long)T) ++log2T;
        const unsigned shift = 31 + log2T;
        return {(unsigned)T, (unsigned)(((1ull << shift) + T - 1) / T), shift};
    }
    __device__ __forceinline__ void operator()(unsigned m, unsigned* quotient, unsigned* rest) const {
        *quotient = (unsigned)(((unsigned long long)m * magic) >> shift);
        *rest = m - *quotient * T;
    }
};

inline int group_lanes(int d) {  // the smallest power of two >= d / 8
    int g = 2;
    while (g * 8 < d) g *= 2;
    return g;
}

// rows.cu: out[c] = sum over the rows of part[rows][cols], in a fixed order, for up to
// two such pairs at once (a null out is left out).
cudaError_t launch_partial_sum(const float* part0, int rows0, float* out0, const float* part1, int rows1,
                               float* out1, int cols, cudaStream_t s);

// rows.cu: multiprocessors of the current device
int sm_count();

}  // namespace la
