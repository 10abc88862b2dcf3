// The gradients of the selective scan, chunk by chunk.  With du = dy gate sigmoid(gate),
// u = c_t . h_t + skip x and e_t = exp(delta_t A), walking backward from the gradient of
// the state that leaves the chunk:
//
//   g_t = c_t du_t + e_(t+1) g_(t+1)
//   s = sum_n g b,  q = (e_t g_t) h_(t-1),  r = sum_n q A
//   dx = delta s + skip du,  ddt = (x s + r) softplus'(dt + dt_bias),  dgate = dy u silu'(gate)
//   dA = sum_t q delta,  db_n = sum over channels g delta x,  dc_n = sum over channels du h_t
//
// The walk over a chunk's blocks of kBlock tokens goes backward; a block's states are
// computed again from the state before it (the local one the summary walk left, plus what
// the chunk's entering state has become) and kept in registers while the block is walked
// backward.
//
// A lane holds four states of two channels.  Sums over n cross L = N / 4 lanes, sums over
// channels (for db, dc) the other 32 / L: both give away half of what they hold at each
// step.  Which state a register holds is turned with the lane (n = 4 j + (i ^ turn)), and
// which channel, so that the halves to keep and to give have fixed registers.
#pragma once

#include "ssm.cuh"

namespace la {
namespace ssm {

constexpr int kBwdWarps = 4;

template <typename T, int N>
struct BwdShape {
    static constexpr int L = N / 4, CL = 32 / L, CW = 2 * CL;  // lanes of a channel, pairs and channels of a warp
    static constexpr int kTurns = CL < 4 ? CL : 4;             // ways the four states are turned
    static constexpr int M = L / 2, K = kBlock / M;            // own tokens: every M-th, K of a block
    static constexpr int kThreads = kBwdWarps * 32;
};

template <typename T, int N>
__global__ void __launch_bounds__(kBwdWarps * 32) ssm_gradients_kernel(const __grid_constant__ SsmBwdParams bp) {
    using S = BwdShape<T, N>;
    constexpr int CL = S::CL, U = kBlock, M = S::M, K = S::K;
    constexpr int kColumns = N == 64 ? 1 : 2;  // 48 KB of shared memory hold one set of N = 64
    const SsmParams& p = bp.f;
    tc::griddep_launch_dependents();
    __shared__ __align__(16) float bc[2][S::kTurns][U][2 * N];
    __shared__ __align__(16) float4 vals[kBwdWarps][U][S::CW];  // delta, delta x, du of a token and channel
    __shared__ float columns[kColumns][kBwdWarps][U][2 * N];
    __shared__ unsigned starts[2];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, j = lane / CL, cl = lane % CL;
    unsigned unit = blockIdx.x;
    const unsigned tile = unit % (unsigned)(p.tiles * p.G);
    unit /= (unsigned)(p.tiles * p.G);
    const int chunk = (int)(unit % (unsigned)p.chunks);
    const long long b = unit / (unsigned)p.chunks;
    const int g_at = (int)(tile / (unsigned)p.tiles);
    const int first = (int)(tile % (unsigned)p.tiles) * (kBwdWarps * S::CW) + w * S::CW;
    const int turn = cl & (S::kTurns - 1);
    // register q of two: channel 2 cl + (q ^ (j & 1)), so that register 0 is the lane's own
    int c[2];
    bool on[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int in_group = first + 2 * cl + (q ^ (j & 1));
        on[q] = in_group < p.channels;
        c[q] = g_at * p.channels + (on[q] ? in_group : 0);
    }
    const int t0 = chunk * p.chunk, t1 = (int)min((long long)t0 + p.chunk, (long long)p.T);
    float A[2][4], hin[2][4], g[2][4], dA[2][4];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const long long at = ((b * p.chunks + chunk) * p.D + c[q]) * N;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = 4 * j + (i ^ turn);
            A[q][i] = on[q] ? __ldg(p.A + (size_t)c[q] * N + n) * kLog2e : 0.f;
            hin[q][i] = on[q] ? p.chunk_h[at + n] : 0.f;
            g[q][i] = on[q] ? p.chunk_g[at + n] : 0.f;
            dA[q][i] = 0.f;
        }
    }
    const float skip = p.skip ? p.skip[c[0]] : 0.f, bias = p.bias ? p.bias[c[0]] : 0.f;
    float dskip = 0.f, dbias = 0.f;
    const bool gated = p.gate.p != nullptr;

    // own tokens of a block: t + k M + (j >> 1), own channel c[0]
    const int own = j >> 1;
    const T* x_at = (const T*)p.x.p + b * p.x.b + c[0];
    const T* dt_at = (const T*)p.dt.p + b * p.dt.b + c[0];
    const T* gate_at = gated ? (const T*)p.gate.p + b * p.gate.b + c[0] : nullptr;
    const T* dy_at = (const T*)p.dy.p + b * p.dy.b + c[0];
    T* dx_at = (T*)bp.dx.p + b * bp.dx.b + c[0];
    T* ddt_at = (T*)bp.ddt.p + b * bp.ddt.b + c[0];
    T* dgate_at = gated ? (T*)bp.dgate.p + b * bp.dgate.b + c[0] : nullptr;
    T nx[K] = {}, ndt[K] = {}, ngate[K] = {}, ndy[K] = {};
    float nh[2][4], ns[2];  // the next block's local state and sum of delta
    SharedRows<T, N, S::kThreads, U> rows;
    int position = 1;
    auto fetch = [&](int t) {
        if (t < t0) return;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int at = t + k * M + own;
            if (on[0] && at < t1) {
                nx[k] = x_at[at * p.x.t];
                ndt[k] = dt_at[at * p.dt.t];
                if (gated) ngate[k] = gate_at[at * p.gate.t];
                ndy[k] = dy_at[at * p.dy.t];
            }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const long long at = (b * p.blocks + t / U) * p.D + c[q];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                nh[q][i] = on[q] && t > t0 ? p.block_h[at * N + 4 * j + (i ^ turn)] : 0.f;
            ns[q] = on[q] && t > t0 ? p.block_s[at] : 0.f;
        }
        rows.load(p, b, g_at, t, t1);
        if (p.positions && w == 0) position = lane < U && t + lane < t1 ? p.positions[b * p.T + t + lane] : 1;
    };
    // b and c of a block into shared memory, once for each turn: entry i of a group of
    // four is entry i ^ turn
    auto store_rows = [&](int buf) {
#pragma unroll
        for (int i = 0; i < decltype(rows)::kEach; ++i) {
            const int q = i * S::kThreads + threadIdx.x;
            if (q < decltype(rows)::kPieces) {
                float2 v[4];
                floats8<false>(rows.raw[i], v);
#pragma unroll
                for (int k = 0; k < S::kTurns; ++k) {
                    float* to = &bc[buf][k][0][0] + q * 8;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const float f[4] = {v[2 * half].x, v[2 * half].y, v[2 * half + 1].x, v[2 * half + 1].y};
                        *reinterpret_cast<float4*>(to + 4 * half) = make_float4(f[0 ^ k], f[1 ^ k], f[2 ^ k], f[3 ^ k]);
                    }
                }
            }
        }
        if (w == 0) {
            const unsigned m = __ballot_sync(0xffffffffu, position == 0);
            if (lane == 0) starts[buf] = m;
        }
    };
    // the warps' sums over channels of the block at t
    auto add_up = [&](int t, int from) {
        for (int i = threadIdx.x; i < U * 2 * N; i += S::kThreads) {
            const int tok = i / (2 * N), col = i % (2 * N);
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < kBwdWarps; ++k) v += columns[from % kColumns][k][tok][col];
            if (t + tok < t1) bp.part_bc[(((long long)tile * p.B + b) * p.T + t + tok) * (2 * N) + col] = v;
        }
    };
    const int last = t0 + (t1 - t0 - 1) / U * U;
    fetch(last);
    int buf = 0;
    for (int t = last; t >= t0; t -= U, buf ^= 1) {
        // the block's own elementwise values
        float xs[K], d[K], du[K], f_gate[K], slope[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const bool there = on[0] && t + k * M + own < t1;
            xs[k] = there ? load_elem(nx, k) : 0.f;
            const float v = load_elem(ndt, k) + bias;
            d[k] = there ? (p.softplus ? softplus<T>(v) : v) : 0.f;
            slope[k] = there ? (p.softplus ? sigmoid<T>(v) : 1.f) : 0.f;
            du[k] = there ? load_elem(ndy, k) : 0.f;
            f_gate[k] = 0.f;
            if (gated) {
                const float z = there ? load_elem(ngate, k) : 0.f, s = sigmoid<T>(z), a = z * s;
                f_gate[k] = du[k] * fmaf(a, 1.f - s, s);
                du[k] *= a;
            }
            vals[w][k * M + own][2 * cl + (j & 1)] = make_float4(d[k], d[k] * xs[k], du[k], 0.f);
        }
        store_rows(buf);
        // states entering the block: the local one and the chunk's entering one, decayed
        float hs[U + 1][2][4];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                hs[0][q][i] = ns[q] == INFINITY ? nh[q][i] : fmaf(exp2_fast(ns[q] * A[q][i]), hin[q][i], nh[q][i]);
        fetch(t - U);
        __syncthreads();
        if (t != last) {
            add_up(t + U, buf ^ 1);  // of the block before this one
            if (kColumns == 1) __syncthreads();
        }
        const unsigned block_starts = starts[buf];
        const int c0 = 2 * cl + (j & 1), c1 = 2 * cl + (1 ^ (j & 1));
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float bv[4];
            *reinterpret_cast<float4*>(bv) = *reinterpret_cast<const float4*>(&bc[buf][turn][u][4 * j]);
            const float2 v0 = *reinterpret_cast<const float2*>(&vals[w][u][c0]);
            const float2 v1 = *reinterpret_cast<const float2*>(&vals[w][u][c1]);
            const bool start = block_starts >> u & 1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float i0 = v0.y * bv[i], i1 = v1.y * bv[i];
                hs[u + 1][0][i] = start ? i0 : fmaf(exp2_fast(v0.x * A[0][i]), hs[u][0][i], i0);
                hs[u + 1][1][i] = start ? i1 : fmaf(exp2_fast(v1.x * A[1][i]), hs[u][1][i], i1);
            }
        }
        float sv[U], rv[U], uv[U];
#pragma unroll
        for (int u = U - 1; u >= 0; --u) {
            float bv[4], cv[4], db[4], dc[4];
            *reinterpret_cast<float4*>(bv) = *reinterpret_cast<const float4*>(&bc[buf][turn][u][4 * j]);
            *reinterpret_cast<float4*>(cv) = *reinterpret_cast<const float4*>(&bc[buf][turn][u][N + 4 * j]);
            const float4 val[2] = {vals[w][u][c0], vals[w][u][c1]};
            const bool start = block_starts >> u & 1;
            float s[2] = {0.f, 0.f}, r[2] = {0.f, 0.f}, y[2] = {0.f, 0.f};
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float h = hs[u + 1][q][i];
                    g[q][i] = fmaf(cv[i], val[q].z, g[q][i]);
                    s[q] = fmaf(g[q][i], bv[i], s[q]);
                    y[q] = fmaf(cv[i], h, y[q]);
                    db[i] = q == 0 ? g[q][i] * val[q].y : fmaf(g[q][i], val[q].y, db[i]);
                    dc[i] = q == 0 ? h * val[q].z : fmaf(h, val[q].z, dc[i]);
                    g[q][i] = start ? 0.f : g[q][i] * exp2_fast(val[q].x * A[q][i]);
                    const float qq = start ? 0.f : g[q][i] * hs[u][q][i];
                    r[q] = fmaf(qq, A[q][i], r[q]);
                    dA[q][i] = fmaf(qq, val[q].x, dA[q][i]);
                }
            // over n: the own channel's register is kept
            sv[u] = s[0] + __shfl_xor_sync(0xffffffffu, s[1], CL);
            rv[u] = r[0] + __shfl_xor_sync(0xffffffffu, r[1], CL);
            uv[u] = y[0] + __shfl_xor_sync(0xffffffffu, y[1], CL);
            // over channels
            if (CL >= 4) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    db[i] += __shfl_xor_sync(0xffffffffu, db[i + 2], 2);
                    dc[i] += __shfl_xor_sync(0xffffffffu, dc[i + 2], 2);
                }
            }
#pragma unroll
            for (int i = 0; i < (CL >= 4 ? 1 : 3); i += 2) {
                db[i] += __shfl_xor_sync(0xffffffffu, db[i + 1], 1);
                dc[i] += __shfl_xor_sync(0xffffffffu, dc[i + 1], 1);
            }
#pragma unroll
            for (int gap = 4; gap < CL; gap *= 2) {
                db[0] += __shfl_xor_sync(0xffffffffu, db[0], gap);
                dc[0] += __shfl_xor_sync(0xffffffffu, dc[0], gap);
            }
            float* to = &columns[buf % kColumns][w][u][4 * j];
            if (CL >= 4) {
                if (CL == 4 || cl < 4) to[turn] = db[0];
                if (CL == 4 || (cl >= 4 && cl < 8)) to[N + turn] = dc[0];
            } else {
                to[turn] = db[0];
                to[2 + turn] = db[2];
                to[N + turn] = dc[0];
                to[N + 2 + turn] = dc[2];
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float s[M], r[M], y[M];
#pragma unroll
            for (int i = 0; i < M; ++i) s[i] = sv[k * M + i], r[i] = rv[k * M + i], y[i] = uv[k * M + i];
            const float into = share_sums<M>(s, own, 2 * CL), along = share_sums<M>(r, own, 2 * CL);
            const float u = fmaf(skip, xs[k], share_sums<M>(y, own, 2 * CL));
            const int at = t + k * M + own;
            if (on[0] && at < t1) {
                constexpr float kLn2 = 0.69314718055994531f;  // A holds log2 e
                const float ddt = fmaf(xs[k], into, along * kLn2) * slope[k];
                store_elem(dx_at + at * bp.dx.t, 0, fmaf(d[k], into, skip * du[k]));
                store_elem(ddt_at + at * bp.ddt.t, 0, ddt);
                if (gated) store_elem(dgate_at + at * bp.dgate.t, 0, f_gate[k] * u);
                dskip = fmaf(du[k], xs[k], dskip);
                dbias += ddt;
            }
        }
    }
    __syncthreads();
    add_up(t0, buf ^ 1);
    const long long part = b * p.chunks + chunk;
#pragma unroll
    for (int q = 0; q < 2; ++q)
        if (on[q]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = 4 * j + (i ^ turn);
                if (bp.part_A) bp.part_A[(part * p.D + c[q]) * N + n] = dA[q][i];
                if (bp.dh0 && chunk == 0) bp.dh0[(b * p.D + c[q]) * N + n] = g[q][i];
            }
        }
#pragma unroll
    for (int gap = 1; gap < M; gap *= 2) {
        dskip += __shfl_xor_sync(0xffffffffu, dskip, gap * 2 * CL);
        dbias += __shfl_xor_sync(0xffffffffu, dbias, gap * 2 * CL);
    }
    if (on[0] && own == 0) {
        if (bp.part_skip) bp.part_skip[part * p.D + c[0]] = dskip;
        if (bp.part_bias) bp.part_bias[part * p.D + c[0]] = dbias;
    }
}



template <typename T>
cudaError_t launch_gradients_here(const SsmBwdParams& p, unsigned grid, cudaStream_t s) {
    TraceScope trace("ssm_gradients_kernel", s);
    const int threads = kBwdWarps * 32;
    switch (p.f.N) {
        case 8: ssm_gradients_kernel<T, 8><<<grid, threads, 0, s>>>(p); break;
        case 16: ssm_gradients_kernel<T, 16><<<grid, threads, 0, s>>>(p); break;
        case 32: ssm_gradients_kernel<T, 32><<<grid, threads, 0, s>>>(p); break;
        default: ssm_gradients_kernel<T, 64><<<grid, threads, 0, s>>>(p); break;
    }
    return cudaGetLastError();
}

}  // namespace ssm
}  // namespace la
