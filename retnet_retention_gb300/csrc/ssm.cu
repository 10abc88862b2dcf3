// The selective scan: a state of N numbers for each of D channels,
//
//   delta = softplus(dt + dt_bias),  h_t = exp(delta A) h_(t-1) + delta x b_t,
//   y_t = (c_t . h_t + skip x) gate sigmoid(gate),
//
// with A [D][N], and b_t, c_t [N] shared by a group's channels; its gradients
// (csrc/ssm_bwd.cuh) and its single step.  A document's first token (positions = 0) drops
// the old state by a selection.
//
// Bound by the instructions of the state: for each of its entries and tokens one 2^x and four
// fp32 operations (delta A, delta x b, h, c h); x, dt, gate and y are 8 bytes (bf16) for N of
// them.  A walk goes token by token with the state in registers (csrc/ssm.cuh).  Where the
// channels are too few for the card a sequence is cut into chunks: one walk leaves each
// chunk's state from zero and its sum of delta (the decay over a chunk is exp(A sum)), a
// small kernel puts them together, and a second walk writes y from the state entering each
// chunk.  The gradients always work chunk by chunk.
#include <algorithm>
#include <climits>

#include "ssm.cuh"

namespace la {

namespace ssm {

namespace {

// ---- the chunks of a sequence put together ---------------------------------------------

constexpr int kJoinWarps = 16;

// A run of chunks: the sum of its delta (infinity: a document starts in it, what enters is
// dropped) and the state it reaches from zero.
struct Run4 {
    float4 b;
    float sum;
};

// v[b][chunk][D][N]: what a chunk adds becomes what enters it, in place; from the first
// chunk with s0 before it, or from the last with s0 behind it.  A CTA per 128 columns of [D][N] of
// a sequence, four a lane (of one channel); each warp puts a run of chunks together, then walks
// them again.  Chunks come in batches whose loads are in flight together (a store in between
// would hold the next one's back).
__global__ void __launch_bounds__(kJoinWarps * 32) ssm_join_kernel(
    float* forward, const float* forward_s0, float* backward, const float* backward_s0, const float* chunk_s,
    const float* __restrict__ A, int D, int N, int chunks) {
    __shared__ Run4 runs[kJoinWarps][32];
    const bool back = forward == nullptr || blockIdx.z == 1;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const long long quad = (long long)blockIdx.x * 32 + lane, quads = (long long)D * N / 4, b = blockIdx.y;
    float4* const v = reinterpret_cast<float4*>(back ? backward : forward);
    const float4* const s0 = reinterpret_cast<const float4*>(back ? backward_s0 : forward_s0);
    const int d = (int)(quad * 4 / N);
    const float4 a = __ldg(reinterpret_cast<const float4*>(A) + quad);
    const int each = (chunks + warps - 1) / warps;
    const int k0 = min(w * each, chunks), k1 = min(k0 + each, chunks);
    auto at = [&](int k) { return b * chunks + (back ? chunks - 1 - k : k); };
    constexpr int kBatch = 4;
    float sum[kBatch];
    float4 add[kBatch];
    auto load = [&](int k) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            sum[i] = 0.f, add[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k + i < k1) {
                sum[i] = chunk_s[at(k + i) * D + d] * kLog2e;
                add[i] = v[at(k + i) * quads + quad];
            }
        }
    };
    // The state behind a chunk or run from s.  A decay that underflows drops nothing: what is not a number
    // stays so, as in an uncut walk.
    auto step = [&](float d_sum, const float4& b4, const float4& s) {
        if (d_sum == INFINITY) return b4;
        return make_float4(carry(d_sum * a.x, s.x, b4.x), carry(d_sum * a.y, s.y, b4.y), carry(d_sum * a.z, s.z, b4.z),
                           carry(d_sum * a.w, s.w, b4.w));
    };
    load(k0);
    float4 s = s0 ? s0[b * quads + quad] : make_float4(0.f, 0.f, 0.f, 0.f);
    if (warps > 1) {
        Run4 run = {make_float4(0.f, 0.f, 0.f, 0.f), 0.f};
        for (int k = k0; k < k1; k += kBatch) {
            if (k > k0) load(k);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                run.b = step(sum[i], add[i], run.b);
                run.sum = run.sum == INFINITY || sum[i] == INFINITY ? INFINITY : run.sum + sum[i];  // NaN too ends there
            }
        }
        runs[w][lane] = run;
        __syncthreads();
        for (int k = 0; k < w; ++k) s = step(runs[k][lane].sum, runs[k][lane].b, s);
    }
    for (int k = k0; k < k1; k += kBatch) {
        if (k > k0 || k1 - k0 > kBatch) load(k);
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (k + i < k1) {
                v[at(k + i) * quads + quad] = s;
                s = step(sum[i], add[i], s);
            }
    }
}

// ---- db, dc from the tiles' sums -------------------------------------------------------

template <typename T>
__global__ void __launch_bounds__(256) ssm_shared_grad_kernel(const float* part, long long tokens, int T_, int N,
                                                              int tiles, SsmRows db, SsmRows dc) {
    const int g = blockIdx.y;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;  // of [tokens][2 N / 4]
    const int quads = 2 * N / 4;
    if (i >= tokens * quads) return;
    const long long m = i / quads, b = m / T_, t = m - b * T_;
    const int col = (int)(i % quads) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < tiles; ++k) {
        const float4 r = *reinterpret_cast<const float4*>(part + (((long long)g * tiles + k) * tokens + m) * (2 * N) + col);
        v.x += r.x; v.y += r.y; v.z += r.z; v.w += r.w;
    }
    const SsmRows& to = col >= N ? dc : db;
    T* out = (T*)to.p + b * to.b + t * to.t + g * N + col % N;
    store_elem(out, 0, v.x);
    store_elem(out, 1, v.y);
    store_elem(out, 2, v.z);
    store_elem(out, 3, v.w);
}

// ---- one token -------------------------------------------------------------------------

__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
    *reinterpret_cast<float4*>(v) = __ldg(reinterpret_cast<const float4*>(p));
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&v)[4]) {
    const uint2 r = __ldg(reinterpret_cast<const uint2*>(p));
    v[0] = __uint_as_float(r.x << 16);
    v[1] = __uint_as_float(r.x & 0xffff0000u);
    v[2] = __uint_as_float(r.y << 16);
    v[3] = __uint_as_float(r.y & 0xffff0000u);
}

// Four states a lane: a channel's L = N / 4 lanes lie side by side; a CTA keeps its channels and
// walks sequences, four at a time, so that A is read once.  The elementwise work of a sequence's
// channel is one lane's, as in the walk over tokens.
template <typename T, int N>
__global__ void __launch_bounds__(128) ssm_step_kernel(const __grid_constant__ SsmParams p) {
    constexpr int L = N / 4, R = 4, M = L < R ? L : R, K = R / M;  // own sequences: every M-th of R
    const int j = threadIdx.x % L, own = j % M, base = (threadIdx.x & 31) - j;
    const int c = (int)((blockIdx.x * 128u + threadIdx.x) / (unsigned)L);
    const bool on = c < p.D;
    const int cc = on ? c : 0, g = cc / p.channels;
    float A[4];
    load4(p.A + (size_t)cc * N + 4 * j, A);
    const float skip = p.skip ? p.skip[cc] : 0.f, bias = p.bias ? p.bias[cc] : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) A[i] *= kLog2e;
    const T* const bm = (const T*)p.bm.p + g * N + 4 * j;
    const T* const cm = (const T*)p.cm.p + g * N + 4 * j;
    for (int b0 = blockIdx.y * R; b0 < p.B; b0 += gridDim.y * R) {
        float h[R][4], bv[R][4], cv[R][4], x[K], dt[K], z[K], d[K], dx[K];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const long long b = min(b0 + r, p.B - 1);
            *reinterpret_cast<float4*>(h[r]) = *reinterpret_cast<const float4*>(p.h0 + (b * p.D + cc) * N + 4 * j);
            load4(bm + b * p.bm.b, bv[r]);
            load4(cm + b * p.cm.b, cv[r]);
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const long long b = min(b0 + k * M + own, p.B - 1);
            x[k] = load_elem((const T*)p.x.p + b * p.x.b, cc);
            dt[k] = load_elem((const T*)p.dt.p + b * p.dt.b, cc);
            z[k] = p.gate.p ? load_elem((const T*)p.gate.p + b * p.gate.b, cc) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float v = dt[k] + bias;
            d[k] = p.softplus ? softplus<T>(v) : v;
            dx[k] = d[k] * x[k];
            if (p.gate.p) z[k] *= sigmoid<T>(z[k]);
        }
        float y[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float delta = __shfl_sync(0xffffffffu, d[r / M], base + r % M);
            const float in = __shfl_sync(0xffffffffu, dx[r / M], base + r % M);
            y[r] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[r][i] = fmaf(exp2_fast(fmaf(delta, A[i], kRaise)), h[r][i], in * bv[r][i]);
                y[r] = fmaf(cv[r][i], h[r][i], y[r]);
            }
            if (on && b0 + r < p.B)
                *reinterpret_cast<float4*>(p.h_out + ((long long)(b0 + r) * p.D + cc) * N + 4 * j) =
                    *reinterpret_cast<float4*>(h[r]);
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float v[M];
#pragma unroll
            for (int i = 0; i < M; ++i) v[i] = y[k * M + i];
            float u = share_sums<M>(v, own, 1);
#pragma unroll
            for (int gap = M; gap < L; gap *= 2) u += __shfl_xor_sync(0xffffffffu, u, gap);
            u = fmaf(skip, x[k], u);
            if (p.gate.p) u *= z[k];
            const int b = b0 + k * M + own;
            if (on && j < M && b < p.B) store_elem((T*)p.y.p, (long long)b * p.D + c, u);
        }
    }
}

template <typename T>
cudaError_t launch_step(const SsmParams& p, dim3 grid, cudaStream_t s) {
    switch (p.N) {
        case 8: ssm_step_kernel<T, 8><<<grid, 128, 0, s>>>(p); break;
        case 16: ssm_step_kernel<T, 16><<<grid, 128, 0, s>>>(p); break;
        case 32: ssm_step_kernel<T, 32><<<grid, 128, 0, s>>>(p); break;
        default: ssm_step_kernel<T, 64><<<grid, 128, 0, s>>>(p); break;
    }
    return cudaGetLastError();
}

// ---- plans -----------------------------------------------------------------------------

SsmParams params(const SsmArgs& a) {
    auto rows = [](const void* p, const long long* s) { return SsmRows{p, s[0], s[1]}; };
    SsmParams p = {};
    p.x = rows(a.x, a.x_strides);
    p.dt = rows(a.dt, a.dt_strides);
    p.gate = rows(a.gate, a.gate_strides);
    p.bm = rows(a.bm, a.b_strides);
    p.cm = rows(a.cm, a.c_strides);
    p.dy = rows(a.dy, a.dy_strides);
    p.y = rows(a.y, a.y_strides);
    p.A = a.A; p.skip = a.skip; p.bias = a.dt_bias;
    p.positions = a.positions;
    p.h0 = a.h0; p.h_out = a.h_out;
    p.B = a.B; p.T = a.T; p.D = a.D; p.N = a.N; p.G = a.G;
    p.channels = a.D / a.G;
    p.softplus = a.softplus;
    return p;
}

// How channels lie in warps, and chunks.
struct Plan {
    Split split;
    int tiles, chunks, chunk;
};

// Sixteen states a lane in two channels (N = 8: eight in one).
Split wide_split(int N) { return N == 8 ? Split{1, 1} : Split{N / 8, 2}; }

Plan plan_of(const SsmArgs& a, Split split, int channels_cta, long long chunks) {
    Plan p;
    p.split = split;
    p.tiles = (a.D / a.G + channels_cta - 1) / channels_cta;
    const long long chunk = ((a.T + chunks - 1) / chunks + kTile - 1) / kTile * kTile;
    p.chunk = (int)std::min<long long>(chunk, INT_MAX / 2 / kTile * kTile);
    p.chunks = (int)((a.T + (long long)p.chunk - 1) / p.chunk);
    return p;
}

// One walk where the channels give a scheduler more than half a warp: a warp alone takes 203 cycles
// a token, two together 322.  With fewer the sequences are cut, down to chunks of 32 tokens, which
// costs a second walk (8 x 2048 tokens of 16 states: 1024 channels 144 us cut, 169 not; 1280 175 and 202;
// 1536 205 and 202; 2048 271 and 203; 5 x 8192 of 4096 channels 1296 and 1258, although eight SMs hold
// two CTAs and the others one; 8 x 8192 of 1536, at the border, 755 and 800).  Below 512 tokens one launch
// instead of three (3 x 256 of 208 channels 17 us, cut 12 in a graph, where the caller's two more
// launches do not count).  Where even that leaves few warps, four states a lane (3 x 512 tokens of 208
// channels: 13.6 us, with sixteen 14.4).
Plan forward_plan(const SsmArgs& a) {
    const long long sms = sm_count();
    Split split = wide_split(a.N);
    auto warps = [&](Split s) { return (long long)a.B * a.G * ((a.D / a.G + s.cta() - 1) / s.cta()) * kWarps; };
    const long long w = warps(split);
    long long chunks = 1;
    if (2 * w < 5 * sms && a.T >= 512) chunks = std::min<long long>(a.T / 32, (16 * sms + w - 1) / w);
    if (a.N < 64 && w * chunks <= 2 * sms) split = {a.N / 4, 1};
    return plan_of(a, split, split.cta(), chunks);
}

// As many chunks as give an SM 28 CTAs of the gradients' walk, of 64 tokens at least: more chunks fill
// the last turn of the card better and cost the join (4 x 4096 tokens of 2048 channels: 28 CTAs an SM 916 us,
// 14 950, 8 1001, 56 954).  Chunks of 32 tokens would shorten small calls (1 x 512 of 1024 channels 40 us, with
// 64 52, 128 86; 1 x 2048 of 512 channels 56, 59, 85; 4 x 512 of 2048 152, 154, 174) and take their part of the
// workspace twice.
Plan backward_plan(const SsmArgs& a, int channels) {
    const long long tiles = (a.D / a.G + channels - 1) / channels;
    const long long ctas = (long long)a.B * a.G * tiles, want = (long long)sm_count() * 28;
    const long long chunks = std::max<long long>(1, std::min<long long>((want + ctas - 1) / ctas, a.T / 64));
    return plan_of(a, wide_split(a.N), channels, chunks);
}

void use(SsmParams* p, const Plan& plan) {
    p->chunks = plan.chunks;
    p->chunk = plan.chunk;
    p->tiles = plan.tiles;
}

// Regions of a workspace, one behind the other, each at a multiple of 256 bytes.
struct Workspace {
    char* at;
    size_t used = 0;
    float* take(size_t floats) {
        float* p = at ? (float*)(at + used) : nullptr;
        used += (floats * sizeof(float) + 255) / 256 * 256;
        return p;
    }
};

size_t forward_workspace(const SsmArgs& a, const Plan& plan, SsmParams* p) {
    Workspace w{(char*)a.workspace};
    if (plan.chunks > 1) {
        p->chunk_h = w.take((size_t)a.B * plan.chunks * a.D * a.N);
        p->chunk_s = w.take((size_t)a.B * plan.chunks * a.D);
    }
    return w.used;
}

size_t backward_workspace(const SsmArgs& a, const Plan& plan, SsmBwdParams* bp) {
    Workspace w{(char*)a.workspace};
    SsmParams& p = bp->f;
    const size_t chunks = (size_t)a.B * plan.chunks, D = a.D, N = a.N, blocks = (size_t)a.B * ((a.T + kBlock - 1) / kBlock);
    p.chunk_h = w.take(chunks * D * N);
    p.chunk_g = w.take(chunks * D * N);
    p.chunk_s = w.take(chunks * D);
    p.block_h = w.take(blocks * D * N);
    p.block_s = w.take(blocks * D);
    bp->part_A = w.take(chunks * D * N);
    bp->part_skip = w.take(chunks * D);
    bp->part_bias = w.take(chunks * D);
    bp->part_bc = w.take((size_t)a.G * plan.tiles * a.B * a.T * 2 * N);
    return w.used;
}

cudaError_t join(const SsmParams& p, bool forward, bool backward, const float* dh_T, cudaStream_t s) {
    const int warps = std::min(kJoinWarps, (p.chunks + 3) / 4);
    const dim3 grid((unsigned)((long long)p.D * p.N / 128), p.B, forward && backward ? 2 : 1);
    TraceScope trace("ssm_join_kernel", s);
    ssm_join_kernel<<<grid, warps * 32, 0, s>>>(forward ? p.chunk_h : nullptr, p.h0, p.chunk_g, dh_T, p.chunk_s, p.A,
                                                p.D, p.N, p.chunks);
    return cudaGetLastError();
}

unsigned grid_of(const SsmParams& p) { return (unsigned)((long long)p.tiles * p.G * p.chunks * p.B); }

int bwd_channels(int N) { return 4 * 2 * (128 / N); }  // of a CTA of the gradients' walk

template <typename T>
cudaError_t forward(const SsmArgs& a, cudaStream_t s) {
    SsmParams p = params(a);
    const Plan plan = forward_plan(a);
    use(&p, plan);
    forward_workspace(a, plan, &p);
    if (plan.chunks > 1) {
        cudaError_t e = launch_scan<T, kState>(p, plan.split, grid_of(p), s);
        if (e == cudaSuccess) e = join(p, true, false, nullptr, s);
        if (e != cudaSuccess) return e;
    }
    return launch_scan<T, kForward>(p, plan.split, grid_of(p), s);
}

template <typename T>
cudaError_t backward(const SsmArgs& a, cudaStream_t s) {
    SsmBwdParams bp = {};
    bp.f = params(a);
    SsmParams& p = bp.f;
    const Plan plan = backward_plan(a, bwd_channels(a.N));
    use(&p, plan);
    backward_workspace(a, plan, &bp);
    p.blocks = (a.T + kBlock - 1) / kBlock;
    SsmParams summary = p;
    const int cta = plan.split.cta();
    summary.tiles = (p.channels + cta - 1) / cta;
    cudaError_t e = launch_scan<T, kSummary>(summary, plan.split, grid_of(summary), s);
    if (e == cudaSuccess) e = join(p, true, true, a.dh_T, s);
    if (e != cudaSuccess) return e;
    auto rows = [](void* q, const long long* st) { return SsmRows{q, st[0], st[1]}; };
    bp.dx = rows(a.dx, a.dx_strides);
    bp.ddt = rows(a.ddt, a.ddt_strides);
    bp.dgate = rows(a.dgate, a.dgate_strides);
    bp.dh0 = a.dh0;
    if (!a.dA) bp.part_A = nullptr;
    if (!a.dskip) bp.part_skip = nullptr;
    if (!a.ddt_bias) bp.part_bias = nullptr;
    e = launch_gradients<T>(bp, grid_of(p), s);
    if (e != cudaSuccess) return e;
    const int parts = p.B * p.chunks;
    const PartialSum sums[3] = {{bp.part_A, a.dA, parts, a.D * a.N},
                                {bp.part_skip, a.dskip, parts, a.D},
                                {bp.part_bias, a.ddt_bias, parts, a.D}};
    e = launch_partial_sums(sums, 3, s);
    if (e != cudaSuccess) return e;
    const long long tokens = (long long)a.B * a.T, quads = tokens * (2 * a.N / 4);
    TraceScope trace("ssm_shared_grad_kernel", s);
    ssm_shared_grad_kernel<T><<<dim3((unsigned)((quads + 255) / 256), a.G), 256, 0, s>>>(
        bp.part_bc, tokens, a.T, a.N, p.tiles, rows(a.db, a.db_strides), rows(a.dc, a.dc_strides));
    return cudaGetLastError();
}

}  // namespace
}  // namespace ssm

size_t ssm_workspace_bytes(const SsmArgs& a) {
    SsmParams p = {};
    return ssm::forward_workspace(a, ssm::forward_plan(a), &p);
}

size_t ssm_bwd_workspace_bytes(const SsmArgs& a) {
    SsmBwdParams p = {};
    return ssm::backward_workspace(a, ssm::backward_plan(a, ssm::bwd_channels(a.N)), &p);
}

cudaError_t launch_ssm_fwd(const SsmArgs& a, cudaStream_t s) {
    return a.bf16 ? ssm::forward<__nv_bfloat16>(a, s) : ssm::forward<float>(a, s);
}

cudaError_t launch_ssm_bwd(const SsmArgs& a, cudaStream_t s) {
    return a.bf16 ? ssm::backward<__nv_bfloat16>(a, s) : ssm::backward<float>(a, s);
}

cudaError_t launch_ssm_step(const SsmArgs& a, cudaStream_t s) {
    const SsmParams p = ssm::params(a);
    const long long threads = (long long)a.D * (a.N / 4);
    const unsigned blocks = (unsigned)((threads + 127) / 128);
    const long long rows = (a.B + 3) / 4, want = ((long long)sm_count() * 16 + blocks - 1) / blocks;
    const dim3 grid(blocks, (unsigned)std::max(1ll, std::min(rows, std::min(want, 65535ll))));
    TraceScope trace("ssm_step_kernel", s);
    return a.bf16 ? ssm::launch_step<__nv_bfloat16>(p, grid, s) : ssm::launch_step<float>(p, grid, s);
}

}  // namespace la
