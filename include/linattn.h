/*
 * linattn.h - C ABI of the GB300 (sm_103a) causal decayed linear attention
 * library, liblinattn.so.
 *
 * The operator (one head, one sequence):
 *
 *   S_t = gamma * S_{t-1} + phi(k_t) v_t^T        S: d_k x d_v, fp32
 *   z_t = gamma * z_{t-1} + phi(k_t)              z: d_k,       fp32
 *   o_t = phi(q_t)^T S_t  [ / (phi(q_t)^T z_t + eps)  when normalising ]
 *
 * which equals the masked parallel form O = (Q K^T . D) V, D_nm = gamma^(n-m)
 * for n >= m and 0 otherwise.
 *   - "RetNet" (bembew): "Parallel Representation" (O = (QK^T . D)V and D),
 *     "Recurrent Representation" (S_n = gamma S_{n-1} + K_n^T V_n,
 *     O_n = Q_n S_n), "Chunked Recurrent Representation" (chunks computed in
 *     parallel, the state carried between them), "Multi-Scale Retention"
 *     (one gamma per head).
 *   - "Linear attention" (zerotofrontier 21.2): box "Causal linear attention,
 *     recurrent form" (phi, the normaliser z, eps in the denominator, rows of
 *     S index features and columns value dimensions) and box "Linear
 *     attention" (the non-causal form).
 *   - "Efficient and Sparse Transformers" (temporalbook 12.5), subsection 6:
 *     linear attention is the gamma = 1 case; phi(x) = elu(x) + 1.
 *
 * Conventions for every entry point:
 *   - Tensors are dense, row-major, caller-owned DEVICE memory (allocated by
 *     the caller, e.g. PyTorch); the library allocates nothing, keeps no
 *     state between calls and never synchronises the stream.
 *   - Layouts: Q, K [B][H][T][d_k]; V, O [B][H][T][d_v]; S [B][H][d_k][d_v]
 *     (rows = features, columns = value dims); z [B][H][d_k].
 *   - Q/K/V/O hold `dtype` elements (fp32 or bf16); states are always fp32.
 *   - Every device pointer must be 16-byte aligned; d_k and d_v must be
 *     multiples of 16 in [16, 256].
 *   - `gamma` is a HOST array of H fp32 decays, each in (0, 1]; it is read
 *     during the call (its values travel in the kernel parameters), so the
 *     array may be reused as soon as the call returns.
 *   - Calls run on the CURRENT device (cudaSetDevice): it must own `stream`
 *     and every buffer passed; the segment plans and workspace sizes are the
 *     current device's too (its SM count).
 *   - Work is enqueued asynchronously on `stream` (a cudaStream_t; NULL is the
 *     legacy default stream).  The return code covers host-side argument
 *     checks and launch errors only.  `dev_status`, if not NULL, is a device
 *     int the kernels set to a nonzero la_status when they detect a problem
 *     on the device (a bounded wait that ran out); the caller zeroes it
 *     beforehand and reads it after synchronising.
 *   - Arguments are checked before anything is enqueued: a call that returns
 *     LA_ERR_INVALID_ARG or LA_ERR_UNSUPPORTED has launched nothing and
 *     written nothing.
 */
#ifndef LINATTN_H
#define LINATTN_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Symbols of the shared library (the library is built with hidden default
 * visibility; only these are exported). */
#if defined(__GNUC__)
#define LA_API __attribute__((visibility("default")))
#else
#define LA_API
#endif

/* Same object as cudaStream_t. */
typedef struct CUstream_st* la_stream_t;

typedef enum {
    LA_OK = 0,
    LA_ERR_INVALID_ARG = 1,  /* bad size, pointer, alignment, gamma or workspace */
    LA_ERR_UNSUPPORTED = 2,  /* a combination the method does not define */
    LA_ERR_CUDA = 3,         /* a CUDA runtime call or launch failed */
    LA_ERR_TIMEOUT = 4       /* device side only: a bounded wait ran out */
} la_status;

typedef enum { LA_DTYPE_F32 = 0, LA_DTYPE_BF16 = 1 } la_dtype;

/* flags */
#define LA_PHI_ELU1  1u  /* apply phi(x) = elu(x) + 1 to q and k (not v) */
#define LA_NORMALIZE 2u  /* divide by phi(q)^T z + eps */
#define LA_NONCAUSAL 4u  /* every query reads the whole sequence; gamma must be 1 */
/* Divide by max(|phi(q)^T z|, 1) instead of phi(q)^T z + eps (implies normalising;
 * eps unused): the matrix LSTM's floored normaliser, box "An LSTM whose cell is
 * linear attention" on the "Linear attention" page, which equals RetNet's
 * division of each score row by the absolute value of its sum clamped below at 1
 * (same page, "Its normalizer is unstable").  Defined for signed features too. */
#define LA_NORM_FLOOR 8u
/* Per-token decay (la_chunk_fwd_gated): only the planning queries
 * la_workspace_size and la_chunk_fwd_launches take this flag, to size a
 * la_chunk_fwd_gated call; la_chunk_fwd rejects it. */
#define LA_GATED 16u
/* Second-order Taylor feature map in place of elu + 1 ("Linear attention" page,
 * section "A Taylor feature map", box "Taylor features"):
 *   phi(x) = (1, x_1 .. x_d, vec(x x^T) / sqrt 2),  1 + d + d^2 entries, vec row-major,
 * so that phi(q)^T phi(k) = 1 + s + s^2/2 with s = q^T k (always >= 1/2, a safe
 * denominator).  d_k = 16 (Based's projected width: 273 features), not with
 * LA_PHI_ELU1, causal.  d_k is the width of Q and K; the states S0 / S_out / S are
 * [B][H][1 + d_k + d_k^2][d_v] fp32 and z0 / z_out / z [B][H][1 + d_k + d_k^2],
 * rows in the order of phi above.  la_chunk_fwd (and la_workspace_size,
 * la_chunk_fwd_launches, la_chunk_fwd_noalloc): bf16, d_v a multiple of 64, chunk
 * 0 or 128, an sm_103 device.  la_recurrent_step: bf16 or fp32, d_v <= 256.
 * la_chunk_bwd: bf16 or fp32, d_v <= 128, per-head decay.  Other calls and
 * shapes answer LA_ERR_UNSUPPORTED. */
#define LA_PHI_TAYLOR 32u

/* Human-readable text of a status code (static storage, never NULL). */
LA_API const char* la_status_string(int status);

/* ABI version of this header: LA_ABI_VERSION. */
#define LA_ABI_VERSION 1
LA_API int la_abi_version(void);

/*
 * Bytes of device workspace la_chunk_fwd needs for these arguments (0 when
 * the chosen path needs none).  Pure host arithmetic; never fails (returns
 * 0 for arguments la_chunk_fwd would reject).  `chunk` as for la_chunk_fwd.
 */
LA_API size_t la_workspace_size(int B, int H, int T, int d_k, int d_v, la_dtype dtype,
                                unsigned flags, int chunk);

/*
 * Number of kernels la_chunk_fwd enqueues for these arguments on the current
 * device (1 for the single-pass paths; 2 or 3 when long sequences are split
 * into segments: segment states, then - for more than four segments per
 * sequence - the scan over them, then the outputs).  LA_GATED adds the decays'
 * preparation.  0 for
 * arguments la_chunk_fwd would reject or T == 0.  Pure host query.
 */
LA_API int la_chunk_fwd_launches(int B, int H, int T, int d_k, int d_v, la_dtype dtype,
                                 unsigned flags, int chunk);

/*
 * Zero-fill a state: S[B][H][d_k][d_v] and, if not NULL, z[B][H][d_k].
 * The empty state S_0 = 0, z_0 = 0 of the "Causal linear attention,
 * recurrent form" box ("Linear attention", zerotofrontier 21.2).
 * Errors: LA_ERR_INVALID_ARG for S == NULL, a negative size, or a misaligned
 * pointer; LA_ERR_CUDA if the launch fails.  B or H == 0 is a no-op.
 */
LA_API la_status la_state_init(float* S, float* z, int B, int H, int d_k, int d_v,
                               la_stream_t stream);

/*
 * Chunkwise forward over whole sequences (prefill / training forward):
 * "Chunked Recurrent Representation" ("RetNet", bembew) - the intra-chunk
 * part in the parallel form, the inter-chunk part through the carried state.
 *
 *   Q, K      [B][H][T][d_k]  dtype      inputs, read only
 *   V         [B][H][T][d_v]  dtype      input, read only
 *   gamma     host float[H]              per-head decay in (0, 1]
 *   flags     LA_PHI_ELU1 | LA_NORMALIZE | LA_NONCAUSAL | LA_NORM_FLOOR
 *   eps       added to the denominator (used only with LA_NORMALIZE and not
 *             LA_NORM_FLOOR; the pages use 1e-6)
 *   S0, z0    [B][H][d_k][d_v], [B][H][d_k] fp32 initial state, or NULL for
 *             zero.  S0 may alias S_out and z0 may alias z_out (in-place
 *             continuation).  The normaliser state z is carried whether or
 *             not LA_NORMALIZE is set, so z_out is valid either way.
 *   O         [B][H][T][d_v]  dtype      output; must not overlap Q, K, V
 *   S_out     [B][H][d_k][d_v] fp32 final state S_T, or NULL
 *   z_out     [B][H][d_k] fp32 final normaliser z_T, or NULL
 *   chunk     chunk length C: 0 = let the library choose, else one of
 *             16, 32, 64, 128 (the result does not depend on it beyond
 *             rounding)
 *   workspace device scratch of at least la_workspace_size(...) bytes
 *             (may be NULL when that size is 0); overwritten by the call
 *   dev_status  device int or NULL (see the conventions above)
 *
 * T == 0 is valid: nothing is written to O and the final state equals the
 * initial one.  B == 0 or H == 0 is a no-op.
 * LA_NONCAUSAL ("Linear attention" box, non-causal form): requires every
 * gamma == 1 and S0 == z0 == NULL, else LA_ERR_UNSUPPORTED; S_out / z_out
 * then receive phi(K)^T V and phi(K)^T 1.
 * Errors: LA_ERR_INVALID_ARG (negative size, d_k/d_v not a multiple of 16
 * in [16, 256], a NULL required pointer, misalignment, gamma outside (0, 1],
 * non-finite or negative eps, an unknown flag, dtype or chunk, workspace
 * too small, O overlapping an input); LA_ERR_UNSUPPORTED; LA_ERR_CUDA.
 */
LA_API la_status la_chunk_fwd(const void* Q, const void* K, const void* V, la_dtype dtype,
                              const float* gamma, int B, int H, int T, int d_k, int d_v,
                              unsigned flags, float eps,
                              const float* S0, const float* z0,
                              void* O, float* S_out, float* z_out,
                              int chunk, void* workspace, size_t workspace_bytes,
                              int* dev_status, la_stream_t stream);

/*
 * One recurrent decode step for every (b, h), updating the state in place:
 * "Recurrent Representation" ("RetNet", bembew) and the decode step of the
 * "Linear attention" page (zerotofrontier 21.2, "Decoding, training, and
 * what each costs"; update first, then read, so the token is in its own sum):
 *
 *   S = gamma S + phi(k) v^T ;  z = gamma z + phi(k)     (z only if normalising)
 *   o = phi(q)^T S  [ / (phi(q)^T z + eps) ]  [ / max(|phi(q)^T z|, 1) ]
 *
 *   q, k   [B][H][d_k] dtype;  v [B][H][d_v] dtype;  o [B][H][d_v] dtype
 *   S      [B][H][d_k][d_v] fp32, read and written in place
 *   z      [B][H][d_k] fp32, in place; required with LA_NORMALIZE or
 *          LA_NORM_FLOOR, else ignored
 *   flags  LA_PHI_ELU1 | LA_NORMALIZE | LA_NORM_FLOOR (LA_NONCAUSAL is
 *          LA_ERR_UNSUPPORTED)
 * Errors: as la_chunk_fwd.
 */
LA_API la_status la_recurrent_step(const void* q, const void* k, const void* v, la_dtype dtype,
                                   const float* gamma, int B, int H, int d_k, int d_v,
                                   unsigned flags, float eps,
                                   float* S, float* z, void* o,
                                   int* dev_status, la_stream_t stream);

/*
 * Chunkwise forward with a per-token (data-dependent) scalar decay in place
 * of the per-head gamma:
 *
 *   S_t = a_t S_{t-1} + phi(k_t) v_t^T,   z_t = a_t z_{t-1} + phi(k_t),
 *   o_t = phi(q_t)^T S_t  [ normalised as in la_chunk_fwd ]
 *
 * with a_t = exp(log_a[b][h][t]).  The generic "decay the old state, add the
 * new contribution, read out" recurrence of "Linear Attention, RWKV, and
 * RetNet" (temporalbook 13.3, subsection 4 "The Unifying Picture"), whose
 * decay G_t depends on the input in the selective case, with G_t = a_t 1 a
 * scalar per head and token; "Efficient and Sparse Transformers"
 * (temporalbook 12.5, "Gated Linear Attention: Toward Input-Dependent
 * Forgetting") has RetNet as the constant case G_t = gamma 1.  The chunkwise
 * form uses cumulative log-decays inside each chunk instead of powers of
 * gamma (the state between chunks decays by the product of the chunk's a_t).
 *
 *   log_a  DEVICE fp32 [B][H][T], natural log of each decay, finite and <= 0
 *          (a_t in (0, 1]); read only; not checked (device memory)
 *   other arguments as la_chunk_fwd (no gamma); flags as la_chunk_fwd, with
 *          or without LA_GATED; LA_NONCAUSAL is LA_ERR_UNSUPPORTED
 *   workspace: at least la_workspace_size(..., flags | LA_GATED, chunk)
 *          bytes (the tensor-core path always needs some: the per-chunk
 *          cumulative decays)
 * Errors: as la_chunk_fwd; LA_ERR_INVALID_ARG also for log_a == NULL or
 * misaligned when T > 0.
 */
LA_API la_status la_chunk_fwd_gated(const void* Q, const void* K, const void* V,
                                    la_dtype dtype, const float* log_a, int B, int H, int T,
                                    int d_k, int d_v, unsigned flags, float eps,
                                    const float* S0, const float* z0,
                                    void* O, float* S_out, float* z_out,
                                    int chunk, void* workspace, size_t workspace_bytes,
                                    int* dev_status, la_stream_t stream);

/*
 * One decode step with a per-token decay: la_recurrent_step with
 * S = a S + phi(k) v^T, z = a z + phi(k), a = exp(log_a[b][h]).
 *   log_a  DEVICE fp32 [B][H] (this step's decays), finite and <= 0
 * Errors: as la_recurrent_step; LA_ERR_INVALID_ARG also for log_a == NULL or
 * misaligned.
 */
LA_API la_status la_recurrent_step_gated(const void* q, const void* k, const void* v,
                                         la_dtype dtype, const float* log_a, int B, int H,
                                         int d_k, int d_v, unsigned flags, float eps,
                                         float* S, float* z, void* o,
                                         int* dev_status, la_stream_t stream);

/*
 * Backward pass: the gradients of la_chunk_fwd's outputs, for the loss
 *   L = sum_t dO_t . o_t + <dS_T, S_T> + <dz_T, z_T>
 * with respect to Q, K, V and the initial state.  "Linear attention"
 * (zerotofrontier 21.2), "Decoding, training, and what each costs": the
 * gradients are cumulative sums too, forward in time for the queries and
 * backward in time for the keys and values, so no intermediate state is
 * stored (the states are recomputed, chunk by chunk).
 *
 *   Q, K, V, gamma, flags, eps, S0, z0   as the forward call that made O (flags:
 *          LA_PHI_ELU1, LA_NORMALIZE, LA_NORM_FLOOR; LA_NONCAUSAL is
 *          LA_ERR_UNSUPPORTED)
 *   dO     [B][H][T][d_v] dtype: the loss's gradient with respect to O
 *   dS_T   [B][H][d_k][d_v] fp32 or NULL (zero); dz_T [B][H][d_k] fp32 or NULL
 *   dQ, dK [B][H][T][d_k] dtype, dV [B][H][T][d_v] dtype: outputs (may not
 *          overlap any input)
 *   dS0    [B][H][d_k][d_v] fp32 or NULL, dz0 [B][H][d_k] fp32 or NULL: the
 *          initial state's gradients
 *   workspace: at least la_bwd_workspace_size(...) bytes (the sweeps'
 *          segment states and, when normalising, per-token denominators; the
 *          tensor-core passes' operands where they run)
 * d_k and d_v must be at most 128 (LA_ERR_UNSUPPORTED otherwise).  Paths: bf16
 * calls with per-head decay, no normaliser and LA_PHI_ELU1 or no feature map
 * run as three tensor-core forward passes; normalised bf16 calls with per-head decay
 * and d_v = 64 take dq from the CUDA cores in fp32 and dk, dv from two
 * tensor-core passes (dq of the normalised form cancels too much for bf16
 * operands); everything else runs in fp32 on the CUDA cores.
 * LA_PHI_TAYLOR: the Taylor feature map as in la_chunk_fwd (d_k = 16, not with
 * LA_PHI_ELU1, not with per-token decays); S0, z0, dS_T, dz_T, dS0 and dz0 then
 * have 1 + d_k + d_k^2 = 273 rows in the map's order, and dQ, dK are the
 * gradients of the raw 16-wide q and k (through the map's transpose Jacobian).
 * Errors as la_chunk_fwd.
 */
LA_API la_status la_chunk_bwd(const void* Q, const void* K, const void* V, const void* dO,
                              la_dtype dtype, const float* gamma, int B, int H, int T, int d_k,
                              int d_v, unsigned flags, float eps, const float* S0,
                              const float* z0, const float* dS_T, const float* dz_T, void* dQ,
                              void* dK, void* dV, float* dS0, float* dz0, void* workspace,
                              size_t workspace_bytes, int* dev_status, la_stream_t stream);

/* la_chunk_bwd with the per-token decay of la_chunk_fwd_gated (log_a: DEVICE
 * fp32 [B][H][T]) in place of gamma.  The decays themselves get no gradient. */
LA_API la_status la_chunk_bwd_gated(const void* Q, const void* K, const void* V, const void* dO,
                                    la_dtype dtype, const float* log_a, int B, int H, int T,
                                    int d_k, int d_v, unsigned flags, float eps,
                                    const float* S0, const float* z0, const float* dS_T,
                                    const float* dz_T, void* dQ, void* dK, void* dV,
                                    float* dS0, float* dz0, void* workspace,
                                    size_t workspace_bytes, int* dev_status, la_stream_t stream);

/* Bytes of workspace la_chunk_bwd needs (pure host arithmetic; 0 for arguments
 * it would reject). */
LA_API size_t la_bwd_workspace_size(int B, int H, int T, int d_k, int d_v, la_dtype dtype,
                                    unsigned flags);

/*
 * Queries and keys made ready for retention, in one pass: the norm of every
 * head's row, the rotation by its token's position, a scale, and the layout
 * la_chunk_fwd and la_recurrent_step read.
 *
 *   n = x r w,  r = (mean(x^2) + eps)^(-1/2)     with LA_QK_NORM, else n = x
 *   (y_i, y_j) = s (n_i cos - n_j sin, n_i sin + n_j cos),  angle p inv_freq[m],
 *       for pair m = 0 .. rot/2 - 1 of the first rot entries: (m, m + rot/2), or
 *       (2m, 2m + 1) with LA_QK_ADJACENT;  y = s n for the other entries
 *
 * RetNet rotates its queries and keys by their position before the retention;
 * decode is the same call with T = 1.
 *
 *   q, k      [B][T][Hq][d], [B][T][Hk][d] dtype, rows of d entries dense, the
 *             other strides free (slices of a packed projection; a stride of 0
 *             repeats a row).  q_strides, k_strides: HOST arrays of 3 strides
 *             (batch, token, head) in elements, each >= 0 and a multiple of 16
 *             bytes, or NULL for the dense layout.  The stride of a dimension of
 *             size 1 is not read.
 *   d         a multiple of 16 in [16, 256];  rot a multiple of 16 in [0, d]
 *   inv_freq  HOST double[rot/2], radians per position (rot > 0); below 2^64 in size
 *   positions DEVICE int32 [B][T], any values, or NULL: token t stands at pos0 + t,
 *             0 <= pos0 and pos0 + T - 1 < 2^31.  The angle keeps fp32 accuracy at
 *             every position (its fraction of a turn is taken in 64-bit integers).
 *   q_weight, k_weight  DEVICE fp32 [d] or NULL (ones); NULL without LA_QK_NORM
 *   eps       > 0, finite (with LA_QK_NORM)
 *   q_scale, k_scale    finite
 *   flags     LA_QK_NORM | LA_QK_ADJACENT
 *   q_out, k_out  [B][Hq][T][d], [B][Hk][T][d] dtype, dense; their memory may overlap
 *             no input's (first to last row) and not each other's
 *
 * Sums, norms and angles are fp32, rounded once to dtype at the end; the sum of a
 * row's squares must stay below the fp32 range (|x| below about 1e18).
 * B or T == 0 is a no-op; Hq, Hk in [1, 65536]; B * T < 2^31.
 * Errors: LA_ERR_INVALID_ARG, LA_ERR_CUDA.
 */
#define LA_QK_NORM 1u
#define LA_QK_ADJACENT 2u
LA_API la_status la_qk_rotate_fwd(const void* q, const long long* q_strides, const void* k,
                                  const long long* k_strides, la_dtype dtype, int B, int T, int Hq,
                                  int Hk, int d, int rot, const double* inv_freq,
                                  const int* positions, int pos0, const float* q_weight,
                                  const float* k_weight, float eps, float q_scale, float k_scale,
                                  unsigned flags, void* q_out, void* k_out, la_stream_t stream);

/*
 * Gradients of la_qk_rotate_fwd.
 *
 *   q, k .. flags   as the forward call
 *   dq_out, dk_out  [B][Hq][T][d], [B][Hk][T][d] dtype, dense: the loss's gradient
 *             with respect to q_out, k_out (la_chunk_bwd's dQ, dK)
 *   dq, dk    [B][T][Hq][d], [B][T][Hk][d] dtype with strides as q's; they may be
 *             slices of one packed row (side by side, or interleaved head by head,
 *             the outer strides then multiples of the heads'), their rows apart, and
 *             their memory (first to last row) may overlap no input's
 *   dq_weight, dk_weight  fp32 [d] or NULL: the weights' gradients, summed over
 *             batch, tokens and heads in a fixed order; overwritten
 *   workspace at least la_qk_rotate_bwd_workspace_size(...) bytes when a weight
 *             gradient is asked for, else may be NULL; overwritten.  Calls that may
 *             run at the same time need a workspace each.
 * A row repeated by a stride of 0 gets a gradient for each of its uses: the caller
 * adds them up.  B or T == 0: the weight gradients are zeroed, nothing else is done.
 * Errors as la_qk_rotate_fwd.
 */
LA_API la_status la_qk_rotate_bwd(const void* q, const long long* q_strides, const void* k,
                                  const long long* k_strides, const void* dq_out,
                                  const void* dk_out, la_dtype dtype, int B, int T, int Hq, int Hk,
                                  int d, int rot, const double* inv_freq, const int* positions,
                                  int pos0, const float* q_weight, const float* k_weight, float eps,
                                  float q_scale, float k_scale, unsigned flags, void* dq,
                                  const long long* dq_strides, void* dk, const long long* dk_strides,
                                  float* dq_weight, float* dk_weight, void* workspace,
                                  size_t workspace_bytes, la_stream_t stream);
LA_API size_t la_qk_rotate_bwd_workspace_size(int B, int T, int Hq, int Hk, int d, la_dtype dtype);

/*
 * The norm and gate of each head's output, retention's [B][H][T][d] to the layer's
 * row [B][T][H][d]:
 *
 *   n = o r, r = (mean(o^2) + eps)^(-1/2)     (o less its mean with LA_GATE_CENTER)
 *   y = n w  [ g sigmoid(g) ]
 *
 * RetNet's per-head norm and swish gate: raw retention outputs grow with the sum
 * of the decays.  Decode is the same call with T = 1.
 *
 *   o         [B][H][T][d] dtype; o_strides: HOST array of 3 strides (batch, head,
 *             token) in elements or NULL for dense.  The per-channel recurrence's
 *             [B][T][H d] is read with strides (T H d, d, H d).
 *   gate      [B][T][H][d] dtype or NULL; gate_strides (batch, token, head) or NULL
 *   weight    DEVICE fp32 [H][d] or NULL (ones)
 *   flags     LA_GATE_CENTER;  eps > 0, finite
 *   y         [B][T][H][d] dtype, y_strides (batch, token, head) or NULL; its rows
 *             may not overlap each other, nor its memory (first to last row) an input's
 *   A gate of -infinity makes its entry NaN (0 times infinity), the type's lowest
 *   value makes it 0.
 * Strides as la_qk_rotate_fwd: rows dense, strides >= 0 and multiples of 16 bytes.
 * d a multiple of 16 in [16, 256], H in [1, 65536], B * T < 2^31; sums in fp32 (as
 * la_qk_rotate_fwd).  B or T == 0 is a no-op.  Errors: LA_ERR_INVALID_ARG,
 * LA_ERR_CUDA.
 */
#define LA_GATE_CENTER 1u
LA_API la_status la_head_gate_fwd(const void* o, const long long* o_strides, const void* gate,
                                  const long long* gate_strides, la_dtype dtype,
                                  const float* weight, int B, int H, int T, int d, unsigned flags,
                                  float eps, void* y, const long long* y_strides,
                                  la_stream_t stream);

/*
 * Gradients of la_head_gate_fwd.
 *   o, gate, weight, flags, eps   as the forward call
 *   dy        [B][T][H][d] dtype, dy_strides (batch, token, head) or NULL
 *   d_o       [B][H][T][d] dtype, do_strides (batch, head, token) or NULL (dense:
 *             what la_chunk_bwd reads as dO)
 *   dgate     [B][T][H][d] dtype, dgate_strides or NULL; NULL exactly when gate is
 *   dweight   fp32 [H][d] or NULL: summed over batch and tokens in a fixed order;
 *             overwritten
 *   workspace at least la_head_gate_bwd_workspace_size(...) bytes when dweight is
 *             asked for, else may be NULL; one for each call that may run at once
 * Each output's rows lie apart, in memory (first to last row) that overlaps no
 * input's and no other output's.  B or T == 0: dweight is zeroed, nothing else is
 * done.  Errors as la_head_gate_fwd.
 */
LA_API la_status la_head_gate_bwd(const void* o, const long long* o_strides, const void* gate,
                                  const long long* gate_strides, const void* dy,
                                  const long long* dy_strides, la_dtype dtype, const float* weight,
                                  int B, int H, int T, int d, unsigned flags, float eps, void* d_o,
                                  const long long* do_strides, void* dgate,
                                  const long long* dgate_strides, float* dweight, void* workspace,
                                  size_t workspace_bytes, la_stream_t stream);
LA_API size_t la_head_gate_bwd_workspace_size(int B, int H, int T, int d, la_dtype dtype);

/*
 * The per-channel gated recurrence, the member of the family "decay the old state,
 * add, read out" ("Linear Attention, RWKV, and RetNet", temporalbook 13.3,
 * subsection 4) with a decay for each token and channel and a state of one number
 * a channel:
 *
 *   h_t = a_t h_(t-1) + x_t,   a_t = exp(log_a[b][t][c])
 *
 *   x       [B][T][D] dtype, dense;  D a multiple of 16
 *   log_a   DEVICE fp32 [B][T][D], natural logs, <= 0 (not checked).  -inf (and
 *           any value whose exponential is zero in fp32) restarts the channel at its
 *           token: h_t = x_t whatever came before, infinities and NaN included.
 *   h0      [B][D] fp32 initial state or NULL for zero; may be h_out itself
 *           (in-place continuation), else may not overlap it
 *   h       [B][T][D] dtype, output; may overlap no input
 *   h_out   [B][D] fp32 final state h_T, or NULL
 *   dev_status  device int or NULL (see the conventions above)
 *
 * The state is fp32 throughout; h is rounded where it is stored.  An infinity or NaN
 * lasts in the state until a restart.  T == 0: h_out is the initial state.  B == 0
 * is a no-op.  B * D at most 2^33, B * T * D at most 2^44.  No workspace.
 * Errors: LA_ERR_INVALID_ARG, LA_ERR_CUDA.
 */
LA_API la_status la_scan_fwd(const void* x, la_dtype dtype, const float* log_a, int B, int T, int D,
                             const float* h0, void* h, float* h_out, int* dev_status,
                             la_stream_t stream);

/*
 * Gradients of la_scan_fwd for the loss sum_t dh_t . h_t + <dh_T, h_T>:
 *
 *   c_t = a_t (dh_t + c_(t+1)), c_T = dh_T;  dx_t = dh_t + c_(t+1),
 *   dlog_a_t = c_t h_(t-1),  dh0 = c_0
 *
 *   log_a, h0   as the forward call;  h: its output
 *   dh      [B][T][D] dtype;  dh_T [B][D] fp32 or NULL (zero)
 *   dx      [B][T][D] dtype, dlog_a [B][T][D] fp32: outputs, overlapping nothing
 *   dh0     [B][D] fp32 or NULL; may be dh_T itself
 * dlog_a reads h as it was rounded to dtype.  A restarted token passes nothing to
 * the tokens before it and has dlog_a = 0.  T == 0: dh0 is dh_T.
 * Errors as la_scan_fwd.
 */
LA_API la_status la_scan_bwd(const float* log_a, const void* h, const void* dh, la_dtype dtype,
                             int B, int T, int D, const float* h0, const float* dh_T, void* dx,
                             float* dlog_a, float* dh0, int* dev_status, la_stream_t stream);

/*
 * One token of la_scan_fwd: h_out = exp(log_a) h_in + x, h its rounding to dtype.
 *   x, h [B][D] dtype;  log_a, h_in, h_out [B][D] fp32.  h_out may be h_in itself
 *   (in place) and otherwise overlaps nothing; h overlaps nothing.
 * Errors as la_scan_fwd.
 */
LA_API la_status la_scan_step(const void* x, la_dtype dtype, const float* log_a, int B, int D,
                              const float* h_in, float* h_out, void* h, la_stream_t stream);

/*
 * The short causal convolution over each channel, as it stands before a state space or
 * gated mixer:
 *
 *   u_t = bias + sum_j w[c][j] x_(t-W+1+j),   y = u,  or  u sigmoid(u) with LA_CONV_SILU
 *
 *   x, y      [B][T][D] dtype, rows of D entries dense, x_strides, y_strides: HOST arrays
 *             of 2 strides (batch, token) in elements or NULL for dense, each >= 0 and a
 *             multiple of 16 bytes (x may be a slice of a packed projection; y's rows lie
 *             apart).  The stride of a dimension of size 1 is not read.
 *   weight    DEVICE fp32 [D][W], W from 2 to 4, the last tap the token's own;
 *             bias DEVICE fp32 [D] or NULL
 *   state     [B][W-1][D] dtype: the rows before token 0, oldest first, or NULL (zeros)
 *   positions DEVICE int32 [B][T], each token's place in its document, or NULL: a tap k
 *             tokens back counts only where k <= positions[b][t] (documents packed one
 *             behind another, or padding before a sequence).  What does not count is not
 *             read into the sum, infinities and NaN included.  Taps that count and lie
 *             before token 0 read the state.
 *   state_out [B][W-1][D] dtype: the last W - 1 rows of state and x as they are, those of
 *             another document or of padding among them, or NULL; may be state itself,
 *             else may not overlap it.  A call that goes on from there gives its tokens'
 *             positions (la_short_conv_step_at for single ones).
 *   flags     LA_CONV_SILU
 * No output may overlap an input (state_out: but state itself) or another output.  Sums in
 * fp32, rounded once.  D a multiple of 16, B * T at most 2^31 - 256, B * D at most 2^33,
 * D * W < 2^31.
 * T == 0: state_out is the state.  B == 0 is a no-op.
 * Errors: LA_ERR_INVALID_ARG, LA_ERR_CUDA.
 */
#define LA_CONV_SILU 1u
LA_API la_status la_short_conv_fwd(const void* x, const long long* x_strides, la_dtype dtype,
                                   const float* weight, const float* bias, int B, int T, int D,
                                   int W, unsigned flags, const void* state, const int* positions,
                                   void* y, const long long* y_strides, void* state_out,
                                   la_stream_t stream);

/*
 * Gradients of la_short_conv_fwd.
 *   x .. positions  as the forward call
 *   dy        [B][T][D] dtype, dy_strides as x's;  dstate_T [B][W-1][D] dtype or NULL: the
 *             gradient with respect to state_out
 *   dx        [B][T][D] dtype, dx_strides (rows apart; may be a slice of a packed gradient)
 *   dweight   fp32 [D][W] or NULL, dbias fp32 [D] or NULL: summed over batch and tokens
 *             in a fixed order; overwritten
 *   dstate    [B][W-1][D] dtype or NULL: with respect to state (given or not)
 *   workspace at least la_short_conv_bwd_workspace_size(...) bytes when dweight or dbias is
 *             asked for, else may be NULL; one for each call that may run at once
 * No output may overlap an input or another output.  B or T == 0: dweight and dbias are
 * zeroed, dstate is dstate_T.  Errors as la_short_conv_fwd.
 */
LA_API la_status la_short_conv_bwd(const void* x, const long long* x_strides, const void* dy,
                                   const long long* dy_strides, la_dtype dtype,
                                   const float* weight, const float* bias, int B, int T, int D,
                                   int W, unsigned flags, const void* state, const int* positions,
                                   const void* dstate_T, void* dx, const long long* dx_strides,
                                   float* dweight, float* dbias, void* dstate, void* workspace,
                                   size_t workspace_bytes, la_stream_t stream);
LA_API size_t la_short_conv_bwd_workspace_size(int B, int T, int D, int W, la_dtype dtype);

/*
 * One token of la_short_conv_fwd: x [B][D] dtype with x_stride elements from sequence to
 * sequence, y [B][D] dense.  state [B][W-1][D], every row of which counts, and state_out as
 * there (state_out may be state itself).  Errors as la_short_conv_fwd.
 */
LA_API la_status la_short_conv_step(const void* x, long long x_stride, la_dtype dtype,
                                    const float* weight, const float* bias, int B, int D, int W,
                                    unsigned flags, const void* state, void* state_out, void* y,
                                    la_stream_t stream);

/*
 * la_short_conv_step of tokens at their places in their documents: positions DEVICE int32 [B],
 * as la_short_conv_fwd's, or NULL: a tap k tokens back counts only where k <= positions[b].
 * The state behind a packed or padded prompt holds its last W - 1 rows whatever they belong
 * to, and la_short_conv_step counts them all: tokens at positions below W - 1 need this
 * call.  The state moves up all the same.
 */
LA_API la_status la_short_conv_step_at(const void* x, long long x_stride, la_dtype dtype,
                                       const float* weight, const float* bias, int B, int D, int W,
                                       unsigned flags, const void* state, const int* positions,
                                       void* state_out, void* y, la_stream_t stream);

/*
 * The selective scan: "decay the old state, add, read out" with N numbers of state a
 * channel, their decay chosen by each token:
 *
 *   delta = softplus(dt + dt_bias)    with LA_SSM_SOFTPLUS, else dt + dt_bias
 *   h_t = exp(delta A) h_(t-1) + delta x_t b_t       (entry by entry over [D][N])
 *   y_t = c_t . h_t + skip x_t    [ times gate sigmoid(gate) ]
 *
 *   x, dt, gate, y  [B][T][D] dtype;  gate may be NULL
 *   b, c      [B][T][G][N] dtype, shared by the D / G channels of a group, a multiple
 *             of 8; N is 8, 16, 32 or 64
 *   strides   HOST array of 6 pairs of strides (batch, token) in elements, for x, dt, b,
 *             c, gate and y in this order, or NULL (all dense): rows (of D or G N entries)
 *             dense, strides >= 0 and multiples of 16 bytes, y's rows apart.  The stride of a
 *             dimension of size 1 is not read.
 *   A         DEVICE fp32 [D][N], finite (as a rule below 0; each token's exp(delta A)
 *             inside the fp32 range);  skip, dt_bias DEVICE fp32 [D] or NULL (zero)
 *   h0        [B][D][N] fp32 initial state or NULL for zero; may be h_out itself, else may
 *             not overlap it
 *   positions DEVICE int32 [B][T] or NULL: a token with position 0 starts a document: the old state
 *             is dropped, infinities and NaN included
 *   h_out     [B][D][N] fp32 final state or NULL
 *   flags     LA_SSM_SOFTPLUS
 *   workspace at least la_ssm_workspace_size(...) bytes (which may be 0); overwritten;
 *             one for each call that may run at once
 * States, decays and sums are fp32; y is rounded where it is stored.  A decay is one hardware 2^x (2 ulp);
 * with dtype bf16 the softplus and the gate's sigmoid take theirs too, off by 2^-22 |v| of
 * themselves, which h_out and the fp32 gradients inherit.  No output may overlap an
 * input or another output.  D a multiple of 16, B and G < 65536, B * T at most 2^31 - 256,
 * D * N < 2^31, B * D * N at most 2^33.  T == 0: h_out is the initial state.  B == 0 is a no-op.
 * Errors: LA_ERR_INVALID_ARG, LA_ERR_CUDA.
 */
#define LA_SSM_SOFTPLUS 1u
LA_API la_status la_ssm_fwd(const void* x, const void* dt, const float* A, const void* b,
                            const void* c, const float* skip, const void* gate,
                            const float* dt_bias, const long long* strides, la_dtype dtype, int B,
                            int T, int D, int N, int G, unsigned flags, const float* h0,
                            const int* positions, void* y, float* h_out, void* workspace,
                            size_t workspace_bytes, la_stream_t stream);
LA_API size_t la_ssm_workspace_size(int B, int T, int D, int N, int G, la_dtype dtype);

/*
 * Gradients of la_ssm_fwd for the loss sum dy . y + <dh_T, h_T>; the states are computed
 * again from the inputs.
 *   x .. positions  as the forward call
 *   dy        [B][T][D] dtype;  dh_T [B][D][N] fp32 or NULL (zero)
 *   strides   HOST array of 11 pairs, for x, dt, b, c, gate, dy, dx, ddt, db, dc and
 *             dgate, or NULL (all dense); the outputs' rows lie apart
 *   dx, ddt, dgate  [B][T][D], db, dc [B][T][G][N] dtype; dgate is NULL exactly when gate
 *             is.  ddt is with respect to dt as given (through the softplus).
 *   dA        fp32 [D][N], dskip, ddt_bias fp32 [D], or NULL: summed over batch and tokens
 *             in a fixed order; overwritten
 *   dh0       [B][D][N] fp32 or NULL
 *   workspace at least la_ssm_bwd_workspace_size(...) bytes; overwritten; one for each
 *             call that may run at once
 * A token that starts a document passes nothing to the tokens before it.  db and dc are summed
 * in fp32 over a group's channels and rounded once.  No output may overlap an input or another
 * output.  B or T == 0: dA, dskip and ddt_bias are zeroed, dh0 is dh_T.  Errors as la_ssm_fwd.
 */
LA_API la_status la_ssm_bwd(const void* x, const void* dt, const float* A, const void* b,
                            const void* c, const float* skip, const void* gate,
                            const float* dt_bias, const void* dy, const long long* strides,
                            la_dtype dtype, int B, int T, int D, int N, int G, unsigned flags,
                            const float* h0, const int* positions, const float* dh_T, void* dx,
                            void* ddt, float* dA, void* db, void* dc, float* dskip, void* dgate,
                            float* ddt_bias, float* dh0, void* workspace, size_t workspace_bytes,
                            la_stream_t stream);
LA_API size_t la_ssm_bwd_workspace_size(int B, int T, int D, int N, int G, la_dtype dtype);

/*
 * One token of la_ssm_fwd: x, dt, gate [B][D], b, c [B][G][N] dtype; strides: HOST array
 * of 5 strides from sequence to sequence, for x, dt, b, c and gate, or NULL (dense);
 * h_in, h_out [B][D][N] fp32, h_out may be h_in itself (a sequence that starts here begins
 * from zeros); y [B][D] dense.
 * Errors as la_ssm_fwd.
 */
LA_API la_status la_ssm_step(const void* x, const void* dt, const float* A, const void* b,
                             const void* c, const float* skip, const void* gate,
                             const float* dt_bias, const long long* strides, la_dtype dtype, int B,
                             int D, int N, int G, unsigned flags, const float* h_in, float* h_out,
                             void* y, la_stream_t stream);

/*
 * The seam between two blocks of a residual stream: the norm after a block, its gate, the
 * residual, and the norm before the next block, in one pass over the rows:
 *
 *   p  = norm(o) post_weight  with LA_BLOCK_POST_NORM, else o
 *   h' = residual_scale h + scale gate p
 *   y  = norm(h') pre_weight  with LA_BLOCK_PRE_NORM
 *   norm(v) = v (mean(v^2) + eps)^(-1/2)       (v less its mean with LA_BLOCK_CENTER)
 *
 *   o, y      [B][T][D] dtype;  h, h_out [B][T][D] residual_dtype: dtype or fp32.  h may be
 *             NULL (no residual), h_out may be NULL (not kept), y is NULL exactly without
 *             LA_BLOCK_PRE_NORM.  Each with 2 strides (batch, token) as la_short_conv_fwd's
 *             x, or NULL for dense; the outputs' rows lie apart.
 *   post_weight, pre_weight  DEVICE fp32 [D] or NULL (ones); NULL without their norm
 *   gate      DEVICE fp32 [D], or [B][D] with LA_BLOCK_GATE_EACH, or NULL (ones)
 *   scale, residual_scale    finite;  eps > 0, finite
 * h_out may be h itself with the same strides; else no output may overlap an input or another
 * output.  y is the norm of h' before its rounding.  Sums in fp32; a row's squares must stay
 * below its range.  D a multiple of 16 up to 8192, B < 65536, B * T at most 2^31 - 256.
 * B or T == 0 is a no-op.  Errors: LA_ERR_INVALID_ARG, LA_ERR_CUDA.
 */
#define LA_BLOCK_POST_NORM 1u
#define LA_BLOCK_PRE_NORM 2u
#define LA_BLOCK_CENTER 4u
#define LA_BLOCK_GATE_EACH 8u
LA_API la_status la_block_norm_fwd(const void* o, const long long* o_strides, la_dtype dtype,
                                   const void* h, const long long* h_strides,
                                   la_dtype residual_dtype, const float* post_weight,
                                   const float* gate, const float* pre_weight, int B, int T, int D,
                                   unsigned flags, float scale, float residual_scale, float eps,
                                   void* h_out, const long long* h_out_strides, void* y,
                                   const long long* y_strides, la_stream_t stream);

/*
 * Gradients of la_block_norm_fwd from its output h_out.
 *   o, post_weight .. eps  as the forward call;  h_out as it left it (read with
 *             LA_BLOCK_PRE_NORM only)
 *   dy        [B][T][D] dtype, NULL exactly without LA_BLOCK_PRE_NORM;  dh_out [B][T][D]
 *             residual_dtype or NULL (zero): the gradient with respect to h_out; one of the
 *             two is given
 *   d_o       [B][T][D] dtype;  dh [B][T][D] residual_dtype or NULL: with respect to h; may
 *             be dh_out itself with the same strides
 *   dpost_weight, dpre_weight fp32 [D], dgate like gate, or NULL: summed over the rows they
 *             are shared by in a fixed order; overwritten
 *   workspace at least la_block_norm_bwd_workspace_size(...) bytes when one of these is asked
 *             for, else may be NULL; one for each call that may run at once
 * No other output may overlap an input or another output.  B or T == 0: the sums are zeroed.
 * Errors as la_block_norm_fwd.
 */
LA_API la_status la_block_norm_bwd(const void* o, const long long* o_strides, la_dtype dtype,
                                   const void* h_out, const long long* h_out_strides,
                                   la_dtype residual_dtype, const void* dy,
                                   const long long* dy_strides, const void* dh_out,
                                   const long long* dh_out_strides, const float* post_weight,
                                   const float* gate, const float* pre_weight, int B, int T, int D,
                                   unsigned flags, float scale, float residual_scale, float eps,
                                   void* d_o, const long long* d_o_strides, void* dh,
                                   const long long* dh_strides, float* dpost_weight, float* dgate,
                                   float* dpre_weight, void* workspace, size_t workspace_bytes,
                                   la_stream_t stream);
LA_API size_t la_block_norm_bwd_workspace_size(int B, int T, int D, la_dtype dtype, unsigned flags);

/*
 * la_chunk_fwd for callers that cannot allocate device memory.  The source
 * pages have no counterpart to this entry point.
 *
 * la_chunk_fwd may need caller-provided scratch (la_workspace_size).  Some
 * callers cannot call cudaMalloc: a plugin inside a host framework that owns
 * every device allocation and passes the plugin only its inputs and outputs,
 * or a serving loop that must not allocate once running (cudaMalloc can
 * synchronise the device and can fail under memory pressure).  This entry
 * point takes the same arguments as la_chunk_fwd minus the workspace and
 * uses instead a fixed scratch array compiled into the library: a file-scope
 * device array of LA_NOALLOC_SCRATCH_BYTES bytes that every GPU loading the
 * library holds until the process exits.  It allocates nothing.
 *
 *   - The first call on a device looks up the array's device address (with
 *     that device current) and caches it.  The cached address holds until the
 *     device is reset (cudaDeviceReset); calls after a reset in the same
 *     process are not supported.
 *   - Calls whose la_workspace_size exceeds LA_NOALLOC_SCRATCH_BYTES return
 *     LA_ERR_INVALID_ARG without launching anything.
 *   - Every call shares the one array, and the array keeps whatever the last
 *     call left in it.  Nothing needs clearing: within a call every scratch
 *     byte is written before it is read (the state walk writes each segment's
 *     contribution, zeros included where no normaliser is carried, before the
 *     scan or the output walk reads it).  Calls that overlap on the GPU
 *     (different streams, or host threads) race on the array and give wrong
 *     results; serialise them.
 *   - Errors otherwise as la_chunk_fwd; LA_ERR_CUDA if the address lookup fails.
 */
#define LA_NOALLOC_SCRATCH_BYTES (16u << 20)
LA_API la_status la_chunk_fwd_noalloc(const void* Q, const void* K, const void* V,
                                      la_dtype dtype, const float* gamma, int B, int H, int T,
                                      int d_k, int d_v, unsigned flags, float eps,
                                      const float* S0, const float* z0,
                                      void* O, float* S_out, float* z_out, int chunk,
                                      int* dev_status, la_stream_t stream);

/*
 * la_chunk_fwd on HOST buffers, the copies included: the end-to-end call for a
 * caller whose inputs and outputs live in host memory (the operation is
 * la_chunk_fwd's; the pages have no counterpart to the copies).
 *
 *   Q, K, V, S0, z0   as la_chunk_fwd, in HOST memory (pinned, e.g. by
 *                     cudaHostAlloc, for the copies to run asynchronously and
 *                     overlap; pageable memory works, with serialised copies)
 *   O, S_out, z_out   as la_chunk_fwd, in HOST memory; written when the call's
 *                     work on `stream` completes
 *   pieces            the batch is cut into `pieces` groups of whole sequences
 *                     (1 <= pieces <= B); piece i is copied in, computed and
 *                     copied out in order on one of two streams the call creates
 *                     (i mod 2), into slot i mod 2 of the arena, so one piece's
 *                     copies overlap another's compute
 *   arena, arena_bytes  caller-owned DEVICE memory of at least
 *                     la_host_arena_size(...) bytes (16-byte aligned): two
 *                     slots of one piece's inputs, outputs and workspace; the
 *                     library allocates nothing
 *   stream            the call's work starts after the work already on `stream`,
 *                     and work enqueued on `stream` afterwards starts after the
 *                     call's (events); the call returns without waiting: the host
 *                     buffers must stay valid, and the outputs are not read, until
 *                     `stream` has passed the call's work
 * gamma and the flags as la_chunk_fwd (the per-token decay is not taken here).
 * Every check of the per-piece calls runs before anything is enqueued.
 * Errors: as la_chunk_fwd; LA_ERR_INVALID_ARG also for pieces outside [1, B],
 * a NULL host input or output when T > 0, or an arena that is too small or
 * misaligned; LA_ERR_CUDA if a copy, stream or event call fails.
 */
LA_API size_t la_host_arena_size(int B, int H, int T, int d_k, int d_v, la_dtype dtype,
                                 unsigned flags, int chunk, int pieces);
LA_API la_status la_chunk_fwd_host(const void* Q, const void* K, const void* V, la_dtype dtype,
                                   const float* gamma, int B, int H, int T, int d_k, int d_v,
                                   unsigned flags, float eps, const float* S0, const float* z0,
                                   void* O, float* S_out, float* z_out, int chunk, int pieces,
                                   void* arena, size_t arena_bytes, int* dev_status,
                                   la_stream_t stream);

/*
 * Test and diagnostic switches (no counterpart on the pages).  Process-wide,
 * all 0 by default; they steer no call unless a test sets them.
 *
 *   LA_OPT_PATH           0: automatic path choice.  1: la_chunk_fwd and
 *                         la_chunk_bwd run on the fp32 CUDA-core kernels
 *                         (la_workspace_size and la_bwd_workspace_size answer
 *                         for that path).  2: la_chunk_fwd runs on the
 *                         tensor-core kernels or answers LA_ERR_UNSUPPORTED.
 *   LA_OPT_TC_LOCKSTEP    1: the tensor-core forward uses its lockstep kernel
 *                         where it would use the pipelined one.
 *   LA_OPT_FORCE_TIMEOUT  1: the tensor-core forward kernels first wait 1 ms on
 *                         a barrier nothing arrives on, then record
 *                         LA_ERR_TIMEOUT in dev_status and return without
 *                         computing (the device status path, exercised with
 *                         neither a hang nor a fault).
 *                         la_scan_fwd and la_scan_bwd on long sequences: the CTAs
 *                         of a cluster send each other nothing, each waits 1 ms,
 *                         and the status is recorded.
 *
 * Returns the option's previous value, or -1 (nothing changed) for an unknown
 * option or an out-of-range value.  Set a switch before enqueuing the calls it
 * should affect; it is read when a call is made, not when its kernels run.
 */
#define LA_OPT_PATH 1
#define LA_OPT_TC_LOCKSTEP 2
#define LA_OPT_FORCE_TIMEOUT 3
LA_API int la_debug_set(int option, int value);

/*
 * Launch tracing (profiling aid; no counterpart on the pages).  While enabled,
 * the library records a pair of CUDA events on the launching stream around
 * every kernel it enqueues, for up to `capacity` launches (capacity <= 0
 * disables tracing and frees the events).  la_trace_collect waits for the
 * recorded launches, writes up to max_records {kernel name, device ms}
 * records (names are static strings) and resets the log; it returns the
 * number written, or -LA_ERR_CUDA.  Not thread-safe across concurrent
 * streams' interleaved calls beyond keeping each record's pair consistent.
 */
typedef struct {
    const char* kernel;
    float ms;
} la_trace_record;

LA_API int la_trace_enable(int capacity);
LA_API int la_trace_collect(la_trace_record* out, int max_records);

#ifdef __cplusplus
}
#endif

#endif /* LINATTN_H */
