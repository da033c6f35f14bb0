/*
 * selscan.h -- C ABI of the selective state space scan in libkda: a diagonal
 * recurrence whose step sizes, input and output projections come with each
 * token.
 *
 * Per (sequence, group, channel), with a state h of n values,
 *
 *     D_t = softplus(dt_t + dt_bias)  (SELSCAN_SOFTPLUS)  or  dt_t + dt_bias,
 *     h_t = exp(D_t A) h_{t-1} + D_t x_t B_t         (over the n values),
 *     y_t = (C_t . h_t + skip x_t) silu(z_t)
 *
 * B and C are shared by the d channels of a group (H groups; H = 1 for one
 * projection of all channels).  Conventions as in kda.h: device pointers owned
 * by the caller, 16-byte aligned, dense row-major tensors, work enqueued on
 * `stream`, argument errors returned synchronously before any launch.  Layouts:
 *
 *     x, dt, z     [T] rows of H x d channels (dtype: KDA_BF16 or KDA_FP32)
 *     B, C         [T] rows of H x n values (dtype)
 *     y, dy        [T][H][d] (dtype)
 *     A            [H][d][n] fp32
 *     skip, dt_bias  [H][d] fp32 or NULL (zeros)
 *     z            or NULL (no gate)
 *     state        [N][H][d][n] fp32
 *
 * x, dt, B, C and z have a distance between rows, in elements (selscan_rows):
 * they may start at any element and be any distance apart that holds a row (slices
 * of a wider projection); rows on a 16-byte grid are read fastest.
 *
 * The state, step sizes, decays and every sum are fp32; y is rounded once to
 * dtype.  D_t A is meant to be <= 0; any finite one gives the recurrence's
 * result as long as the states, and the decays' products over the tokens of a
 * sequence, stay finite, and backward their gradients, the products of both and
 * of those with a rate.  A decay below 2^-126 may count as 0, and so may a step
 * below that and what products of decays below that leave of a state.  Rates
 * beyond 2.3e38 in size (the type's lowest value, -inf) count as that: they leave
 * nothing of a state at any step that is not 0.
 * A sequence whose values are not finite never reaches another sequence's
 * outputs.  Results do not depend on timing: the same call on the same inputs
 * gives the same bits.
 */
#ifndef SELSCAN_H_
#define SELSCAN_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SELSCAN_LINEAR_STEP = 0,
    SELSCAN_SOFTPLUS = 1
} selscan_step;

/* Tokens between two stored states of selscan_prefill (`states`). */
#define SELSCAN_CHUNK 16

/* The token inputs and the distances between their rows, in elements. */
typedef struct {
    const void *x, *dt, *B, *C, *z;
    int64_t ldx, lddt, ldB, ldC, ldz;
} selscan_rows;

/*
 * Bytes of device workspace selscan_prefill needs on the current device.
 * Returns 0 for a size it does not support.  Contents need no initialisation
 * and are overwritten by every call.
 */
size_t selscan_prefill_workspace_size(int32_t num_seqs, int64_t total_tokens, int32_t H,
                                      int32_t d, int32_t n);

/*
 * The scan over a packed (varlen) batch: for every sequence s (tokens
 * cu_seqlens[s] .. cu_seqlens[s+1]-1) from S0[s] (zeros when S0 is NULL).
 * Writes y for every token of every sequence and the final states S_T; a
 * zero-length sequence gives S_T[s] = S0[s].  Values of tokens at or past
 * cu_seqlens[num_seqs] have no effect and their y is not written.
 *
 *   cu_seqlens   device int32 [num_seqs+1], as for kda_prefill (checked on the
 *                device: no output is written for a malformed one)
 *   S_T          output [N][H][d][n] fp32; may equal S0; may be NULL only when
 *                num_seqs == 0
 *   states       output [ceil(T / SELSCAN_CHUNK)][H][d][n] fp32 or NULL: for
 *                selscan_backward, the state that reaches token
 *                i x SELSCAN_CHUNK (before its decay), where that token lies
 *                inside a sequence, behind its first; other rows are not
 *                written
 *   workspace    selscan_prefill_workspace_size bytes, 16-byte aligned, not
 *                shared by calls that may run concurrently
 *
 * Long sequences are spread over the GPU by their tokens where num_seqs x H x d is
 * too small to fill it, whatever their lengths: in a batch of many, one that is far
 * longer than the rest is walked by itself (some 125 ns a token, backward 525), and is
 * done sooner by a call of its own.
 *
 * kda_prefill_device_status(workspace) reports device-detected errors
 * (KDA_ERR_DEVICE_INPUT).  Supported: H >= 1, d >= 1, 1 <= n <= 64,
 * H x d <= 2^20, total_tokens <= 2^31 - 1 - 4096, num_seqs <= 2^30,
 * distances between rows < 2^40, T x H x d x n < 2^46, num_seqs x H x d x n < 2^42.
 */
kda_status selscan_prefill(const selscan_rows* rows, const float* A, const float* skip,
                           const float* dt_bias, const float* S0, const int32_t* cu_seqlens,
                           int32_t num_seqs, int64_t total_tokens, int32_t H, int32_t d,
                           int32_t n, kda_dtype dtype, selscan_step step, void* y, float* S_T,
                           float* states, void* workspace, size_t workspace_bytes,
                           kda_stream_t stream);

/* Bytes of device workspace selscan_backward needs on the current device; `with_states` is
 * 0 when the call passes no `states` (they are then recomputed into the workspace).
 * Where a group's channels take several CTAs (128, 64, 32 or 16 channels each, for n up
 * to 8, 16, 32 or 64) their sums for dB and dC come first: 8 T H n bytes a CTA of a group
 * (1.1 GB for 131072 x 4096 channels of 16 values, 17 GB of 64).
 * Returns 0 for a size it does not support. */
size_t selscan_backward_workspace_size(int32_t num_seqs, int64_t total_tokens, int32_t H,
                                       int32_t d, int32_t n, int32_t with_states);

/* Gradients of selscan_backward, all fp32 and dense. */
typedef struct {
    float *dx, *ddt;        /* [T][H][d]; ddt with respect to dt (before softplus) */
    float *dB, *dC;         /* [T][H][n] */
    float *dz;              /* [T][H][d]; NULL without a gate, and only then */
    float *dA;              /* [H][d][n] */
    float *dskip, *ddt_bias;  /* [H][d], or NULL (not written) */
    float *dS0;             /* [N][H][d][n], or NULL (not written) */
} selscan_grads;

/*
 * Backward pass of selscan_prefill on the same inputs, given dy = dL/dy and
 * dS_T = dL/dS_T.  With dr_t = dy_t silu(z_t) and g_t the gradient of h_t,
 *
 *     g_t  = C_t dr_t + exp(D_{t+1} A) g_{t+1}    (the last token: + dS_T)
 *     dB_t = sum over channels of g_t D_t x_t,    dC_t = of h_t dr_t,
 *     dA   = sum_t g_t exp(D_t A) h_{t-1} D_t,    dx_t = D_t B_t . g_t + skip dr_t,
 *     dD_t = x_t B_t . g_t + A . (g_t exp(D_t A) h_{t-1})
 *
 *   dy           [T][H][d] (dtype)
 *   dS_T         [N][H][d][n] fp32 or NULL (zeros)
 *   states       selscan_prefill's `states` for these inputs, or NULL: the
 *                forward scan is run again
 *   grads        the outputs
 *   workspace    selscan_backward_workspace_size bytes, 16-byte aligned
 *
 * Gradients of tokens at or past cu_seqlens[num_seqs] are not written.  No
 * output may overlap an input or another output.  Device-detected errors and
 * supported sizes as selscan_prefill.
 */
kda_status selscan_backward(const selscan_rows* rows, const float* A, const float* skip,
                            const float* dt_bias, const float* S0, const int32_t* cu_seqlens,
                            int32_t num_seqs, int64_t total_tokens, int32_t H, int32_t d,
                            int32_t n, kda_dtype dtype, selscan_step step, const void* dy,
                            const float* dS_T, const float* states, const selscan_grads* grads,
                            void* workspace, size_t workspace_bytes, kda_stream_t stream);

/*
 * One token for each of B sequences, from row p = parents ? parents[b] : b of S:
 *
 *     S_out[b] = exp(D[b] A) S[p] + D[b] x[b] B[b],
 *     y[b] = (C[b] . S_out[b] + skip x[b]) silu(z[b])
 *
 *   rows      with B in T's place        y  [B][H][d] (dtype)
 *   S         [num_rows][H][d][n] fp32 (num_rows == B when parents is NULL)
 *   parents   device int32 [B] or NULL: the row of S each sequence continues
 *             (beam search: several may name one row); an entry outside
 *             [0, num_rows) starts from a zero state
 *   S_out     [B][H][d][n] fp32; may equal S when parents is NULL, else it must
 *             not overlap S
 *
 * Supported: as selscan_prefill with B in T's place and B or num_rows in num_seqs'; B x H x d
 * < 2^35 and ceil(B / 4) x H x ceil(d / 32) <= 2^33 - 4 (which groups of one channel can pass
 * by itself); B == 0 is a valid no-op.
 */
kda_status selscan_decode_step(const selscan_rows* rows, const float* A, const float* skip,
                               const float* dt_bias, const float* S, int32_t num_rows,
                               const int32_t* parents, int32_t B, int32_t H, int32_t d,
                               int32_t n, kda_dtype dtype, selscan_step step, void* y,
                               float* S_out, kda_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SELSCAN_H_ */
