/*
 * linrec.h -- C ABI of the gated linear recurrence in libkda: the elementwise
 * sibling of the matrix-state recurrence of kda.h.
 *
 * Per (sequence, head, channel), with a_t the forget gate and u_t the input,
 *
 *     h_t = a_t h_{t-1} + u_t,     y_t = h_t,
 *     u_t = x_t               (LINREC_PLAIN)
 *     u_t = (1 - a_t) x_t     (LINREC_COMPLEMENT: a leaky average)
 *
 * Conventions as in kda.h: device pointers owned by the caller, 16-byte
 * aligned, dense row-major tensors, work enqueued on `stream`, argument errors
 * returned synchronously before any launch.  Layouts:
 *
 *     x, y, dy    [T][H][d]   (dtype: KDA_BF16 or KDA_FP32)
 *     gate        by kda_gate_format: [T][H][d] fp32, [T][H] fp32 (one gate
 *                 for all channels of a head), or log a [T][H][d] bf16
 *     state       [N][H][d] fp32
 *
 * The state, the products of gates and every sum are fp32; y is rounded once
 * to dtype.  Gates are meant to lie in [0, 1] (log a <= 0); any finite gates
 * whose products over LINREC_MAX_TILE tokens stay finite give the recurrence's
 * result (beyond that, only a state of zero does: it stays zero).  Of a state
 * that the gates of up to LINREC_MAX_TILE tokens multiply by less than 2^-126,
 * what is left may count as 0.
 * Inputs and states are meant to be finite.  A sequence whose values are not
 * never reaches another sequence's outputs.  Results do not depend on timing:
 * the same call on the same inputs gives the same bits.
 */
#ifndef LINREC_H_
#define LINREC_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    LINREC_PLAIN = 0,
    LINREC_COMPLEMENT = 1
} linrec_input;

/* Tokens between two stored states of linrec_prefill (`states`). */
#define LINREC_CHUNK 128

/* Tokens whose gates' product is formed by itself, at most. */
#define LINREC_MAX_TILE 256

/*
 * Bytes of device workspace linrec_prefill needs: about total_tokens x H x d / 32
 * + num_seqs x H x d x 4.  Returns 0 for a size it does not support.
 * Contents need no initialisation and are overwritten by every call.
 */
size_t linrec_prefill_workspace_size(int32_t num_seqs, int64_t total_tokens, int32_t H,
                                     int32_t d);

/*
 * The recurrence over a packed (varlen) batch: for every sequence n (tokens
 * cu_seqlens[n] .. cu_seqlens[n+1]-1) from S0[n] (zeros when S0 is NULL).
 * Writes y for every token of every sequence and the final states S_T; a
 * zero-length sequence gives S_T[n] = S0[n].  Values of tokens at or past
 * cu_seqlens[num_seqs] have no effect and their y is not written.
 *
 *   cu_seqlens   device int32 [num_seqs+1], as for kda_prefill (checked on the
 *                device: no output is written for a malformed one)
 *   y            output [T][H][d] (dtype)
 *   S_T          output [N][H][d] fp32; may equal S0; may be NULL only when
 *                num_seqs == 0
 *   states       output [ceil(T / LINREC_CHUNK)][H][d] fp32 or NULL: for
 *                linrec_backward, the state that reaches token
 *                i x LINREC_CHUNK (before its gate; 0 where that token starts
 *                a sequence or lies past the last one)
 *   workspace    linrec_prefill_workspace_size bytes, 16-byte aligned, not
 *                shared by calls that may run concurrently
 *
 * kda_prefill_device_status(workspace) reports device-detected errors
 * (KDA_ERR_DEVICE_INPUT; KDA_ERR_DEVICE_TIMEOUT if a wait of the time-axis
 * scan ran out).  Supported: H >= 1, 1 <= d <= 65536, H x d <= 2^20 (odd widths
 * too), total_tokens <= 2^31 - 1 - 128, total_tokens x H x d < 2^45, num_seqs <= 2^30,
 * num_seqs x H x d < 2^40.
 */
kda_status linrec_prefill(const void* x, const void* gate, kda_gate_format gate_format,
                          const float* S0, const int32_t* cu_seqlens, int32_t num_seqs,
                          int64_t total_tokens, int32_t H, int32_t d, kda_dtype dtype,
                          linrec_input input, void* y, float* S_T, float* states,
                          void* workspace, size_t workspace_bytes, kda_stream_t stream);

/* Bytes of device workspace linrec_backward needs; `with_states` is 0 when the
 * call passes no `states` (they are then recomputed into the workspace).
 * Returns 0 for a size or layout it does not support. */
size_t linrec_backward_workspace_size(int32_t num_seqs, int64_t total_tokens, int32_t H,
                                      int32_t d, kda_gate_format gate_format,
                                      int32_t with_states);

/*
 * Backward pass of linrec_prefill on the same inputs, given dy = dL/dy and
 * dS_T = dL/dS_T:
 *
 *     g_t = dy_t + a_{t+1} g_{t+1}        (the last token: dy_t + dS_T)
 *     dx_t = g_t  or  (1 - a_t) g_t,      da_t = g_t (h_{t-1} [- x_t]),
 *     dS0 = a_1 g_1
 *
 *   dy           [T][H][d] (dtype)
 *   dS_T         [N][H][d] fp32 or NULL (zeros)
 *   states       linrec_prefill's `states` for these inputs, or NULL: the
 *                forward scan is run again
 *   dx           output [T][H][d] fp32
 *   dgate        output fp32, the gradient with respect to the gate in its own
 *                layout: [T][H][d], [T][H] (summed over the head's channels),
 *                or [T][H][d] with respect to log a
 *   dS0          output [N][H][d] fp32 or NULL (not written)
 *   workspace    linrec_backward_workspace_size bytes, 16-byte aligned
 *
 * Gradients of tokens at or past cu_seqlens[num_seqs] are not written.  No
 * output may overlap an input or another output.  Device-detected errors and
 * supported sizes as linrec_prefill.
 */
kda_status linrec_backward(const void* x, const void* gate, kda_gate_format gate_format,
                           const float* S0, const int32_t* cu_seqlens, int32_t num_seqs,
                           int64_t total_tokens, int32_t H, int32_t d, kda_dtype dtype,
                           linrec_input input, const void* dy, const float* dS_T,
                           const float* states, float* dx, float* dgate, float* dS0,
                           void* workspace, size_t workspace_bytes, kda_stream_t stream);

/*
 * One token for each of B sequences:
 *
 *     S_out[b] = a[b] S[p] + u[b],  y[b] = S_out[b],  p = parents ? parents[b] : b
 *
 *   x, y      [B][H][d] (dtype)       gate  as above with B in T's place
 *   S         [num_rows][H][d] fp32 (num_rows == B when parents is NULL)
 *   parents   device int32 [B] or NULL: the row of S each sequence continues
 *             (beam search: several may name one row); an entry outside
 *             [0, num_rows) starts from a zero state
 *   S_out     [B][H][d] fp32; may equal S when parents is NULL, else it must
 *             not overlap S
 *
 * Supported: as linrec_prefill; B == 0 is a valid no-op.
 */
kda_status linrec_decode_step(const void* x, const void* gate, kda_gate_format gate_format,
                              const float* S, int32_t num_rows, const int32_t* parents,
                              int32_t B, int32_t H, int32_t d, kda_dtype dtype,
                              linrec_input input, void* y, float* S_out, kda_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LINREC_H_ */
