/*
 * causalconv.h -- C ABI of the short causal convolution in libkda: the
 * depthwise filter over the last few tokens that a layer applies to the inputs
 * of its recurrence (q, k and v of kda.h, x of selscan.h).
 *
 * Per (sequence, channel), with x_t = 0 or the stored inputs before the
 * sequence's first token,
 *
 *     v_t = b + sum_{j=0}^{W-1} w_j x_{t-W+1+j},     y_t = v_t  or  silu(v_t)
 *
 * Conventions as in kda.h: device pointers owned by the caller, 16-byte
 * aligned, dense row-major tensors, work enqueued on `stream`, argument errors
 * returned synchronously before any launch.  Layouts:
 *
 *     x         [T] rows of D channels, ldx elements apart (dtype: KDA_BF16 or
 *               KDA_FP32).  x alone may start at any element and ldx >= D may
 *               be any distance (a slice of a wider projection); rows on a
 *               16-byte grid are read fastest.
 *     y, dy     [T][D] (dtype)
 *     w         [D][W] fp32, w[c][W-1] the weight of the token itself
 *     b         [D] fp32 or NULL (zeros)
 *     state     [N][W-1][D] (dtype): the last W-1 inputs, oldest first
 *
 * Sums are fp32; y is rounded once to dtype.  States are copies of inputs.  A
 * sequence whose values are not finite never reaches another sequence's
 * outputs.  Results do not depend on timing: the same call on the same inputs
 * gives the same bits.
 */
#ifndef CAUSALCONV_H_
#define CAUSALCONV_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    CAUSALCONV_LINEAR = 0,
    CAUSALCONV_SILU = 1
} causalconv_activation;

/*
 * Bytes of device workspace causalconv_prefill needs (a status word and room
 * for the states).  Returns 0 for a size it does not support.  Contents need no
 * initialisation and are overwritten by every call.
 */
size_t causalconv_prefill_workspace_size(int32_t num_seqs, int64_t total_tokens, int32_t D,
                                         int32_t W, kda_dtype dtype);

/*
 * The convolution over a packed (varlen) batch: for every sequence n (tokens
 * cu_seqlens[n] .. cu_seqlens[n+1]-1) behind the inputs S0[n] (zeros when S0 is
 * NULL).  Writes y for every token of every sequence and the final states S_T: a
 * sequence shorter than W-1 keeps the end of S0[n].  Values of tokens at or past
 * cu_seqlens[num_seqs] have no effect and their y is not written.
 *
 *   cu_seqlens   device int32 [num_seqs+1], as for kda_prefill (checked on the
 *                device: no output is written for a malformed one)
 *   S_T          output [N][W-1][D] (dtype); may equal S0; may be NULL only when
 *                num_seqs == 0
 *   workspace    causalconv_prefill_workspace_size bytes, 16-byte aligned, not
 *                shared by calls that may run concurrently
 *
 * kda_prefill_device_status(workspace) reports device-detected errors
 * (KDA_ERR_DEVICE_INPUT).  Supported: 2 <= W <= 4, 1 <= D <= 2^20,
 * total_tokens <= 2^31 - 1 - 4096, num_seqs <= 2^30, ldx < 2^40, T x D < 2^42,
 * num_seqs x D < 2^36.
 */
kda_status causalconv_prefill(const void* x, int64_t ldx, const float* w, const float* b,
                              const void* S0, const int32_t* cu_seqlens, int32_t num_seqs,
                              int64_t total_tokens, int32_t D, int32_t W, kda_dtype dtype,
                              causalconv_activation activation, void* y, void* S_T,
                              void* workspace, size_t workspace_bytes, kda_stream_t stream);

/* Bytes of device workspace causalconv_backward needs: at most about T x D x (W + 1) / 8.
 * Returns 0 for a size it does not support. */
size_t causalconv_backward_workspace_size(int32_t num_seqs, int64_t total_tokens, int32_t D,
                                          int32_t W);

/*
 * Backward pass of causalconv_prefill on the same inputs, given dy = dL/dy and
 * dS_T = dL/dS_T:
 *
 *     dv_t = dy_t  or  dy_t silu'(v_t)
 *     dx_t = sum_j w_j dv_{t+W-1-j}  [+ dS_T's row of token t],
 *     dw_j = sum_t dv_t x_{t-W+1+j},   db = sum_t dv_t,
 *     dS0  = the same sums for the inputs before the first token
 *
 *   dy           [T][D] (dtype)
 *   dS_T         [N][W-1][D] fp32 or NULL (zeros)
 *   dx           output [T][D] fp32
 *   dw           output [D][W] fp32
 *   db           output [D] fp32 or NULL (not written)
 *   dS0          output [N][W-1][D] fp32 or NULL (not written)
 *   workspace    causalconv_backward_workspace_size bytes, 16-byte aligned
 *
 * Gradients of tokens at or past cu_seqlens[num_seqs] are not written.  No
 * output may overlap an input or another output.  Device-detected errors and
 * supported sizes as causalconv_prefill.
 */
kda_status causalconv_backward(const void* x, int64_t ldx, const float* w, const float* b,
                               const void* S0, const int32_t* cu_seqlens, int32_t num_seqs,
                               int64_t total_tokens, int32_t D, int32_t W, kda_dtype dtype,
                               causalconv_activation activation, const void* dy,
                               const float* dS_T, float* dx, float* dw, float* db, float* dS0,
                               void* workspace, size_t workspace_bytes, kda_stream_t stream);

/*
 * One token for each of B sequences: y[b] behind the inputs S[p], p = parents ?
 * parents[b] : b, and S_out[b] = the last W-1 of S[p] and x[b].
 *
 *   x         [B] rows, ldx apart        y  [B][D] (dtype)
 *   S         [num_rows][W-1][D] (dtype) (num_rows == B when parents is NULL)
 *   parents   device int32 [B] or NULL: the row of S each sequence continues
 *             (beam search: several may name one row); an entry outside
 *             [0, num_rows) starts from zeros
 *   S_out     [B][W-1][D] (dtype); may equal S when parents is NULL, else it
 *             must not overlap S
 *
 * Supported: as causalconv_prefill; B == 0 is a valid no-op.
 */
kda_status causalconv_decode_step(const void* x, int64_t ldx, const float* w, const float* b,
                                  const void* S, int32_t num_rows, const int32_t* parents,
                                  int32_t B, int32_t D, int32_t W, kda_dtype dtype,
                                  causalconv_activation activation, void* y, void* S_out,
                                  kda_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CAUSALCONV_H_ */
