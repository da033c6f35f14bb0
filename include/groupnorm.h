/*
 * groupnorm.h -- C ABI of the gated group norm in libkda: the norm of each
 * head's output behind a recurrence (kda.h, linrec.h, selscan.h), with its gate
 * or activation in the same pass.
 *
 * Channels last: per (token, head), over the head's d channels,
 *
 *     m = mean(x) or 0 (GROUPNORM_RMS),   r = 1 / sqrt(mean((x - m)^2) + eps),
 *     v = w (x - m) r + b,
 *     y = v act(z)  with a gate z,  or  act(v)  without
 *
 * Conventions as in kda.h: device pointers owned by the caller, 16-byte
 * aligned, dense row-major tensors, work enqueued on `stream`, argument errors
 * returned synchronously before any launch.  Layouts:
 *
 *     x, z      [T] rows of H x d channels, ldx and ldz elements apart (dtype:
 *               KDA_BF16 or KDA_FP32).  Both may start at any element and be
 *               any distance >= H x d apart; rows on a 16-byte grid are read
 *               fastest.
 *     y, dy     [T][H][d] (dtype)
 *     w, b      [H][d] fp32, or [d] for all heads (param_heads == 1); NULL:
 *               ones and zeros
 *
 * Statistics and sums are fp32, the deviations from the mean themselves; y is
 * rounded once to dtype.  A row whose values are not finite never reaches
 * another row's y.  Results do not depend on timing.
 */
#ifndef GROUPNORM_H_
#define GROUPNORM_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GROUPNORM_RMS = 0,    /* the mean stays in */
    GROUPNORM_CENTER = 1  /* the mean is taken off */
} groupnorm_kind;

typedef enum {
    GROUPNORM_IDENTITY = 0,
    GROUPNORM_SILU = 1,
    GROUPNORM_SIGMOID = 2
} groupnorm_activation;

/*
 * The norm of T tokens.
 *
 *   z             gate or NULL (then the activation takes v itself)
 *   param_heads   1 or H: heads of w and b
 *   eps           >= 0, finite (with 0, a head without deviations gives NaN)
 *   y             output [T][H][d] (dtype); may equal x, or z, where those rows
 *                 are dense
 *
 * Supported: H >= 1, 1 <= d <= 16384, H x d <= 2^20, T <= 2^31 - 1,
 * ldx, ldz < 2^40, T x H < 2^40; T == 0 is a valid no-op.
 */
kda_status groupnorm_forward(const void* x, int64_t ldx, const float* w, const float* b,
                             int32_t param_heads, const void* z, int64_t ldz, int64_t T,
                             int32_t H, int32_t d, kda_dtype dtype, groupnorm_kind kind,
                             groupnorm_activation activation, float eps, void* y,
                             kda_stream_t stream);

/* Bytes of device workspace groupnorm_backward needs for these sizes (partial sums of
 * the parameters' gradients).  Returns 0 for a size it does not support. */
size_t groupnorm_backward_workspace_size(int64_t T, int32_t H, int32_t d);

/*
 * Backward pass of groupnorm_forward on the same inputs, given dy = dL/dy.
 *
 *   dx            output [T][H][d] fp32
 *   dz            output [T][H][d] fp32, or NULL (not written; without a gate
 *                 it must be NULL)
 *   dw, db        outputs shaped like w and b (param_heads x d) fp32, or NULL
 *                 (not written); T == 0 gives zeros
 *   workspace     groupnorm_backward_workspace_size bytes, 16-byte aligned, not
 *                 shared by calls that may run concurrently; may be NULL when dw
 *                 and db are
 *
 * No output may overlap an input or another output.  Supported sizes as
 * groupnorm_forward.
 */
kda_status groupnorm_backward(const void* x, int64_t ldx, const float* w, const float* b,
                              int32_t param_heads, const void* z, int64_t ldz, int64_t T,
                              int32_t H, int32_t d, kda_dtype dtype, groupnorm_kind kind,
                              groupnorm_activation activation, float eps, const void* dy,
                              float* dx, float* dz, float* dw, float* db, void* workspace,
                              size_t workspace_bytes, kda_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GROUPNORM_H_ */
