/*
 * beam.h -- C ABI of beam search over recurrent states in libkda: selection
 * over beams and vocabulary, and the moves of the states that follow from it.
 *
 * A batch holds B requests of K beams; row b K + k of every per-beam tensor
 * (logits, states) is beam k of request b, and a parent is such a row.
 *
 * Conventions as in kda.h: device pointers owned by the caller, 16-byte
 * aligned, work enqueued on `stream`, argument errors returned synchronously
 * before any launch.
 */
#ifndef BEAM_H_
#define BEAM_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

#define BEAM_MAX_BEAMS 32     /* K */
#define BEAM_MAX_SELECT 64    /* num_out */

/* Bytes of device workspace beam_select needs; 0 for a size it does not
 * support.  Contents need no initialisation. */
size_t beam_select_workspace_size(int32_t B, int32_t K, int32_t V, int32_t num_out);

/*
 * The num_out best continuations of each request over its K beams and V tokens.
 * Candidate (k, v) has the value
 *
 *     scores[b][k] + logits[b K + k][v] - log sum_w exp(logits[b K + k][w]),
 *
 * formed in 64 bits from the fp32 or bf16 logits and a logarithm of the sum of
 * 32-bit exponentials relative to one near the row's largest: off by 1e-7 as a
 * rule and by less than 3e-6 at worst, wherever the logits lie (equal rows get
 * equal ones).  A finished beam has one candidate, token `eos` at
 * scores[b][k], and its logits are not read.  Candidates are ordered
 * by value, larger first, equal values by k V + v, smaller first.
 *
 *   logits       [B K][ld] (dtype), the first V entries of each row used
 *                (ld >= V, ld x element size a multiple of 16 bytes or ld == V).
 *                -inf masks a token; NaN counts as -inf and +inf as the largest
 *                finite float
 *   scores       [B][K] fp32; -inf for a beam that is not there, NaN counts as
 *                -inf, +inf as the largest finite float
 *   finished     uint8 [B][K], nonzero for a finished beam, or NULL (none is)
 *   eos          token of a finished beam's candidate, 0 <= eos < V (used only
 *                with `finished`)
 *   out_scores   [B][num_out] fp32: the values, best first.  Where fewer than
 *                num_out candidates are above -inf, the rest are -inf, still
 *                in the order of k V + v
 *   out_parents  int32 [B][num_out]: rows b K + k
 *   out_tokens   int32 [B][num_out]
 *   workspace    beam_select_workspace_size bytes, 16-byte aligned, not shared
 *                by calls that may run concurrently
 *
 * Supported: 1 <= K <= BEAM_MAX_BEAMS, 1 <= num_out <= BEAM_MAX_SELECT and
 * num_out <= K V, 1 <= V <= 2^20, B K <= 2^20.  B == 0 is a valid no-op.
 */
kda_status beam_select(const void* logits, int64_t ld, const float* scores,
                       const uint8_t* finished, int32_t B, int32_t K, int32_t V,
                       int32_t num_out, int32_t eos, kda_dtype dtype, float* out_scores,
                       int32_t* out_parents, int32_t* out_tokens, void* workspace,
                       size_t workspace_bytes, kda_stream_t stream);

/* One per-beam tensor of beam_reorder: B K rows of row_bytes bytes. */
typedef struct {
    void* data;
    int64_t row_bytes;
} beam_state;

/*
 * Moves per-beam rows to the beams that continue them, in place and for several
 * tensors at once: row i of each becomes the old row parents[i].  Rows whose
 * parent is themselves are neither read nor written.
 *
 *   states    host array of num_states tensors (any element type and row size)
 *   parents   device int32 [B K]: parents[b K + k] is a row of the same request
 *             (b K .. b K + K - 1); a row whose entry is anything else stays as
 *             it is
 *
 * The tensors must not overlap one another or `parents`.  Supported:
 * 1 <= K <= BEAM_MAX_BEAMS, B K <= 2^20, any row_bytes up to 2^40.
 */
kda_status beam_reorder(const beam_state* states, int32_t num_states, const int32_t* parents,
                        int32_t B, int32_t K, kda_stream_t stream);

/*
 * kda_decode_step_gates with each sequence's state read from its parent's row:
 * S_out[b] = one step from S_in[parents[b]], so that beams move without a pass
 * over the states of their own.
 *
 *   S_in      [num_rows][H][d_v][d_k] fp32
 *   parents   device int32 [B]; several may name one row; an entry outside
 *             [0, num_rows) starts from a zero state
 *   S_out     [B][H][d_v][d_k] fp32, must not overlap S_in
 *
 * Everything else as kda_decode_step_gates.
 */
kda_status kda_decode_step_parents(const void* q, const void* k, const void* v,
                                   const void* alpha, kda_gate_format gate_format,
                                   const float* beta, const float* S_in, int32_t num_rows,
                                   const int32_t* parents, float* S_out, int32_t B, int32_t H,
                                   int32_t d_k, int32_t d_v, kda_dtype dtype, void* o,
                                   kda_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BEAM_H_ */
