// C ABI of the operators around a layer's recurrence: argument validation and dispatch.
// Every entry point is declared and documented in include/causalconv.h, groupnorm.h and
// selscan.h.
#include "layer_ops.h"

#include <math.h>

namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 40;

bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

struct Span {
    const void* p;
    size_t bytes;
};
bool overlaps(const Span& a, const Span& b) {
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}
// Whether an output overlaps an input or another output.  same_out/same_in: a pair that may
// be the same buffer (-1: none).
bool any_overlap(const Span* outs, int n_out, const Span* ins, int n_in, int same_out = -1,
                 int same_in = -1) {
    for (int o = 0; o < n_out; ++o) {
        for (int i = 0; i < n_in; ++i) {
            if (o == same_out && i == same_in && outs[o].p == ins[i].p) continue;
            if (overlaps(outs[o], ins[i])) return true;
        }
        for (int q = o + 1; q < n_out; ++q)
            if (overlaps(outs[o], outs[q])) return true;
    }
    return false;
}
bool all_aligned16(const void* const* ps, int n) {
    for (int i = 0; i < n; ++i)
        if (ps[i] && !aligned(ps[i], 16)) return false;
    return true;
}
size_t elem_bytes(kda_dtype dtype) { return dtype == KDA_BF16 ? 2 : 4; }
bool known(kda_dtype dtype) { return dtype == KDA_BF16 || dtype == KDA_FP32; }
// Bytes from the first to behind the last element of strided rows.
size_t row_bytes(int64_t rows, int64_t ld, int64_t width, size_t esz) {
    return rows > 0 ? ((size_t)(rows - 1) * ld + width) * esz : 0;
}
kda_status launched(cudaError_t err) { return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

kda_status conv_check(int64_t rows, int32_t num_seqs, int32_t D, int32_t W, kda_dtype dtype,
                      causalconv_activation act) {
    if (rows < 0 || num_seqs < 0 || D < 1 || W < 1 || !known(dtype)) return KDA_ERR_INVALID_ARG;
    if (act != CAUSALCONV_LINEAR && act != CAUSALCONV_SILU) return KDA_ERR_INVALID_ARG;
    if (W < 2 || W > 4 || D > (1 << 20) || rows > (int64_t)INT32_MAX - 4096 ||
        num_seqs > (1 << 30))
        return KDA_ERR_UNSUPPORTED;
    // CTAs are counted in 32 bits
    if (rows * D >= (int64_t)1 << 42 || (int64_t)num_seqs * D >= (int64_t)1 << 36)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}
kda_status stride_check(int64_t ld, int64_t width) {
    if (ld < width) return KDA_ERR_INVALID_ARG;
    return ld >= kMaxStride ? KDA_ERR_UNSUPPORTED : KDA_OK;
}

kda_status norm_check(int64_t T, int32_t H, int32_t d, int32_t param_heads, int64_t ldx,
                      int64_t ldz, bool gated, kda_dtype dtype, groupnorm_kind kind,
                      groupnorm_activation act, float eps) {
    if (T < 0 || H < 1 || d < 1 || !known(dtype)) return KDA_ERR_INVALID_ARG;
    if (kind != GROUPNORM_RMS && kind != GROUPNORM_CENTER) return KDA_ERR_INVALID_ARG;
    if (act != GROUPNORM_IDENTITY && act != GROUPNORM_SILU && act != GROUPNORM_SIGMOID)
        return KDA_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || isinf(eps)) return KDA_ERR_INVALID_ARG;
    if (param_heads != 1 && param_heads != H) return KDA_ERR_INVALID_ARG;
    if (d > 16384 || (int64_t)H * d > (1 << 20) || T > (int64_t)INT32_MAX)
        return KDA_ERR_UNSUPPORTED;
    if (T * H >= (int64_t)1 << 40) return KDA_ERR_UNSUPPORTED;
    kda_status st = stride_check(ldx, (int64_t)H * d);
    if (st == KDA_OK && gated) st = stride_check(ldz, (int64_t)H * d);
    return st;
}

}  // namespace

// ---------------------------------------------------------------- causalconv

size_t causalconv_prefill_workspace_size(int32_t num_seqs, int64_t total_tokens, int32_t D,
                                         int32_t W, kda_dtype dtype) {
    if (conv_check(total_tokens, num_seqs, D, W, dtype, CAUSALCONV_LINEAR) != KDA_OK) return 0;
    return kda::conv_prefill_bytes(num_seqs, D, W, dtype);
}

kda_status causalconv_prefill(const void* x, int64_t ldx, const float* w, const float* b,
                              const void* S0, const int32_t* cu_seqlens, int32_t num_seqs,
                              int64_t total_tokens, int32_t D, int32_t W, kda_dtype dtype,
                              causalconv_activation activation, void* y, void* S_T,
                              void* workspace, size_t workspace_bytes, kda_stream_t stream) {
    kda_status st = conv_check(total_tokens, num_seqs, D, W, dtype, activation);
    if (st == KDA_OK) st = stride_check(ldx, D);
    if (st != KDA_OK) return st;
    if (!w || !cu_seqlens || !workspace || (num_seqs > 0 && !S_T)) return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0 && (!x || !y)) return KDA_ERR_INVALID_ARG;
    if (workspace_bytes < kda::conv_prefill_bytes(num_seqs, D, W, dtype))
        return KDA_ERR_INVALID_ARG;
    const size_t esz = elem_bytes(dtype);
    const void* ptrs[] = {w, b, S0, cu_seqlens, y, S_T, workspace};
    if (!all_aligned16(ptrs, 7) || !aligned(x, esz)) return KDA_ERR_INVALID_ARG;
    const size_t n_s = (size_t)num_seqs * (W - 1) * D * esz;
    const Span ins[] = {{x, row_bytes(total_tokens, ldx, D, esz)},
                        {w, (size_t)D * W * 4},
                        {b, (size_t)D * 4},
                        {S0, n_s},
                        {cu_seqlens, ((size_t)num_seqs + 1) * 4},
                        {workspace, workspace_bytes}};
    const Span outs[] = {{y, (size_t)total_tokens * D * esz}, {S_T, n_s}};
    if (any_overlap(outs, 2, ins, 6, 1, 3)) return KDA_ERR_INVALID_ARG;

    kda::ConvArgs a = {};
    a.x = x; a.ldx = ldx; a.w = w; a.b = b; a.S0 = S0; a.cu_seqlens = cu_seqlens;
    a.total_tokens = total_tokens; a.num_seqs = num_seqs; a.D = D; a.W = W; a.dtype = dtype;
    a.silu = activation == CAUSALCONV_SILU; a.y = y; a.S_T = S_T;
    return launched(kda::launch_conv_prefill(a, static_cast<char*>(workspace),
                                             static_cast<cudaStream_t>(stream)));
}

size_t causalconv_backward_workspace_size(int32_t num_seqs, int64_t total_tokens, int32_t D,
                                          int32_t W) {
    if (conv_check(total_tokens, num_seqs, D, W, KDA_BF16, CAUSALCONV_LINEAR) != KDA_OK) return 0;
    return kda::conv_backward_bytes(total_tokens, D, W);
}

kda_status causalconv_backward(const void* x, int64_t ldx, const float* w, const float* b,
                               const void* S0, const int32_t* cu_seqlens, int32_t num_seqs,
                               int64_t total_tokens, int32_t D, int32_t W, kda_dtype dtype,
                               causalconv_activation activation, const void* dy,
                               const float* dS_T, float* dx, float* dw, float* db, float* dS0,
                               void* workspace, size_t workspace_bytes, kda_stream_t stream) {
    kda_status st = conv_check(total_tokens, num_seqs, D, W, dtype, activation);
    if (st == KDA_OK) st = stride_check(ldx, D);
    if (st != KDA_OK) return st;
    if (!w || !cu_seqlens || !workspace || !dw) return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0 && (!x || !dy || !dx)) return KDA_ERR_INVALID_ARG;
    if (workspace_bytes < kda::conv_backward_bytes(total_tokens, D, W)) return KDA_ERR_INVALID_ARG;
    const size_t esz = elem_bytes(dtype);
    const void* ptrs[] = {w, b, S0, cu_seqlens, dy, dS_T, dx, dw, db, dS0, workspace};
    if (!all_aligned16(ptrs, 11) || !aligned(x, esz)) return KDA_ERR_INVALID_ARG;
    const size_t n_s = (size_t)num_seqs * (W - 1) * D, n_x = (size_t)total_tokens * D;
    const Span ins[] = {{x, row_bytes(total_tokens, ldx, D, esz)},
                        {w, (size_t)D * W * 4},
                        {b, (size_t)D * 4},
                        {S0, n_s * esz},
                        {cu_seqlens, ((size_t)num_seqs + 1) * 4},
                        {dy, n_x * esz},
                        {dS_T, n_s * 4},
                        {workspace, workspace_bytes}};
    const Span outs[] = {{dx, n_x * 4}, {dw, (size_t)D * W * 4}, {db, (size_t)D * 4},
                         {dS0, n_s * 4}};
    if (any_overlap(outs, 4, ins, 8)) return KDA_ERR_INVALID_ARG;

    kda::ConvArgs a = {};
    a.x = x; a.ldx = ldx; a.w = w; a.b = b; a.S0 = S0; a.cu_seqlens = cu_seqlens;
    a.total_tokens = total_tokens; a.num_seqs = num_seqs; a.D = D; a.W = W; a.dtype = dtype;
    a.silu = activation == CAUSALCONV_SILU;
    a.dy = dy; a.dS_T = dS_T; a.dx = dx; a.dw = dw; a.db = db; a.dS0 = dS0;
    return launched(kda::launch_conv_backward(a, static_cast<char*>(workspace),
                                              static_cast<cudaStream_t>(stream)));
}

kda_status causalconv_decode_step(const void* x, int64_t ldx, const float* w, const float* b,
                                  const void* S, int32_t num_rows, const int32_t* parents,
                                  int32_t B, int32_t D, int32_t W, kda_dtype dtype,
                                  causalconv_activation activation, void* y, void* S_out,
                                  kda_stream_t stream) {
    if (num_rows < 0) return KDA_ERR_INVALID_ARG;
    kda_status st = conv_check(B, B > num_rows ? B : num_rows, D, W, dtype, activation);
    if (st == KDA_OK) st = stride_check(ldx, D);
    if (st != KDA_OK) return st;
    if (B == 0) return KDA_OK;
    if (!parents && num_rows != B) return KDA_ERR_INVALID_ARG;
    if (!x || !w || (num_rows > 0 && !S) || !y || !S_out) return KDA_ERR_INVALID_ARG;
    const size_t esz = elem_bytes(dtype);
    const void* ptrs[] = {w, b, S, parents, y, S_out};
    if (!all_aligned16(ptrs, 6) || !aligned(x, esz)) return KDA_ERR_INVALID_ARG;
    const size_t n_s = (size_t)(W - 1) * D * esz;
    const Span ins[] = {{x, row_bytes(B, ldx, D, esz)}, {w, (size_t)D * W * 4},
                        {b, (size_t)D * 4},             {parents, (size_t)B * 4},
                        {S, (size_t)num_rows * n_s}};
    const Span outs[] = {{y, (size_t)B * D * esz}, {S_out, (size_t)B * n_s}};
    if (any_overlap(outs, 2, ins, 5, parents ? -1 : 1, 4)) return KDA_ERR_INVALID_ARG;

    kda::ConvStepArgs a = {};
    a.x = x; a.ldx = ldx; a.w = w; a.b = b; a.S = S; a.parents = parents; a.num_rows = num_rows;
    a.B = B; a.D = D; a.W = W; a.dtype = dtype; a.silu = activation == CAUSALCONV_SILU;
    a.y = y; a.S_out = S_out;
    return launched(kda::launch_conv_step(a, static_cast<cudaStream_t>(stream)));
}

// ---------------------------------------------------------------- groupnorm

kda_status groupnorm_forward(const void* x, int64_t ldx, const float* w, const float* b,
                             int32_t param_heads, const void* z, int64_t ldz, int64_t T,
                             int32_t H, int32_t d, kda_dtype dtype, groupnorm_kind kind,
                             groupnorm_activation activation, float eps, void* y,
                             kda_stream_t stream) {
    const kda_status st = norm_check(T, H, d, param_heads, ldx, ldz, z != nullptr, dtype, kind,
                                     activation, eps);
    if (st != KDA_OK) return st;
    if (T == 0) return KDA_OK;
    if (!x || !y) return KDA_ERR_INVALID_ARG;
    const size_t esz = elem_bytes(dtype);
    const int64_t D = (int64_t)H * d;
    const void* ptrs[] = {w, b, y};
    if (!all_aligned16(ptrs, 3) || !aligned(x, esz) || !aligned(z, esz)) return KDA_ERR_INVALID_ARG;
    const size_t n_p = (size_t)param_heads * d * 4;
    const Span out = {y, (size_t)T * D * esz};
    const Span rows[] = {{x, row_bytes(T, ldx, D, esz)}, {z, row_bytes(T, ldz, D, esz)}};
    for (int i = 0; i < 2; ++i) {   // y may take the place of dense rows
        const bool same = rows[i].p == y && (i == 0 ? ldx : ldz) == D;
        if (!same && overlaps(out, rows[i])) return KDA_ERR_INVALID_ARG;
    }
    if (overlaps(out, {w, n_p}) || overlaps(out, {b, n_p})) return KDA_ERR_INVALID_ARG;

    kda::NormArgs a = {};
    a.x = x; a.z = z; a.ldx = ldx; a.ldz = z ? ldz : 0; a.T = T; a.w = w; a.b = b;
    a.param_heads = param_heads; a.H = H; a.d = d; a.dtype = dtype;
    a.center = kind == GROUPNORM_CENTER; a.act = activation; a.eps = eps; a.y = y;
    return launched(kda::launch_norm_forward(a, static_cast<cudaStream_t>(stream)));
}

size_t groupnorm_backward_workspace_size(int64_t T, int32_t H, int32_t d) {
    if (norm_check(T, H, d, 1, (int64_t)H * d, 0, false, KDA_BF16, GROUPNORM_RMS,
                   GROUPNORM_IDENTITY, 0.f) != KDA_OK)
        return 0;
    return kda::norm_backward_bytes(T, H, d);
}

kda_status groupnorm_backward(const void* x, int64_t ldx, const float* w, const float* b,
                              int32_t param_heads, const void* z, int64_t ldz, int64_t T,
                              int32_t H, int32_t d, kda_dtype dtype, groupnorm_kind kind,
                              groupnorm_activation activation, float eps, const void* dy,
                              float* dx, float* dz, float* dw, float* db, void* workspace,
                              size_t workspace_bytes, kda_stream_t stream) {
    const kda_status st = norm_check(T, H, d, param_heads, ldx, ldz, z != nullptr, dtype, kind,
                                     activation, eps);
    if (st != KDA_OK) return st;
    if (dz && !z) return KDA_ERR_INVALID_ARG;
    if (T > 0 && (!x || !dy || !dx)) return KDA_ERR_INVALID_ARG;
    if (dw || db) {
        if (!workspace || workspace_bytes < kda::norm_backward_bytes(T, H, d))
            return KDA_ERR_INVALID_ARG;
    }
    const size_t esz = elem_bytes(dtype);
    const int64_t D = (int64_t)H * d;
    const void* ptrs[] = {w, b, dy, dx, dz, dw, db, workspace};
    if (!all_aligned16(ptrs, 8) || !aligned(x, esz) || !aligned(z, esz)) return KDA_ERR_INVALID_ARG;
    const size_t n_p = (size_t)param_heads * d * 4, n_x = (size_t)T * D;
    const Span ins[] = {{x, row_bytes(T, ldx, D, esz)}, {z, row_bytes(T, ldz, D, esz)},
                        {w, n_p}, {b, n_p}, {dy, n_x * esz}, {workspace, workspace_bytes}};
    const Span outs[] = {{dx, n_x * 4}, {dz, n_x * 4}, {dw, n_p}, {db, n_p}};
    if (any_overlap(outs, 4, ins, 6)) return KDA_ERR_INVALID_ARG;

    kda::NormArgs a = {};
    a.x = x; a.z = z; a.dy = dy; a.ldx = ldx; a.ldz = z ? ldz : 0; a.T = T; a.w = w; a.b = b;
    a.param_heads = param_heads; a.H = H; a.d = d; a.dtype = dtype;
    a.center = kind == GROUPNORM_CENTER; a.act = activation; a.eps = eps;
    a.dx = dx; a.dz = dz; a.dw = dw; a.db = db;
    return launched(kda::launch_norm_backward(a, static_cast<char*>(workspace),
                                              static_cast<cudaStream_t>(stream)));
}

// ---------------------------------------------------------------- selscan

static kda_status scan_check(int64_t rows, int32_t num_seqs, int32_t H, int32_t d, int32_t n) {
    if (rows < 0 || num_seqs < 0 || H < 1 || d < 1 || n < 1) return KDA_ERR_INVALID_ARG;
    if (n > 64 || d > (1 << 20) || (int64_t)H * d > (1 << 20) ||
        rows > (int64_t)INT32_MAX - 4096 || num_seqs > (1 << 30))
        return KDA_ERR_UNSUPPORTED;
    const int64_t D = (int64_t)H * d;
    if (rows * D * n >= (int64_t)1 << 46 || (int64_t)num_seqs * D * n >= (int64_t)1 << 42)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}
static kda_status scan_rows_check(const selscan_rows* r, int64_t T, int32_t H, int32_t d,
                                  int32_t n, kda_dtype dtype, selscan_step step) {
    if (!r || !known(dtype)) return KDA_ERR_INVALID_ARG;
    if (step != SELSCAN_LINEAR_STEP && step != SELSCAN_SOFTPLUS) return KDA_ERR_INVALID_ARG;
    const int64_t D = (int64_t)H * d, P = (int64_t)H * n;
    if (T > 0 && (!r->x || !r->dt || !r->B || !r->C)) return KDA_ERR_INVALID_ARG;
    const size_t esz = elem_bytes(dtype);
    const void* ps[] = {r->x, r->dt, r->B, r->C, r->z};
    for (const void* p : ps)
        if (!aligned(p, esz)) return KDA_ERR_INVALID_ARG;
    const int64_t ld[] = {r->ldx, r->lddt, r->ldB, r->ldC, r->z ? r->ldz : D};
    const int64_t width[] = {D, D, P, P, D};
    for (int i = 0; i < 5; ++i) {
        const kda_status st = stride_check(ld[i], width[i]);
        if (st != KDA_OK) return st;
    }
    return KDA_OK;
}
static void scan_row_spans(const selscan_rows* r, int64_t T, int32_t H, int32_t d, int32_t n,
                           kda_dtype dtype, Span* s) {
    const size_t esz = elem_bytes(dtype);
    const int64_t D = (int64_t)H * d, P = (int64_t)H * n;
    s[0] = {r->x, row_bytes(T, r->ldx, D, esz)};
    s[1] = {r->dt, row_bytes(T, r->lddt, D, esz)};
    s[2] = {r->B, row_bytes(T, r->ldB, P, esz)};
    s[3] = {r->C, row_bytes(T, r->ldC, P, esz)};
    s[4] = {r->z, row_bytes(T, r->ldz, D, esz)};
}

size_t selscan_prefill_workspace_size(int32_t num_seqs, int64_t total_tokens, int32_t H,
                                      int32_t d, int32_t n) {
    if (scan_check(total_tokens, num_seqs, H, d, n) != KDA_OK) return 0;
    return kda::scan_prefill_bytes(num_seqs, total_tokens, H, d, n);
}

kda_status selscan_prefill(const selscan_rows* rows, const float* A, const float* skip,
                           const float* dt_bias, const float* S0, const int32_t* cu_seqlens,
                           int32_t num_seqs, int64_t total_tokens, int32_t H, int32_t d,
                           int32_t n, kda_dtype dtype, selscan_step step, void* y, float* S_T,
                           float* states, void* workspace, size_t workspace_bytes,
                           kda_stream_t stream) {
    kda_status st = scan_check(total_tokens, num_seqs, H, d, n);
    if (st == KDA_OK) st = scan_rows_check(rows, total_tokens, H, d, n, dtype, step);
    if (st != KDA_OK) return st;
    if (!A || !cu_seqlens || !workspace || (num_seqs > 0 && !S_T)) return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0 && !y) return KDA_ERR_INVALID_ARG;
    if (workspace_bytes < kda::scan_prefill_bytes(num_seqs, total_tokens, H, d, n))
        return KDA_ERR_INVALID_ARG;
    const void* ptrs[] = {A, skip, dt_bias, S0, cu_seqlens, y, S_T, states, workspace};
    if (!all_aligned16(ptrs, 9)) return KDA_ERR_INVALID_ARG;
    const size_t D = (size_t)H * d, n_s = (size_t)num_seqs * D * n * 4;
    Span ins[11];
    scan_row_spans(rows, total_tokens, H, d, n, dtype, ins);
    ins[5] = {A, D * n * 4};
    ins[6] = {skip, D * 4};
    ins[7] = {dt_bias, D * 4};
    ins[8] = {S0, n_s};
    ins[9] = {cu_seqlens, ((size_t)num_seqs + 1) * 4};
    ins[10] = {workspace, workspace_bytes};
    const size_t chunks = (size_t)(total_tokens + SELSCAN_CHUNK - 1) / SELSCAN_CHUNK;
    const Span outs[] = {{y, (size_t)total_tokens * D * elem_bytes(dtype)}, {S_T, n_s},
                         {states, chunks * D * n * 4}};
    if (any_overlap(outs, 3, ins, 11, 1, 8)) return KDA_ERR_INVALID_ARG;

    kda::ScanArgs a = {};
    a.in = *rows; a.A = A; a.skip = skip; a.dt_bias = dt_bias; a.S0 = S0;
    a.cu_seqlens = cu_seqlens; a.total_tokens = total_tokens; a.num_seqs = num_seqs; a.H = H;
    a.d = d; a.n = n; a.dtype = dtype; a.softplus = step == SELSCAN_SOFTPLUS;
    a.y = y; a.S_T = S_T; a.states = states;
    return launched(kda::launch_scan_prefill(a, static_cast<char*>(workspace),
                                             static_cast<cudaStream_t>(stream)));
}

size_t selscan_backward_workspace_size(int32_t num_seqs, int64_t total_tokens, int32_t H,
                                       int32_t d, int32_t n, int32_t with_states) {
    if (scan_check(total_tokens, num_seqs, H, d, n) != KDA_OK) return 0;
    return kda::scan_backward_bytes(num_seqs, total_tokens, H, d, n, with_states != 0);
}

kda_status selscan_backward(const selscan_rows* rows, const float* A, const float* skip,
                            const float* dt_bias, const float* S0, const int32_t* cu_seqlens,
                            int32_t num_seqs, int64_t total_tokens, int32_t H, int32_t d,
                            int32_t n, kda_dtype dtype, selscan_step step, const void* dy,
                            const float* dS_T, const float* states, const selscan_grads* grads,
                            void* workspace, size_t workspace_bytes, kda_stream_t stream) {
    kda_status st = scan_check(total_tokens, num_seqs, H, d, n);
    if (st == KDA_OK) st = scan_rows_check(rows, total_tokens, H, d, n, dtype, step);
    if (st != KDA_OK) return st;
    if (!A || !cu_seqlens || !workspace || !grads || !grads->dA) return KDA_ERR_INVALID_ARG;
    const selscan_grads& g = *grads;
    if (total_tokens > 0 && (!dy || !g.dx || !g.ddt || !g.dB || !g.dC || (rows->z && !g.dz)))
        return KDA_ERR_INVALID_ARG;
    if (g.dz && !rows->z) return KDA_ERR_INVALID_ARG;
    if (workspace_bytes < kda::scan_backward_bytes(num_seqs, total_tokens, H, d, n,
                                                   states != nullptr))
        return KDA_ERR_INVALID_ARG;
    const void* ptrs[] = {A, skip, dt_bias, S0, cu_seqlens, dy, dS_T, states, workspace, g.dx,
                          g.ddt, g.dB, g.dC, g.dz, g.dA, g.dskip, g.ddt_bias, g.dS0};
    if (!all_aligned16(ptrs, 18)) return KDA_ERR_INVALID_ARG;
    const size_t D = (size_t)H * d, n_s = (size_t)num_seqs * D * n * 4;
    const size_t n_x = (size_t)total_tokens * D, n_p = (size_t)total_tokens * H * n * 4;
    const size_t chunks = (size_t)(total_tokens + SELSCAN_CHUNK - 1) / SELSCAN_CHUNK;
    Span ins[14];
    scan_row_spans(rows, total_tokens, H, d, n, dtype, ins);
    ins[5] = {A, D * n * 4};
    ins[6] = {skip, D * 4};
    ins[7] = {dt_bias, D * 4};
    ins[8] = {S0, n_s};
    ins[9] = {cu_seqlens, ((size_t)num_seqs + 1) * 4};
    ins[10] = {dy, n_x * elem_bytes(dtype)};
    ins[11] = {dS_T, n_s};
    ins[12] = {states, chunks * D * n * 4};
    ins[13] = {workspace, workspace_bytes};
    const Span outs[] = {{g.dx, n_x * 4}, {g.ddt, n_x * 4}, {g.dB, n_p}, {g.dC, n_p},
                         {g.dz, n_x * 4}, {g.dA, D * n * 4}, {g.dskip, D * 4},
                         {g.ddt_bias, D * 4}, {g.dS0, n_s}};
    if (any_overlap(outs, 9, ins, 14)) return KDA_ERR_INVALID_ARG;

    kda::ScanArgs a = {};
    a.in = *rows; a.A = A; a.skip = skip; a.dt_bias = dt_bias; a.S0 = S0;
    a.cu_seqlens = cu_seqlens; a.total_tokens = total_tokens; a.num_seqs = num_seqs; a.H = H;
    a.d = d; a.n = n; a.dtype = dtype; a.softplus = step == SELSCAN_SOFTPLUS;
    a.states = const_cast<float*>(states); a.dy = dy; a.dS_T = dS_T; a.g = g;
    return launched(kda::launch_scan_backward(a, static_cast<char*>(workspace),
                                              static_cast<cudaStream_t>(stream)));
}

kda_status selscan_decode_step(const selscan_rows* rows, const float* A, const float* skip,
                               const float* dt_bias, const float* S, int32_t num_rows,
                               const int32_t* parents, int32_t B, int32_t H, int32_t d,
                               int32_t n, kda_dtype dtype, selscan_step step, void* y,
                               float* S_out, kda_stream_t stream) {
    if (num_rows < 0) return KDA_ERR_INVALID_ARG;
    kda_status st = scan_check(B, B > num_rows ? B : num_rows, H, d, n);
    if (st == KDA_OK) st = scan_rows_check(rows, B, H, d, n, dtype, step);
    if (st != KDA_OK) return st;
    if (B == 0) return KDA_OK;
    if ((int64_t)B * H * d >= (int64_t)1 << 35) return KDA_ERR_UNSUPPORTED;
    int32_t rows_a_warp;
    if (kda::scan_step_blocks(B, H, d, &rows_a_warp) > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (!parents && num_rows != B) return KDA_ERR_INVALID_ARG;
    if (!A || (num_rows > 0 && !S) || !y || !S_out) return KDA_ERR_INVALID_ARG;
    const void* ptrs[] = {A, skip, dt_bias, S, parents, y, S_out};
    if (!all_aligned16(ptrs, 7)) return KDA_ERR_INVALID_ARG;
    const size_t D = (size_t)H * d;
    Span ins[10];
    scan_row_spans(rows, B, H, d, n, dtype, ins);
    ins[5] = {A, D * n * 4};
    ins[6] = {skip, D * 4};
    ins[7] = {dt_bias, D * 4};
    ins[8] = {parents, (size_t)B * 4};
    ins[9] = {S, (size_t)num_rows * D * n * 4};
    const Span outs[] = {{y, (size_t)B * D * elem_bytes(dtype)}, {S_out, (size_t)B * D * n * 4}};
    if (any_overlap(outs, 2, ins, 10, parents ? -1 : 1, 9)) return KDA_ERR_INVALID_ARG;

    kda::ScanStepArgs a = {};
    a.in = *rows; a.A = A; a.skip = skip; a.dt_bias = dt_bias; a.S = S; a.parents = parents;
    a.num_rows = num_rows; a.B = B; a.H = H; a.d = d; a.n = n; a.dtype = dtype;
    a.softplus = step == SELSCAN_SOFTPLUS; a.y = y; a.S_out = S_out;
    return launched(kda::launch_scan_step(a, static_cast<cudaStream_t>(stream)));
}
