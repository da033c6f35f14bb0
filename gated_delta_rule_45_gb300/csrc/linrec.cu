// Gated linear recurrence h_t = a_t h_{t-1} + u_t (include/linrec.h): prefill,
// backward and decode step.
//
// First form: one thread per (sequence, channel) walks its tokens in order.
#include "kda_internal.h"

#include <type_traits>

namespace kda {
namespace {

constexpr int kThreads = 128;

// Gate of token row t, channel c (H x d channels a row): a and 1 - a.
template <int GATE>
__device__ __forceinline__ void gate_at(const void* gate, int64_t t, int c, int H, int d, float& a,
                                        float& na) {
    const int64_t D = (int64_t)H * d;
    if (GATE == KDA_GATE_HEAD_F32) {
        a = static_cast<const float*>(gate)[t * H + c / d];
        na = 1.f - a;
    } else if (GATE == KDA_GATE_CHANNEL_LOG_BF16) {
        const float la = __bfloat162float(static_cast<const __nv_bfloat16*>(gate)[t * D + c]);
        a = expf(la);
        na = -expm1f(la);
    } else {
        a = static_cast<const float*>(gate)[t * D + c];
        na = 1.f - a;
    }
}

template <typename T, int GATE>
__global__ void linrec_fwd_kernel(const LinrecArgs p) {
    if (*p.status) return;
    const int D = p.H * p.d;
    const int c = blockIdx.x * kThreads + threadIdx.x;
    const int n = blockIdx.y;
    if (c >= D) return;
    const T* x = static_cast<const T*>(p.x);
    T* y = static_cast<T*>(p.y);
    float h = p.S0 ? p.S0[(int64_t)n * D + c] : 0.f;
    const int64_t lo = p.cu_seqlens[n], hi = p.cu_seqlens[n + 1];
    for (int64_t t = lo; t < hi; ++t) {
        float a, na;
        gate_at<GATE>(p.gate, t, c, p.H, p.d, a, na);
        if (p.states && t % LINREC_CHUNK == 0)
            p.states[t / LINREC_CHUNK * D + c] = t == lo ? 0.f : h;
        const float xv = Elem<T>::load(x + t * D + c);
        h = fmaf(a, h, p.complement ? na * xv : xv);
        if (y) Elem<T>::store(y + t * D + c, h);
    }
    if (p.S_T) p.S_T[(int64_t)n * D + c] = h;
    if (p.states && n == p.num_seqs - 1)
        for (int64_t i = (hi + LINREC_CHUNK - 1) / LINREC_CHUNK; i * LINREC_CHUNK < p.total_tokens; ++i)
            p.states[i * D + c] = 0.f;
}

// hbuf: fp32 [T][D] states; da: fp32 [T][D], the gradient of each channel's gate.
template <typename T, int GATE>
__global__ void linrec_bwd_kernel(const LinrecArgs p, float* hbuf, float* da_out) {
    if (*p.status) return;
    const int D = p.H * p.d;
    const int c = blockIdx.x * kThreads + threadIdx.x;
    const int n = blockIdx.y;
    if (c >= D) return;
    const T* x = static_cast<const T*>(p.x);
    const T* dy = static_cast<const T*>(p.dy);
    const float h0 = p.S0 ? p.S0[(int64_t)n * D + c] : 0.f;
    const int64_t lo = p.cu_seqlens[n], hi = p.cu_seqlens[n + 1];
    float h = h0;
    for (int64_t t = lo; t < hi; ++t) {
        float a, na;
        gate_at<GATE>(p.gate, t, c, p.H, p.d, a, na);
        const float xv = Elem<T>::load(x + t * D + c);
        h = fmaf(a, h, p.complement ? na * xv : xv);
        hbuf[t * D + c] = h;
    }
    float r = p.dS_T ? p.dS_T[(int64_t)n * D + c] : 0.f;
    for (int64_t t = hi - 1; t >= lo; --t) {
        float a, na;
        gate_at<GATE>(p.gate, t, c, p.H, p.d, a, na);
        const float prev = t == lo ? h0 : hbuf[(t - 1) * D + c];
        const float xv = Elem<T>::load(x + t * D + c);
        const float g = Elem<T>::load(dy + t * D + c) + r;
        p.dx[t * D + c] = p.complement ? na * g : g;
        const float da = g * (p.complement ? prev - xv : prev);
        da_out[t * D + c] = GATE == KDA_GATE_CHANNEL_LOG_BF16 ? a * da : da;
        r = a * g;
    }
    if (p.dS0) p.dS0[(int64_t)n * D + c] = r;
}

__global__ void linrec_head_sum_kernel(const float* da, const int32_t* cu, int32_t num_seqs,
                                       int H, int d, float* dgate, const int32_t* status) {
    if (*status || num_seqs == 0) return;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;   // t * H + h
    if (i >= (int64_t)cu[num_seqs] * H) return;
    float s = 0.f;
    for (int j = 0; j < d; ++j) s += da[i * d + j];
    dgate[i] = s;
}

template <typename T, int GATE>
__global__ void linrec_step_kernel(const LinrecStepArgs p) {
    const int D = p.H * p.d;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (int64_t)p.B * D) return;
    const int b = (int)(i / D), c = (int)(i % D);
    const int row = p.parents ? p.parents[b] : b;
    const float h = row >= 0 && row < p.num_rows ? p.S[(int64_t)row * D + c] : 0.f;
    float a, na;
    gate_at<GATE>(p.gate, b, c, p.H, p.d, a, na);
    const float xv = Elem<T>::load(static_cast<const T*>(p.x) + i);
    const float out = fmaf(a, h, p.complement ? na * xv : xv);
    p.S_out[i] = out;
    Elem<T>::store(static_cast<T*>(p.y) + i, out);
}

template <typename F>
cudaError_t by_type(kda_dtype dtype, int gate, F&& f) {
    if (dtype == KDA_BF16) {
        if (gate == KDA_GATE_HEAD_F32) return f((__nv_bfloat16*)0, std::integral_constant<int, 1>());
        if (gate == KDA_GATE_CHANNEL_LOG_BF16) return f((__nv_bfloat16*)0, std::integral_constant<int, 2>());
        return f((__nv_bfloat16*)0, std::integral_constant<int, 0>());
    }
    if (gate == KDA_GATE_HEAD_F32) return f((float*)0, std::integral_constant<int, 1>());
    if (gate == KDA_GATE_CHANNEL_LOG_BF16) return f((float*)0, std::integral_constant<int, 2>());
    return f((float*)0, std::integral_constant<int, 0>());
}

size_t pad(size_t b) { return (b + 255) & ~(size_t)255; }

cudaError_t plan(const LinrecArgs& a, char* ws, cudaStream_t stream) {
    PrefillArgs pa = {};
    pa.cu_seqlens = a.cu_seqlens; pa.num_seqs = a.num_seqs; pa.total_tokens = a.total_tokens;
    pa.status = reinterpret_cast<int32_t*>(ws + WorkspaceLayout::kStatus);
    pa.counter = reinterpret_cast<int32_t*>(ws + WorkspaceLayout::kCounter);
    pa.order = reinterpret_cast<int32_t*>(ws + WorkspaceLayout::kOrder);
    return launch_planner(pa, stream);
}

}  // namespace

size_t linrec_prefill_bytes(int32_t num_seqs, int64_t, int64_t) {
    return WorkspaceLayout::bytes(num_seqs);
}

size_t linrec_backward_bytes(int32_t num_seqs, int64_t T, int32_t H, int32_t d, int, bool) {
    return WorkspaceLayout::bytes(num_seqs) + 2 * pad((size_t)T * H * d * 4);
}

cudaError_t launch_linrec_prefill(LinrecArgs a, char* ws, cudaStream_t stream) {
    a.status = reinterpret_cast<int32_t*>(ws);
    cudaError_t err = plan(a, ws, stream);
    if (err != cudaSuccess || a.num_seqs == 0) return err;
    const dim3 grid((a.H * a.d + kThreads - 1) / kThreads, a.num_seqs);
    return by_type(a.dtype, a.gate_format, [&](auto* t, auto g) {
        using T = std::remove_pointer_t<decltype(t)>;
        linrec_fwd_kernel<T, decltype(g)::value><<<grid, kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    });
}

cudaError_t launch_linrec_backward(LinrecArgs a, char* ws, cudaStream_t stream) {
    a.status = reinterpret_cast<int32_t*>(ws);
    cudaError_t err = plan(a, ws, stream);
    if (err != cudaSuccess || a.num_seqs == 0) return err;
    const int64_t D = (int64_t)a.H * a.d;
    float* hbuf = reinterpret_cast<float*>(ws + WorkspaceLayout::bytes(a.num_seqs));
    const bool head = a.gate_format == KDA_GATE_HEAD_F32;
    float* da = head ? hbuf + pad((size_t)a.total_tokens * D * 4) / 4 : a.dgate;
    const dim3 grid((unsigned)((D + kThreads - 1) / kThreads), a.num_seqs);
    err = by_type(a.dtype, a.gate_format, [&](auto* t, auto g) {
        using T = std::remove_pointer_t<decltype(t)>;
        linrec_bwd_kernel<T, decltype(g)::value><<<grid, kThreads, 0, stream>>>(a, hbuf, da);
        return cudaGetLastError();
    });
    if (err != cudaSuccess || !head || a.total_tokens == 0) return err;
    const int64_t rows = a.total_tokens * a.H;
    linrec_head_sum_kernel<<<(unsigned)((rows + kThreads - 1) / kThreads), kThreads, 0, stream>>>(
        da, a.cu_seqlens, a.num_seqs, a.H, a.d, a.dgate, a.status);
    return cudaGetLastError();
}

cudaError_t launch_linrec_step(const LinrecStepArgs& a, cudaStream_t stream) {
    const int64_t n = (int64_t)a.B * a.H * a.d;
    return by_type(a.dtype, a.gate_format, [&](auto* t, auto g) {
        using T = std::remove_pointer_t<decltype(t)>;
        linrec_step_kernel<T, decltype(g)::value>
            <<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    });
}

}  // namespace kda
