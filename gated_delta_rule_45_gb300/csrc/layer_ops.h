// Arguments, launchers and device helpers of the operators around a layer's recurrence:
// the short causal convolution, the selective scan and the gated group norm.
#pragma once

#include "causalconv.h"
#include "groupnorm.h"
#include "kda_internal.h"
#include "selscan.h"

namespace kda {

// Arguments as in causalconv.h.
struct ConvArgs {
    const void* x;
    int64_t ldx;
    const float *w, *b;
    const void* S0;
    const int32_t* cu_seqlens;
    int64_t total_tokens;
    int32_t num_seqs, D, W;
    kda_dtype dtype;
    int32_t silu;
    // prefill
    void *y = nullptr, *S_T = nullptr;
    // backward
    const void* dy = nullptr;
    const float* dS_T = nullptr;
    float *dx = nullptr, *dw = nullptr, *db = nullptr, *dS0 = nullptr;
};
struct ConvStepArgs {
    const void* x;
    int64_t ldx;
    const float *w, *b;
    const void* S;
    const int32_t* parents;   // or null
    int32_t num_rows, B, D, W;
    kda_dtype dtype;
    int32_t silu;
    void *y, *S_out;
};
size_t conv_prefill_bytes(int32_t num_seqs, int32_t D, int32_t W, kda_dtype dtype);
size_t conv_backward_bytes(int64_t total_tokens, int32_t D, int32_t W);
cudaError_t launch_conv_prefill(const ConvArgs& a, char* ws, cudaStream_t stream);
cudaError_t launch_conv_backward(const ConvArgs& a, char* ws, cudaStream_t stream);
cudaError_t launch_conv_step(const ConvStepArgs& a, cudaStream_t stream);

// Arguments as in groupnorm.h.
struct NormArgs {
    const void *x, *z, *dy;
    int64_t ldx, ldz, T;
    const float *w, *b;
    int32_t param_heads, H, d;
    kda_dtype dtype;
    int32_t center, act;
    float eps;
    void* y;
    float *dx, *dz, *dw, *db;
};
size_t norm_backward_bytes(int64_t T, int32_t H, int32_t d);
cudaError_t launch_norm_forward(const NormArgs& a, cudaStream_t stream);
cudaError_t launch_norm_backward(const NormArgs& a, char* ws, cudaStream_t stream);

// Arguments as in selscan.h.
struct ScanArgs {
    selscan_rows in;
    const float *A, *skip, *dt_bias, *S0;
    const int32_t* cu_seqlens;
    int64_t total_tokens;
    int32_t num_seqs, H, d, n;
    kda_dtype dtype;
    int32_t softplus;
    // prefill
    void* y = nullptr;
    float *S_T = nullptr, *states = nullptr;   // backward: states is an input
    // backward
    const void* dy = nullptr;
    const float* dS_T = nullptr;
    selscan_grads g = {};
};
struct ScanStepArgs {
    selscan_rows in;
    const float *A, *skip, *dt_bias, *S;
    const int32_t* parents;   // or null
    int32_t num_rows, B, H, d, n;
    kda_dtype dtype;
    int32_t softplus;
    void* y;
    float* S_out;
};
size_t scan_prefill_bytes(int32_t num_seqs, int64_t total_tokens, int32_t H, int32_t d, int32_t n);
size_t scan_backward_bytes(int32_t num_seqs, int64_t total_tokens, int32_t H, int32_t d, int32_t n,
                           bool with_states);
cudaError_t launch_scan_prefill(const ScanArgs& a, char* ws, cudaStream_t stream);
cudaError_t launch_scan_backward(const ScanArgs& a, char* ws, cudaStream_t stream);
cudaError_t launch_scan_step(const ScanStepArgs& a, cudaStream_t stream);

// Sums of the rows of part [rows][n1 + n2] in a fixed order: the first n1 columns to out1, the
// others to out2, either of which may be null.  Nothing is written when *status (may be
// null) says that the offsets are malformed.  (causalconv.cu)
cudaError_t launch_column_sums(const float* part, int64_t rows, int64_t n1, int64_t n2,
                               float* out1, float* out2, const int32_t* status,
                               cudaStream_t stream);
// status = whether the offsets are well formed; nothing for up to kSelfCheck sequences, unless
// `always`.
cudaError_t launch_offsets_check(const int32_t* cu, int32_t N, int64_t T, int32_t* status,
                                 cudaStream_t stream, bool always = false);

constexpr int kSelfCheck = 1024;   // most sequences whose offsets every CTA checks by itself

#ifdef __CUDACC__

// Whether cu_seqlens is well formed; all threads of the CTA call it.  The first CTA leaves the
// outcome in *status (for large batches launch_offsets_check has).
__device__ __forceinline__ bool offsets_ok(const int32_t* cu, int32_t N, int64_t T,
                                           int32_t* status) {
    if (N > kSelfCheck) return *reinterpret_cast<volatile int32_t*>(status) == KDA_OK;
    bool bad = false;
    for (int i = threadIdx.x; i <= N; i += blockDim.x) {
        const int32_t c = cu[i];
        bad |= i == 0 ? c != 0 : c < cu[i - 1];
        bad |= i == N && (int64_t)c > T;
    }
    bad = __syncthreads_or(bad);
    if (blockIdx.x == 0 && threadIdx.x == 0) *status = bad ? KDA_ERR_DEVICE_INPUT : KDA_OK;
    return !bad;
}

// The sequence of token t < cu[N]: cu[n] <= t < cu[n + 1].
__device__ __forceinline__ int32_t sequence_of(const int32_t* cu, int32_t N, int64_t t) {
    int32_t lo = 0, hi = N;   // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
        const int32_t m = lo + (hi - lo) / 2;
        if (cu[m] <= t) lo = m; else hi = m;
    }
    return lo;
}

// V neighbouring values as stored: 16, 8 or 4 bytes at once, or one by one.
template <typename T, int V>
struct Pack {
    static constexpr int kWords = V * sizeof(T) / 4;
    uint32_t w[kWords > 0 ? kWords : 1];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (V * sizeof(T) == 16) {
            const uint4 u = *reinterpret_cast<const uint4*>(p);
            w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
        } else if constexpr (V * sizeof(T) == 8) {
            const uint2 u = *reinterpret_cast<const uint2*>(p);
            w[0] = u.x; w[1] = u.y;
        } else if constexpr (V * sizeof(T) == 4) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
            w[0] = *reinterpret_cast<const uint16_t*>(p);
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (kWords > 0 ? kWords : 1); ++i) w[i] = 0;
    }
    __device__ __forceinline__ float get(int i) const {   // i known at compile time
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
    __device__ __forceinline__ void set(const float (&v)[V]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] = __float_as_uint(v[i]);
        } else if constexpr (V == 1) {
            w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (V * sizeof(T) == 16)
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (V * sizeof(T) == 8)
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else if constexpr (V * sizeof(T) == 4)
            *reinterpret_cast<uint32_t*>(p) = w[0];
        else
            *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
    }
};

// 1 / (1 + e^-v).  e^-v overflows to inf below -88, where the quotient is 0.
__device__ __forceinline__ float sigmoid(float v) {
    return __fdividef(1.f, 1.f + __expf(-v));
}
__device__ __forceinline__ float silu(float v) { return __fdividef(v, 1.f + __expf(-v)); }
// silu and its slope s (1 + v (1 - s)).
__device__ __forceinline__ float silu_grad(float v) {
    const float s = sigmoid(v);
    return s * fmaf(v, 1.f - s, 1.f);
}

#endif  // __CUDACC__

// Whether rows of `width` elements, `ld` apart, can be read V elements at a time.
inline bool rows_fit(const void* p, int64_t ld, int64_t width, size_t esz, int V) {
    return reinterpret_cast<uintptr_t>(p) % (V * esz) == 0 && ld % V == 0 && width % V == 0;
}

}  // namespace kda
