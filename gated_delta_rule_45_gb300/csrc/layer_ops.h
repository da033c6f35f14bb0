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
// CTAs that launch_scan_step starts, at most INT32_MAX for a call that it can make, and the rows
// of the batch that a warp of theirs takes.
int64_t scan_step_blocks(int32_t B, int32_t H, int32_t d, int32_t* rows);
cudaError_t launch_scan_step(const ScanStepArgs& a, cudaStream_t stream);

// Sums of the rows of part in a fixed order.  A row holds n[0], n[1] and n[2] columns for out[0],
// out[1] and out[2], any of which may be null, and is whole vectors of four long.  Nothing is
// written when *status (may be null) says that the offsets are malformed.  The first columns are a
// [turned][n[0] / turned] matrix that goes to out[0] transposed.  (causalconv.cu)
struct SumColumns {
    int64_t n[3];
};
struct SumOutputs {
    float* out[3];
};
cudaError_t launch_column_sums(const float* part, int64_t rows, SumColumns n, SumOutputs out,
                               const int32_t* status, cudaStream_t stream, int32_t turned = 1);
__host__ __device__ inline int64_t sum_row(const SumColumns& n) { return (n.n[0] + n.n[1] + n.n[2] + 3) / 4 * 4; }
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

// Two floats for the packed instructions.
using F2 = unsigned long long;
__device__ __forceinline__ F2 pack2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(F2 r) {
    float2 a;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
    return a;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {   // one unit in the last place; 0 for x beyond 2^126
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float sum2(F2 a) {
    const float2 v = unpack2(a);
    return v.x + v.y;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 both(float a) { return pack2(a, a); }
constexpr float kLog2e = 1.4426950408889634f;

// V channels in fp32, in pairs for the packed instructions (a single one in the low half).
template <int V>
struct Lane {
    static constexpr int kPairs = (V + 1) / 2;
    F2 v[kPairs];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) v[i] = 0;
    }
    template <typename T>
    __device__ __forceinline__ void from(const Pack<T, V>& k) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
            v[i] = pack2(k.get(2 * i), V > 1 ? k.get(2 * i + (V > 1 ? 1 : 0)) : 0.f);
    }
    template <typename T>
    __device__ __forceinline__ Pack<T, V> to() const {
        float f[V];
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = i % 2 ? unpack2(v[i / 2]).y : unpack2(v[i / 2]).x;
        Pack<T, V> k;
        k.set(f);
        return k;
    }
    __device__ __forceinline__ void fma(const Lane& a, const Lane& b) {   // this += a b
#pragma unroll
        for (int i = 0; i < kPairs; ++i) v[i] = fma2(a.v[i], b.v[i], v[i]);
    }
    __device__ __forceinline__ float sum() const {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const float2 u = unpack2(v[i]);
            t += V > 1 ? u.x + u.y : u.x;
        }
        return t;
    }
    __device__ __forceinline__ void add(const Lane& a) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) v[i] = add2(v[i], a.v[i]);
    }
};
template <typename T, int V>
__device__ __forceinline__ Lane<V> load_lane(const void* p, int64_t at) {
    Pack<T, V> k;
    k.load(static_cast<const T*>(p) + at);
    Lane<V> l;
    l.from(k);
    return l;
}

// 1 / (1 + e^-v): the exponential as 2^(-v log2 e), off by the rounding of its argument (2^-24
// of |v| log2 e), which counts where the exponential is not small against 1.  It overflows to inf
// below -88, where the quotient is 0.
__device__ __forceinline__ float sigmoid(float v) {
    return rcp(1.f + ex2(-kLog2e * v));
}
__device__ __forceinline__ F2 sigmoid2(F2 v) {
    const float2 t = unpack2(mul2(v, both(-kLog2e)));
    const float2 u = unpack2(add2(pack2(ex2(t.x), ex2(t.y)), both(1.f)));
    return pack2(rcp(u.x), rcp(u.y));
}
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }
__device__ __forceinline__ F2 silu2(F2 v) { return mul2(v, sigmoid2(v)); }
// silu and its slope s (1 + v (1 - s)).
__device__ __forceinline__ float silu_grad(float v) {
    const float s = sigmoid(v);
    return s * fmaf(v, 1.f - s, 1.f);
}
__device__ __forceinline__ F2 silu_grad2(F2 v) {
    const F2 s = sigmoid2(v), vs = mul2(v, s);           // s + v s - v s s
    return fma2(vs, fma2(s, both(-1.f), both(1.f)), s);
}

#endif  // __CUDACC__

// Whether rows of `width` elements, `ld` apart, can be read V elements at a time.
inline bool rows_fit(const void* p, int64_t ld, int64_t width, size_t esz, int V) {
    return reinterpret_cast<uintptr_t>(p) % (V * esz) == 0 && ld % V == 0 && width % V == 0;
}

}  // namespace kda
