// Beam search over recurrent states (include/beam.h): selection over beams and
// vocabulary, and the reordering of per-beam rows.
//
// First form: one CTA a request, num_out rounds of a search for the best
// candidate after the one chosen before.
#include "kda_internal.h"

#include <cfloat>
#include <climits>
#include <cmath>

namespace kda {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float logit_at(const T* row, int v) {
    const float x = Elem<T>::load(row + v);
    return isnan(x) ? -INFINITY : fminf(x, FLT_MAX);
}

template <typename T>
__global__ void beam_select_kernel(const BeamSelectArgs p) {
    __shared__ double lse[BEAM_MAX_BEAMS];
    __shared__ double red[kThreads];
    __shared__ long long redi[kThreads];
    const int b = blockIdx.x, tid = threadIdx.x;
    const T* logits = static_cast<const T*>(p.logits);
    for (int k = 0; k < p.K; ++k) {
        const T* row = logits + ((int64_t)b * p.K + k) * p.ld;
        float m = -INFINITY;
        for (int v = tid; v < p.V; v += kThreads) m = fmaxf(m, logit_at(row, v));
        red[tid] = m;
        __syncthreads();
        for (int o = kThreads / 2; o > 0; o >>= 1) {
            if (tid < o) red[tid] = fmax(red[tid], red[tid + o]);
            __syncthreads();
        }
        m = (float)red[0];
        __syncthreads();
        double s = 0.0;
        if (m != -INFINITY)
            for (int v = tid; v < p.V; v += kThreads) s += (double)expf(logit_at(row, v) - m);
        red[tid] = s;
        __syncthreads();
        for (int o = kThreads / 2; o > 0; o >>= 1) {
            if (tid < o) red[tid] += red[tid + o];
            __syncthreads();
        }
        if (tid == 0) lse[k] = m == -INFINITY ? 0.0 : (double)m + log(red[0]);
        __syncthreads();
    }
    double last = INFINITY;
    long long lasti = -1;
    for (int i = 0; i < p.num_out; ++i) {
        double best = -INFINITY;
        long long besti = LLONG_MAX;
        for (int k = 0; k < p.K; ++k) {
            const T* row = logits + ((int64_t)b * p.K + k) * p.ld;
            const bool fin = p.finished && p.finished[(int64_t)b * p.K + k];
            float sc = p.scores[(int64_t)b * p.K + k];
            sc = isnan(sc) ? -INFINITY : fminf(sc, FLT_MAX);
            for (int v = tid; v < p.V; v += kThreads) {
                const double c = fin ? (v == p.eos ? (double)sc : -INFINITY)
                                     : (double)sc + ((double)logit_at(row, v) - lse[k]);
                const long long at = (long long)k * p.V + v;
                const bool after = c < last || (c == last && at > lasti);
                if (after && (c > best || (c == best && at < besti))) { best = c; besti = at; }
            }
        }
        red[tid] = best;
        redi[tid] = besti;
        __syncthreads();
        for (int o = kThreads / 2; o > 0; o >>= 1) {
            if (tid < o && (red[tid + o] > red[tid] ||
                            (red[tid + o] == red[tid] && redi[tid + o] < redi[tid]))) {
                red[tid] = red[tid + o];
                redi[tid] = redi[tid + o];
            }
            __syncthreads();
        }
        last = red[0];
        lasti = redi[0];
        __syncthreads();
        if (tid == 0) {
            const int64_t at = (int64_t)b * p.num_out + i;
            p.out_scores[at] = (float)last;
            p.out_parents[at] = b * p.K + (int)(lasti / p.V);
            p.out_tokens[at] = (int)(lasti % p.V);
        }
    }
}

// One thread per 4- or 1-byte column of a request's K rows: all moved rows are
// read before any is written.
template <typename U>
__global__ void beam_reorder_kernel(U* data, int64_t c0, int64_t cols, const int32_t* parents, int K) {
    const int64_t c = c0 + (int64_t)blockIdx.y * kThreads + threadIdx.x;
    if (c >= cols) return;
    const int base = blockIdx.x * K;
    U old[BEAM_MAX_BEAMS];
    for (int k = 0; k < K; ++k) {
        const int p = parents[base + k];
        if (p >= base && p < base + K) old[k] = data[(int64_t)p * cols + c];
        else old[k] = data[(int64_t)(base + k) * cols + c];
    }
    for (int k = 0; k < K; ++k) data[(int64_t)(base + k) * cols + c] = old[k];
}

}  // namespace

size_t beam_select_bytes(int32_t, int32_t, int32_t, int32_t) { return 256; }

cudaError_t launch_beam_select(const BeamSelectArgs& a, char*, cudaStream_t stream) {
    if (a.dtype == KDA_BF16)
        beam_select_kernel<__nv_bfloat16><<<a.B, kThreads, 0, stream>>>(a);
    else
        beam_select_kernel<float><<<a.B, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_beam_reorder(const beam_state* states, int32_t num_states,
                                const int32_t* parents, int32_t B, int32_t K,
                                cudaStream_t stream) {
    for (int i = 0; i < num_states; ++i) {
        const int64_t bytes = states[i].row_bytes;
        const bool w = bytes % 4 == 0;
        const int64_t cols = w ? bytes / 4 : bytes;
        for (int64_t c0 = 0; c0 < cols; c0 += 65535LL * kThreads) {
            const int64_t left = (cols - c0 + kThreads - 1) / kThreads;
            const dim3 grid(B, (unsigned)(left < 65535 ? left : 65535));
            if (w) beam_reorder_kernel<<<grid, kThreads, 0, stream>>>(static_cast<uint32_t*>(states[i].data), c0, cols, parents, K);
            else beam_reorder_kernel<<<grid, kThreads, 0, stream>>>(static_cast<uint8_t*>(states[i].data), c0, cols, parents, K);
            const cudaError_t err = cudaGetLastError();
            if (err != cudaSuccess) return err;
        }
    }
    return cudaSuccess;
}

}  // namespace kda
