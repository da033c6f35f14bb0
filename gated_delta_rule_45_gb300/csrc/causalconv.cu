// Short causal convolution (include/causalconv.h): prefill, backward and decode step.
//
// Mathematics.  v_t = b + sum_j w_j x_{t-W+1+j} per channel; backward, every dv_t = dy_t
// silu'(v_t) goes to the W inputs it was formed from.  A thread owns V neighbouring channels of
// a run of tokens and walks it with the last W - 1 inputs in registers (backward: and the
// gradients of the last W - 1 inputs, which later tokens still add to), so every row is read
// once but for W - 1 rows at the edges of a run.
//
// The packed token axis is cut into runs regardless of sequences; at a sequence's first
// token the window is replaced by the stored state.
//
// Bound: HBM.
#include "layer_ops.h"

#include <type_traits>

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kRun = 32;        // tokens a thread, forward
constexpr int kBatch = 8;       // rows loaded at once
constexpr int64_t kMaxParts = 2048;   // runs of the backward pass, at most

struct ConvGrid {
    int32_t nvec;      // vectors of V channels in a row
    int32_t cw;        // of them side by side in a CTA (a power of two)
    int32_t cblocks;   // CTAs along the channels
    int32_t run;       // tokens of a run
    int64_t runs;
    int64_t main;      // CTAs of the runs; the forward pass's later ones copy states
};

ConvGrid conv_grid(int64_t T, int32_t D, int V, int run) {
    ConvGrid g;
    g.nvec = (D + V - 1) / V;
    g.cw = 1;
    while (g.cw < kThreads && g.cw < g.nvec) g.cw *= 2;
    g.cblocks = (g.nvec + g.cw - 1) / g.cw;
    g.run = run;
    g.runs = (T + run - 1) / run;
    const int64_t rows = kThreads / g.cw;
    g.main = (g.runs + rows - 1) / rows * g.cblocks;
    return g;
}

// Where a thread works: its channels and its run.
struct Place {
    int32_t c;       // first channel, or -1
    int64_t run;
};
template <int V>
__device__ __forceinline__ Place place(const ConvGrid& g, int64_t block) {
    const int64_t rb = block / g.cblocks;
    const int32_t v = (int32_t)(block - rb * g.cblocks) * g.cw + (threadIdx.x & (g.cw - 1));
    Place p;
    p.c = v < g.nvec ? v * V : -1;
    p.run = rb * (kThreads / g.cw) + threadIdx.x / g.cw;
    return p;
}

template <int W, int V>
struct Window {
    float x[W - 1][V];   // the last W - 1 inputs, oldest first
    __device__ __forceinline__ void push(const float (&v)[V]) {
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) x[j][i] = x[j + 1][i];
#pragma unroll
        for (int i = 0; i < V; ++i) x[W - 2][i] = v[i];
    }
};

template <typename T, int V>
__device__ __forceinline__ void load_row(const void* p, int64_t at, float (&v)[V]) {
    Pack<T, V> k;
    k.load(static_cast<const T*>(p) + at);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = k.get(i);
}

// The inputs before token t of sequence n (first token `start`).
template <typename T, int W, int V>
__device__ __forceinline__ void enter(const ConvArgs& p, int32_t n, int64_t start, int64_t t,
                                      int32_t c, Window<W, V>& win) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int64_t row = t - (W - 1) + j;
        if (row >= start) {
            load_row<T, V>(p.x, row * p.ldx + c, win.x[j]);
        } else if (p.S0) {
            const int64_t r = (int64_t)n * (W - 1) + (row - start + W - 1);
            load_row<T, V>(p.S0, r * p.D + c, win.x[j]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) win.x[j][i] = 0.f;
        }
    }
}

template <int W, int V>
struct Filter {
    float w[W][V], b[V];
    __device__ __forceinline__ void load(const float* wp, const float* bp, int32_t c) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][i] = wp[(int64_t)(c + i) * W + j];
            b[i] = bp ? bp[c + i] : 0.f;
        }
    }
    __device__ __forceinline__ void apply(const Window<W, V>& win, const float (&x)[V],
                                          float (&v)[V]) const {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[i] = b[i];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) v[i] = fmaf(w[j][i], win.x[j][i], v[i]);
            v[i] = fmaf(w[W - 1][i], x[i], v[i]);
        }
    }
};

template <typename T, int W, int V>
__global__ void __launch_bounds__(kThreads)
conv_fwd_kernel(const ConvArgs p, const ConvGrid g, int32_t* status) {
    const int32_t* cu = p.cu_seqlens;
    if (!offsets_ok(cu, p.num_seqs, p.total_tokens, status)) return;
    if ((int64_t)blockIdx.x >= g.main) {
        // final states: row j of sequence n is input end - (W - 1) + j
        const int64_t i = ((int64_t)blockIdx.x - g.main) * kThreads + threadIdx.x;
        const int64_t r = i / g.nvec;
        const int32_t c = (int32_t)(i - r * g.nvec) * V, n = (int32_t)(r / (W - 1));
        if (n >= p.num_seqs) return;
        const int64_t start = cu[n], row = cu[n + 1] - (W - 1) + (r - (int64_t)n * (W - 1));
        Pack<T, V> k;
        if (row >= start) k.load(static_cast<const T*>(p.x) + row * p.ldx + c);
        else if (p.S0) k.load(static_cast<const T*>(p.S0) +
                              ((int64_t)n * (W - 1) + (row - start + W - 1)) * p.D + c);
        else k.zero();
        k.store(static_cast<T*>(p.S_T) + r * p.D + c);
        return;
    }
    const Place at = place<V>(g, blockIdx.x);
    const int64_t last = cu[p.num_seqs];
    int64_t t = at.run * g.run;
    const int64_t stop = t + g.run < last ? t + g.run : last;
    if (at.c < 0 || t >= stop) return;
    const int32_t c = at.c;
    int32_t n = sequence_of(cu, p.num_seqs, t);
    Filter<W, V> f;
    f.load(p.w, p.b, c);
    Window<W, V> win;
    enter<T, W, V>(p, n, cu[n], t, c, win);
    auto step = [&](const float (&x)[V], int64_t row) {
        float v[V];
        f.apply(win, x, v);
        win.push(x);
        if (p.silu) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = silu(v[i]);
        }
        Pack<T, V> k;
        k.set(v);
        k.store(static_cast<T*>(p.y) + row * p.D + c);
    };
    while (true) {
        const int64_t end = cu[n + 1], to = end < stop ? end : stop;
        for (; t + kBatch <= to; t += kBatch) {
            Pack<T, V> k[kBatch];
#pragma unroll
            for (int r = 0; r < kBatch; ++r)
                k[r].load(static_cast<const T*>(p.x) + (t + r) * p.ldx + c);
#pragma unroll
            for (int r = 0; r < kBatch; ++r) {
                float x[V];
#pragma unroll
                for (int i = 0; i < V; ++i) x[i] = k[r].get(i);
                step(x, t + r);
            }
        }
        for (; t < to; ++t) {
            float x[V];
            load_row<T, V>(p.x, t * p.ldx + c, x);
            step(x, t);
        }
        if (t >= stop) return;
        while (cu[n + 1] <= t) ++n;
        enter<T, W, V>(p, n, t, t, c, win);
    }
}

// A run's gradients.  Token t's dv reaches the inputs of tokens t - W + 1 .. t, so the
// gradient of an input is complete W - 1 tokens later: a run walks on that far behind its end
// (within the sequence) and leaves the parameters' sums of those tokens to the next run.
template <typename T, int W, int V>
__global__ void __launch_bounds__(kThreads)
conv_bwd_kernel(const ConvArgs p, const ConvGrid g, float* part, int32_t* status) {
    const int32_t* cu = p.cu_seqlens;
    if (!offsets_ok(cu, p.num_seqs, p.total_tokens, status)) return;
    const Place at = place<V>(g, blockIdx.x);
    if (at.c < 0 || at.run >= g.runs) return;
    const int32_t c = at.c;
    const int64_t last = cu[p.num_seqs], first = at.run * g.run;
    const int64_t stop = first + g.run < last ? first + g.run : last;
    float dw[W][V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = 0.f;
    }
    if (first < stop) {
        int64_t t = first;
        int32_t n = sequence_of(cu, p.num_seqs, t);
        Filter<W, V> f;
        f.load(p.w, p.b, c);
        Window<W, V> win;
        enter<T, W, V>(p, n, cu[n], t, c, win);
        while (true) {
            const int64_t end = cu[n + 1];
            // tokens whose inputs' gradients this run writes: from `from` on, up to `to`
            const int64_t from = t, to = end < stop ? end : stop;
            const int64_t walk = to + W - 1 < end ? to + W - 1 : end;
            float acc[W][V];   // gradients of inputs t - W + 1 .. t, not complete yet
#pragma unroll
            for (int j = 0; j < W; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) acc[j][i] = 0.f;
            auto emit = [&](const float (&v)[V], int64_t row) {
                Pack<float, V> k;
                k.set(v);
                k.store(p.dx + row * p.D + c);
            };
            auto step = [&](const float (&x)[V], const float (&dy)[V], bool own) {
                float v[V], dv[V];
                f.apply(win, x, v);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    dv[i] = p.silu ? dy[i] * silu_grad(v[i]) : dy[i];
                    if (own) {
                        db[i] += dv[i];
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) dw[j][i] = fmaf(dv[i], win.x[j][i], dw[j][i]);
                        dw[W - 1][i] = fmaf(dv[i], x[i], dw[W - 1][i]);
                    }
#pragma unroll
                    for (int j = 0; j + 1 < W; ++j) acc[j][i] = acc[j + 1][i];
                    acc[W - 1][i] = 0.f;
#pragma unroll
                    for (int j = 0; j < W; ++j) acc[j][i] = fmaf(f.w[j][i], dv[i], acc[j][i]);
                }
                win.push(x);
            };
            for (; t < walk; ++t) {
                if (t - (W - 1) >= from && t + kBatch / 2 <= to) {
                    Pack<T, V> kx[kBatch / 2], kd[kBatch / 2];
#pragma unroll
                    for (int r = 0; r < kBatch / 2; ++r) {
                        kx[r].load(static_cast<const T*>(p.x) + (t + r) * p.ldx + c);
                        kd[r].load(static_cast<const T*>(p.dy) + (t + r) * p.D + c);
                    }
#pragma unroll
                    for (int r = 0; r < kBatch / 2; ++r) {
                        float x[V], dy[V];
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            x[i] = kx[r].get(i);
                            dy[i] = kd[r].get(i);
                        }
                        step(x, dy, true);
                        emit(acc[0], t + r - (W - 1));
                    }
                    t += kBatch / 2 - 1;
                    continue;
                }
                float x[V], dy[V];
                load_row<T, V>(p.x, t * p.ldx + c, x);
                load_row<T, V>(p.dy, t * p.D + c, dy);
                step(x, dy, t < to);
                if (t - (W - 1) >= from) emit(acc[0], t - (W - 1));
            }
            // at a sequence's end nothing more is added to its last inputs
            if (walk == end) {
#pragma unroll
                for (int j = 1; j < W; ++j) {
                    const int64_t row = end - W + j;
                    if (row >= from && row < to) emit(acc[j], row);
                }
            }
            if (to >= stop) break;
            t = to;
            while (cu[n + 1] <= t) ++n;
            enter<T, W, V>(p, n, t, t, c, win);
        }
    }
    float* row = part + at.run * ((int64_t)p.D * (W + 1));
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) row[(int64_t)(c + i) * W + j] = dw[j][i];
        row[(int64_t)p.D * W + c + i] = db[i];
    }
}

// The ends of the sequences: dS_T goes to the last inputs, be they tokens or stored ones, and
// the stored ones get what the first tokens took from them.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads)
conv_edge_kernel(const ConvArgs p, const int32_t* status) {
    if (*status != KDA_OK) return;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int32_t n = (int32_t)(i / p.D), c = (int32_t)(i - (int64_t)n * p.D);
    if (n >= p.num_seqs) return;
    const int64_t start = p.cu_seqlens[n], end = p.cu_seqlens[n + 1], len = end - start;
    float gS[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        gS[k] = p.dS_T ? p.dS_T[((int64_t)n * (W - 1) + k) * p.D + c] : 0.f;
        const int64_t row = end - (W - 1) + k;
        if (p.dS_T && row >= start) p.dx[row * p.D + c] += gS[k];
    }
    if (!p.dS0) return;
    Filter<W, 1> f;
    f.load(p.w, p.b, c);
    Window<W, 1> win;
    enter<T, W, 1>(p, n, start, start, c, win);
    float g[W - 1];
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
        g[r] = 0.f;
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            if (r - len == k) g[r] = gS[k];   // a row that the sequence did not push out
    }
#pragma unroll
    for (int t = 0; t < W - 1; ++t) {
        if (t >= len) break;
        float x[1], dy[1], v[1];
        load_row<T, 1>(p.x, (start + t) * p.ldx + c, x);
        load_row<T, 1>(p.dy, (start + t) * p.D + c, dy);
        f.apply(win, x, v);
        win.push(x);
        const float dv = p.silu ? dy[0] * silu_grad(v[0]) : dy[0];
#pragma unroll
        for (int r = t; r < W - 1; ++r) g[r] = fmaf(f.w[r - t][0], dv, g[r]);
    }
#pragma unroll
    for (int r = 0; r < W - 1; ++r) p.dS0[((int64_t)n * (W - 1) + r) * p.D + c] = g[r];
}

// One token a row.  A thread reads all it needs of the state before it writes any.
template <typename T, int W, int V>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(const ConvStepArgs p, int32_t nvec) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int32_t b = (int32_t)(i / nvec), c = (int32_t)(i - (int64_t)b * nvec) * V;
    if (b >= p.B) return;
    const int32_t row = p.parents ? p.parents[b] : b;
    const bool live = row >= 0 && row < p.num_rows;
    Pack<T, V> s[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        if (live) s[j].load(static_cast<const T*>(p.S) + ((int64_t)row * (W - 1) + j) * p.D + c);
        else s[j].zero();
    }
    s[W - 1].load(static_cast<const T*>(p.x) + b * p.ldx + c);
    Filter<W, V> f;
    f.load(p.w, p.b, c);
    float v[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        v[k] = f.b[k];
#pragma unroll
        for (int j = 0; j < W; ++j) v[k] = fmaf(f.w[j][k], s[j].get(k), v[k]);
        if (p.silu) v[k] = silu(v[k]);
    }
    Pack<T, V> y;
    y.set(v);
    y.store(static_cast<T*>(p.y) + (int64_t)b * p.D + c);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        s[j + 1].store(static_cast<T*>(p.S_out) + ((int64_t)b * (W - 1) + j) * p.D + c);
}

constexpr int kSumCols = 32, kSumRows = 8;
// A CTA sums 32 columns: eight threads a column take every eighth row, in order, and their
// sums are added in order.
__global__ void __launch_bounds__(kSumCols * kSumRows)
column_sum_kernel(const float* __restrict__ part, int64_t rows, int64_t n1, int64_t n2,
                  float* out1, float* out2, const int32_t* status) {
    if (status && *status != KDA_OK) return;
    __shared__ float s[kSumRows][kSumCols];
    const int cl = threadIdx.x % kSumCols, rl = threadIdx.x / kSumCols;
    const int64_t col = (int64_t)blockIdx.x * kSumCols + cl, n = n1 + n2;
    float sum = 0.f;
    if (col < n) {
        int64_t r = rl;
        for (; r + 3 * kSumRows < rows; r += 4 * kSumRows) {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = part[(r + k * kSumRows) * n + col];
            sum += (v[0] + v[1]) + (v[2] + v[3]);
        }
        for (; r < rows; r += kSumRows) sum += part[r * n + col];
    }
    s[rl][cl] = sum;
    __syncthreads();
    if (rl != 0 || col >= n) return;
#pragma unroll
    for (int k = 1; k < kSumRows; ++k) sum += s[k][cl];
    float* out = col < n1 ? out1 : out2;
    if (out) out[col < n1 ? col : col - n1] = sum;
}

__global__ void __launch_bounds__(1024)
offsets_check_kernel(const int32_t* cu, int32_t N, int64_t T, int32_t* status) {
    bool bad = false;
    for (int64_t i = threadIdx.x; i <= N; i += 1024) {
        const int32_t c = cu[i];
        bad |= i == 0 ? c != 0 : c < cu[i - 1];
        bad |= i == N && (int64_t)c > T;
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *status = bad ? KDA_ERR_DEVICE_INPUT : KDA_OK;
}

size_t pad(size_t b) { return (b + 255) & ~(size_t)255; }
constexpr size_t kHead = 256;   // the status word's part of the workspace

template <typename F>
cudaError_t by_type(kda_dtype dtype, int W, F&& f) {
    auto pick = [&](auto* t) {
        switch (W) {
            case 2: return f(t, std::integral_constant<int, 2>());
            case 3: return f(t, std::integral_constant<int, 3>());
            default: return f(t, std::integral_constant<int, 4>());
        }
    };
    return dtype == KDA_BF16 ? pick((__nv_bfloat16*)nullptr) : pick((float*)nullptr);
}

// Tokens of a backward run.
int backward_run(int64_t T) {
    const int64_t r = (T + kMaxParts - 1) / kMaxParts;
    return (int)(r < 32 ? 32 : r);
}

}  // namespace

cudaError_t launch_column_sums(const float* part, int64_t rows, int64_t n1, int64_t n2,
                               float* out1, float* out2, const int32_t* status,
                               cudaStream_t stream) {
    const int64_t blocks = (n1 + n2 + kSumCols - 1) / kSumCols;
    column_sum_kernel<<<(unsigned)blocks, kSumCols * kSumRows, 0, stream>>>(part, rows, n1, n2,
                                                                            out1, out2, status);
    return cudaGetLastError();
}

cudaError_t launch_offsets_check(const int32_t* cu, int32_t N, int64_t T, int32_t* status,
                                 cudaStream_t stream, bool always) {
    if (N <= kSelfCheck && !always) return cudaSuccess;
    offsets_check_kernel<<<1, 1024, 0, stream>>>(cu, N, T, status);
    return cudaGetLastError();
}

size_t conv_prefill_bytes(int32_t num_seqs, int32_t D, int32_t W, kda_dtype dtype) {
    return kHead + pad((size_t)num_seqs * (W - 1) * D * (dtype == KDA_BF16 ? 2 : 4));
}
size_t conv_backward_bytes(int64_t T, int32_t D, int32_t W) {
    const int run = backward_run(T);
    return kHead + pad((size_t)((T + run - 1) / run) * D * (W + 1) * sizeof(float));
}

cudaError_t launch_conv_prefill(const ConvArgs& a, char* ws, cudaStream_t stream) {
    int32_t* status = reinterpret_cast<int32_t*>(ws);
    cudaError_t err = launch_offsets_check(a.cu_seqlens, a.num_seqs, a.total_tokens, status, stream);
    if (err != cudaSuccess) return err;
    ConvArgs b = a;
    const size_t esz = a.dtype == KDA_BF16 ? 2 : 4;
    if (a.S0 && a.S0 == a.S_T && a.num_seqs > 0) {   // in place: S_T is written while S0 is read
        b.S0 = ws + kHead;
        err = cudaMemcpyAsync(ws + kHead, a.S0, (size_t)a.num_seqs * (a.W - 1) * a.D * esz,
                              cudaMemcpyDeviceToDevice, stream);
        if (err != cudaSuccess) return err;
    }
    return by_type(a.dtype, a.W, [&](auto* t, auto w) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int W = decltype(w)::value;
        const bool wide = rows_fit(a.x, a.ldx, a.D, esz, 4);
        const ConvGrid g = conv_grid(a.total_tokens, a.D, wide ? 4 : 1, kRun);
        const int64_t copies = (int64_t)a.num_seqs * (W - 1) * g.nvec;
        const int64_t blocks = g.main + (copies + kThreads - 1) / kThreads;
        auto kernel = wide ? conv_fwd_kernel<T, W, 4> : conv_fwd_kernel<T, W, 1>;
        kernel<<<(unsigned)(blocks > 0 ? blocks : 1), kThreads, 0, stream>>>(b, g, status);
        return cudaGetLastError();
    });
}

cudaError_t launch_conv_backward(const ConvArgs& a, char* ws, cudaStream_t stream) {
    int32_t* status = reinterpret_cast<int32_t*>(ws);
    float* part = reinterpret_cast<float*>(ws + kHead);
    cudaError_t err = launch_offsets_check(a.cu_seqlens, a.num_seqs, a.total_tokens, status, stream);
    if (err != cudaSuccess) return err;
    const size_t esz = a.dtype == KDA_BF16 ? 2 : 4;
    err = by_type(a.dtype, a.W, [&](auto* t, auto w) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int W = decltype(w)::value;
        const bool wide = rows_fit(a.x, a.ldx, a.D, esz, 4);
        const ConvGrid g = conv_grid(a.total_tokens, a.D, wide ? 4 : 1,
                                     backward_run(a.total_tokens));
        auto kernel = wide ? conv_bwd_kernel<T, W, 4> : conv_bwd_kernel<T, W, 1>;
        kernel<<<(unsigned)(g.main > 0 ? g.main : 1), kThreads, 0, stream>>>(a, g, part, status);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess || a.num_seqs == 0 || (!a.dS_T && !a.dS0)) return e;
        const int64_t blocks = ((int64_t)a.num_seqs * a.D + kThreads - 1) / kThreads;
        conv_edge_kernel<T, W><<<(unsigned)blocks, kThreads, 0, stream>>>(a, status);
        return cudaGetLastError();
    });
    if (err != cudaSuccess) return err;
    const int run = backward_run(a.total_tokens);
    return launch_column_sums(part, (a.total_tokens + run - 1) / run, (int64_t)a.D * a.W, a.D, a.dw,
                              a.db, status, stream);
}

cudaError_t launch_conv_step(const ConvStepArgs& a, cudaStream_t stream) {
    const size_t esz = a.dtype == KDA_BF16 ? 2 : 4;
    return by_type(a.dtype, a.W, [&](auto* t, auto w) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int W = decltype(w)::value;
        const bool wide = rows_fit(a.x, a.ldx, a.D, esz, 4);
        const int32_t nvec = a.D / (wide ? 4 : 1);
        const int64_t blocks = ((int64_t)a.B * nvec + kThreads - 1) / kThreads;
        auto kernel = wide ? conv_step_kernel<T, W, 4> : conv_step_kernel<T, W, 1>;
        kernel<<<(unsigned)blocks, kThreads, 0, stream>>>(a, nvec);
        return cudaGetLastError();
    });
}

}  // namespace kda
