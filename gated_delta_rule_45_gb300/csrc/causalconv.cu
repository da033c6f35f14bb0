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
// Bound: HBM.  Measured, bf16, W = 4 with silu: 64 ragged prompts of 266240 x 4096 692 us (4.4 GB,
// 6.3 TB/s; 735 with a division in the sigmoid instead of the reciprocal, with that 791 in runs of
// 64 tokens, 906 with 8-byte loads and single instructions instead of pairs), 8 x 4096 x 4096
// forward 102 us (5.3), backward 226 us (1.07 GB, 4.8; waits for loads with 16 warps an SM, the
// activation's slope and 13 multiply-adds a value; 128 tokens a run).  Rows loaded one by one, each
// where the one eight before was used, instead of eight at once: 916 us for 735 (registers leave
// one CTA an SM).
#include "layer_ops.h"

#include <type_traits>

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRun = 256;    // tokens a thread, forward
constexpr int kBatch = 8;       // rows loaded at once
constexpr int kBackBatch = 4;   // and of both tensors, backward
constexpr int kMinParts = 256;  // runs of the backward pass, where there are tokens for them

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
    Lane<V> x[W - 1];   // the last W - 1 inputs, oldest first
    __device__ __forceinline__ void push(const Lane<V>& v) {
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) x[j] = x[j + 1];
        x[W - 2] = v;
    }
};

// The inputs before token t of sequence n (first token `start`).
template <typename T, int W, int V>
__device__ __forceinline__ void enter(const ConvArgs& p, int32_t n, int64_t start, int64_t t,
                                      int32_t c, Window<W, V>& win) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int64_t row = t - (W - 1) + j;
        if (row >= start) {
            win.x[j] = load_lane<T, V>(p.x, row * p.ldx + c);
        } else if (p.S0) {
            const int64_t r = (int64_t)n * (W - 1) + (row - start + W - 1);
            win.x[j] = load_lane<T, V>(p.S0, r * p.D + c);
        } else {
            win.x[j].zero();
        }
    }
}

template <int W, int V>
struct Filter {
    Lane<V> w[W], b;
    __device__ __forceinline__ void load(const float* wp, const float* bp, int32_t c) {
        float f[V][W];
        const float* from = wp + (int64_t)c * W;
        if constexpr (W == 4) {   // one vector a channel
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float4 u = reinterpret_cast<const float4*>(from)[i];
                f[i][0] = u.x; f[i][1] = u.y; f[i][2] = u.z; f[i][W - 1] = u.w;
            }
        } else if constexpr (V % 4 == 0) {
            float4 u[V * W / 4];
#pragma unroll
            for (int i = 0; i < V * W / 4; ++i) u[i] = reinterpret_cast<const float4*>(from)[i];
#pragma unroll
            for (int i = 0; i < V * W; ++i) {
                const float4 t = u[i / 4];
                f[i / W][i % W] = i % 4 == 0 ? t.x : i % 4 == 1 ? t.y : i % 4 == 2 ? t.z : t.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V * W; ++i) f[i / W][i % W] = from[i];
        }
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int i = 0; i < Lane<V>::kPairs; ++i)
                w[j].v[i] = pack2(f[2 * i][j], V > 1 ? f[2 * i + (V > 1 ? 1 : 0)][j] : 0.f);
        b.zero();
        if (!bp) return;
        constexpr int U = V < 4 ? V : 4;
#pragma unroll
        for (int i = 0; i < V; i += U) {
            Pack<float, U> k;
            k.load(bp + c + i);
#pragma unroll
            for (int q = 0; q < U; q += 2)
                b.v[(i + q) / 2] = pack2(k.get(q), U > 1 ? k.get(q + (U > 1 ? 1 : 0)) : 0.f);
        }
    }
    __device__ __forceinline__ Lane<V> apply(const Window<W, V>& win, const Lane<V>& x) const {
        Lane<V> v = b;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) v.fma(w[j], win.x[j]);
        v.fma(w[W - 1], x);
        return v;
    }
};
template <int V>
__device__ __forceinline__ void activate(Lane<V>& v, int32_t on) {
    if (!on) return;
#pragma unroll
    for (int i = 0; i < Lane<V>::kPairs; ++i) v.v[i] = silu2(v.v[i]);
}
// dy's way through the activation of v.
template <int V>
__device__ __forceinline__ Lane<V> activate_back(const Lane<V>& v, const Lane<V>& dy, int32_t on) {
    if (!on) return dy;
    Lane<V> d;
#pragma unroll
    for (int i = 0; i < Lane<V>::kPairs; ++i) d.v[i] = mul2(dy.v[i], silu_grad2(v.v[i]));
    return d;
}

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
    auto step = [&](const Lane<V>& x, int64_t row) {
        Lane<V> v = f.apply(win, x);
        win.push(x);
        activate(v, p.silu);
        v.template to<T>().store(static_cast<T*>(p.y) + row * p.D + c);
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
                Lane<V> x;
                x.from(k[r]);
                step(x, t + r);
            }
        }
        for (; t < to; ++t) step(load_lane<T, V>(p.x, t * p.ldx + c), t);
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
    Lane<V> dw[W], db;
    db.zero();
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j].zero();
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
            Lane<V> acc[W];   // gradients of inputs t - W + 1 .. t, not complete yet
#pragma unroll
            for (int j = 0; j < W; ++j) acc[j].zero();
            auto emit = [&](const Lane<V>& v, int64_t row) {
                v.template to<float>().store(p.dx + row * p.D + c);
            };
            auto step = [&](const Lane<V>& x, const Lane<V>& dy, bool own) {
                const Lane<V> dv = activate_back(f.apply(win, x), dy, p.silu);
                if (own) {
                    db.add(dv);
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) dw[j].fma(dv, win.x[j]);
                    dw[W - 1].fma(dv, x);
                }
#pragma unroll
                for (int j = 0; j + 1 < W; ++j) acc[j] = acc[j + 1];
                acc[W - 1].zero();
#pragma unroll
                for (int j = 0; j < W; ++j) acc[j].fma(f.w[j], dv);
                win.push(x);
            };
            auto one = [&]() {
                step(load_lane<T, V>(p.x, t * p.ldx + c), load_lane<T, V>(p.dy, t * p.D + c), t < to);
                if (t - (W - 1) >= from) emit(acc[0], t - (W - 1));
                ++t;
            };
            while (t < walk && t - (W - 1) < from) one();
            for (; t + kBackBatch <= to; t += kBackBatch) {
                Pack<T, V> kx[kBackBatch], kd[kBackBatch];
#pragma unroll
                for (int r = 0; r < kBackBatch; ++r) {
                    kx[r].load(static_cast<const T*>(p.x) + (t + r) * p.ldx + c);
                    kd[r].load(static_cast<const T*>(p.dy) + (t + r) * p.D + c);
                }
#pragma unroll
                for (int r = 0; r < kBackBatch; ++r) {
                    Lane<V> x, dy;
                    x.from(kx[r]);
                    dy.from(kd[r]);
                    step(x, dy, true);
                    emit(acc[0], t + r - (W - 1));
                }
            }
            while (t < walk) one();
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
    // part[run]: dw by weight, then db
    float* row = part + at.run * sum_row(SumColumns{{(int64_t)p.D * W, p.D, 0}}) + c;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j].template to<float>().store(row + (int64_t)j * p.D);
    db.template to<float>().store(row + (int64_t)W * p.D);
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
        const Lane<1> x = load_lane<T, 1>(p.x, (start + t) * p.ldx + c);
        const Lane<1> dy = load_lane<T, 1>(p.dy, (start + t) * p.D + c);
        const Lane<1> dv = activate_back(f.apply(win, x), dy, p.silu);
        win.push(x);
#pragma unroll
        for (int r = t; r < W - 1; ++r)
            g[r] = fmaf(unpack2(f.w[r - t].v[0]).x, unpack2(dv.v[0]).x, g[r]);
    }
#pragma unroll
    for (int r = 0; r < W - 1; ++r) p.dS0[((int64_t)n * (W - 1) + r) * p.D + c] = g[r];
}

// One token a row, kStepRows rows a thread with the same weights.  A thread reads all it needs of
// a state before it writes any.
constexpr int kStepRows = 2;
template <typename T, int W, int V>
__global__ void __launch_bounds__(kThreads)
conv_step_kernel(const ConvStepArgs p, int32_t nvec, int32_t rows) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int32_t r = (int32_t)(i / nvec), c = (int32_t)(i - (int64_t)r * nvec) * V;
    if (r >= rows) return;
    Pack<T, V> s[kStepRows][W];
#pragma unroll
    for (int q = 0; q < kStepRows; ++q) {
        const int64_t b = (int64_t)q * rows + r;
        if (b >= p.B) break;
        const int32_t row = p.parents ? p.parents[b] : (int32_t)b;
        const bool live = row >= 0 && row < p.num_rows;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            if (live)
                s[q][j].load(static_cast<const T*>(p.S) + ((int64_t)row * (W - 1) + j) * p.D + c);
            else s[q][j].zero();
        }
        s[q][W - 1].load(static_cast<const T*>(p.x) + b * p.ldx + c);
    }
    Filter<W, V> f;
    f.load(p.w, p.b, c);
#pragma unroll
    for (int q = 0; q < kStepRows; ++q) {
        const int64_t b = (int64_t)q * rows + r;
        if (b >= p.B) break;
        Window<W, V> win;
        Lane<V> x;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) win.x[j].from(s[q][j]);
        x.from(s[q][W - 1]);
        Lane<V> v = f.apply(win, x);
        activate(v, p.silu);
        v.template to<T>().store(static_cast<T*>(p.y) + b * p.D + c);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            s[q][j + 1].store(static_cast<T*>(p.S_out) + (b * (W - 1) + j) * p.D + c);
    }
}

constexpr int kSumCols = 32, kSumRows = 8;
// A CTA sums 32 columns: eight threads a column take every eighth row, in order, and their
// sums are added in order.
__global__ void __launch_bounds__(kSumCols * kSumRows)
column_sum_kernel(const float* __restrict__ part, int64_t rows, int64_t row, const SumColumns cols,
                  const SumOutputs outs, const int32_t* status, int32_t turned) {
    if (status && *status != KDA_OK) return;
    __shared__ float s[kSumRows][kSumCols];
    const int cl = threadIdx.x % kSumCols, rl = threadIdx.x / kSumCols;
    int64_t col = (int64_t)blockIdx.x * kSumCols + cl;
    const bool on = col < cols.n[0] + cols.n[1] + cols.n[2];
    float sum = 0.f;
    if (on) {
        int64_t r = rl;
        for (; r + 3 * kSumRows < rows; r += 4 * kSumRows) {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = part[(r + k * kSumRows) * row + col];
            sum += (v[0] + v[1]) + (v[2] + v[3]);
        }
        for (; r < rows; r += kSumRows) sum += part[r * row + col];
    }
    s[rl][cl] = sum;
    __syncthreads();
    if (rl != 0 || !on) return;
#pragma unroll
    for (int k = 1; k < kSumRows; ++k) sum += s[k][cl];
    float* out = outs.out[0];
    if (col < cols.n[0]) {
        if (turned > 1)
            col = col % (cols.n[0] / turned) * turned + col / (cols.n[0] / turned);
    } else {
        col -= cols.n[0];
        out = outs.out[1];
        if (col >= cols.n[1]) {
            col -= cols.n[1];
            out = outs.out[2];
        }
    }
    if (out) out[col] = sum;
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

// Tokens of a backward run: 32, or more where that leaves kMinParts runs or more, so that their
// partial sums are few.
int backward_run(int64_t T) {
    int64_t r = 32;
    while (r < 128 && T / (2 * r) >= kMinParts) r *= 2;
    while (T / r > 8 * kMinParts) r *= 2;
    return (int)r;
}

}  // namespace

cudaError_t launch_column_sums(const float* part, int64_t rows, SumColumns n, SumOutputs out,
                               const int32_t* status, cudaStream_t stream, int32_t turned) {
    const int64_t blocks = (n.n[0] + n.n[1] + n.n[2] + kSumCols - 1) / kSumCols;
    column_sum_kernel<<<(unsigned)blocks, kSumCols * kSumRows, 0, stream>>>(
        part, rows, sum_row(n), n, out, status, turned);
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
    return kHead + pad((size_t)((T + run - 1) / run) * sum_row({(int64_t)D * W, D, 0}) * sizeof(float));
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
        constexpr int V = 16 / sizeof(T);
        const bool wide = rows_fit(a.x, a.ldx, a.D, esz, V);
        // the longest runs that leave each SM 512 threads or more: a run reads W - 1 rows of
        // the one before it again, short ones spread few tokens over the GPU
        int run = kMaxRun;
        while (run > kBatch && (a.total_tokens + run - 1) / run * ((a.D + (wide ? V - 1 : 0)) / (wide ? V : 1)) <
                                   512 * (int64_t)(sm_count() > 0 ? sm_count() : 1))
            run /= 2;
        const ConvGrid g = conv_grid(a.total_tokens, a.D, wide ? V : 1, run);
        const int64_t copies = (int64_t)a.num_seqs * (W - 1) * g.nvec;
        const int64_t blocks = g.main + (copies + kThreads - 1) / kThreads;
        auto kernel = wide ? conv_fwd_kernel<T, W, V> : conv_fwd_kernel<T, W, 1>;
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
    const int64_t D = a.D;
    return launch_column_sums(part, (a.total_tokens + run - 1) / run, {D * a.W, D, 0},
                              {a.dw, a.db, nullptr}, status, stream, a.W);
}

cudaError_t launch_conv_step(const ConvStepArgs& a, cudaStream_t stream) {
    const size_t esz = a.dtype == KDA_BF16 ? 2 : 4;
    return by_type(a.dtype, a.W, [&](auto* t, auto w) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int W = decltype(w)::value;
        const bool wide = rows_fit(a.x, a.ldx, a.D, esz, 4);
        const int32_t nvec = a.D / (wide ? 4 : 1);
        const int32_t rows = (a.B + kStepRows - 1) / kStepRows;
        const int64_t blocks = ((int64_t)rows * nvec + kThreads - 1) / kThreads;
        auto kernel = wide ? conv_step_kernel<T, W, 4> : conv_step_kernel<T, W, 1>;
        kernel<<<(unsigned)blocks, kThreads, 0, stream>>>(a, nvec, rows);
        return cudaGetLastError();
    });
}

}  // namespace kda
