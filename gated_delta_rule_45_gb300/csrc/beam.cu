// Beam search over recurrent states (include/beam.h): selection over beams and
// vocabulary, and the reordering of per-beam rows.
//
// Selection.  The value of candidate (beam k, token v) is
// score_k + x_kv - log sum_w exp(x_kw); within a beam the order is that of the
// logits.  One pass over the logits, cut into pieces of at most 64 values a thread:
// each CTA leaves, for its piece, the maximum, the sum of exponentials relative to it
// and its num_out largest logits, sorted.  A second kernel, one CTA a request, joins
// the sums in 64 bits and picks the num_out best of all pieces' candidates by their
// values in 64 bits (candidates of different beams can lie closer than fp32 resolves).
//
// Both pick by threshold.  Keys order value and index together, so no two are equal.
// With t the num_out-th largest of the threads' own maxima, exactly num_out threads
// hold keys >= t, all of the num_out largest keys are among theirs, and their list is
// short (num_out times a thread's share at the very most); it is ranked by counting.
//
// Bound: HBM (each logit is read once); at 64 x 8 x 128000 bf16 logits SELECT.
#include "kda_internal.h"

#include <cfloat>
#include <cmath>

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kShare = 64;   // most values a thread looks at

// 16 bytes of logits.
template <typename T>
struct Logits;
template <>
struct Logits<float> {
    static constexpr int N = 4;
    uint4 u;
    __device__ __forceinline__ float get(int i) const {
        return __uint_as_float(i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w);
    }
    __device__ __forceinline__ void set(int i, float x) {
        (i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w) = __float_as_uint(x);
    }
};
template <>
struct Logits<__nv_bfloat16> {
    static constexpr int N = 8;
    uint4 u;
    __device__ __forceinline__ float get(int i) const {
        const uint32_t w = i < 2 ? u.x : i < 4 ? u.y : i < 6 ? u.z : u.w;
        return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
    }
    __device__ __forceinline__ void set(int i, float x) {
        uint32_t& w = i < 2 ? u.x : i < 4 ? u.y : i < 6 ? u.z : u.w;
        const uint32_t b = __float_as_uint(x);   // a bf16 value already
        w = i & 1 ? (w & 0xffffu) | (b & 0xffff0000u) : (w & 0xffff0000u) | b >> 16;
    }
};

// 16 bytes from bit `shift` (16 .. 112) of a and the vector after it.
__device__ __forceinline__ uint4 shifted(const uint4 a, const uint4 b, int shift) {
    uint64_t w0 = (uint64_t)a.y << 32 | a.x, w1 = (uint64_t)a.w << 32 | a.z;
    uint64_t w2 = (uint64_t)b.y << 32 | b.x;
    if (shift & 64) {
        w0 = w1;
        w1 = w2;
        w2 = (uint64_t)b.w << 32 | b.z;
    }
    const int s = shift & 63;
    if (s) {
        w0 = w0 >> s | w1 << (64 - s);
        w1 = w1 >> s | w2 << (64 - s);
    }
    return make_uint4((uint32_t)w0, (uint32_t)(w0 >> 32), (uint32_t)w1, (uint32_t)(w1 >> 32));
}

// NaN counts as -inf, +inf as the largest finite float.
__device__ __forceinline__ float tame(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX); }

// Whole numbers that sort as floats do (-0 as +0); 0 is below every one of them.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ uint64_t ordered(double x) {
    const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
    return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ double unordered(uint64_t u) {
    return __longlong_as_double((long long)(u >> 63 ? u & ~(1ull << 63) : ~u));
}

// A logit and its token, larger logits first, then lower tokens.  0: none.
__device__ __forceinline__ uint64_t logit_key(float x, int v) {
    return (uint64_t)ordered(x) << 32 | (0xffffffffu - (uint32_t)v);
}

// A value in 64 bits and the candidate's index.
struct ValueKey {
    uint64_t value;
    uint64_t index;   // ~0u - index; 0: none
};
__device__ __forceinline__ bool above(uint64_t a, uint64_t b) { return a > b; }
__device__ __forceinline__ bool above(const ValueKey& a, const ValueKey& b) {
    return a.value > b.value || (a.value == b.value && a.index > b.index);
}
__device__ __forceinline__ bool exists(uint64_t a) { return a != 0; }
__device__ __forceinline__ bool exists(const ValueKey& a) { return a.index != 0; }

// The num-th largest of the threads' best keys, Key{} when fewer threads have one.
// Returns whether this thread's best is among the num largest.
template <int THREADS, typename Key>
__device__ bool threshold(Key* best, Key* limit, const Key& mine, int num) {
    best[threadIdx.x] = mine;
    if (threadIdx.x == 0) *limit = Key{};
    __syncthreads();
    int rank = 0;   // a thread without a key ranks behind all that have one
    if (__any_sync(0xffffffffu, exists(mine))) {
#pragma unroll 8
        for (int j = 0; j < THREADS; ++j) rank += above(best[j], mine);
    }
    if (exists(mine) && rank == num - 1) *limit = mine;
    __syncthreads();
    return exists(mine) && rank < num;
}

// One piece of one row.  pieces: of a row; span: 16-byte vectors of a piece.
template <typename T>
__global__ void __launch_bounds__(kThreads)
beam_piece_kernel(const BeamSelectArgs p, int pieces, int span, uint64_t* __restrict__ keys,
                  float2* __restrict__ sums) {
    constexpr int N = Logits<T>::N;
    extern __shared__ __align__(16) uint64_t list[];   // num_out x kShare
    __shared__ uint64_t best_of[kThreads];
    __shared__ uint64_t limit;
    __shared__ float2 part[kWarps];
    __shared__ int count;
    asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x / pieces, piece = blockIdx.x % pieces;
    const int num = p.num_out;
    uint64_t* out = keys + (int64_t)blockIdx.x * num;

    // Rows need not start on a 16-byte boundary.  Which tokens a thread takes does not
    // depend on where the row starts, so equal rows have equal sums and tie exactly.
    const T* r = static_cast<const T*>(p.logits) + row * p.ld;
    const int shift = (int)(reinterpret_cast<uintptr_t>(r) & 15) * 8;   // bits
    const int lo = piece * span * N, hi = min(lo + span * N, p.V);      // tokens

    const float score = tame(p.scores[row]);
    const bool finished = p.finished && p.finished[row];
    if (finished || score == -INFINITY) {
        // nothing to read: `eos` of a finished beam, then the lowest tokens at -inf
        const bool has = finished && score != -INFINITY && p.eos >= lo && p.eos < hi;
        for (int j = tid; j < num; j += kThreads) {
            int v = lo + j;
            uint64_t key = 0;
            if (has) {
                if (j == 0) key = logit_key(0.f, p.eos);
                else if (--v >= p.eos) ++v;   // the tokens without eos
            }
            if (!key && v < hi) key = logit_key(-INFINITY, v);
            out[j] = key;
        }
        if (tid == 0) sums[blockIdx.x] = has ? make_float2(0.f, 1.f) : make_float2(-INFINITY, 0.f);
        return;
    }

    // A thread's j-th N values, -inf past the row's end.  Off the boundary they come from
    // the two aligned vectors they lie in (the next values of the row have to be there).
    auto load = [&](int j) {
        Logits<T> q;
        const int v = lo + (j * kThreads + tid) * N;
        if (v + (shift ? 2 * N : N) <= p.V) {
            const uint4* w = reinterpret_cast<const uint4*>(
                reinterpret_cast<uintptr_t>(r + v) & ~(uintptr_t)15);
            q.u = __ldg(w);
            if (shift) q.u = shifted(q.u, __ldg(w + 1), shift);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) q.set(i, v + i < p.V ? Elem<T>::load(r + v + i) : -INFINITY);
        }
        return q;
    };
    const int mine = (span + kThreads - 1) / kThreads;   // vectors a thread

    float m = -INFINITY, s = 0.f;   // running maximum and sum of exponentials
    uint64_t best = 0;
    // clean: values are known to be no NaN and no +inf
    auto look = [&](const Logits<T>& q, int j, bool clean) {
        const int v = lo + (j * kThreads + tid) * N;
        float x[N], top = -INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] = clean ? q.get(i) : tame(q.get(i));
            top = fmaxf(top, x[i]);
        }
        if (top > m || best == 0) {   // a new best: its first place
            s *= m == -INFINITY ? 0.f : __expf(m - top);
            m = top;
            int at = -1;
#pragma unroll
            for (int i = N - 1; i >= 0; --i)
                if (x[i] == top && v + i < hi) at = i;
            if (at >= 0) best = logit_key(top, v + at);
        }
        if (m != -INFINITY) {
            float e = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) e += __expf(x[i] - m);
            s += e;
        }
    };
    for (int j0 = 0; j0 < mine; j0 += 4) {
        Logits<T> q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j0 + j < mine) q[j] = load(j0 + j);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j0 + j < mine) look(q[j], j0 + j, true);
    }
    // a NaN or +inf among them, or (where m is -inf) perhaps a NaN: again, replaced
    if (!(s < INFINITY) || m == -INFINITY) {
        m = -INFINITY;
        s = 0.f;
        best = 0;
        for (int j = 0; j < mine; ++j) look(load(j), j, false);
    }

    // the piece's maximum and sum
    float M = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float S = m == -INFINITY ? 0.f : s * __expf(m - M);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
    if (lane == 0) part[warp] = make_float2(M, S);
    if (tid == 0) count = 0;
    const bool among = threshold<kThreads>(best_of, &limit, best, num);
    if (tid == 0) {
        float top = -INFINITY, sum = 0.f;
        for (int j = 0; j < kWarps; ++j) top = fmaxf(top, part[j].x);
        for (int j = 0; j < kWarps; ++j)
            if (part[j].y > 0.f) sum += part[j].y * __expf(part[j].x - top);
        sums[blockIdx.x] = make_float2(top, sum);
    }
    // the keys from the limit on, then their ranks
    if (among) {
        const uint64_t from = limit;
        for (int j = 0; j < mine; ++j) {
            const Logits<T> q = load(j);
            const int v = lo + (j * kThreads + tid) * N;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint64_t key = logit_key(tame(q.get(i)), v + i);
                if (v + i < hi && key >= from) list[atomicAdd(&count, 1)] = key;
            }
        }
    }
    __syncthreads();
    const int have = count;
    for (int i = tid; i < have; i += kThreads) {
        const uint64_t key = list[i];
        int rank = 0;
        for (int j = 0; j < have; ++j) rank += list[j] > key;
        if (rank < num) out[rank] = key;
    }
    for (int i = have + tid; i < num; i += kThreads) out[i] = 0;
}

// One request: joins its rows' pieces.
template <int THREADS>
__global__ void __launch_bounds__(THREADS)
beam_join_kernel(const BeamSelectArgs p, int pieces, const uint64_t* __restrict__ keys,
                 const float2* __restrict__ sums) {
    extern __shared__ __align__(16) ValueKey candidates[];   // num_out x a thread's share
    __shared__ ValueKey best_of[THREADS];
    __shared__ ValueKey limit;
    __shared__ double lse[BEAM_MAX_BEAMS];
    __shared__ double score[BEAM_MAX_BEAMS];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x, num = p.num_out;
    if (tid == 0) count = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int k = warp; k < p.K; k += THREADS / 32) {
        const float2* q = sums + ((int64_t)b * p.K + k) * pieces;
        float M = -INFINITY;
        for (int j = lane; j < pieces; j += 32) M = fmaxf(M, q[j].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        double s = 0.0;
        for (int j = lane; j < pieces; j += 32)
            if (q[j].y > 0.f) s += (double)q[j].y * exp((double)q[j].x - (double)M);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) {
            lse[k] = s > 0.0 ? (double)M + log(s) : 0.0;
            score[k] = (double)tame(p.scores[(int64_t)b * p.K + k]);
        }
    }
    __syncthreads();

    const int per_beam = pieces * num, all = p.K * per_beam;
    const uint64_t* mine = keys + (int64_t)b * all;
    auto value = [&](int i) {
        const uint64_t key = mine[i];
        ValueKey q{0, 0};
        if (key) {
            const int k = i / per_beam;
            const float x = unordered((uint32_t)(key >> 32));
            const uint32_t v = 0xffffffffu - (uint32_t)key;
            const double val = x == -INFINITY || score[k] == -INFINITY
                                   ? -INFINITY : score[k] + ((double)x - lse[k]);
            q.value = ordered(val);
            q.index = 0xffffffffu - ((uint32_t)k * (uint32_t)p.V + v);
        }
        return q;
    };
    ValueKey best{0, 0};
    for (int i = tid; i < all; i += THREADS) {
        const ValueKey q = value(i);
        if (above(q, best)) best = q;
    }
    if (threshold<THREADS>(best_of, &limit, best, num)) {
        const ValueKey from = limit;
        for (int i = tid; i < all; i += THREADS) {
            const ValueKey q = value(i);
            if (exists(q) && !above(from, q)) candidates[atomicAdd(&count, 1)] = q;
        }
    }
    __syncthreads();
    const int have = count;
    for (int i = tid; i < have; i += THREADS) {
        const ValueKey key = candidates[i];
        int rank = 0;
        for (int j = 0; j < have; ++j) rank += above(candidates[j], key);
        if (rank < num) {
            const uint32_t at = 0xffffffffu - (uint32_t)key.index;
            const int64_t o = (int64_t)b * num + rank;
            p.out_scores[o] = (float)unordered(key.value);
            p.out_parents[o] = b * p.K + (int)(at / (uint32_t)p.V);
            p.out_tokens[o] = (int)(at % (uint32_t)p.V);
        }
    }
}

struct Pieces {
    int pieces, span;   // of a row; 16-byte vectors of one
};
// A thread takes up to kShare values; fewer when that would leave SMs without a CTA
// (four CTAs an SM keep enough loads in flight).
Pieces split_row(int64_t rows, int32_t V, kda_dtype dtype) {
    const int N = dtype == KDA_BF16 ? 8 : 4;
    const int64_t vectors = (V + N - 1) / N;
    const int64_t most = kShare / N;                // vectors a thread
    const int64_t ctas = 4 * (int64_t)(sm_count() > 0 ? sm_count() : 148);
    int64_t each = (vectors * rows + ctas * kThreads - 1) / (ctas * kThreads);
    each = each < 1 ? 1 : each > most ? most : each;
    Pieces s;
    s.span = (int)(each * kThreads);
    s.pieces = (int)((vectors + s.span - 1) / s.span);
    return s;
}

// Candidates a thread of the joining kernel may hold.
int join_share(const Pieces& s, int K, int num_out, int threads) {
    return (K * s.pieces * num_out + threads - 1) / threads;
}

size_t pad(size_t b) { return (b + 255) & ~(size_t)255; }

template <int THREADS>
cudaError_t launch_join(const BeamSelectArgs& a, const Pieces& s, const uint64_t* keys,
                        const float2* sums, cudaStream_t stream) {
    const size_t smem =
        (size_t)join_share(s, a.K, a.num_out, THREADS) * a.num_out * sizeof(ValueKey);
    if (smem > 16 * 1024) {   // with the static part perhaps above the default limit
        const cudaError_t err =
            cudaFuncSetAttribute(beam_join_kernel<THREADS>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (err != cudaSuccess) return err;
    }
    // its launch overlaps the pieces' kernel; it waits for their results itself
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(a.B);
    c.blockDim = dim3(THREADS);
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    c.attrs = &early;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, beam_join_kernel<THREADS>, a, s.pieces, keys, sums);
}

// ---------------------------------------------------------------- reordering
//
// A thread owns one column (16, 4 or 1 bytes) of a request's K rows: it reads the
// rows that move, all before it writes any, so the permutation needs no second copy
// of the tensor and no barrier, and rows that stay cost nothing.  Bound: HBM.

constexpr int kMaxStates = 64;    // tensors a launch
constexpr int kColumns = 4;       // columns a thread, one after the other

struct ReorderArgs {
    char* data[kMaxStates];
    int64_t cols[kMaxStates];           // columns of a row
    uint32_t first[kMaxStates + 1];     // first block of each tensor
    int32_t count;
    const int32_t* parents;
    int32_t K;
};

template <typename U, int KMAX>
__global__ void __launch_bounds__(kThreads) beam_reorder_kernel(const ReorderArgs p) {
    int t = 0;
    while (t + 1 < p.count && blockIdx.x >= p.first[t + 1]) ++t;
    const int64_t cols = p.cols[t];
    const uint32_t per = (uint32_t)((cols + kThreads * kColumns - 1) / (kThreads * kColumns));
    const uint32_t block = blockIdx.x - p.first[t];
    const int base = (int)(block / per) * p.K;
    const int64_t c0 = (int64_t)(block % per) * (kThreads * kColumns) + threadIdx.x;
    U* rows = reinterpret_cast<U*>(p.data[t]) + (int64_t)base * cols;

    int from[KMAX];   // the row of the request that row k becomes, -1: itself
#pragma unroll
    for (int k = 0; k < KMAX; ++k) {
        from[k] = -1;
        if (k < p.K) {
            const int q = __ldg(p.parents + base + k) - base;
            if (q >= 0 && q < p.K && q != k) from[k] = q;
        }
    }
#pragma unroll 1
    for (int i = 0; i < kColumns; ++i) {
        const int64_t c = c0 + (int64_t)i * kThreads;
        if (c >= cols) return;
        U old[KMAX];
#pragma unroll
        for (int k = 0; k < KMAX; ++k)
            if (from[k] >= 0) old[k] = rows[from[k] * cols + c];
#pragma unroll
        for (int k = 0; k < KMAX; ++k)
            if (from[k] >= 0) rows[k * cols + c] = old[k];
    }
}

template <typename U>
cudaError_t reorder_by(ReorderArgs& a, uint32_t blocks, cudaStream_t stream) {
    if (a.K <= 4) beam_reorder_kernel<U, 4><<<blocks, kThreads, 0, stream>>>(a);
    else if (a.K <= 8) beam_reorder_kernel<U, 8><<<blocks, kThreads, 0, stream>>>(a);
    else if (a.K <= 16) beam_reorder_kernel<U, 16><<<blocks, kThreads, 0, stream>>>(a);
    else beam_reorder_kernel<U, 32><<<blocks, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

// The tensors whose rows are whole columns of U (and not of a wider type).
template <typename U>
cudaError_t reorder_columns(const beam_state* states, int32_t num_states, int wider,
                            const int32_t* parents, int32_t B, int32_t K, cudaStream_t stream) {
    ReorderArgs a;
    a.parents = parents;
    a.K = K;
    a.count = 0;
    uint32_t blocks = 0;
    for (int i = 0; i <= num_states; ++i) {
        int64_t need = 0, cols = 0;
        if (i < num_states) {
            const int64_t n = states[i].row_bytes;
            if (n == 0 || n % sizeof(U) != 0 || (wider && n % wider == 0)) continue;
            cols = n / (int64_t)sizeof(U);
            need = (cols + kThreads * kColumns - 1) / (kThreads * kColumns) * B;
            if (need > INT32_MAX) return cudaErrorInvalidValue;
        }
        if (a.count > 0 && (i == num_states || a.count == kMaxStates ||
                            (int64_t)blocks + need > INT32_MAX)) {
            a.first[a.count] = blocks;
            const cudaError_t err = reorder_by<U>(a, blocks, stream);
            if (err != cudaSuccess) return err;
            a.count = 0;
            blocks = 0;
        }
        if (i == num_states) break;
        a.data[a.count] = static_cast<char*>(states[i].data);
        a.cols[a.count] = cols;
        a.first[a.count] = blocks;
        ++a.count;
        blocks += (uint32_t)need;
    }
    return cudaSuccess;
}

}  // namespace

size_t beam_select_bytes(int32_t B, int32_t K, int32_t V, int32_t num_out) {
    const int64_t rows = (int64_t)B * K;
    size_t most = 256;
    for (kda_dtype t : {KDA_BF16, KDA_FP32}) {
        const Pieces s = split_row(rows, V, t);
        const size_t n = (size_t)rows * s.pieces;
        const size_t b = pad(n * num_out * sizeof(uint64_t)) + pad(n * sizeof(float2));
        most = b > most ? b : most;
    }
    return most;
}

cudaError_t launch_beam_select(const BeamSelectArgs& a, char* ws, cudaStream_t stream) {
    const int64_t rows = (int64_t)a.B * a.K;
    const Pieces s = split_row(rows, a.V, a.dtype);
    uint64_t* keys = reinterpret_cast<uint64_t*>(ws);
    float2* sums = reinterpret_cast<float2*>(ws + pad((size_t)rows * s.pieces * a.num_out * 8));
    const unsigned grid = (unsigned)(rows * s.pieces);
    const int share = s.span / kThreads * (a.dtype == KDA_BF16 ? 8 : 4);
    const size_t smem = (size_t)a.num_out * share * sizeof(uint64_t);
    if (a.dtype == KDA_BF16)
        beam_piece_kernel<__nv_bfloat16><<<grid, kThreads, smem, stream>>>(a, s.pieces, s.span, keys, sums);
    else
        beam_piece_kernel<float><<<grid, kThreads, smem, stream>>>(a, s.pieces, s.span, keys, sums);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    // 16 candidates a thread at most where 256 threads will do
    if (join_share(s, a.K, a.num_out, kThreads) <= 16)
        return launch_join<kThreads>(a, s, keys, sums, stream);
    return launch_join<1024>(a, s, keys, sums, stream);
}

cudaError_t launch_beam_reorder(const beam_state* states, int32_t num_states,
                                const int32_t* parents, int32_t B, int32_t K,
                                cudaStream_t stream) {
    if (K == 1) return cudaSuccess;   // a beam alone is its own parent
    cudaError_t err = reorder_columns<uint4>(states, num_states, 0, parents, B, K, stream);
    if (err == cudaSuccess)
        err = reorder_columns<uint32_t>(states, num_states, 16, parents, B, K, stream);
    if (err == cudaSuccess)
        err = reorder_columns<uint8_t>(states, num_states, 4, parents, B, K, stream);
    return err;
}

}  // namespace kda
