// Beam search over recurrent states (include/beam.h): selection over beams and
// vocabulary, and the reordering of per-beam rows.
//
// Selection.  The value of candidate (beam k, token v) is
// score_k + x_kv - log sum_w exp(x_kw); within a beam the order is that of the
// logits.  One pass over the logits, cut into pieces: each CTA leaves, for its piece,
// the maximum, the sum of exponentials relative to it and its num_out largest logits,
// sorted.  A second kernel, one CTA a request, joins the sums in 64 bits and picks the
// num_out best of all pieces' candidates by their values in 64 bits (candidates of
// different beams can lie closer than fp32 resolves).
//
// Both pick by threshold: a bound that at least num_out threads' own maxima reach
// leaves a short list of candidates, which is ranked by counting.  Keys order value and
// index together, so no two are equal.  Rows of equal or masked logits, where the bound
// would leave a long list, go through the exact num_out-th largest of the threads'
// maximum keys: exactly num_out threads hold keys from there on, so the list is
// num_out times a thread's share at the most.
//
// Bound: HBM (each logit is read once, 19 us for 64 x 8 x 128000 bf16, 16 of them);
// measured 38 us: 31 for the pieces, whose warps issue in three cycles of five, and 7 to
// join.  For the best one alone it is 30 us: the rest is the listing.
#include "kda_internal.h"

#include <cfloat>
#include <cmath>

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kList = 1024;  // logits the fast pass may list
constexpr int kJoin = 16;    // candidates a thread of the joining kernel, with 256 threads
constexpr int kParts = 8;    // most vectors a thread of a piece's first part
constexpr int kCtas = 3;     // an SM

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

// Exponentials are taken as 2^(x log2 e - c) with c = M log2 e rounded once, M the
// maximum of the piece's first part: one multiply-add and one special-function instruction
// a logit.  The term of x = M is then 2^r and not 1, r = M log2 e - c what the rounding
// left out (6e-8 of c: at M = 1000, 6e-5), so the sum is divided by 2^r.  (log2 e is
// itself rounded, by 2e-8 of x log2 e; in terms relative to e^M that is 2e-8 of x - M,
// which does not show.)  A later logit far above M has a large argument, whose rounding
// shows (6.6e-7 of the term up to 22 above, 2.6e-6 from 44 on, and at 88 sums overflow): a
// piece whose sum says that some lie 22 above is summed again relative to the largest.
// (Taking a new reference on the way would save that, but cost every piece 3 %: 41.5 us
// for 40.3 at 64 x 8 x 128000 bf16.)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMostSum = 0x1p32f;   // the terms of a piece at M or below add to 2^20 at most
constexpr float kMostRest = 0.5f;   // beyond (logits of 1e7 and more): the careful path
__device__ __forceinline__ float exp2_ftz(float x) {   // below the normal numbers: 0
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
    return e;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// (2^(a log2 e - c), 2^(b log2 e - c)), both halves at once
__device__ __forceinline__ uint64_t both_exp2(float a, float b, uint64_t log2e2, uint64_t c2) {
    uint64_t t;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(t) : "l"(pack2(a, b)), "l"(log2e2), "l"(c2));
    float x, y;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(t));
    return pack2(exp2_ftz(x), exp2_ftz(y));
}

// The sum of n values (a power of two) in pairs: of equal ones without rounding.  Rows with
// one logit many times over have equal terms, whose roundings do not cancel.
template <int n>
__device__ __forceinline__ float sum_pairs(float (&v)[n]) {
#pragma unroll
    for (int h = n / 2; h > 0; h /= 2) {
#pragma unroll
        for (int i = 0; i < h; ++i) v[i] += v[i + h];
    }
    return v[0];
}

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

// Upper bits of a key: larger or equal for a larger key, 0 only for none.
__device__ __forceinline__ uint32_t coarse(uint64_t a) { return (uint32_t)(a >> 32); }
__device__ __forceinline__ uint32_t coarse(const ValueKey& a) { return (uint32_t)(a.value >> 32); }

// The r-th largest of a warp's values (0: none), equal ones counted one by one.
__device__ __forceinline__ uint32_t warp_nth(uint32_t c, int r, int lane) {
    uint32_t top = 0;
    for (int i = 0; i < r; ++i) {
        top = __reduce_max_sync(0xffffffffu, c);
        if (lane == __ffs(__ballot_sync(0xffffffffu, c == top)) - 1) c = 0;
    }
    return top;
}

// The num-th largest of the threads' best keys (Key{} when fewer threads have one) goes
// to `limit`; returns whether this thread's best is among the num largest, and then its
// rank.  A first bound, from every warp's own largest, leaves few keys to rank by counting.
template <int THREADS, typename Key>
struct Threshold {
    Key best[THREADS];
    Key limit;
    uint32_t bound[THREADS / 32];
    int count;

    __device__ bool find(const Key& mine, int num, int& rank) {
        constexpr int kW = THREADS / 32;
        const int lane = threadIdx.x & 31;
        const uint32_t c = exists(mine) ? coarse(mine) : 0;
        const uint32_t nth = warp_nth(c, (num + kW - 1) / kW, lane);
        if (lane == 0) bound[threadIdx.x >> 5] = nth;
        if (threadIdx.x == 0) {
            limit = Key{};
            count = 0;
        }
        __syncthreads();
        uint32_t least = bound[0];
#pragma unroll
        for (int j = 1; j < kW; ++j) least = min(least, bound[j]);
        const bool in = exists(mine) && c >= least;
        if (in) best[atomicAdd(&count, 1)] = mine;
        __syncthreads();
        rank = 0;
        if (in) {
            const int have = count;
            for (int j = 0; j < have; ++j) rank += above(best[j], mine);
            if (rank == num - 1) limit = mine;
        }
        __syncthreads();
        return in && rank < num;
    }
};

// Sorts the `have` keys of a list by counting; rank r < num goes to put(r, key).
template <typename Key, typename F>
__device__ __forceinline__ void rank_list(const Key* list, int have, int num, F&& put) {
    for (int i = threadIdx.x; i < have; i += blockDim.x) {
        const Key key = list[i];
        int rank = 0;
        for (int j = 0; j < have; ++j) rank += above(list[j], key);
        if (rank < num) put(rank, key);
    }
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Largest of a vector's values, NaN left out; -inf of none.
__device__ __forceinline__ float largest(const Logits<float>& q) {
    return fmaxf(fmaxf(q.get(0), q.get(1)), fmaxf(q.get(2), q.get(3)));
}
__device__ __forceinline__ float largest(const Logits<__nv_bfloat16>& q) {
    const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(&q.u);
    const __nv_bfloat162 m = __hmax2(__hmax2(w[0], w[1]), __hmax2(w[2], w[3]));
    return fmaxf(fmaxf(__low2float(m), __high2float(m)), -INFINITY);
}

// A piece of a row as its CTA sees it: `vectors` of N values a thread.
template <typename T>
struct Piece {
    static constexpr int N = Logits<T>::N;
    const T* r;       // the row
    int lo, hi;       // tokens [lo, hi)
    int V, shift;     // shift: bits the row starts past a 16-byte boundary
    int vectors;

    // Which tokens a thread takes does not depend on where the row starts, so equal rows
    // have equal sums and tie exactly.
    __device__ __forceinline__ Piece(const BeamSelectArgs& p, int row, int piece, int each) {
        r = static_cast<const T*>(p.logits) + row * p.ld;
        V = p.V;
        shift = (int)(reinterpret_cast<uintptr_t>(r) & 15) * 8;
        vectors = each;
        lo = piece * each * kThreads * N;
        hi = min(lo + each * kThreads * N, V);
    }
    __device__ __forceinline__ int token(int j) const {
        return lo + (j * kThreads + (int)threadIdx.x) * N;
    }
    // A thread's j-th N values, -inf past the row's end.  Off the boundary they come from
    // the two aligned vectors they lie in (the next values of the row have to be there).
    __device__ __forceinline__ Logits<T> load(int j) const {
        Logits<T> q;
        const int v = token(j);
        if (v + (shift ? 2 * N : N) <= V) {
            const uint4* w = reinterpret_cast<const uint4*>(
                reinterpret_cast<uintptr_t>(r + v) & ~(uintptr_t)15);
            q.u = __ldg(w);
            if (shift) q.u = shifted(q.u, __ldg(w + 1), shift);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) q.set(i, v + i < V ? Elem<T>::load(r + v + i) : -INFINITY);
        }
        return q;
    }
    // All threads' vectors j0 .. j0 + n - 1, j0 > 0, on their way into L2 (called by one
    // thread): whole 16 bytes inside the row.
    __device__ __forceinline__ void prefetch(int j0, int n) const {
        const int from = lo + j0 * kThreads * N, to = min(from + n * kThreads * N, hi);
        if (from >= to) return;
        const uintptr_t a = reinterpret_cast<uintptr_t>(r + from) & ~(uintptr_t)15;
        const uintptr_t b = reinterpret_cast<uintptr_t>(r + to) & ~(uintptr_t)15;
        if (a < b)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a),
                         "r"((uint32_t)(b - a)));
    }
    // Vectors j0 .. j0 + U - 1 (those past the piece: -inf).
    template <int U>
    __device__ __forceinline__ void load_some(Logits<T> (&q)[U], int j0) const {
        if (shift == 0 && lo + (j0 + U) * kThreads * N <= hi) {
            const uint4* w = reinterpret_cast<const uint4*>(r + token(j0));
#pragma unroll
            for (int j = 0; j < U; ++j) q[j].u = __ldg(w + j * kThreads);
        } else {
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (j0 + j < vectors) {
                    q[j] = load(j0 + j);
                } else {
#pragma unroll
                    for (int i = 0; i < N; ++i) q[j].set(i, -INFINITY);
                }
            }
        }
    }
};

// The sum of a part's exponentials, in a thread's two halves: few additions one after the
// other (a vector's are in pairs).
template <typename T, int U>
__device__ __forceinline__ uint64_t part_sum(const Logits<T> (&q)[U], uint64_t log2e2,
                                             uint64_t c2) {
    constexpr int N = Logits<T>::N;
    uint64_t sum = 0;
#pragma unroll
    for (int j = 0; j < U; ++j) {
        uint64_t pair[N / 4];
#pragma unroll
        for (int i = 0; i < N; i += 4)
            pair[i / 4] = add2(both_exp2(q[j].get(i), q[j].get(i + 1), log2e2, c2),
                               both_exp2(q[j].get(i + 2), q[j].get(i + 3), log2e2, c2));
        sum = add2(sum, N == 4 ? pair[0] : add2(pair[0], pair[N / 4 - 1]));
    }
    return sum;
}
// The sum of all threads' halves; a barrier.
__device__ __forceinline__ float piece_sum(uint64_t acc, float (&total)[kWarps]) {
    float s, s1;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(s), "=f"(s1) : "l"(acc));
    s = warp_sum(s + s1);
    if ((threadIdx.x & 31) == 0) total[threadIdx.x >> 5] = s;
    __syncthreads();
    float each[kWarps];
#pragma unroll
    for (int j = 0; j < kWarps; ++j) each[j] = total[j];
    return sum_pairs(each);
}

// A piece whose logits lie far above those of its first part: the sum once more, relative to
// the largest of the list.  Returns that and the sum.
template <typename T, int U>
__device__ __noinline__ float2 sum_again(const Piece<T>& w, const uint64_t* list, int have) {
    __shared__ uint32_t largest_of[kWarps];
    __shared__ float total[kWarps];
    uint32_t m = 0;
    for (int i = threadIdx.x; i < have; i += kThreads) m = max(m, (uint32_t)(list[i] >> 32));
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) largest_of[threadIdx.x >> 5] = m;
    __syncthreads();
    for (int j = 0; j < kWarps; ++j) m = max(m, largest_of[j]);
    const float M = unordered(m), c = M * kLog2e;
    uint64_t acc = 0;
    for (int j0 = 0; j0 < w.vectors; j0 += U) {
        Logits<T> q[U];
        w.load_some(q, j0);
        acc = add2(acc, part_sum<T, U>(q, pack2(kLog2e, kLog2e), pack2(-c, -c)));
    }
    return make_float2(M, piece_sum(acc, total));
}

// Pieces whose fast pass gave up: a NaN or +inf, nothing above -inf in the first part, logits
// of 1e7 and more, or so many equal logits that the list ran over.  Values are replaced as
// documented and the threads' maxima carry their tokens: of a step of U vectors a thread,
// at most num_out x U N keys are listed, after the num_out best of the steps before.
template <typename T, int U>
__device__ __noinline__ void careful_piece(const Piece<T>& w, int num, uint64_t* list,
                                           uint64_t* out, float2* sum_out) {
    constexpr int N = Logits<T>::N;
    __shared__ Threshold<kThreads, uint64_t> pick;
    __shared__ uint64_t kept[BEAM_MAX_SELECT];
    __shared__ float part[kWarps];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float M = -INFINITY, S = 0.f;
    int held = 0;
    for (int j0 = 0; j0 < w.vectors; j0 += U) {
        const int j1 = min(j0 + U, w.vectors);
        float m = -INFINITY;
        uint64_t best = 0;
        for (int j = j0; j < j1; ++j) {
            const Logits<T> q = w.load(j);
            const int v = w.token(j);
            for (int i = 0; i < N; ++i) {
                if (v + i >= w.hi) break;
                const float x = tame(q.get(i));
                m = fmaxf(m, x);
                best = max(best, logit_key(x, v + i));
            }
        }
        m = warp_max(m);
        if (lane == 0) part[warp] = m;
        if (tid == 0) count = held;
        if (tid < held) list[tid] = kept[tid];
        int rank;
        const bool among = pick.find(best, num, rank);
        float top = M;
        for (int j = 0; j < kWarps; ++j) top = fmaxf(top, part[j]);
        float s = 0.f;
        const uint64_t from = pick.limit;
        for (int j = j0; j < j1; ++j) {
            const Logits<T> q = w.load(j);
            const int v = w.token(j);
            float e[N];
            for (int i = 0; i < N; ++i) {
                e[i] = 0.f;
                if (v + i >= w.hi) continue;
                const float x = tame(q.get(i));
                if (top != -INFINITY) e[i] = exp2_ftz((x - top) * kLog2e);
                if (among && logit_key(x, v + i) >= from)
                    list[atomicAdd(&count, 1)] = logit_key(x, v + i);
            }
            s += sum_pairs(e);
        }
        s = warp_sum(s);
        __syncthreads();   // the parts are read, the list is complete
        if (lane == 0) part[warp] = s;
        const int have = count;
        rank_list(list, have, num, [&](int rank, uint64_t key) { kept[rank] = key; });
        held = min(have, num);
        __syncthreads();
        if (M != -INFINITY) S *= exp2_ftz((M - top) * kLog2e);
        float e[kWarps];
        for (int j = 0; j < kWarps; ++j) e[j] = part[j];
        S += sum_pairs(e);
        M = top;
        __syncthreads();
    }
    if (tid == 0) *sum_out = make_float2(M, S);
    for (int i = tid; i < num; i += kThreads) out[i] = i < held ? kept[i] : 0;
}

// One piece of one row.  Its first U vectors a thread give the reference of the
// exponentials and, ranked, the num_out best so far: the bound for all that follows.
// The rest then streams by without a barrier, few of its logits reaching the bound; the
// next part is on its way into L2 while one is worked on (64 x 8 x 128000 bf16 39.2 us
// instead of 41.2; two parts ahead 39.7).  Four CTAs an SM leave 64 registers: with five,
// of 48, values spill (42.2).
template <typename T, int U>
__global__ void __launch_bounds__(kThreads, 4)
beam_piece_kernel(const BeamSelectArgs p, int pieces, int each, uint64_t* __restrict__ keys,
                  float2* __restrict__ sums) {
    constexpr int N = Logits<T>::N;
    extern __shared__ __align__(16) uint64_t list[];   // num_out (U N + 1), at least kList
    __shared__ uint32_t bound[kWarps];
    __shared__ float part[kWarps];
    __shared__ float total[kWarps];
    __shared__ float limit;
    __shared__ int count;
    asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x / pieces;
    const int num = p.num_out;
    uint64_t* out = keys + (int64_t)blockIdx.x * num;
    const Piece<T> w(p, row, blockIdx.x - row * pieces, each);
    const float score = tame(p.scores[row]);
    const bool finished = p.finished && p.finished[row];
    if (finished || score == -INFINITY) {
        // nothing to read: `eos` of a finished beam, then the lowest tokens at -inf
        const bool has = finished && score != -INFINITY && p.eos >= w.lo && p.eos < w.hi;
        for (int j = tid; j < num; j += kThreads) {
            int v = w.lo + j;
            uint64_t key = 0;
            if (has) {
                if (j == 0) key = logit_key(0.f, p.eos);
                else if (--v >= p.eos) ++v;   // the tokens without eos
            }
            if (!key && v < w.hi) key = logit_key(-INFINITY, v);
            out[j] = key;
        }
        if (tid == 0) sums[blockIdx.x] = has ? make_float2(0.f, 1.f) : make_float2(-INFINITY, 0.f);
        return;
    }

    Logits<T> q[U];
    w.load_some(q, 0);
    if (tid == 0) w.prefetch(U, U);
    // their maximum, and a bound that at least num_out threads reach
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < U; ++j) m = fmaxf(m, largest(q[j]));
    const int warps = min((w.hi - w.lo) / (32 * N), kWarps);   // whose threads all have values
    const uint32_t nth = warp < warps ? warp_nth(ordered(m), (num + warps - 1) / warps, lane) : 0;
    m = warp_max(m);
    if (lane == 0) {
        part[warp] = m;
        bound[warp] = nth;
    }
    if (tid == 0) {
        count = 0;
        limit = -INFINITY;
    }
    __syncthreads();
    uint32_t least = warps > 0 ? bound[0] : 0;
    float M = part[0];
#pragma unroll
    for (int j = 1; j < kWarps; ++j) {
        if (j < warps) least = min(least, bound[j]);
        M = fmaxf(M, part[j]);
    }
    const float c = M * kLog2e;
    const uint64_t log2e2 = pack2(kLog2e, kLog2e), c2 = pack2(-c, -c);
    uint64_t acc = 0;
    // the sum of exponentials; the vectors with a logit at or above the bound are read
    // again, in a loop that is short code (unrolled over the registers a third of the
    // time went to instruction fetches), and those logits listed
    auto look = [&](int j0, float from) {
        uint32_t hits = 0;
        acc = add2(acc, part_sum<T, U>(q, log2e2, c2));
#pragma unroll
        for (int j = 0; j < U; ++j) hits |= (largest(q[j]) >= from ? 1u : 0u) << j;
        for (; hits; hits &= hits - 1) {
            const int j = j0 + __ffs(hits) - 1, v = w.token(j);
            if (j >= w.vectors) break;
            const Logits<T> x = w.load(j);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (x.get(i) >= from && v + i < w.hi) {
                    const int place = atomicAdd(&count, 1);
                    if (place < kList) list[place] = logit_key(x.get(i), v + i);
                }
            }
        }
    };
    look(0, least ? unordered(least) : -INFINITY);
    if (each > U) {
        // the num_out-th best so far: at least num_out logits of the piece reach it
        __syncthreads();
        const int have = min(count, kList);
        rank_list(list, have, num, [&](int rank, uint64_t key) {
            if (rank == num - 1) limit = unordered((uint32_t)(key >> 32));
        });
        __syncthreads();
        for (int j0 = U; j0 < each; j0 += U) {
            w.load_some(q, j0);
            if (tid == 0) w.prefetch(j0 + U, U);
            look(j0, limit);
        }
    }
    float s = piece_sum(acc, total);   // the list is complete, too
    const int have = count;
    if (s >= kMostSum && have <= kList) {
        const float2 again = sum_again<T, U>(w, list, have);
        M = again.x;
        s = again.y;
    }
    const float rest = fmaf(M, kLog2e, -(M * kLog2e));
    // the same in all threads; a NaN in either fails its comparison
    if (!(s > 0.f && s < kMostSum) || !(fabsf(rest) <= kMostRest) || have > kList) {
        __syncthreads();
        careful_piece<T, U>(w, num, list, out, sums + blockIdx.x);
        return;
    }
    // s 2^-rest, the factor's distance from 1 by itself: a factor near 1 would be rounded (by
    // the last thread: the first ones rank the list)
    if (tid == kThreads - 1) sums[blockIdx.x] = make_float2(M, fmaf(s, expm1f(-rest * kLn2), s));
    rank_list(list, have, num, [&](int rank, uint64_t key) { out[rank] = key; });
    for (int i = have + tid; i < num; i += kThreads) out[i] = 0;
}

// ln t for t > 0 to about 2^-25, as two addends of which the first is exact: t = 2^e f,
// e ln 2 in two parts and ln f of an f near 1.  (The 64-bit functions took half of the
// joining kernel's time: this card's 64-bit rate is low.)
__device__ __forceinline__ double log_of_sum(float t) {
    int e = (int)(__float_as_uint(t) >> 23) - 127;
    float f = __uint_as_float((__float_as_uint(t) & 0x7fffffu) | 0x3f800000u);   // [1, 2)
    if (f > 1.4142135f) {
        f *= 0.5f;
        ++e;
    }
    // ln 2 = 0.693145751953125 (17 bits, so times e it is exact) + the rest
    return (double)(e * 0.693145751953125f) + (double)(fmaf((float)e, 1.42860677e-6f, logf(f)));
}

// One request: joins its rows' pieces.
template <int THREADS>
__global__ void __launch_bounds__(THREADS)
beam_join_kernel(const BeamSelectArgs p, int pieces, uint32_t per_beam_inv,
                 const uint64_t* __restrict__ keys, const float2* __restrict__ sums) {
    extern __shared__ __align__(16) ValueKey candidates[];   // num_out x a thread's share
    __shared__ Threshold<THREADS, ValueKey> pick;
    __shared__ double lse[BEAM_MAX_BEAMS], score[BEAM_MAX_BEAMS];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x, num = p.num_out;
    if (tid == 0) count = 0;
    if (tid < p.K) score[tid] = (double)tame(p.scores[(int64_t)b * p.K + tid]);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int per_beam = pieces * num, all = p.K * per_beam;
    const uint64_t* mine = keys + (int64_t)b * all;
    // neighbouring candidates, of one beam and good or bad together, go to different warps:
    // the first bound is the worst warp's, and would be loose otherwise
    const int first = lane * (THREADS / 32) + warp;
    const uint64_t first_key = first < all ? mine[first] : 0;   // under way with the sums
    // a row's maximum, then its pieces' sums relative to it; a warp a row
    for (int k = warp; k < p.K; k += THREADS / 32) {
        const float2* q = sums + ((int64_t)b * p.K + k) * pieces;
        const float2 own = lane < pieces ? q[lane] : make_float2(-INFINITY, 0.f);
        float M = own.x;
        for (int j = lane + 32; j < pieces; j += 32) M = fmaxf(M, q[j].x);
        M = warp_max(M);
        float s = own.y > 0.f ? own.y * expf(own.x - M) : 0.f;
        for (int j = lane + 32; j < pieces; j += 32)
            if (q[j].y > 0.f) s = fmaf(q[j].y, expf(q[j].x - M), s);
        s = warp_sum(s);
        if (lane == 0) lse[k] = s > 0.f ? (double)M + log_of_sum(s) : 0.0;
    }
    __syncthreads();

    auto value = [&](int i, uint64_t key) {
        ValueKey q{0, 0};
        if (key) {
            const int k = per_beam == 1 ? i : (int)__umulhi((uint32_t)i, per_beam_inv);
            const float x = unordered((uint32_t)(key >> 32));
            const uint32_t v = 0xffffffffu - (uint32_t)key;
            const double val = x == -INFINITY || score[k] == -INFINITY
                                   ? -INFINITY : score[k] + ((double)x - lse[k]);
            q.value = ordered(val);
            q.index = 0xffffffffu - ((uint32_t)k * (uint32_t)p.V + v);
        }
        return q;
    };
    auto put = [&](int rank, const ValueKey& key) {
        const uint32_t at = 0xffffffffu - (uint32_t)key.index;
        const int64_t o = (int64_t)b * num + rank;
        p.out_scores[o] = (float)unordered(key.value);
        p.out_parents[o] = b * p.K + (int)(at / (uint32_t)p.V);
        p.out_tokens[o] = (int)(at % (uint32_t)p.V);
    };
    ValueKey best = value(first, first_key);
    for (int i = first + THREADS; i < all; i += THREADS) {
        const ValueKey q = value(i, mine[i]);
        if (above(q, best)) best = q;
    }
    int rank;
    const bool among = pick.find(best, num, rank);
    if (all <= THREADS) {   // a candidate a thread: the ranks are final
        if (among) put(rank, best);
        return;
    }
    if (among) {
        const ValueKey from = pick.limit;
        for (int i = first; i < all; i += THREADS) {
            const ValueKey q = value(i, i == first ? first_key : mine[i]);
            if (exists(q) && !above(from, q)) candidates[atomicAdd(&count, 1)] = q;
        }
    }
    __syncthreads();
    rank_list(candidates, count, num, put);
}

struct Pieces {
    int pieces, each;   // of a row; 16-byte vectors a thread
};
// Pieces for kCtas CTAs an SM, none shorter than one vector a thread: more pieces leave
// more candidates to join, fewer leave SMs idle (16 x 8 x 128000 bf16 logits: 23.1 us with 2
// CTAs an SM, 22.2 with 3, 27.9 with 4; 32 x 8 x 32000: 15.7, 15.7, 22.0; 64 x 8 x 128000:
// 39, 39, 43).  Nor so long that the logits above the bound of a piece's first part,
// num_out a part on average, outgrow its list (64 x 8 x 250000 in one piece a row: 410 us,
// in two 110).
Pieces split_row(int64_t rows, int32_t K, int32_t V, int32_t num_out, kda_dtype dtype) {
    const int N = dtype == KDA_BF16 ? 8 : 4;
    const int64_t blocks = ((int64_t)(V + N - 1) / N + kThreads - 1) / kThreads;   // one vector a thread
    const int64_t ctas = kCtas * (int64_t)(sm_count() > 0 ? sm_count() : 148);
    const int64_t longest = kParts * kList / 4 / num_out;
    int64_t pieces = rows > 0 ? (ctas + rows - 1) / rows : 1;
    pieces = pieces < blocks ? pieces : blocks;
    const int64_t joined = kJoin * kThreads / (K * num_out);   // 32 beams, 64 of 260000: 136 us without
    if (pieces > joined) pieces = joined > 1 ? joined : 1;
    Pieces s;
    s.each = (int)((blocks + pieces - 1) / pieces);
    if (s.each > longest) s.each = (int)longest;
    s.pieces = (int)((blocks + s.each - 1) / s.each);
    return s;
}

// Candidates a thread of the joining kernel may hold.
int join_share(const Pieces& s, int K, int num_out, int threads) {
    return (K * s.pieces * num_out + threads - 1) / threads;
}

size_t pad(size_t b) { return (b + 255) & ~(size_t)255; }

// Allows a kernel `most` bytes of dynamic shared memory, its largest use by any call.  The
// limit is the kernel's, for all host threads: with each call's own size, one call could
// lower it between another's setting and its launch.
template <typename K>
cudaError_t allow_shared(K kernel, size_t most) {
    if (most <= 16 * 1024) return cudaSuccess;   // with the static part below the default limit
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
}

// Bytes of a piece's list: that of a careful step, at least the fast pass's.
constexpr size_t list_bytes(int num_out, int values) {
    const size_t most = (size_t)num_out * (values + 1);
    return (most > kList ? most : kList) * sizeof(uint64_t);
}
// Bytes of the joining kernel's candidates at most.  kJoin a thread with 256 threads.  With
// 1024 more than that come from pieces kept short (see split_row): of 2^20 fp32 logits, 32
// pieces of 32 vectors a thread, 32 beams, 64 of them: 64 a thread.
template <int THREADS>
constexpr size_t kMostJoin = (THREADS == kThreads ? kJoin : 64) * BEAM_MAX_SELECT *
                             sizeof(ValueKey);

template <typename T, int U>
cudaError_t launch_pieces(const BeamSelectArgs& a, const Pieces& s, uint64_t* keys, float2* sums,
                          cudaStream_t stream) {
    if constexpr (U > 1) {
        if (s.each <= U / 2) return launch_pieces<T, U / 2>(a, s, keys, sums, stream);
    }
    constexpr int kValues = U * Logits<T>::N;
    const cudaError_t err =
        allow_shared(beam_piece_kernel<T, U>, list_bytes(BEAM_MAX_SELECT, kValues));
    if (err != cudaSuccess) return err;
    const size_t smem = list_bytes(a.num_out, kValues);
    const unsigned grid = (unsigned)((int64_t)a.B * a.K * s.pieces);
    beam_piece_kernel<T, U><<<grid, kThreads, smem, stream>>>(a, s.pieces, s.each, keys, sums);
    return cudaGetLastError();
}

template <int THREADS>
cudaError_t launch_join(const BeamSelectArgs& a, const Pieces& s, const uint64_t* keys,
                        const float2* sums, cudaStream_t stream) {
    const size_t smem =
        (size_t)join_share(s, a.K, a.num_out, THREADS) * a.num_out * sizeof(ValueKey);
    if (smem > kMostJoin<THREADS>) return cudaErrorInvalidValue;
    const cudaError_t err = allow_shared(beam_join_kernel<THREADS>, kMostJoin<THREADS>);
    if (err != cudaSuccess) return err;
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
    // i / (pieces num_out) as a product: exact for i below 2^32 over the divisor
    const uint32_t inv = (uint32_t)(((1ull << 32) + s.pieces * a.num_out - 1) / (s.pieces * a.num_out));
    return cudaLaunchKernelEx(&c, beam_join_kernel<THREADS>, a, s.pieces, inv, keys, sums);
}

// ---------------------------------------------------------------- reordering
//
// A thread owns one column (16, 4 or 1 bytes) of a request's K rows: it reads the
// rows that move, all before it writes any, so the permutation needs no second copy
// of the tensor and no barrier, and rows that stay cost nothing.  Bound: HBM; 32 requests
// of 8 rows of 2.1 MB, 0.80 GB: 119-123 us (6.5 TB/s).

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
        const Pieces s = split_row(rows, K, V, num_out, t);
        const size_t n = (size_t)rows * s.pieces;
        const size_t b = pad(n * num_out * sizeof(uint64_t)) + pad(n * sizeof(float2));
        most = b > most ? b : most;
    }
    return most;
}

cudaError_t launch_beam_select(const BeamSelectArgs& a, char* ws, cudaStream_t stream) {
    const int64_t rows = (int64_t)a.B * a.K;
    const Pieces s = split_row(rows, a.K, a.V, a.num_out, a.dtype);
    uint64_t* keys = reinterpret_cast<uint64_t*>(ws);
    float2* sums = reinterpret_cast<float2*>(ws + pad((size_t)rows * s.pieces * a.num_out * 8));
    const cudaError_t err = a.dtype == KDA_BF16
                                ? launch_pieces<__nv_bfloat16, kParts>(a, s, keys, sums, stream)
                                : launch_pieces<float, kParts>(a, s, keys, sums, stream);
    if (err != cudaSuccess) return err;
    if (join_share(s, a.K, a.num_out, kThreads) <= kJoin)
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
