// Gated linear recurrence h_t = a_t h_{t-1} + u_t (include/linrec.h): prefill,
// backward and decode step.
//
// Mathematics.  Every channel is a chain of affine maps h -> a h + u, and maps
// compose: over a run of tokens h_out = A h_in + B with A the product of the
// gates and B the run's result from zero.  A tile of 256 tokens (backward 128) x 64
// channels belongs to one CTA: each of its eight warps takes 32 (16) tokens, two
// channels a lane, with the gates in registers and the rows in shared memory, forms
// its (A, B), and once the state that enters the tile is known every warp starts from
// its own entry state and walks its tokens again.  So x and the gate are read from
// memory once and y is written once.
//
// The packed token axis is cut into tiles regardless of sequences.  At a
// sequence's first token the carried state is replaced by S0 (replaced, not
// multiplied by zero: a state that is not finite stays in its sequence), and a
// tile with such a token needs nothing from before it for what follows.
//
// Between tiles: each publishes its (A, B) as one 8-byte record a channel, and once
// the state that leaves it is known, that state as the map (0, h).  A tile reads
// the records of the eight tiles before it (a warp each) and applies them in token
// order from a map with A = 0 on: the arithmetic is the same whichever that is, so
// results do not depend on timing.  A record is one
// atomic word that is valid as soon as it is not the pattern the workspace was
// filled with, so neither side needs a fence (with flags and fences a tile took
// 13.7 us instead of 4.4).  Tiles are handed out in time order by a ticket, so a
// tile's predecessors are always running or done; every wait is bounded all the same.
//
// The backward pass is the same recurrence on reversed tokens:
// r_t = a_t (dy_t + r_{t+1}), g_t = dy_t + r_{t+1}, with dS_T replacing r at a
// sequence's last token; the states it multiplies are rebuilt in registers from
// the tile's entry state (`states`).
//
// Bound: HBM.  Measured, bf16: prefill of one sequence of 131072 x 4096 with log gates 557
// us for 3.2 GB (5.8 TB/s), of 64 ragged ones, 266240 x 4096, 1343 us for 8.7 GB (6.5);
// backward of 8 x 4096 x 4096 380 us for 2.1 GB (5.7).  32 tokens a warp and two CTAs an SM
// hold 192 KB of inputs on an SM, which covers the waits for the tiles before; 16 tokens
// and three CTAs took 10 % longer.  With one gate a head there are fewer bytes for the same
// instructions: 8 x 4096 x 4096 forward 140 us for 0.54 GB (3.9 TB/s), backward 363 us for
// 1.1 GB (3.0), issue slots 55 and 53 % busy, the rest waits.
#include "kda_internal.h"

#include <cfloat>
#include <type_traits>

namespace kda {
namespace {

constexpr int kWarps = 8;
constexpr int kFwdRows = 32;   // tokens a warp
constexpr int kBwdRows = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kSelfCheck = 1024;   // most sequences whose offsets every CTA checks by itself
constexpr uint64_t kWaitNs = 2000000000ull;
static_assert(kWarps * kFwdRows % LINREC_CHUNK == 0 && kWarps * kBwdRows == LINREC_CHUNK,
              "the forward tiles hold whole chunks, a backward tile is one");
static_assert(kWarps * kFwdRows <= LINREC_MAX_TILE, "the header says over how many tokens the "
              "products of gates have to be finite");

// The workspace, filled with 0xff bytes before each launch whose time axis has
// several tiles (so the first ticket is 2^32 - 1, and a record that is all ones has
// not been published: a computed NaN never has that pattern).
//   [0, 4) status, [4, 8) ticket, [256, ..) uint64 record[tiles][Dp], Dp the
//   channels padded to whole tiles: A in the low half, B in the high half
struct TileSpace {
    int32_t* status;
    uint32_t* ticket;
    uint64_t* record;
    int32_t nt, ct;      // tiles along tokens and channels
    int64_t Dp;
    uint64_t wait_ns;    // limit of a wait for another tile
};
constexpr size_t kRecords = 256;

__device__ __forceinline__ uint64_t now_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// VEC neighbouring channels in fp32; two take the packed instructions.
template <int VEC>
struct Vec {
    float v[VEC];
};
template <int VEC>
__device__ __forceinline__ Vec<VEC> fill(float x) {
    Vec<VEC> r;
#pragma unroll
    for (int i = 0; i < VEC; ++i) r.v[i] = x;
    return r;
}
__device__ __forceinline__ uint64_t pack2(const Vec<2>& a) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.v[0]), "f"(a.v[1]));
    return r;
}
__device__ __forceinline__ Vec<2> unpack2(uint64_t r) {
    Vec<2> a;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a.v[0]), "=f"(a.v[1]) : "l"(r));
    return a;
}
__device__ __forceinline__ Vec<2> fma(const Vec<2>& a, const Vec<2>& b, const Vec<2>& c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pack2(a)), "l"(pack2(b)), "l"(pack2(c)));
    return unpack2(r);
}
__device__ __forceinline__ Vec<2> mul(const Vec<2>& a, const Vec<2>& b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack2(a)), "l"(pack2(b)));
    return unpack2(r);
}
__device__ __forceinline__ Vec<2> add(const Vec<2>& a, const Vec<2>& b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack2(a)), "l"(pack2(b)));
    return unpack2(r);
}
__device__ __forceinline__ Vec<1> fma(const Vec<1>& a, const Vec<1>& b, const Vec<1>& c) {
    return {fmaf(a.v[0], b.v[0], c.v[0])};
}
__device__ __forceinline__ Vec<1> mul(const Vec<1>& a, const Vec<1>& b) {
    return {a.v[0] * b.v[0]};
}
__device__ __forceinline__ Vec<1> add(const Vec<1>& a, const Vec<1>& b) {
    return {a.v[0] + b.v[0]};
}

template <int VEC>
__device__ __forceinline__ Vec<VEC> choose(bool first, const Vec<VEC>& a, const Vec<VEC>& b) {
    Vec<VEC> r;
#pragma unroll
    for (int i = 0; i < VEC; ++i) r.v[i] = first ? a.v[i] : b.v[i];
    return r;
}

// VEC neighbouring values of a row as stored.
template <typename T, int VEC>
struct Piece;
template <>
struct Piece<__nv_bfloat16, 2> {
    uint32_t v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        v = *reinterpret_cast<const uint32_t*>(p);
    }
    __device__ __forceinline__ Vec<2> get() const {
        return {__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)};
    }
};
template <>
struct Piece<__nv_bfloat16, 1> {
    __nv_bfloat16 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *p; }
    __device__ __forceinline__ Vec<1> get() const { return {__bfloat162float(v)}; }
};
template <>
struct Piece<float, 2> {
    Vec<2> v;
    __device__ __forceinline__ void load(const float* p) {
        const float2 u = *reinterpret_cast<const float2*>(p);
        v = {u.x, u.y};
    }
    __device__ __forceinline__ Vec<2> get() const { return v; }
};
template <>
struct Piece<float, 1> {
    Vec<1> v;
    __device__ __forceinline__ void load(const float* p) { v = {*p}; }
    __device__ __forceinline__ Vec<1> get() const { return v; }
};

__device__ __forceinline__ void store(float* p, const Vec<2>& x) {
    *reinterpret_cast<float2*>(p) = make_float2(x.v[0], x.v[1]);
}
__device__ __forceinline__ void store(float* p, const Vec<1>& x) { *p = x.v[0]; }
__device__ __forceinline__ void store(__nv_bfloat16* p, const Vec<2>& x) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x.v[0], x.v[1]);
}
__device__ __forceinline__ void store(__nv_bfloat16* p, const Vec<1>& x) {
    *p = __float2bfloat16_rn(x.v[0]);
}
template <int VEC>
__device__ __forceinline__ Vec<VEC> load_f32(const float* p) {
    Piece<float, VEC> q;
    q.load(p);
    return q.get();
}

// The gate of VEC channels of one token.
template <int GATE, int VEC>
struct Gate {
    Vec<VEC> f;
    __device__ __forceinline__ Vec<VEC> a() const { return f; }
    __device__ __forceinline__ Vec<VEC> na() const {
        Vec<VEC> r;
#pragma unroll
        for (int i = 0; i < VEC; ++i) r.v[i] = 1.f - f.v[i];
        return r;
    }
};
// One gate a head: a lane's channels share it (see lane_channels).
template <int VEC>
struct Gate<KDA_GATE_HEAD_F32, VEC> {
    float f;
    __device__ __forceinline__ Vec<VEC> a() const { return fill<VEC>(f); }
    __device__ __forceinline__ Vec<VEC> na() const { return fill<VEC>(1.f - f); }
};
// a = e^(log a) as 2^(log a log2 e + s) 2^-s, three instructions where the full function
// takes nine (625 -> 562 us for 131072 x 4096).  The special-function unit cuts its
// argument off after 24 fractional bits, which by itself leaves gates near 1, of which a
// state multiplies hundreds, 2e-8 too small on average; s moves their argument to where
// the multiply-add has rounded it to those bits already.  s is one of the values whose
// 2^-s is a float to 1e-12.  Measured over all bf16 inputs down to log a = -1: at most
// 1.6e-7 of the gate, 1e-8 or less on average (the full function: 1.1e-7 and 1.5e-8); a
// log gate of 0 gives exactly 1, and none more than 1.  Below the normal numbers the gate
// is 0.
__device__ __forceinline__ float gate_exp(float la) {
    float a;
    asm("ex2.approx.ftz.f32 %0, %1;"
        : "=f"(a) : "f"(fmaf(la, 1.4426950408889634f, 0x1.8ca934p-1f)));
    return a * 0x1.2b4368p-1f;
}
// log a in bf16; 1 - a from expm1, since 1 - exp would lose it near 1.
template <int VEC>
struct Gate<KDA_GATE_CHANNEL_LOG_BF16, VEC> {
    Piece<__nv_bfloat16, VEC> raw;
    Vec<VEC> f;
    __device__ __forceinline__ Vec<VEC> a() const { return f; }
    __device__ __forceinline__ Vec<VEC> na() const {
        const Vec<VEC> la = raw.get();
        Vec<VEC> r;
#pragma unroll
        for (int i = 0; i < VEC; ++i) r.v[i] = -expm1f(la.v[i]);
        return r;
    }
};

// A warp's rows of x and dy lie in its own part of shared memory (R rows of 32
// lanes x VEC channels; every lane reads back its own channels only), the gates in
// registers: with both in registers only three CTAs fit an SM, which is enough to
// keep HBM busy without the look-back but not with it.
__device__ __forceinline__ uint32_t shared_addr(const void* p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES)
                     : "memory");
}
__device__ __forceinline__ void copies_done() {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
}

// Starts the copies of rows [0, left) of src from element row0 (first row, first
// channel of the tile; the same in all lanes) to dst.  Whole tiles on a 16-byte grid
// go in 16-byte pieces, others by each lane's own channels.
template <int R, typename T, int VEC>
__device__ __forceinline__ void stage_rows(T* dst, const void* src, int64_t row0, int64_t D,
                                           bool wide, int left, bool on, int lane) {
    constexpr int E = sizeof(T);
    if (VEC == 2 && wide) {
        constexpr int kPieces = 64 * E / 16;     // 16-byte pieces a row
        constexpr int kStep = 32 / kPieces;      // rows a pass
        const int row = lane / kPieces, piece = lane % kPieces;
        const char* q = static_cast<const char*>(src) + (row0 + row * D) * E + piece * 16;
        const uint32_t at = shared_addr(dst) + lane * 16;
#pragma unroll
        for (int j = 0; j < R / kStep; ++j)
            copy_async<16>(at + j * 512, q + j * kStep * D * E);
        return;
    }
    const T* q = static_cast<const T*>(src) + row0 + lane * VEC;
    T* d = dst + lane * VEC;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (on && r < left) {
            if constexpr (VEC * E >= 4) copy_async<VEC * E>(shared_addr(d + r * 32 * VEC), q + r * D);
            else d[r * 32 * VEC] = q[r * D];
        }
    }
}
template <typename T, int VEC>
__device__ __forceinline__ Vec<VEC> staged(const T* rows, int r, int lane) {
    Piece<T, VEC> q;
    q.load(rows + r * 32 * VEC + lane * VEC);
    return q.get();
}

// The gates of a warp's rows, in registers.
template <int R, int GATE, int VEC>
__device__ __forceinline__ void take_gate(Gate<GATE, VEC> (&a)[R], const LinrecArgs& p,
                                          int64_t t0, int64_t D, int c0, bool full, int left,
                                          bool on, int lane) {
    if constexpr (GATE == KDA_GATE_HEAD_F32) {
        const float* g = static_cast<const float*>(p.gate) + t0 * p.H +
                         min(c0 + lane * VEC, (int)D - 1) / p.d;
#pragma unroll
        for (int r = 0; r < R; ++r) a[r].f = full || r < left ? g[r * p.H] : 0.f;
    } else {
        using G = std::conditional_t<GATE == KDA_GATE_CHANNEL_LOG_BF16, __nv_bfloat16, float>;
        const G* g = static_cast<const G*>(p.gate) + t0 * D + c0;
        Piece<G, VEC> q[R];
        if (full) {
#pragma unroll
            for (int r = 0; r < R; ++r) q[r].load(g + r * D + lane * VEC);
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                q[r] = Piece<G, VEC>{};
                if (on && r < left) q[r].load(g + r * D + lane * VEC);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if constexpr (GATE == KDA_GATE_CHANNEL_LOG_BF16) a[r].raw = q[r];
            else a[r].f = q[r].get();
        }
    }
}
// Once all loads are under way: a from log a.
template <int R, int GATE, int VEC>
__device__ __forceinline__ void expand_gate(Gate<GATE, VEC> (&a)[R]) {
    if constexpr (GATE == KDA_GATE_CHANNEL_LOG_BF16) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const Vec<VEC> la = a[r].raw.get();
#pragma unroll
            for (int v = 0; v < VEC; ++v) a[r].f.v[v] = gate_exp(la.v[v]);
        }
    }
}

// The inputs u = (1 - a) x of the complement, in fp32 over the 4 bytes a value that
// the warp's rows have (bf16 values were copied into the upper half, and the lower
// rows are written before the upper ones are read).
template <int R, typename T, int GATE, int VEC>
__device__ __forceinline__ void complement_rows(float* u, const T* x, const Gate<GATE, VEC> (&a)[R],
                                                int lane) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        Piece<T, VEC> q[R / 2];
#pragma unroll
        for (int r = 0; r < R / 2; ++r)
            q[r].load(x + (half * (R / 2) + r) * 32 * VEC + lane * VEC);
        __syncwarp();
#pragma unroll
        for (int r = 0; r < R / 2; ++r) {
            const int row = half * (R / 2) + r;
            store(u + row * 32 * VEC + lane * VEC, mul(a[row].na(), q[r].get()));
        }
    }
}

// Offsets of the sequences: checked once a CTA, sampled into shared memory.
struct Offsets {
    int32_t sample[kSelfCheck + 2];
    int32_t stride, count;   // sample[j] = cu[min(j * stride, N)], j < count
};

// True when the offsets are valid.  Up to kSelfCheck sequences are checked here
// (every CTA for itself), more by linrec_check_kernel before the launch.  Waits for that
// one and for the fill of the workspace: nothing of it is touched before.
__device__ bool read_offsets(Offsets& o, const int32_t* cu, int N, int64_t T,
                             const int32_t* status) {
    bool bad = false;
    const int stride = (N + 1 + kSelfCheck) / (kSelfCheck + 1);
    const int count = N / stride + 1 + (N % stride != 0);
    if (N <= kSelfCheck) {
        for (int i = threadIdx.x; i <= N; i += kThreads) {
            const int32_t c = cu[i];
            o.sample[i] = c;
            bad |= i == 0 ? c != 0 : c < cu[i - 1];
            if (i == N) bad |= (int64_t)c > T;
        }
        asm volatile("griddepcontrol.wait;" ::: "memory");
    } else {
        for (int j = threadIdx.x; j < count; j += kThreads)
            o.sample[j] = cu[min((int64_t)j * stride, (int64_t)N)];
        asm volatile("griddepcontrol.wait;" ::: "memory");
        bad = *reinterpret_cast<const volatile int32_t*>(status) == KDA_ERR_DEVICE_INPUT;
    }
    if (threadIdx.x == 0) {
        o.stride = stride;
        o.count = count;
    }
    return !__syncthreads_or(bad);
}

// The sequence that token t < cu[N] belongs to: the last n with cu[n] <= t.
__device__ __forceinline__ int sequence_of(const Offsets& o, const int32_t* cu, int N, int32_t t) {
    int lo = 0, hi = o.count - 1;   // sample[lo] <= t < sample[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (o.sample[mid] <= t) lo = mid;
        else hi = mid;
    }
    if (o.stride == 1) return lo;
    int a = lo * o.stride, b = min(a + o.stride, N);
    while (b - a > 1) {
        const int mid = (a + b) >> 1;
        if (cu[mid] <= t) a = mid;
        else b = mid;
    }
    return a;
}

// First and last tokens of sequences among a warp's rows (bit r: row r), the
// sequence of row `lane`, and how many rows lie before the end.
struct Rows {
    uint32_t start, last;
    int n, live;
};
template <int R>
__device__ __forceinline__ Rows rows_of(const Offsets& o, const int32_t* cu, int N, int64_t t0,
                                        int64_t end, int lane) {
    Rows w;
    const int64_t t = t0 + lane;
    const bool live = lane < R && t < end;
    bool s = false, l = false;
    w.n = 0;
    if (live) {
        w.n = sequence_of(o, cu, N, (int32_t)t);
        s = (o.stride == 1 ? o.sample[w.n] : cu[w.n]) == t;
        l = (o.stride == 1 ? o.sample[w.n + 1] : cu[w.n + 1]) - 1 == t;
    }
    w.start = __ballot_sync(0xffffffffu, s);
    w.last = __ballot_sync(0xffffffffu, l);
    w.live = end <= t0 ? 0 : end - t0 < R ? (int)(end - t0) : R;
    return w;
}

// The status word: without a fill of the workspace it is simply set; else it turns
// from the fill's pattern to OK unless an error was recorded before.
__device__ __forceinline__ void clear_status(const TileSpace& w, int N) {
    if (w.nt == 1 && N <= kSelfCheck) *w.status = KDA_OK;
    else atomicCAS(reinterpret_cast<uint32_t*>(w.status), ~0u, (uint32_t)KDA_OK);
}

// True when every row of the tile is an inner token of one sequence: no boundary in it.
__device__ __forceinline__ bool inner_tile(const Offsets& o, const int32_t* cu, int N, int64_t first,
                                           int tile, int64_t end) {
    if (first + tile >= end) return false;
    const int n = sequence_of(o, cu, N, (int32_t)first);
    const int32_t lo = o.stride == 1 ? o.sample[n] : cu[n];
    const int32_t hi = o.stride == 1 ? o.sample[n + 1] : cu[n + 1];
    return lo < first && hi > first + tile;
}

// dst[n] = src[n] (zeros without src) for the sequences without tokens.
__device__ void copy_empty(const int32_t* cu, int N, int64_t D, const float* src, float* dst) {
    if (!dst || dst == src) return;
    for (int n = blockIdx.x; n < N; n += gridDim.x) {
        if (cu[n] != cu[n + 1]) continue;
        for (int64_t c = threadIdx.x; c < D; c += kThreads)
            dst[n * D + c] = src ? src[n * D + c] : 0.f;
    }
}

// Records of a lane's VEC channels.
template <int VEC>
struct Record {
    uint64_t r[VEC];
    __device__ __forceinline__ void read(const uint64_t* p) {
        if constexpr (VEC == 2)
            asm volatile("ld.relaxed.gpu.global.v2.b64 {%0, %1}, [%2];"
                         : "=l"(r[0]), "=l"(r[1]) : "l"(p) : "memory");
        else
            asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(r[0]) : "l"(p) : "memory");
    }
    __device__ __forceinline__ void write(uint64_t* p) const {
        if constexpr (VEC == 2)
            asm volatile("st.relaxed.gpu.global.v2.b64 [%0], {%1, %2};"
                         ::"l"(p), "l"(r[0]), "l"(r[1]) : "memory");
        else
            asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(p), "l"(r[0]) : "memory");
    }
    __device__ __forceinline__ bool ready() const {
        bool all = true;
#pragma unroll
        for (int v = 0; v < VEC; ++v) all &= r[v] != ~0ull;
        return all;
    }
    __device__ __forceinline__ void set(const Vec<VEC>& A, const Vec<VEC>& B) {
#pragma unroll
        for (int v = 0; v < VEC; ++v)
            r[v] = (uint64_t)__float_as_uint(B.v[v]) << 32 | __float_as_uint(A.v[v]);
    }
    __device__ __forceinline__ float A(int v) const { return __uint_as_float((uint32_t)r[v]); }
    __device__ __forceinline__ float B(int v) const {
        return __uint_as_float((uint32_t)(r[v] >> 32));
    }
};

// A product of gates as published: finite, so that a state of zero stays zero behind gates
// above 1 whose product over the tile overflows, and no NaN, so that the record is not all
// ones (where a gate is NaN, B is as well, and says so).  Handing on only the state where a
// product is infinite would make every finite state right, but the test for it stands
// between a tile's state and the next: 9 % of a narrow sequence's time (200000 x 64).
template <int VEC>
__device__ __forceinline__ Vec<VEC> finite(Vec<VEC> A) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) A.v[v] = fminf(fmaxf(A.v[v], -FLT_MAX), FLT_MAX);
    return A;
}

// Publishes a tile's map, or with A = 0 the state that leaves it (one warp).
template <int VEC>
__device__ __forceinline__ void publish(const TileSpace& w, int i, int64_t ch,
                                        const Vec<VEC>& A, const Vec<VEC>& B) {
    Record<VEC> r;
    r.set(A, B);
    r.write(w.record + (int64_t)i * w.Dp + ch);
}

// True once a wait that began at t0 (0: now) is over its limit, here or in another CTA.
__device__ __noinline__ bool expired(const TileSpace& w, uint64_t& t0) {
    const uint64_t t = now_ns();
    if (t0 == 0) t0 = t;
    if (t - t0 > w.wait_ns) atomicExch(w.status, (int32_t)KDA_ERR_DEVICE_TIMEOUT);
    return *reinterpret_cast<volatile int32_t*>(w.status) == KDA_ERR_DEVICE_TIMEOUT;
}

// The state that enters tile i, for the lane's VEC channels from ch: warp j waits
// for the record of the tile j + 1 steps before (step = -1: towards lower indices,
// +1: higher), then every warp applies the eight from the farthest to the nearest.
// A map with A = 0 is where the walk starts; while none of the eight is one, the
// eight are read again (with few channels a tile has hundreds of others before it that
// are still unresolved, and a walk over all of them costs more than waiting for the
// nearest).  Tiles from `tiles` on hold no sequence and publish nothing.  All warps call it together.  When
// a wait runs out, here or elsewhere, the status word says so and the result is 0.
template <int VEC>
__device__ Vec<VEC> look_back(const TileSpace& w, int i, int step, int64_t tiles, int64_t ch,
                              int warp, int lane, Record<VEC> (*records)[32]) {
    const int64_t idx = i + (int64_t)step * (warp + 1);
    const bool there = idx >= 0 && idx < tiles;
    const uint64_t* p = w.record + (there ? idx * w.Dp + ch : 0);
    uint64_t t0 = 0;
    for (uint32_t round = 0;; ++round) {
        Record<VEC> r;
        r.set(fill<VEC>(0.f), fill<VEC>(0.f));
        bool stop = (round & 63) == 63 && expired(w, t0);
        if (there) {
            r.read(p);
            for (uint32_t spin = 1; !stop && !r.ready(); ++spin) {
                stop = (spin & 63) == 0 && expired(w, t0);
                r.read(p);
            }
        }
        __syncwarp();
        records[warp][lane] = r;
        if (__syncthreads_or(stop)) return fill<VEC>(0.f);
        bool open = false;   // a channel whose walk has no start among the eight
        Vec<VEC> H = fill<VEC>(0.f);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            bool met = false;
#pragma unroll
            for (int j = kWarps - 1; j >= 0; --j) {
                const Record<VEC>& q = records[j][lane];
                const bool last = q.A(v) == 0.f;
                met |= last;
                H.v[v] = last ? q.B(v) : fmaf(q.A(v), H.v[v], q.B(v));
            }
            open |= !met;
        }
        if (!__any_sync(0xffffffffu, open)) return H;   // the same answer in every warp
        __syncthreads();   // all have read the records
    }
}

// Warp maps of a tile.
template <int VEC>
struct Maps {
    Vec<VEC> A[kWarps][32];
    Vec<VEC> B[kWarps][32];
    uint32_t reset[kWarps];   // the warp's rows hold a boundary: B alone counts

    __device__ __forceinline__ void put(int warp, int lane, const Vec<VEC>& a, const Vec<VEC>& b,
                                        uint32_t boundary) {
        A[warp][lane] = a;
        B[warp][lane] = b;
        if (lane == 0) reset[warp] = boundary;
    }
    // The state after warp j's rows from the state before them.
    __device__ __forceinline__ Vec<VEC> step(int j, int lane, const Vec<VEC>& h) const {
        const Vec<VEC> b = B[j][lane];
        return reset[j] ? b : fma(A[j][lane], h, b);
    }
};

// Tickets count from the filled workspace's 2^32 - 1.
__device__ __forceinline__ uint32_t take_ticket(const TileSpace& w) {
    return atomicAdd(w.ticket, 1u) + 1u;
}
// The first tile of a CTA, broadcast: with several tiles along time by ticket.
__device__ __forceinline__ int64_t first_tile(const TileSpace& w, uint32_t* shared) {
    if (w.nt == 1) return blockIdx.x;
    if (threadIdx.x == 0) *shared = take_ticket(w);
    __syncthreads();
    return *shared;
}

// The value that replaces the carried one at a boundary row (S0 at a first token, dS_T
// at a last one), and the store of a state there.  Calls, not inlined: they stand in
// loops unrolled over the rows, whose code would otherwise outgrow the instruction
// cache (with 128-token sequences a fifth of the time went to instruction fetches).
template <int VEC>
__device__ __noinline__ Vec<VEC> boundary_value(const float* src, int n, int r, int64_t D, int ch) {
    const int64_t seq = __shfl_sync(0xffffffffu, n, r);
    return src && ch < D ? load_f32<VEC>(src + seq * D + ch) : fill<VEC>(0.f);
}
// That of the first boundary among a warp's rows, loaded along with the tile.
template <int VEC>
__device__ __forceinline__ Vec<VEC> first_boundary(const float* src, uint32_t mask, int n,
                                                   int64_t D, int ch) {
    const int64_t seq = __shfl_sync(0xffffffffu, n, mask ? __ffs(mask) - 1 : 0);
    return mask && src && ch < D ? load_f32<VEC>(src + seq * D + ch) : fill<VEC>(0.f);
}
template <int VEC>
__device__ __noinline__ void boundary_store(float* dst, int n, int r, int64_t D, int ch,
                                            Vec<VEC> h) {
    const int64_t seq = __shfl_sync(0xffffffffu, n, r);
    if (dst && ch < D) store(dst + seq * D + ch, h);
}

// Rows of x in shared memory; of the complement the inputs u, in fp32.
template <typename T, bool COMP, int VEC>
struct FwdRows {
    static constexpr int R = kFwdRows;
    static constexpr int kBytes = R * 32 * VEC * (COMP ? 4 : (int)sizeof(T));
    // the copies land in the upper half of a row area twice as large
    static constexpr int kAt = COMP ? kBytes - R * 32 * VEC * (int)sizeof(T) : 0;
};

// CTAs an SM: gates of one value a row leave registers, and bf16 rows shared memory, for
// three (8 x 4096 tokens of 4096 channels: 142 us, with two 151).
template <typename T, int GATE, bool COMP>
constexpr int kFwdCtas = GATE == KDA_GATE_HEAD_F32 && sizeof(T) == 2 && !COMP ? 3 : 2;

template <typename T, int GATE, bool COMP, int VEC>
__global__ void __launch_bounds__(kThreads, (kFwdCtas<T, GATE, COMP>))
linrec_fwd_kernel(const LinrecArgs p, const TileSpace w) {
    constexpr int R = kFwdRows, kTile = kWarps * R;
    using Area = FwdRows<T, COMP, VEC>;
    using U = std::conditional_t<COMP, float, T>;
    extern __shared__ __align__(16) char row_area[];
    __shared__ Offsets off;
    __shared__ Maps<VEC> maps;
    __shared__ Record<VEC> records[kWarps][32];
    __shared__ uint32_t next_ticket;
    const int lane = threadIdx.x & 31;
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);   // uniform
    const int N = p.num_seqs;
    const int64_t D = (int64_t)p.H * p.d;
    const int32_t* cu = p.cu_seqlens;
    U* u = reinterpret_cast<U*>(row_area + warp * Area::kBytes);
    T* x = reinterpret_cast<T*>(row_area + warp * Area::kBytes + Area::kAt);

    const int64_t tiles = (int64_t)w.nt * w.ct;
    const bool valid = read_offsets(off, cu, N, p.total_tokens, w.status);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (valid) clear_status(w, N);
        else *w.status = KDA_ERR_DEVICE_INPUT;
    }
    if (!valid) return;
    int64_t tile = first_tile(w, &next_ticket);
    const int64_t end = cu[N], live_tiles = (end + kTile - 1) / kTile;
    copy_empty(cu, N, D, p.S0, p.S_T);

    while (tile < tiles) {
        const int i = (int)((uint32_t)tile / (uint32_t)w.ct);
        const int64_t t0 = (int64_t)i * kTile + warp * R;
        const int c0 = (int)((uint32_t)tile % (uint32_t)w.ct) * 32 * VEC;
        const int ch = c0 + lane * VEC;   // this lane's channels
        const bool on = ch < D;
        const int left = t0 < end ? (int)min(end - t0, (int64_t)R) : 0;
        const bool full = left == R && c0 + 32 * VEC <= D;

        stage_rows<R, T, VEC>(x, p.x, t0 * D + c0, D, full && D % 8 == 0, left, on, lane);
        // all of the CTA's warps take the plain path or the one with boundaries together:
        // each is unrolled, and the instruction cache holds one of them
        const bool edge = c0 + 32 * VEC > D ||
                          !inner_tile(off, cu, N, (int64_t)i * kTile, kTile, end);
        Rows rows = {};
        if (edge) rows = rows_of<R>(off, cu, N, t0, end, lane);
        const Vec<VEC> start0 = first_boundary<VEC>(p.S0, rows.start, rows.n, D, ch);
        Gate<GATE, VEC> a[R];
        take_gate<R, GATE, VEC>(a, p, t0, D, c0, full, left, on, lane);
        expand_gate<R, GATE, VEC>(a);
        copies_done();
        if constexpr (COMP) complement_rows<R, T, GATE, VEC>(u, x, a, lane);
        auto input = [&](int r) { return staged<U, VEC>(u, r, lane); };
        // Rows with at most one first and one last token take loops without branches: with
        // one at each row the shared-memory reads would wait for one another, and the tiles
        // behind a boundary with them (8 sequences of 4096 tokens: 202 us instead of 188).
        const int at_start = __ffs(rows.start) - 1, at_last = __ffs(rows.last) - 1;
        const bool one = __popc(rows.start) <= 1 && __popc(rows.last) <= 1;
        // the state that replaces the carried one at a sequence's first token
        auto start = [&](int r) {
            return r == at_start ? start0 : boundary_value<VEC>(p.S0, rows.n, r, D, ch);
        };

        Vec<VEC> A = fill<VEC>(1.f), B = fill<VEC>(0.f);
        if (!edge) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                B = fma(a[r].a(), B, input(r));
                A = mul(A, a[r].a());
            }
        } else if (one) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                B = fma(a[r].a(), choose(r == at_start, start0, B), input(r));
                A = mul(A, a[r].a());
            }
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (rows.start >> r & 1) B = start(r);
                B = fma(a[r].a(), B, input(r));
                A = mul(A, a[r].a());
            }
        }
        maps.put(warp, lane, A, B, rows.start);
        __syncthreads();

        // a state enters the tile, unless its first row starts a sequence; the first
        // warp hands the tile's map on, and later the state that leaves it
        const int64_t first = (int64_t)i * kTile;
        const bool needed = first < end && !(maps.reset[0] & 1);
        const bool wanted = w.nt > 1 && first + kTile < end;
        bool reset = false;
        if (warp == 0 && wanted) {
            A = fill<VEC>(1.f);
            B = fill<VEC>(0.f);
#pragma unroll
            for (int j = 0; j < kWarps; ++j) {
                reset |= maps.reset[j] != 0;
                B = maps.step(j, lane, B);
                A = mul(A, maps.A[j][lane]);
            }
            A = reset ? fill<VEC>(0.f) : finite(A);
            publish<VEC>(w, i, ch, A, B);
        }
        Vec<VEC> h = fill<VEC>(0.f);
        if (needed) {
            h = look_back<VEC>(w, i, -1, live_tiles, ch, warp, lane, records);
            if (warp == 0 && wanted && !reset) {
#pragma unroll
                for (int v = 0; v < VEC; ++v)
                    if (A.v[v] != 0.f) B.v[v] = fmaf(A.v[v], h.v[v], B.v[v]);
                publish<VEC>(w, i, ch, fill<VEC>(0.f), B);
            }
        }
        // The next tile is claimed only now: a tile claimed before the look-back would
        // not be started while this CTA waits, and its successors would wait for both
        // (that made the long prefill twice as slow).
        if (threadIdx.x == 0 && w.nt > 1) next_ticket = take_ticket(w);

        for (int j = 0; j < warp; ++j) h = maps.step(j, lane, h);
        if (p.states && on && t0 % LINREC_CHUNK == 0 && t0 < p.total_tokens)
            store(p.states + t0 / LINREC_CHUNK * D + ch,
                  t0 < end && !(rows.start & 1) ? h : fill<VEC>(0.f));
        T* y = p.y ? static_cast<T*>(p.y) + (t0 * D + c0) : nullptr;
        if (!edge) {
            if (y) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    h = fma(a[r].a(), h, input(r));
                    store(y + r * D + lane * VEC, h);
                }
            }
        } else if (const int stored = on && y ? left : 0; one) {
            Vec<VEC> end_state = fill<VEC>(0.f);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                h = fma(a[r].a(), choose(r == at_start, start0, h), input(r));
                if (r < stored) store(y + r * D + lane * VEC, h);
                end_state = choose(r == at_last, h, end_state);
            }
            if (at_last >= 0) boundary_store<VEC>(p.S_T, rows.n, at_last, D, ch, end_state);
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (rows.start >> r & 1) h = start(r);
                h = fma(a[r].a(), h, input(r));
                if (r < stored) store(y + r * D + lane * VEC, h);
                if (rows.last >> r & 1) boundary_store<VEC>(p.S_T, rows.n, r, D, ch, h);
            }
        }
        __syncthreads();   // maps, records and the ticket: this tile is done with them
        tile = w.nt > 1 ? (int64_t)next_ticket : tile + gridDim.x;
    }
}

// Where a head's gate gradient, a sum over its channels, goes.
//   kHeadRow: lanes of a warp that share a head are summed by shuffles; a head
//     of at most 64 channels is done, a wider one leaves d / 64 partial sums
//   kHeadWide: every channel's term goes to a buffer, summed afterwards (widths
//     that neither divide 64 nor are a multiple of it)
enum : int { kNoHead = 0, kHeadRow = 1, kHeadWide = 2 };
constexpr int kFewParts = 8;   // summed by one thread

// Per warp: rows of x and dy as stored, and of f in fp32 (see below).
template <typename T, int VEC>
struct BwdRows {
    static constexpr int R = kBwdRows;
    static constexpr int kRaw = R * 32 * VEC * (int)sizeof(T), kF = R * 32 * VEC * 4;
    static constexpr int kBytes = 2 * kRaw + kF;
    };

template <typename T, int GATE, bool COMP, int VEC>
__global__ void __launch_bounds__(kThreads, 2)
linrec_bwd_kernel(const LinrecArgs p, const TileSpace w, const float* __restrict__ states,
                  float* dgate, int head_mode) {
    constexpr int R = kBwdRows;
    using Area = BwdRows<T, VEC>;
    extern __shared__ __align__(16) char row_area[];
    __shared__ Offsets off;
    __shared__ Maps<VEC> maps;    // of the state, tokens forward
    __shared__ Maps<VEC> rmaps;   // of the gradient, tokens backward
    __shared__ Record<VEC> records[kWarps][32];
    __shared__ uint32_t next_ticket;
    const int lane = threadIdx.x & 31;
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);   // uniform
    const int N = p.num_seqs;
    const int64_t D = (int64_t)p.H * p.d;
    const int32_t* cu = p.cu_seqlens;
    T* x = reinterpret_cast<T*>(row_area + warp * Area::kBytes);
    T* dy = reinterpret_cast<T*>(row_area + warp * Area::kBytes + Area::kRaw);
    float* f = reinterpret_cast<float*>(row_area + warp * Area::kBytes + 2 * Area::kRaw);

    const int64_t tiles = (int64_t)w.nt * w.ct;
    const bool valid = read_offsets(off, cu, N, p.total_tokens, w.status);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (valid) clear_status(w, N);
        else *w.status = KDA_ERR_DEVICE_INPUT;
    }
    if (!valid) return;
    int64_t tile = first_tile(w, &next_ticket);
    const int64_t end = cu[N], live_tiles = (end + LINREC_CHUNK - 1) / LINREC_CHUNK;
    copy_empty(cu, N, D, p.dS_T, p.dS0);

    while (tile < tiles) {
        const int i = w.nt - 1 - (int)((uint32_t)tile / (uint32_t)w.ct);
        const int64_t t0 = (int64_t)i * LINREC_CHUNK + warp * R;
        const int c0 = (int)((uint32_t)tile % (uint32_t)w.ct) * 32 * VEC;
        const int ch = c0 + lane * VEC;
        const bool on = ch < D;
        const int left = t0 < end ? (int)min(end - t0, (int64_t)R) : 0;
        const bool full = left == R && c0 + 32 * VEC <= D;

        stage_rows<R, T, VEC>(x, p.x, t0 * D + c0, D, full && D % 8 == 0, left, on, lane);
        stage_rows<R, T, VEC>(dy, p.dy, t0 * D + c0, D, full && D % 8 == 0, left, on, lane);
        const bool edge = c0 + 32 * VEC > D ||   // as in the forward kernel
                          !inner_tile(off, cu, N, (int64_t)i * LINREC_CHUNK, LINREC_CHUNK, end);
        Rows rows = {};
        if (edge) rows = rows_of<R>(off, cu, N, t0, end, lane);
        const Vec<VEC> start0 = first_boundary<VEC>(p.S0, rows.start, rows.n, D, ch);
        const Vec<VEC> last0 = first_boundary<VEC>(p.dS_T, rows.last, rows.n, D, ch);
        Vec<VEC> H = fill<VEC>(0.f);   // the state that enters the tile
        if (on && (int64_t)i * LINREC_CHUNK < end) H = load_f32<VEC>(states + i * D + ch);
        Gate<GATE, VEC> a[R];
        take_gate<R, GATE, VEC>(a, p, t0, D, c0, full, left, on, lane);
        expand_gate<R, GATE, VEC>(a);
        copies_done();
        auto input = [&](int r) {
            const Vec<VEC> q = staged<T, VEC>(x, r, lane);
            if constexpr (COMP) return mul(a[r].na(), q);
            else return q;
        };
        const int at_start = __ffs(rows.start) - 1, at_last = __ffs(rows.last) - 1;
        const bool one = __popc(rows.start) <= 1 && __popc(rows.last) <= 1;   // as there
        auto start = [&](int r) {
            return r == at_start ? start0 : boundary_value<VEC>(p.S0, rows.n, r, D, ch);
        };
        auto behind = [&](int r) {
            return r == at_last ? last0 : boundary_value<VEC>(p.dS_T, rows.n, r, D, ch);
        };

        // maps of the warp's rows, both ways
        Vec<VEC> A = fill<VEC>(1.f), B = fill<VEC>(0.f), RB = fill<VEC>(0.f), RA = fill<VEC>(1.f);
        if (!edge) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                B = fma(a[r].a(), B, input(r));
                A = mul(A, a[r].a());
            }
#pragma unroll
            for (int r = R - 1; r >= 0; --r)
                RB = mul(a[r].a(), add(staged<T, VEC>(dy, r, lane), RB));
            RA = A;
        } else if (one) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                B = fma(a[r].a(), choose(r == at_start, start0, B), input(r));
                A = mul(A, a[r].a());
            }
#pragma unroll
            for (int r = R - 1; r >= 0; --r) {
                RB = choose(r == at_last, last0, RB);
                // rows past the end hand on nothing
                RB = choose(r < left, mul(a[r].a(), add(staged<T, VEC>(dy, r, lane), RB)), RB);
                RA = choose(r < left, mul(RA, a[r].a()), RA);
            }
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (rows.start >> r & 1) B = start(r);
                B = fma(a[r].a(), B, input(r));
                A = mul(A, a[r].a());
            }
#pragma unroll
            for (int r = R - 1; r >= 0; --r) {
                if (rows.last >> r & 1) RB = behind(r);
                if (r < left) {   // rows past the end hand on nothing
                    RB = mul(a[r].a(), add(staged<T, VEC>(dy, r, lane), RB));
                    RA = mul(RA, a[r].a());
                }
            }
        }
        maps.put(warp, lane, A, B, rows.start);
        rmaps.put(warp, lane, RA, RB, rows.last);
        __syncthreads();

        // a gradient enters the tile from behind, unless its last row ends a sequence
        // (or lies past the last one); the last warp hands the tile's map on
        const int64_t first = (int64_t)i * LINREC_CHUNK;
        const bool needed = first + LINREC_CHUNK < end &&
                            !(rmaps.reset[kWarps - 1] >> (R - 1) & 1);
        const bool wanted = i > 0 && first < end;
        bool reset = false;
        if (warp == kWarps - 1 && wanted) {
            A = fill<VEC>(1.f);
            B = fill<VEC>(0.f);
#pragma unroll
            for (int j = kWarps - 1; j >= 0; --j) {
                reset |= rmaps.reset[j] != 0;
                B = rmaps.step(j, lane, B);
                A = mul(A, rmaps.A[j][lane]);
            }
            A = reset ? fill<VEC>(0.f) : finite(A);
            publish<VEC>(w, i, ch, A, B);
        }
        // what the gate multiplies at each row, before the wait: the state before the
        // row, less x for the complement
        for (int j = 0; j < warp; ++j) H = maps.step(j, lane, H);
        auto put_f = [&](int r) {
            Vec<VEC> q = H;
            if constexpr (COMP) {
                const Vec<VEC> xr = staged<T, VEC>(x, r, lane);
#pragma unroll
                for (int v = 0; v < VEC; ++v) q.v[v] = H.v[v] - xr.v[v];
            }
            store(f + r * 32 * VEC + lane * VEC, q);
            H = fma(a[r].a(), H, input(r));
        };
        if (!edge) {
#pragma unroll
            for (int r = 0; r < R; ++r) put_f(r);
        } else if (one) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                H = choose(r == at_start, start0, H);
                put_f(r);
            }
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (rows.start >> r & 1) H = start(r);
                put_f(r);
            }
        }
        Vec<VEC> G = fill<VEC>(0.f);   // the gradient that comes from behind
        if (needed) {
            G = look_back<VEC>(w, i, +1, live_tiles, ch, warp, lane, records);
            if (warp == kWarps - 1 && wanted && !reset) {
#pragma unroll
                for (int v = 0; v < VEC; ++v)
                    if (A.v[v] != 0.f) B.v[v] = fmaf(A.v[v], G.v[v], B.v[v]);
                publish<VEC>(w, i, ch, fill<VEC>(0.f), B);
            }
        }
        if (threadIdx.x == 0 && w.nt > 1) next_ticket = take_ticket(w);   // as in the forward kernel

        for (int j = kWarps - 1; j > warp; --j) G = rmaps.step(j, lane, G);
        float* dx = p.dx + (t0 * D + c0);
        float* dg = dgate + (t0 * D + c0);
        const bool sum_lanes = GATE == KDA_GATE_HEAD_F32 && head_mode == kHeadRow;
        // row r's gradients
        auto row = [&](int r, bool out) {
            const Vec<VEC> g = add(staged<T, VEC>(dy, r, lane), G);
            if constexpr (COMP) {
                if (out) store(dx + r * D + lane * VEC, mul(a[r].na(), g));
            } else {
                if (out) store(dx + r * D + lane * VEC, g);
            }
            Vec<VEC> da = mul(g, staged<float, VEC>(f, r, lane));
            G = mul(a[r].a(), g);
            if constexpr (GATE == KDA_GATE_CHANNEL_LOG_BF16) da = mul(a[r].a(), da);
            if (sum_lanes) store(f + r * 32 * VEC + lane * VEC, da);
            else if (out) store(dg + r * D + lane * VEC, da);
        };
        if (!edge) {
#pragma unroll
            for (int r = R - 1; r >= 0; --r) row(r, true);
        } else if (one) {
            Vec<VEC> first_gradient = fill<VEC>(0.f);
#pragma unroll
            for (int r = R - 1; r >= 0; --r) {
                G = choose(r == at_last, last0, G);
                const Vec<VEC> before = G;
                row(r, on && r < left);
                G = choose(r < left, G, before);
                first_gradient = choose(r == at_start, G, first_gradient);
            }
            if (at_start >= 0) boundary_store<VEC>(p.dS0, rows.n, at_start, D, ch, first_gradient);
        } else {
#pragma unroll
            for (int r = R - 1; r >= 0; --r) {
                if (rows.last >> r & 1) G = behind(r);
                if (r < left) row(r, on);
                if (rows.start >> r & 1) boundary_store<VEC>(p.dS0, rows.n, r, D, ch, G);
            }
        }
        if (sum_lanes) {
            // lanes that share a head (or one of its 64-channel parts) add up; [T][H][parts]:
            // the part's index is the channel over its width
            const int part = p.d < 32 * VEC ? p.d : 32 * VEC, width = part / VEC;
            const int64_t out = t0 * (D / part) + ch / part;
            float s[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const Vec<VEC> da = staged<float, VEC>(f, r, lane);
                s[r] = on && r < left ? da.v[0] + (VEC == 2 ? da.v[VEC - 1] : 0.f) : 0.f;
            }
            if (width == 32 && R == 16) {
                // all lanes: each exchange halves the rows a lane carries, so that lanes 2 r
                // and 2 r + 1 end with row r
#pragma unroll
                for (int o = 16, n = R / 2; o > 1; o >>= 1, n >>= 1) {
                    const bool upper = lane & o;
#pragma unroll
                    for (int r = 0; r < n; ++r) {
                        const float give = upper ? s[r] : s[r + n];
                        s[r] = (upper ? s[r + n] : s[r]) + __shfl_xor_sync(0xffffffffu, give, o);
                    }
                }
                s[0] += __shfl_xor_sync(0xffffffffu, s[0], 1);
                if ((lane & 1) == 0 && lane / 2 < left) dgate[out + lane / 2 * (D / part)] = s[0];
            } else {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    if (o < width) {
#pragma unroll
                        for (int r = 0; r < R; ++r) s[r] += __shfl_xor_sync(0xffffffffu, s[r], o);
                    }
                }
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (on && r < left && (lane & (width - 1)) == 0) dgate[out + r * (D / part)] = s[r];
            }
        }
        __syncthreads();
        tile = w.nt > 1 ? (int64_t)next_ticket : tile + gridDim.x;
    }
}

// dgate[t][h] = the sum of the head's `parts` terms: a thread each for few terms, in order,
// a warp each for many.
__global__ void __launch_bounds__(kThreads)
linrec_head_sum_kernel(const float* __restrict__ part, const int32_t* cu, int32_t N, int32_t H,
                       int32_t parts, float* __restrict__ dgate, const int32_t* status) {
    if (N == 0 || *status == KDA_ERR_DEVICE_INPUT) return;
    const int64_t rows = (int64_t)cu[N] * H;
    if (parts <= kFewParts) {
        for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < rows;
             i += (int64_t)gridDim.x * kThreads) {
            float s = 0.f;
            for (int j = 0; j < parts; ++j) s += part[i * parts + j];
            dgate[i] = s;
        }
        return;
    }
    const int lane = threadIdx.x & 31;
    for (int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); i < rows;
         i += (int64_t)gridDim.x * kWarps) {
        float s = 0.f;
        for (int j = lane; j < parts; j += 32) s += part[i * parts + j];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) dgate[i] = s;
    }
}

// Fills the workspace with 0xff bytes, but for the status word when `keep`.
__global__ void __launch_bounds__(kThreads)
linrec_fill_kernel(char* ws, size_t bytes, bool keep) {
    asm volatile("griddepcontrol.launch_dependents;");
    const uint4 ones = make_uint4(~0u, ~0u, ~0u, ~0u);
    for (size_t i = blockIdx.x * (size_t)kThreads + threadIdx.x; i < bytes / 16;
         i += (size_t)gridDim.x * kThreads) {
        if (i == 0 && keep) {
            uint32_t* w = reinterpret_cast<uint32_t*>(ws);
            w[1] = w[2] = w[3] = ~0u;
        } else {
            reinterpret_cast<uint4*>(ws)[i] = ones;
        }
    }
}

// Offsets of more sequences than a CTA checks by itself.
__global__ void linrec_check_kernel(const int32_t* cu, int32_t N, int64_t T, int32_t* status) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i > N) return;
    const int32_t c = cu[i];
    if ((i == 0 ? c != 0 : c < cu[i - 1]) || (i == N && (int64_t)c > T))
        *status = KDA_ERR_DEVICE_INPUT;
}

// A batch of one sequence of kCheckTiles tiles and one channel, in a workspace whose ticket
// stands behind the first tile: nobody takes that, so the others' waits for its record run
// out.  Behind the layout's end: x, gate, y [T], S_T, cu_seqlens.
constexpr int kCheckTiles = 3, kCheckTokens = kCheckTiles * kWarps * kFwdRows;
__global__ void __launch_bounds__(kThreads)
linrec_check_case_kernel(char* ws, size_t end) {
    for (size_t i = threadIdx.x; i < end / 4; i += kThreads)
        reinterpret_cast<uint32_t*>(ws)[i] = i == 1 ? 0u : ~0u;
    float* x = reinterpret_cast<float*>(ws + end);
    for (int i = threadIdx.x; i < 3 * kCheckTokens + 4; i += kThreads) x[i] = 0.5f;
    int32_t* cu = reinterpret_cast<int32_t*>(x + 3 * kCheckTokens + 4);
    if (threadIdx.x < 2) cu[threadIdx.x] = threadIdx.x * kCheckTokens;
}

// One token a row: W neighbouring channels a thread, four where the head width allows
// (16-byte accesses of the state and the fp32 gate), else one.  A streaming pass, bound by
// HBM and, at a few megabytes, by its launch.
template <typename T, int GATE, int W>
__global__ void __launch_bounds__(kThreads) linrec_step_kernel(const LinrecStepArgs p, int blocks) {
    const int D = p.H * p.d;
    const int b = blockIdx.x / blocks;
    const int c = ((blockIdx.x - b * blocks) * kThreads + threadIdx.x) * W;
    if (c >= D) return;
    const int row = p.parents ? p.parents[b] : b;
    const int64_t at = (int64_t)b * D + c;
    const bool live = row >= 0 && row < p.num_rows;
    const float* S = p.S + (live ? (int64_t)row * D + c : 0);
    float h[W], a[W], na[W], x[W];
    if constexpr (W == 4) {
        const float4 s = live ? __ldcs(reinterpret_cast<const float4*>(S))
                              : make_float4(0.f, 0.f, 0.f, 0.f);
        h[0] = s.x; h[1] = s.y; h[2] = s.z; h[3] = s.w;
    } else {
        h[0] = live ? *S : 0.f;
    }
    auto load = [&](const auto* q, float (&out)[W]) {
        using E = std::remove_cv_t<std::remove_pointer_t<decltype(q)>>;
        if constexpr (W == 1) {
            out[0] = Elem<E>::load(q);
        } else if constexpr (sizeof(E) == 4) {
            const float4 u = __ldcs(reinterpret_cast<const float4*>(q));
            out[0] = u.x; out[1] = u.y; out[2] = u.z; out[3] = u.w;
        } else {
            const uint2 u = __ldcs(reinterpret_cast<const uint2*>(q));
            out[0] = __uint_as_float(u.x << 16); out[1] = __uint_as_float(u.x & 0xffff0000u);
            out[2] = __uint_as_float(u.y << 16); out[3] = __uint_as_float(u.y & 0xffff0000u);
        }
    };
    load(static_cast<const T*>(p.x) + at, x);
    if (GATE == KDA_GATE_CHANNEL_LOG_BF16) {
        load(static_cast<const __nv_bfloat16*>(p.gate) + at, a);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            na[i] = -expm1f(a[i]);
            a[i] = gate_exp(a[i]);
        }
    } else {
        if (GATE == KDA_GATE_HEAD_F32) {
#pragma unroll
            for (int i = 0; i < W; ++i) a[i] = static_cast<const float*>(p.gate)[b * (int64_t)p.H + c / p.d];
        } else {
            load(static_cast<const float*>(p.gate) + at, a);
        }
#pragma unroll
        for (int i = 0; i < W; ++i) na[i] = 1.f - a[i];
    }
#pragma unroll
    for (int i = 0; i < W; ++i) h[i] = fmaf(a[i], h[i], p.complement ? na[i] * x[i] : x[i]);
    T* y = static_cast<T*>(p.y) + at;
    if constexpr (W == 4) {
        *reinterpret_cast<float4*>(p.S_out + at) = make_float4(h[0], h[1], h[2], h[3]);
        store(y, Vec<2>{h[0], h[1]});
        store(y + 2, Vec<2>{h[2], h[3]});
    } else {
        p.S_out[at] = h[0];
        Elem<T>::store(y, h[0]);
    }
}

template <typename F>
cudaError_t by_type(kda_dtype dtype, int gate, F&& f) {
    auto pick = [&](auto* t) {
        switch (gate) {
            case KDA_GATE_HEAD_F32: return f(t, std::integral_constant<int, KDA_GATE_HEAD_F32>());
            case KDA_GATE_CHANNEL_LOG_BF16:
                return f(t, std::integral_constant<int, KDA_GATE_CHANNEL_LOG_BF16>());
            default: return f(t, std::integral_constant<int, KDA_GATE_CHANNEL_F32>());
        }
    };
    return dtype == KDA_BF16 ? pick((__nv_bfloat16*)nullptr) : pick((float*)nullptr);
}

size_t pad(size_t b) { return (b + 255) & ~(size_t)255; }

// Two channels a lane need rows on a 4-byte (bf16) grid, an even row width, and with a
// head gate heads of an even width.
int lane_channels(int64_t D) { return D % 2 == 0 ? 2 : 1; }
int lane_channels(int64_t D, int32_t d, int gate_format) {
    return gate_format == KDA_GATE_HEAD_F32 && d % 2 != 0 ? 1 : lane_channels(D);
}

struct TileLayout {
    int64_t nt, ct, Dp;
    size_t end;
};
// rows: tokens a warp; lanes: channels a lane (the wider tiles need the larger workspace).
TileLayout tile_layout(int64_t T, int64_t D, int rows, int lanes) {
    TileLayout L;
    const int64_t tile = kWarps * rows;
    const int64_t width = 32 * lanes;
    L.nt = T > 0 ? (T + tile - 1) / tile : 1;
    L.ct = (D + width - 1) / width;
    L.Dp = L.ct * width;
    L.end = kRecords + (L.nt > 1 ? pad((size_t)L.nt * L.Dp * sizeof(uint64_t)) : 0);
    return L;
}

// Whether the tiles need a workspace filled beforehand.
bool filled(const LinrecArgs& a, const TileLayout& L) { return L.nt > 1 || a.num_seqs > kSelfCheck; }

void set_space(TileSpace& w, const TileLayout& L, char* ws) {
    w.status = reinterpret_cast<int32_t*>(ws);
    w.ticket = reinterpret_cast<uint32_t*>(ws + 4);
    w.record = reinterpret_cast<uint64_t*>(ws + kRecords);
    w.nt = (int32_t)L.nt;
    w.ct = (int32_t)L.ct;
    w.Dp = L.Dp;
    w.wait_ns = kWaitNs;
}

// Fills the workspace (keeping the status word of an earlier pass) and checks the
// offsets of large batches.
cudaError_t start_tiles(const LinrecArgs& a, const TileLayout& L, char* ws, bool keep_status,
                        TileSpace& w, cudaStream_t stream) {
    set_space(w, L, ws);
    if (filled(a, L)) {
        const size_t blocks = (L.end / 16 + kThreads - 1) / kThreads;
        const size_t most = 4 * (size_t)(sm_count() > 0 ? sm_count() : 1);
        linrec_fill_kernel<<<(unsigned)(blocks < most ? blocks : most), kThreads, 0, stream>>>(
            ws, L.end, keep_status);
        const cudaError_t err = cudaGetLastError();
        if (err != cudaSuccess) return err;
    }
    if (a.num_seqs > kSelfCheck && !keep_status) {
        linrec_check_kernel<<<a.num_seqs / kThreads + 1, kThreads, 0, stream>>>(
            a.cu_seqlens, a.num_seqs, a.total_tokens, w.status);
        return cudaGetLastError();
    }
    return cudaSuccess;
}

// f(T, gate, complement, channels a lane) with its arguments as types.
template <int N>
using Int = std::integral_constant<int, N>;
template <typename F>
cudaError_t by_tile(const LinrecArgs& a, F&& f) {
    return by_type(a.dtype, a.gate_format, [&](auto* t, auto g) {
        auto pick = [&](auto comp) {
            return lane_channels((int64_t)a.H * a.d, a.d, a.gate_format) == 2
                       ? f(t, g, comp, Int<2>())
                       : f(t, g, comp, Int<1>());
        };
        return a.complement ? pick(std::true_type()) : pick(std::false_type());
    });
}

// After a fill the kernel starts while that still runs: it reads its offsets meanwhile
// and waits before its first ticket (3 us less a call than after a memset).
template <typename K>
cudaError_t configure_tiles(K kernel, const TileLayout& L, int ctas, bool early, int smem,
                            cudaStream_t stream, cudaLaunchConfig_t& c,
                            cudaLaunchAttribute& attr) {
    if (smem > 32 * 1024) {   // above what every kernel may have with its static part
        const cudaError_t err =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (err != cudaSuccess) return err;
    }
    const int64_t tiles = L.nt * L.ct, most = ctas * (int64_t)sm_count();
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    c.gridDim = dim3((unsigned)(tiles < most ? tiles : most > 0 ? most : 1));
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    c.attrs = &attr;
    c.numAttrs = early ? 1 : 0;
    return cudaSuccess;
}

cudaError_t run_forward(const LinrecArgs& a, char* ws, cudaStream_t stream) {
    const TileLayout L = tile_layout(a.total_tokens, (int64_t)a.H * a.d, kFwdRows,
                                     lane_channels((int64_t)a.H * a.d, a.d, a.gate_format));
    TileSpace w;
    cudaError_t err = start_tiles(a, L, ws, false, w, stream);
    if (err != cudaSuccess) return err;
    return by_tile(a, [&](auto* t, auto g, auto comp, auto vec) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int V = decltype(vec)::value;
        constexpr bool C = decltype(comp)::value;
        auto kernel = linrec_fwd_kernel<T, decltype(g)::value, C, V>;
        cudaLaunchConfig_t c = {};
        cudaLaunchAttribute attr;
        const cudaError_t set =
            configure_tiles(kernel, L, kFwdCtas<T, decltype(g)::value, C>, filled(a, L),
                            kWarps * FwdRows<T, C, V>::kBytes, stream, c, attr);
        return set == cudaSuccess ? cudaLaunchKernelEx(&c, kernel, a, w) : set;
    });
}

int head_mode(int32_t d, int gate_format, int64_t D) {
    if (gate_format != KDA_GATE_HEAD_F32) return kNoHead;
    const int lanes = lane_channels(D, d, gate_format);
    const int width = 32 * lanes;
    if (d >= lanes && (d % width == 0 || width % d == 0)) return kHeadRow;
    return kHeadWide;
}
// Partial sums a head's gate gradient is left in (1: none are).
int32_t head_parts(int32_t d, int gate_format, int64_t D) {
    switch (head_mode(d, gate_format, D)) {
        case kHeadRow: {
            const int32_t width = 32 * lane_channels(D, d, gate_format);
            return d > width ? d / width : 1;
        }
        case kHeadWide: return d;
        default: return 1;
    }
}

}  // namespace

size_t linrec_prefill_bytes(int32_t num_seqs, int64_t total_tokens, int64_t D) {
    return tile_layout(total_tokens, D, kFwdRows, lane_channels(D)).end +
           pad((size_t)num_seqs * D * sizeof(float));
}

// Workspace of the backward pass: the tiles, the states when the caller has
// none, and the partial sums of head gates.
size_t linrec_backward_bytes(int32_t, int64_t total_tokens, int32_t H, int32_t d,
                             int gate_format, bool with_states) {
    const int64_t D = (int64_t)H * d;
    // (the forward scan's tiles need less room than the backward one's)
    const TileLayout L = tile_layout(total_tokens, D, kBwdRows, lane_channels(D));
    size_t b = L.end;
    if (!with_states && total_tokens > 0) b += pad((size_t)L.nt * D * sizeof(float));
    const int32_t parts = head_parts(d, gate_format, D);
    if (parts > 1) b += pad((size_t)total_tokens * H * parts * sizeof(float));
    return b;
}

cudaError_t launch_linrec_prefill(const LinrecArgs& a, char* ws, cudaStream_t stream) {
    if (!a.S0 || a.S0 != a.S_T) return run_forward(a, ws, stream);
    // in place: the kernel reads S0 twice, the second time when another warp may
    // have written S_T, so it reads a copy
    const int64_t D = (int64_t)a.H * a.d;
    LinrecArgs b = a;
    float* copy = reinterpret_cast<float*>(
        ws + tile_layout(a.total_tokens, D, kFwdRows, lane_channels(D)).end);
    const cudaError_t err = cudaMemcpyAsync(copy, a.S0, (size_t)a.num_seqs * D * sizeof(float),
                                            cudaMemcpyDeviceToDevice, stream);
    if (err != cudaSuccess) return err;
    b.S0 = copy;
    return run_forward(b, ws, stream);
}

cudaError_t launch_linrec_wait_check(char* ws, uint64_t timeout_ns, cudaStream_t stream) {
    const TileLayout L = tile_layout(kCheckTokens, 1, kFwdRows, 1);
    static_assert(kRecords + kCheckTiles * 32 * sizeof(uint64_t) + 256 +
                  (3 * kCheckTokens + 8) * sizeof(float) <= KDA_SCAN_CHECK_BYTES, "its workspace");
    linrec_check_case_kernel<<<1, kThreads, 0, stream>>>(ws, L.end);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    TileSpace w;
    set_space(w, L, ws);
    w.wait_ns = timeout_ns;
    float* x = reinterpret_cast<float*>(ws + L.end);
    LinrecArgs a = {};
    a.x = x;
    a.gate = x + kCheckTokens;
    a.y = x + 2 * kCheckTokens;
    a.S_T = x + 3 * kCheckTokens;
    a.cu_seqlens = reinterpret_cast<const int32_t*>(x + 3 * kCheckTokens + 4);
    a.total_tokens = kCheckTokens;
    a.num_seqs = a.H = a.d = 1;
    a.dtype = KDA_FP32;
    a.gate_format = KDA_GATE_CHANNEL_F32;
    linrec_fwd_kernel<float, KDA_GATE_CHANNEL_F32, false, 1>
        <<<kCheckTiles - 1, kThreads, kWarps * FwdRows<float, false, 1>::kBytes, stream>>>(a, w);
    return cudaGetLastError();
}

cudaError_t launch_linrec_backward(const LinrecArgs& a, char* ws, cudaStream_t stream) {
    const int64_t D = (int64_t)a.H * a.d;
    const TileLayout L = tile_layout(a.total_tokens, D, kBwdRows,
                                     lane_channels(D, a.d, a.gate_format));
    size_t at = tile_layout(a.total_tokens, D, kBwdRows, lane_channels(D)).end;
    const float* states = a.states;
    cudaError_t err;
    const bool rerun = !states && a.total_tokens > 0;
    if (rerun) {   // the forward scan once more, for the tiles' entry states alone
        LinrecArgs f = a;
        f.states = reinterpret_cast<float*>(ws + at);
        states = f.states;
        at += pad((size_t)L.nt * D * sizeof(float));
        err = run_forward(f, ws, stream);
        if (err != cudaSuccess) return err;
    }
    TileSpace w;
    err = start_tiles(a, L, ws, rerun, w, stream);
    if (err != cudaSuccess) return err;
    const int mode = head_mode(a.d, a.gate_format, D);
    const int32_t parts = head_parts(a.d, a.gate_format, D);
    float* dgate = parts > 1 ? reinterpret_cast<float*>(ws + at) : a.dgate;
    err = by_tile(a, [&](auto* t, auto g, auto comp, auto vec) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int V = decltype(vec)::value;
        auto kernel = linrec_bwd_kernel<T, decltype(g)::value, decltype(comp)::value, V>;
        cudaLaunchConfig_t c = {};
        cudaLaunchAttribute attr;
        const cudaError_t set = configure_tiles(kernel, L, 2, filled(a, L),
                                             kWarps * BwdRows<T, V>::kBytes, stream, c, attr);
        return set == cudaSuccess ? cudaLaunchKernelEx(&c, kernel, a, w, states, dgate, mode) : set;
    });
    if (err != cudaSuccess || parts == 1 || a.total_tokens == 0) return err;
    const int64_t each = parts <= kFewParts ? kThreads : kWarps;   // rows a block
    const int64_t blocks = (a.total_tokens * a.H + each - 1) / each;
    const int64_t most = 16 * (int64_t)sm_count();
    linrec_head_sum_kernel<<<(unsigned)(blocks < most ? blocks : most), kThreads, 0, stream>>>(
        dgate, a.cu_seqlens, a.num_seqs, a.H, parts, a.dgate, w.status);
    return cudaGetLastError();
}

cudaError_t launch_linrec_step(const LinrecStepArgs& a, cudaStream_t stream) {
    const int D = a.H * a.d;
    const bool wide = a.d % 4 == 0;
    const int blocks = (D / (wide ? 4 : 1) + kThreads - 1) / kThreads;
    if ((int64_t)a.B * blocks > INT32_MAX) return cudaErrorInvalidValue;
    return by_type(a.dtype, a.gate_format, [&](auto* t, auto g) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int G = decltype(g)::value;
        auto kernel = wide ? linrec_step_kernel<T, G, 4> : linrec_step_kernel<T, G, 1>;
        kernel<<<(unsigned)(a.B * blocks), kThreads, 0, stream>>>(a, blocks);
        return cudaGetLastError();
    });
}

}  // namespace kda
