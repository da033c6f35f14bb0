// Gated linear recurrence h_t = a_t h_{t-1} + u_t (include/linrec.h): prefill,
// backward and decode step.
//
// Mathematics.  Every channel is a chain of affine maps h -> a h + u, and maps
// compose: over a run of tokens h_out = A h_in + B with A the product of the
// gates and B the run's result from zero.  A tile of 128 tokens x 64 channels
// lives in the registers of one CTA: each of its eight warps holds 16 tokens
// (two channels a lane), forms its (A, B), and once the state that enters the
// tile is known every warp starts from its own entry state and walks its
// tokens again in registers.  So x and the gate are read from memory once and
// y is written once.
//
// The packed token axis is cut into tiles regardless of sequences.  At a
// sequence's first token the carried state is replaced by S0 (replaced, not
// multiplied by zero: a state that is not finite stays in its sequence), and a
// tile with such a token needs nothing from before it for what follows.
//
// Between tiles: each publishes its (A, B), looks back over the tiles before it
// for the nearest state that is already known, and applies the (A, B) of the
// tiles between in token order.  The arithmetic is the same whichever tile that
// is, so results do not depend on timing.  Tiles are handed out in time order by
// a ticket, so a tile's predecessors are always running or done; every wait is
// bounded all the same.
//
// The backward pass is the same recurrence on reversed tokens:
// r_t = a_t (dy_t + r_{t+1}), g_t = dy_t + r_{t+1}, with dS_T replacing r at a
// sequence's last token; the states it multiplies are rebuilt in registers from
// the tile's entry state (`states`).
#include "kda_internal.h"

#include <type_traits>

namespace kda {
namespace {

constexpr int kWarps = 8;
constexpr int kRows = LINREC_CHUNK / kWarps;   // tokens a warp
constexpr int kThreads = kWarps * 32;
constexpr int kSelfCheck = 1024;   // most sequences whose offsets every CTA checks by itself
constexpr uint64_t kWaitNs = 2000000000ull;
static_assert(kRows == 16, "row masks and the four-row groups are written for 16");

// Head of the workspace: zeroed before each launch whose time axis has several tiles.
//   [0, 4) status, [4, 8) ticket, [16, ..) uint32 flag[tiles][channel tiles]
// then float2 agg[tiles][Dp] and float inc[tiles][Dp] (Dp: channels padded to tiles).
enum : uint32_t { kNone = 0, kAggregate = 1, kInclusive = 2 };

struct TileSpace {
    int32_t* status;
    uint32_t* ticket;
    uint32_t* flag;
    float2* agg;
    float* inc;
    int32_t nt, ct;      // tiles along tokens and channels
    int64_t Dp;
};

__device__ __forceinline__ uint64_t now_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_release(uint32_t* p, uint32_t v) {
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
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
// log a in bf16: exp by the accurate function, since a state multiplies up to
// thousands of gates; 1 - a from expm1, since 1 - exp would lose it near 1.
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

// How a warp's rows reach its registers.
//   kStaged: 16-byte asynchronous copies into the warp's own part of shared
//     memory, issued while the tile before is worked on (rows on a 16-byte
//     grid: D a multiple of 8, and a head gate's d even)
//   kDirect: plain loads
enum : int { kDirect = 0, kStaged = 1 };

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
    const int n = on ? 16 : 0;   // 0: the destination is filled with zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool on) {
    const int n = on ? 4 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void copies_done() {
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Bytes of one warp's rows of an array of E-byte elements in shared memory.
template <int E>
constexpr int staged_bytes() { return kRows * 64 * E; }
template <int GATE>
constexpr int gate_bytes() {
    return GATE == KDA_GATE_HEAD_F32 ? kRows * 32 * 4
                                     : staged_bytes<GATE == KDA_GATE_CHANNEL_LOG_BF16 ? 2 : 4>();
}

// Issues the copies of a warp's 16 rows x 64 channels of src ([T][D], E-byte
// elements) from token t0, channel c0; outside the tensor zeros.
template <int E>
__device__ __forceinline__ void stage_rows(uint32_t dst, const void* src, int64_t t0, int64_t T,
                                           int64_t D, int64_t c0, int lane) {
    constexpr int kPieces = 64 * E / 16;             // 16-byte pieces a row
    constexpr int kStep = 32 / kPieces;              // rows a pass
    const int row = lane / kPieces, piece = lane % kPieces;
    const int64_t c = c0 + piece * (16 / E);
    const char* p = static_cast<const char*>(src) + ((t0 + row) * D + c) * E;
    const int64_t step = D * kStep * E;
    const int left = c < D ? (int)(T - t0 < kRows ? T - t0 : kRows) - row : 0;
    const uint32_t at = dst + row * 64 * E + piece * 16;
#pragma unroll
    for (int j = 0; j < kRows / kStep; ++j) {
        const bool on = j * kStep < left;
        copy16(at + j * kStep * 64 * E, on ? p : src, on);
        p += step;
    }
}
// A head gate: lane's own head, one value a row.
__device__ __forceinline__ void stage_heads(uint32_t dst, const void* src, int64_t t0, int64_t T,
                                            int H, int head, bool on, int lane) {
    const char* p = static_cast<const char*>(src) + (t0 * H + head) * 4;
    const int left = on ? (int)(T - t0 < kRows ? T - t0 : kRows) : 0;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        copy4(dst + (r * 32 + lane) * 4, r < left ? p : src, r < left);
        p += H * 4;
    }
}

// One warp's rows of an array in registers: from its staged copy, or by plain
// loads (left: rows to read, 0 for a lane without channels).
template <int PATH, typename T, int VEC>
__device__ __forceinline__ void take_rows(Piece<T, VEC> (&x)[kRows], const char* staged,
                                          const void* src, int64_t at, int64_t D, int left,
                                          int lane) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (PATH == kStaged) {
            x[r].load(reinterpret_cast<const T*>(staged) + r * 64 + lane * VEC);
        } else {
            x[r] = Piece<T, VEC>{};
            if (r < left) x[r].load(static_cast<const T*>(src) + at + r * D);
        }
    }
}
template <int PATH, int GATE, int VEC>
__device__ __forceinline__ void take_gate(Gate<GATE, VEC> (&a)[kRows], const char* staged,
                                          const void* src, int64_t t0, int64_t D, int64_t ch,
                                          int H, int d, int left, int lane) {
    if constexpr (GATE == KDA_GATE_HEAD_F32) {
        const int h0 = (int)(ch / d), h1 = (int)((ch + VEC - 1) / d);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (PATH == kStaged) {
                a[r].f = fill<VEC>(reinterpret_cast<const float*>(staged)[r * 32 + lane]);
            } else {
                a[r].f = fill<VEC>(0.f);
                if (r < left) {
                    const float* g = static_cast<const float*>(src) + (t0 + r) * H;
                    a[r].f.v[0] = g[h0];
                    a[r].f.v[VEC - 1] = g[h1];
                }
            }
        }
    } else if constexpr (GATE == KDA_GATE_CHANNEL_LOG_BF16) {
        Piece<__nv_bfloat16, VEC> raw[kRows];
        take_rows<PATH, __nv_bfloat16, VEC>(raw, staged, src, t0 * D + ch, D, left, lane);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            a[r].raw = raw[r];
            const Vec<VEC> la = raw[r].get();
#pragma unroll
            for (int v = 0; v < VEC; ++v) a[r].f.v[v] = expf(la.v[v]);
        }
    } else {
        Piece<float, VEC> raw[kRows];
        take_rows<PATH, float, VEC>(raw, staged, src, t0 * D + ch, D, left, lane);
#pragma unroll
        for (int r = 0; r < kRows; ++r) a[r].f = raw[r].get();
    }
}

// Offsets of the sequences: checked once a CTA, sampled into shared memory.
struct Offsets {
    int32_t sample[kSelfCheck + 2];
    int32_t stride, count;   // sample[j] = cu[min(j * stride, N)], j < count
};

// True when the offsets are valid.  Up to kSelfCheck sequences are checked here
// (every CTA for itself), more by linrec_check_kernel before the launch.
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
    } else {
        for (int j = threadIdx.x; j < count; j += kThreads)
            o.sample[j] = cu[min((int64_t)j * stride, (int64_t)N)];
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
__device__ __forceinline__ Rows rows_of(const Offsets& o, const int32_t* cu, int N, int64_t t0,
                                        int64_t end, int lane) {
    Rows w;
    const int64_t t = t0 + lane;
    const bool live = lane < kRows && t < end;
    bool s = false, l = false;
    w.n = 0;
    if (live) {
        w.n = sequence_of(o, cu, N, (int32_t)t);
        s = (o.stride == 1 ? o.sample[w.n] : cu[w.n]) == t;
        l = (o.stride == 1 ? o.sample[w.n + 1] : cu[w.n + 1]) - 1 == t;
    }
    w.start = __ballot_sync(0xffffffffu, s);
    w.last = __ballot_sync(0xffffffffu, l);
    w.live = end <= t0 ? 0 : end - t0 < kRows ? (int)(end - t0) : kRows;
    return w;
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

// One warp finds the state that enters tile i of channel tile c: the nearest tile
// before it (in scan order, step = -1: towards lower indices, +1: higher) whose
// state is known, then the maps of the tiles between.  Lane's VEC channels from
// ch.  Gives zeros when the wait ran out or another warp's did.
template <int VEC>
__device__ Vec<VEC> look_back(const TileSpace& w, int i, int c, int step, int64_t ch, int lane) {
    Vec<VEC> H = fill<VEC>(0.f);
    int base = i + step;   // lane j looks at base + j * step
    int found = -1;
    uint64_t t0 = 0;
    for (uint32_t round = 0;; ++round) {
        const int idx = base + lane * step;
        uint32_t f = kNone;
        if (idx >= 0 && idx < w.nt) f = ld_acquire(w.flag + (int64_t)idx * w.ct + c);
        const uint32_t inc = __ballot_sync(0xffffffffu, f == kInclusive);
        const uint32_t any = __ballot_sync(0xffffffffu, f != kNone);
        if (inc) {
            const int first = __ffs(inc) - 1;
            const uint32_t before = (1u << first) - 1;
            if ((any & before) == before) {
                found = base + first * step;
                break;
            }
        } else if (any == 0xffffffffu) {
            base += 32 * step;
            continue;
        }
        if ((round & 63) == 63) {
            // bounded: give up after kWaitNs, or as soon as another wait has
            const uint64_t t = now_ns();
            if (t0 == 0) t0 = t;
            int stop = 0;
            if (lane == 0) {
                if (t - t0 > kWaitNs) atomicExch(w.status, (int32_t)KDA_ERR_DEVICE_TIMEOUT);
                stop = *reinterpret_cast<volatile int32_t*>(w.status) != 0;
            }
            if (__shfl_sync(0xffffffffu, stop, 0)) return H;
        }
    }
    __syncwarp();
    // the padded channels have entries too, so every lane reads
#pragma unroll
    for (int v = 0; v < VEC; ++v) H.v[v] = __ldcg(w.inc + (int64_t)found * w.Dp + ch + v);
    for (int k = found - step; k != i; k -= step) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float2 m = __ldcg(w.agg + (int64_t)k * w.Dp + ch + v);
            H.v[v] = fmaf(m.x, H.v[v], m.y);
        }
    }
    return H;
}

// Publishes a tile's map or its leaving state (one warp).
template <int VEC>
__device__ __forceinline__ void publish(const TileSpace& w, int i, int c, int64_t ch, int lane,
                                        uint32_t kind, const Vec<VEC>& A, const Vec<VEC>& B) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        if (kind == kInclusive) w.inc[(int64_t)i * w.Dp + ch + v] = B.v[v];
        else w.agg[(int64_t)i * w.Dp + ch + v] = make_float2(A.v[v], B.v[v]);
    }
    __threadfence();
    __syncwarp();
    if (lane == 0) st_release(w.flag + (int64_t)i * w.ct + c, kind);
}

// Warp maps of a tile.  Two buffers, for tiles in turn, save the barrier between
// one tile's last reads and the next one's writes.
template <int VEC, int BUFS>
struct Maps {
    Vec<VEC> A[BUFS][kWarps][32];
    Vec<VEC> B[BUFS][kWarps][32];
    uint32_t reset[BUFS][kWarps];   // the warp's rows hold a boundary: B alone counts

    __device__ __forceinline__ void put(int buf, int warp, int lane, const Vec<VEC>& a,
                                        const Vec<VEC>& b, uint32_t boundary) {
        A[buf][warp][lane] = a;
        B[buf][warp][lane] = b;
        if (lane == 0) reset[buf][warp] = boundary;
    }
    // The state after warp j's rows from the state before them.
    __device__ __forceinline__ Vec<VEC> step(int buf, int j, int lane, const Vec<VEC>& h) const {
        const Vec<VEC> b = B[buf][j][lane];
        return reset[buf][j] ? b : fma(A[buf][j][lane], h, b);
    }
};

// The first tile of a CTA, broadcast: with several tiles along time by ticket.
__device__ __forceinline__ int64_t first_tile(const TileSpace& w, uint32_t* shared) {
    if (w.nt == 1) return blockIdx.x;
    if (threadIdx.x == 0) *shared = atomicAdd(w.ticket, 1u);
    __syncthreads();
    return *shared;
}

// CTAs an SM: 48 registers a thread hold a tile of bf16 inputs (32 of gates, 16 of
// inputs), so that three CTAs fit; fp32 inputs, and log gates with the complement,
// which keep both log a and a, leave room for two.
template <typename T, int GATE, bool COMP, int PATH>
constexpr int fwd_ctas() {
    return PATH == kStaged && sizeof(T) == 2 && !(COMP && GATE == KDA_GATE_CHANNEL_LOG_BF16) ? 3 : 2;
}

template <typename T, int GATE, bool COMP, int VEC, int PATH>
__global__ void __launch_bounds__(kThreads, fwd_ctas<T, GATE, COMP, PATH>())
linrec_fwd_kernel(const LinrecArgs p, const TileSpace w) {
    extern __shared__ __align__(16) char staging[];
    __shared__ Offsets off;
    __shared__ Maps<VEC, 2> maps;
    __shared__ Vec<VEC> carry[32];
    __shared__ uint32_t next_ticket;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int N = p.num_seqs;
    const int64_t D = (int64_t)p.H * p.d;
    const int32_t* cu = p.cu_seqlens;
    constexpr int kX = staged_bytes<sizeof(T)>();
    char* sx = staging + warp * (kX + gate_bytes<GATE>());
    char* sg = sx + kX;
    const uint32_t sx32 = (uint32_t)__cvta_generic_to_shared(sx);

    auto stage = [&](int64_t tile) {
        if constexpr (PATH == kStaged) {
            const int i = (int)(tile / w.ct), c = (int)(tile % w.ct);
            const int64_t t0 = (int64_t)i * LINREC_CHUNK + warp * kRows, c0 = (int64_t)c * 64;
            const int64_t T_ = p.total_tokens;
            stage_rows<sizeof(T)>(sx32, p.x, t0, T_, D, c0, lane);
            if constexpr (GATE == KDA_GATE_HEAD_F32) {
                const int64_t ch = c0 + lane * 2;
                stage_heads(sx32 + kX, p.gate, t0, T_, p.H, ch < D ? (int)(ch / p.d) : 0, ch < D,
                            lane);
            } else {
                stage_rows<GATE == KDA_GATE_CHANNEL_LOG_BF16 ? 2 : 4>(sx32 + kX, p.gate, t0, T_, D,
                                                                      c0, lane);
            }
        }
    };

    const int64_t tiles = (int64_t)w.nt * w.ct;
    int64_t tile = first_tile(w, &next_ticket);
    if (tile < tiles) stage(tile);
    if (!read_offsets(off, cu, N, p.total_tokens, w.status)) {
        copies_done();
        if (blockIdx.x == 0 && threadIdx.x == 0) *w.status = KDA_ERR_DEVICE_INPUT;
        return;
    }
    if (w.nt == 1 && N <= kSelfCheck && blockIdx.x == 0 && threadIdx.x == 0) *w.status = KDA_OK;
    const int64_t end = cu[N];
    copy_empty(cu, N, D, p.S0, p.S_T);

    for (int buf = 0; tile < tiles; buf ^= 1) {
        const int i = (int)(tile / w.ct), c = (int)(tile % w.ct);
        const int64_t t0 = (int64_t)i * LINREC_CHUNK + warp * kRows;
        const int64_t ch = (int64_t)c * 32 * VEC + lane * VEC;   // this lane's channels
        const bool on = ch < D;
        const Rows rows = rows_of(off, cu, N, t0, end, lane);
        const bool edge = (rows.start | rows.last) != 0 || rows.live < kRows;

        // the tile, into registers
        Piece<T, VEC> x[kRows];
        Gate<GATE, VEC> a[kRows];
        if (PATH == kStaged) {
            copies_done();
            __syncwarp();
        }
        const int left = on ? rows.live : 0;
        take_rows<PATH, T, VEC>(x, sx, p.x, t0 * D + ch, D, left, lane);
        take_gate<PATH, GATE, VEC>(a, sg, p.gate, t0, D, ch, p.H, p.d, left, lane);
        auto input = [&](int r) {
            if constexpr (COMP) return mul(a[r].na(), x[r].get());
            else return x[r].get();
        };
        // the state that replaces the carried one at a sequence's first token
        auto start = [&](int r) {
            Vec<VEC> h0 = fill<VEC>(0.f);
            const int n = __shfl_sync(0xffffffffu, rows.n, r);
            if (p.S0 && on) h0 = load_f32<VEC>(p.S0 + n * D + ch);
            return h0;
        };

        Vec<VEC> A = fill<VEC>(1.f), B = fill<VEC>(0.f);
        if (!edge) {
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                B = fma(a[r].a(), B, input(r));
                A = mul(A, a[r].a());
            }
        } else {
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (rows.start >> r & 1) B = start(r);
                B = fma(a[r].a(), B, input(r));
                A = mul(A, a[r].a());
            }
        }
        maps.put(buf, warp, lane, A, B, rows.start);
        if (threadIdx.x == 32 && w.nt > 1) next_ticket = atomicAdd(w.ticket, 1u);
        __syncthreads();
        tile = w.nt > 1 ? (int64_t)next_ticket : tile + gridDim.x;
        if (tile < tiles) stage(tile);   // the warp's rows are in registers: their place is free

        if (warp == 0) {
            bool reset = false;
            A = fill<VEC>(1.f);
            B = fill<VEC>(0.f);
#pragma unroll
            for (int j = 0; j < kWarps; ++j) {
                reset |= maps.reset[buf][j] != 0;
                B = maps.step(buf, j, lane, B);
                A = mul(A, maps.A[buf][j][lane]);
            }
            const bool needed = t0 < end && !(rows.start & 1);   // row 0 continues a sequence
            const bool wanted = w.nt > 1 && t0 + LINREC_CHUNK < end;   // a tile comes after
            Vec<VEC> H = fill<VEC>(0.f);
            if (wanted) publish<VEC>(w, i, c, ch, lane, reset ? kInclusive : kAggregate, A, B);
            if (needed) {
                H = look_back<VEC>(w, i, c, -1, ch, lane);
                if (wanted && !reset)
                    publish<VEC>(w, i, c, ch, lane, kInclusive, A, fma(A, H, B));
            }
            if (p.states && on) store(p.states + i * D + ch, H);
            carry[lane] = H;
        }
        __syncthreads();

        Vec<VEC> h = carry[lane];
        for (int j = 0; j < warp; ++j) h = maps.step(buf, j, lane, h);
        T* y = p.y ? static_cast<T*>(p.y) + t0 * D + ch : nullptr;
        if (!edge) {
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                h = fma(a[r].a(), h, input(r));
                if (on && y) store(y + r * D, h);
            }
        } else {
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (rows.start >> r & 1) h = start(r);
                h = fma(a[r].a(), h, input(r));
                if (on && y && r < rows.live) store(y + r * D, h);
                if (rows.last >> r & 1) {
                    const int n = __shfl_sync(0xffffffffu, rows.n, r);
                    if (p.S_T && on) store(p.S_T + n * D + ch, h);
                }
            }
        }
    }
}

// Where a head's gate gradient, a sum over its channels, goes.
//   kHeadRow: lanes of a warp that share a head are summed by shuffles; a head
//     of at most 64 channels is done, a wider one leaves d / 64 partial sums
//   kHeadWide: every channel's term goes to a buffer, summed afterwards (widths
//     that neither divide 64 nor are a multiple of it)
enum : int { kNoHead = 0, kHeadRow = 1, kHeadWide = 2 };

template <typename T, int GATE, bool COMP, int VEC, int PATH>
__global__ void __launch_bounds__(kThreads, 2)
linrec_bwd_kernel(const LinrecArgs p, const TileSpace w, const float* __restrict__ states,
                  float* dgate, int head_mode) {
    extern __shared__ __align__(16) char staging[];
    __shared__ Offsets off;
    // one buffer: with two, two CTAs of fp32 inputs would not fit an SM
    __shared__ Maps<VEC, 1> maps;    // of the state, tokens forward
    __shared__ Maps<VEC, 1> rmaps;   // of the gradient, tokens backward
    __shared__ Vec<VEC> carry[32];
    __shared__ uint32_t next_ticket;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int N = p.num_seqs;
    const int64_t D = (int64_t)p.H * p.d;
    const int32_t* cu = p.cu_seqlens;
    constexpr int kX = staged_bytes<sizeof(T)>();
    char* sx = staging + warp * (2 * kX + gate_bytes<GATE>());
    char* sy = sx + kX;
    char* sg = sy + kX;
    const uint32_t sx32 = (uint32_t)__cvta_generic_to_shared(sx);

    auto stage = [&](int64_t tile) {
        if constexpr (PATH == kStaged) {
            const int i = w.nt - 1 - (int)(tile / w.ct), c = (int)(tile % w.ct);
            const int64_t t0 = (int64_t)i * LINREC_CHUNK + warp * kRows, c0 = (int64_t)c * 64;
            const int64_t T_ = p.total_tokens;
            stage_rows<sizeof(T)>(sx32, p.x, t0, T_, D, c0, lane);
            stage_rows<sizeof(T)>(sx32 + kX, p.dy, t0, T_, D, c0, lane);
            if constexpr (GATE == KDA_GATE_HEAD_F32) {
                const int64_t ch = c0 + lane * 2;
                stage_heads(sx32 + 2 * kX, p.gate, t0, T_, p.H, ch < D ? (int)(ch / p.d) : 0,
                            ch < D, lane);
            } else {
                stage_rows<GATE == KDA_GATE_CHANNEL_LOG_BF16 ? 2 : 4>(sx32 + 2 * kX, p.gate, t0,
                                                                      T_, D, c0, lane);
            }
        }
    };

    const int64_t tiles = (int64_t)w.nt * w.ct;
    int64_t tile = first_tile(w, &next_ticket);
    if (tile < tiles) stage(tile);
    if (!read_offsets(off, cu, N, p.total_tokens, w.status)) {
        copies_done();
        if (blockIdx.x == 0 && threadIdx.x == 0) *w.status = KDA_ERR_DEVICE_INPUT;
        return;
    }
    if (w.nt == 1 && N <= kSelfCheck && blockIdx.x == 0 && threadIdx.x == 0) *w.status = KDA_OK;
    const int64_t end = cu[N];
    copy_empty(cu, N, D, p.dS_T, p.dS0);

    while (tile < tiles) {
        const int i = w.nt - 1 - (int)(tile / w.ct), c = (int)(tile % w.ct);
        const int64_t t0 = (int64_t)i * LINREC_CHUNK + warp * kRows;
        const int64_t ch = (int64_t)c * 32 * VEC + lane * VEC;
        const bool on = ch < D;
        const Rows rows = rows_of(off, cu, N, t0, end, lane);
        const bool edge = (rows.start | rows.last) != 0 || rows.live < kRows;
        Vec<VEC> H = fill<VEC>(0.f);   // the state that enters the tile
        if (on && (int64_t)i * LINREC_CHUNK < end) H = load_f32<VEC>(states + i * D + ch);

        Piece<T, VEC> x[kRows], dy[kRows];
        Gate<GATE, VEC> a[kRows];
        if (PATH == kStaged) {
            copies_done();
            __syncwarp();
        }
        const int left = on ? rows.live : 0;
        take_rows<PATH, T, VEC>(x, sx, p.x, t0 * D + ch, D, left, lane);
        take_rows<PATH, T, VEC>(dy, sy, p.dy, t0 * D + ch, D, left, lane);
        take_gate<PATH, GATE, VEC>(a, sg, p.gate, t0, D, ch, p.H, p.d, left, lane);
        auto input = [&](int r) {
            if constexpr (COMP) return mul(a[r].na(), x[r].get());
            else return x[r].get();
        };
        auto boundary = [&](const float* src, int r) {   // S0 or dS_T of row r's sequence
            Vec<VEC> h0 = fill<VEC>(0.f);
            const int n = __shfl_sync(0xffffffffu, rows.n, r);
            if (src && on) h0 = load_f32<VEC>(src + n * D + ch);
            return h0;
        };

        // maps of the warp's rows, both ways
        Vec<VEC> A = fill<VEC>(1.f), B = fill<VEC>(0.f), RB = fill<VEC>(0.f), RA = fill<VEC>(1.f);
        if (!edge) {
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                B = fma(a[r].a(), B, input(r));
                A = mul(A, a[r].a());
            }
#pragma unroll
            for (int r = kRows - 1; r >= 0; --r) RB = mul(a[r].a(), add(dy[r].get(), RB));
            RA = A;
        } else {
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (rows.start >> r & 1) B = boundary(p.S0, r);
                B = fma(a[r].a(), B, input(r));
                A = mul(A, a[r].a());
            }
#pragma unroll
            for (int r = kRows - 1; r >= 0; --r) {
                if (rows.last >> r & 1) RB = boundary(p.dS_T, r);
                if (r < rows.live) {   // rows past the end hand on nothing
                    RB = mul(a[r].a(), add(dy[r].get(), RB));
                    RA = mul(RA, a[r].a());
                }
            }
        }
        maps.put(0, warp, lane, A, B, rows.start);
        rmaps.put(0, warp, lane, RA, RB, rows.last);
        if (threadIdx.x == 0 && w.nt > 1) next_ticket = atomicAdd(w.ticket, 1u);
        __syncthreads();
        tile = w.nt > 1 ? (int64_t)next_ticket : tile + gridDim.x;
        if (tile < tiles) stage(tile);

        if (warp == kWarps - 1) {
            bool reset = false;
            A = fill<VEC>(1.f);
            B = fill<VEC>(0.f);
#pragma unroll
            for (int j = kWarps - 1; j >= 0; --j) {
                reset |= rmaps.reset[0][j] != 0;
                B = rmaps.step(0, j, lane, B);
                A = mul(A, rmaps.A[0][j][lane]);
            }
            // the tile's last row goes on in the next tile; a tile comes before
            const bool needed = t0 + kRows < end && !(rows.last >> (kRows - 1) & 1);
            const bool wanted = i > 0 && (int64_t)i * LINREC_CHUNK < end;
            Vec<VEC> R = fill<VEC>(0.f);
            if (wanted) publish<VEC>(w, i, c, ch, lane, reset ? kInclusive : kAggregate, A, B);
            if (needed) {
                R = look_back<VEC>(w, i, c, +1, ch, lane);
                if (wanted && !reset)
                    publish<VEC>(w, i, c, ch, lane, kInclusive, A, fma(A, R, B));
            }
            carry[lane] = R;
        }
        __syncthreads();

        // what the gate multiplies at each row: the state before it, less x for the complement
        Vec<VEC> f[kRows];
        for (int j = 0; j < warp; ++j) H = maps.step(0, j, lane, H);
        auto less_x = [&](const Vec<VEC>& prev, int r) {
            if constexpr (!COMP) return prev;
            Vec<VEC> q = x[r].get();
#pragma unroll
            for (int v = 0; v < VEC; ++v) q.v[v] = prev.v[v] - q.v[v];
            return q;
        };
        if (!edge) {
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                f[r] = less_x(H, r);
                H = fma(a[r].a(), H, input(r));
            }
        } else {
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (rows.start >> r & 1) H = boundary(p.S0, r);
                f[r] = less_x(H, r);
                H = fma(a[r].a(), H, input(r));
            }
        }
        Vec<VEC> R = carry[lane];
        for (int j = kWarps - 1; j > warp; --j) R = rmaps.step(0, j, lane, R);
        __syncthreads();   // the maps are read: the next tile may write them
        float* dx = p.dx + t0 * D + ch;
        // row r's gradients from R, the gradient that comes from behind
        auto row = [&](int r, bool out) {
            const Vec<VEC> g = add(dy[r].get(), R);
            if constexpr (COMP) {
                if (out) store(dx + r * D, mul(a[r].na(), g));
            } else {
                if (out) store(dx + r * D, g);
            }
            f[r] = mul(g, f[r]);
            R = mul(a[r].a(), g);
            if constexpr (GATE == KDA_GATE_CHANNEL_LOG_BF16) f[r] = mul(a[r].a(), f[r]);
            if (GATE != KDA_GATE_HEAD_F32 || head_mode == kHeadWide)
                if (out) store(dgate + (t0 + r) * D + ch, f[r]);
        };
        if (!edge) {
#pragma unroll
            for (int r = kRows - 1; r >= 0; --r) row(r, on);
        } else {
#pragma unroll
            for (int r = kRows - 1; r >= 0; --r) {
                if (rows.last >> r & 1) R = boundary(p.dS_T, r);
                if (r < rows.live) row(r, on);
                if (rows.start >> r & 1) {
                    const int n = __shfl_sync(0xffffffffu, rows.n, r);
                    if (p.dS0 && on) store(p.dS0 + n * D + ch, R);
                }
            }
        }
        if constexpr (GATE == KDA_GATE_HEAD_F32) {
            if (head_mode == kHeadRow) {
                // lanes that share a head (or one of its 64-channel parts) add up
                const int part = p.d < 32 * VEC ? p.d : 32 * VEC, width = part / VEC;
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    float s = on && r < rows.live ? f[r].v[0] + (VEC == 2 ? f[r].v[VEC - 1] : 0.f)
                                                  : 0.f;
                    for (int o = width >> 1; o > 0; o >>= 1)
                        s += __shfl_xor_sync(0xffffffffu, s, o);
                    // [T][H][parts]: the part's index is the channel over its width
                    if (on && r < rows.live && (lane & (width - 1)) == 0)
                        dgate[(t0 + r) * (D / part) + ch / part] = s;
                }
            }
        }
    }
}

// dgate[t][h] = the sum of the head's `parts` terms, one warp each.
__global__ void __launch_bounds__(kThreads)
linrec_head_sum_kernel(const float* __restrict__ part, const int32_t* cu, int32_t N, int32_t H,
                       int32_t parts, float* __restrict__ dgate, const int32_t* status) {
    if (N == 0 || *status == KDA_ERR_DEVICE_INPUT) return;
    const int lane = threadIdx.x & 31;
    const int64_t rows = (int64_t)cu[N] * H;
    for (int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); i < rows;
         i += (int64_t)gridDim.x * kWarps) {
        float s = 0.f;
        for (int j = lane; j < parts; j += 32) s += part[i * parts + j];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) dgate[i] = s;
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

template <typename T, int GATE>
__global__ void __launch_bounds__(kThreads) linrec_step_kernel(const LinrecStepArgs p) {
    const int D = p.H * p.d;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (int64_t)p.B * D) return;
    const int b = (int)(i / D), c = (int)(i % D);
    const int row = p.parents ? p.parents[b] : b;
    const float h = row >= 0 && row < p.num_rows ? p.S[(int64_t)row * D + c] : 0.f;
    float a, na;
    if (GATE == KDA_GATE_CHANNEL_LOG_BF16) {
        const float la = __bfloat162float(static_cast<const __nv_bfloat16*>(p.gate)[i]);
        a = expf(la);
        na = -expm1f(la);
    } else {
        a = static_cast<const float*>(p.gate)[GATE == KDA_GATE_HEAD_F32 ? i / p.d : i];
        na = 1.f - a;
    }
    const float xv = Elem<T>::load(static_cast<const T*>(p.x) + i);
    const float out = fmaf(a, h, p.complement ? na * xv : xv);
    p.S_out[i] = out;
    Elem<T>::store(static_cast<T*>(p.y) + i, out);
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

// Two channels a lane need rows on a 4-byte (bf16) grid: an even row width.
int lane_channels(int64_t D) { return D % 2 == 0 ? 2 : 1; }

struct TileLayout {
    int64_t nt, ct, Dp;
    size_t head, agg, inc, end;
};
TileLayout tile_layout(int64_t T, int64_t D) {
    TileLayout L;
    const int64_t width = 32 * lane_channels(D);
    L.nt = T > 0 ? (T + LINREC_CHUNK - 1) / LINREC_CHUNK : 1;
    L.ct = (D + width - 1) / width;
    L.Dp = L.ct * width;
    L.head = L.nt > 1 ? 16 + (size_t)L.nt * L.ct * sizeof(uint32_t) : 16;
    L.agg = pad(L.head);
    L.inc = L.agg + (L.nt > 1 ? pad((size_t)L.nt * L.Dp * sizeof(float2)) : 0);
    L.end = L.inc + (L.nt > 1 ? pad((size_t)L.nt * L.Dp * sizeof(float)) : 0);
    return L;
}

// Clears the head (keeping the status word of an earlier pass) and checks the
// offsets of large batches.
cudaError_t start_tiles(const LinrecArgs& a, const TileLayout& L, char* ws, bool keep_status,
                        TileSpace& w, cudaStream_t stream) {
    w.status = reinterpret_cast<int32_t*>(ws);
    w.ticket = reinterpret_cast<uint32_t*>(ws + 4);
    w.flag = reinterpret_cast<uint32_t*>(ws + 16);
    w.agg = reinterpret_cast<float2*>(ws + L.agg);
    w.inc = reinterpret_cast<float*>(ws + L.inc);
    w.nt = (int32_t)L.nt;
    w.ct = (int32_t)L.ct;
    w.Dp = L.Dp;
    if (L.nt > 1 || a.num_seqs > kSelfCheck) {
        const size_t from = keep_status ? 4 : 0;
        const cudaError_t err = cudaMemsetAsync(ws + from, 0, L.head - from, stream);
        if (err != cudaSuccess) return err;
    }
    if (a.num_seqs > kSelfCheck && !keep_status) {
        linrec_check_kernel<<<a.num_seqs / kThreads + 1, kThreads, 0, stream>>>(
            a.cu_seqlens, a.num_seqs, a.total_tokens, w.status);
        return cudaGetLastError();
    }
    return cudaSuccess;
}

// Rows on a 16-byte grid take the staged path.  A head gate's two channels a lane
// share a head there, so d is even.
bool staged(const LinrecArgs& a) {
    const int64_t D = (int64_t)a.H * a.d;
    return D % 8 == 0 && (a.gate_format != KDA_GATE_HEAD_F32 || a.d % 2 == 0);
}

// f(T, gate, complement, channels a lane, path) with its arguments as types.
template <int N>
using Int = std::integral_constant<int, N>;
template <typename F>
cudaError_t by_tile(const LinrecArgs& a, F&& f) {
    return by_type(a.dtype, a.gate_format, [&](auto* t, auto g) {
        auto pick = [&](auto comp) {
            if (staged(a)) return f(t, g, comp, Int<2>(), Int<kStaged>());
            if (lane_channels((int64_t)a.H * a.d) == 2) return f(t, g, comp, Int<2>(), Int<kDirect>());
            return f(t, g, comp, Int<1>(), Int<kDirect>());
        };
        return a.complement ? pick(std::true_type()) : pick(std::false_type());
    });
}

template <typename K, typename... A>
cudaError_t launch_tiles(K kernel, const TileLayout& L, int ctas, int smem, cudaStream_t stream,
                         const A&... args) {
    if (smem > 0) {
        const cudaError_t err =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (err != cudaSuccess) return err;
    }
    const int64_t tiles = L.nt * L.ct, most = (int64_t)ctas * sm_count();
    kernel<<<(unsigned)(tiles < most ? tiles : most > 0 ? most : 1), kThreads, smem, stream>>>(args...);
    return cudaGetLastError();
}

cudaError_t run_forward(const LinrecArgs& a, char* ws, cudaStream_t stream) {
    const TileLayout L = tile_layout(a.total_tokens, (int64_t)a.H * a.d);
    TileSpace w;
    cudaError_t err = start_tiles(a, L, ws, false, w, stream);
    if (err != cudaSuccess) return err;
    return by_tile(a, [&](auto* t, auto g, auto comp, auto vec, auto path) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int G = decltype(g)::value, P = decltype(path)::value;
        constexpr bool C = decltype(comp)::value;
        const int smem = P == kStaged ? kWarps * (staged_bytes<sizeof(T)>() + gate_bytes<G>()) : 0;
        return launch_tiles(linrec_fwd_kernel<T, G, C, decltype(vec)::value, P>, L,
                            fwd_ctas<T, G, C, P>(), smem, stream, a, w);
    });
}

int head_mode(int32_t d, int gate_format, int64_t D) {
    if (gate_format != KDA_GATE_HEAD_F32) return kNoHead;
    const int lanes = lane_channels(D);
    const int width = 32 * lanes;
    if (d >= lanes && (d % width == 0 || width % d == 0)) return kHeadRow;
    return kHeadWide;
}
// Partial sums a head's gate gradient is left in (1: none are).
int32_t head_parts(int32_t d, int gate_format, int64_t D) {
    switch (head_mode(d, gate_format, D)) {
        case kHeadRow: return d > 32 * lane_channels(D) ? d / (32 * lane_channels(D)) : 1;
        case kHeadWide: return d;
        default: return 1;
    }
}

}  // namespace

size_t linrec_prefill_bytes(int32_t num_seqs, int64_t total_tokens, int64_t D) {
    return tile_layout(total_tokens, D).end + pad((size_t)num_seqs * D * sizeof(float));
}

// Workspace of the backward pass: the tiles, the states when the caller has
// none, and the partial sums of head gates.
size_t linrec_backward_bytes(int32_t, int64_t total_tokens, int32_t H, int32_t d,
                             int gate_format, bool with_states) {
    const int64_t D = (int64_t)H * d;
    const TileLayout L = tile_layout(total_tokens, D);
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
    float* copy = reinterpret_cast<float*>(ws + tile_layout(a.total_tokens, D).end);
    const cudaError_t err = cudaMemcpyAsync(copy, a.S0, (size_t)a.num_seqs * D * sizeof(float),
                                            cudaMemcpyDeviceToDevice, stream);
    if (err != cudaSuccess) return err;
    b.S0 = copy;
    return run_forward(b, ws, stream);
}

cudaError_t launch_linrec_backward(const LinrecArgs& a, char* ws, cudaStream_t stream) {
    const int64_t D = (int64_t)a.H * a.d;
    const TileLayout L = tile_layout(a.total_tokens, D);
    size_t at = L.end;
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
    err = by_tile(a, [&](auto* t, auto g, auto comp, auto vec, auto path) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int G = decltype(g)::value, P = decltype(path)::value;
        const int smem = P == kStaged ? kWarps * (2 * staged_bytes<sizeof(T)>() + gate_bytes<G>()) : 0;
        return launch_tiles(
            linrec_bwd_kernel<T, G, decltype(comp)::value, decltype(vec)::value, P>, L, 2, smem,
            stream, a, w, states, dgate, mode);
    });
    if (err != cudaSuccess || parts == 1 || a.total_tokens == 0) return err;
    const int64_t blocks = (a.total_tokens * a.H + kWarps - 1) / kWarps;
    const int64_t most = 16 * (int64_t)sm_count();
    linrec_head_sum_kernel<<<(unsigned)(blocks < most ? blocks : most), kThreads, 0, stream>>>(
        dgate, a.cu_seqlens, a.num_seqs, a.H, parts, a.dgate, w.status);
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
