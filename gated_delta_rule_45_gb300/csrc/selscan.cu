// Selective state space scan (include/selscan.h): prefill, backward and decode step.
//
// Mathematics.  Per channel, h_t = exp(D_t A) h_{t-1} + D_t x_t B_t over the n values of its state
// and y_t = C_t . h_t.  Unlike a gate that comes with the token, the decays are formed from one
// step size and n rates: one exponential a (token, channel, value), 16 times as many as there
// are inputs, for two multiply-adds each.
//
// Forward: a channel lies in L lanes of 8 values each (n padded to 8, 16, 32 or 64), its
// rates and state in registers.  A CTA walks its tokens in tiles of 16, on the grid of `states`: the
// step sizes and D x are formed once a (token, channel) into shared memory, the state is carried
// through the tile, and the sums over the state are finished (skip, gate, rounding) by a pass
// over the tile in rows of 16 bytes; the next tile's rows are loaded meanwhile, and two buffers
// make one barrier a tile do.
//
// Work along the tokens: where the sequences are many enough to fill the GPU a CTA walks a whole
// sequence, the longest first.  That goes by their number: a batch of many with one far longer than
// the rest is bound by that one's CTAs (64 x 2048 channels with one of 200000 tokens of 266213: 24.4
// ms for 2.9 of equal ones, backward 105 for 12.4).  Few long ones are cut into segments of the packed axis, regardless of sequences:
// the map of a segment is its end state from zero and the sum of its step sizes (the product of
// its decays is exp(A sum D)), a short pass joins the maps, and the segments are walked from
// their entry states.  The backward pass does the same on reversed tokens.
//
// Backward: from `states` (every 16th token) the states before every 4th token are formed on one
// walk; each four tokens' states are then rebuilt in registers and walked backward.  Sums over
// the values or the channels are halved with each exchange (spread_sum); those over a CTA's
// channels go on in a second kernel.  A tile cut short by a sequence is a whole one with rows of
// steps and inputs of zero around it.
//
// Bound: instructions, with the exponentials at a third of their unit's rate (32 a clock and SM).
// Measured, bf16, n = 16 with gate and skip: 64 ragged prompts of 266240 x 2048 2.71 ms (4.4 GB,
// 1.6 TB/s; 8.7e9 exponentials, which alone take 0.93 ms: issue 2.2 a clock and SM of 4), one of
// 131072 x 4096 4.67 ms (cut: each exponential twice), forward of 8 x 4096 x 4096 with `states` 0.86
// ms, backward 3.5 ms (2.75 exponentials and 31 instructions a value; issue 2.15 a clock and SM, waits
// for shared memory, exchanges and loads in equal parts).  Two channels a lane take a tenth fewer
// instructions but leave half the warps: 10 to 25 % slower.  Warps of their own for the passes
// before and after the walk: 50 % slower.
#include "layer_ops.h"

#include <type_traits>

namespace kda {
namespace {

constexpr int kThreads = 128;   // of the small kernels
constexpr int kTile = SELSCAN_CHUNK;   // tokens of a forward tile; segments are whole tiles
constexpr int kNs = 8;          // state values a lane, forward
constexpr int kBack = SELSCAN_CHUNK;   // tokens of a backward tile
constexpr int kSub = 4;         // tokens whose states lie in registers, backward
constexpr int kParts = kBack / kSub;
constexpr int kSumTokens = 512;   // whose sums for the parameters are added up by themselves
static_assert(kTile == SELSCAN_CHUNK, "tiles hold whole chunks");

constexpr float kLn2 = 0.6931471805599453f;
// Decays 2^(D A log2 e).  The special-function unit cuts its argument off after 24 fractional
// bits, which by itself leaves decays near 1, of which a state multiplies hundreds, 1e-8 to
// 2.5e-8 too small on average; three quarters of half its last bit, added in the multiply-add
// that forms the argument, leave 1e-8 at most either way (measured over steps of 1e-6 to 0.5).  A
// rate of 0 still gives exactly 1: the addend itself is cut off.
constexpr float kNudge = 0x1.8p-26f;
__device__ __forceinline__ float decay(float step, float rate) {
    return ex2(fmaf(step, rate, kNudge));
}
// A log2 e, kept finite: a rate that the factor takes out of range (2.36e38 and more, such as the
// type's lowest value) would give NaN at a step of 0, which the rows around a short tile have too.
__device__ __forceinline__ float scaled_rate(float A) {
    float r;
    asm("{\n\t.reg .f32 t;\n\tmin.NaN.f32 t, %1, 0f7F7FFFFF;\n\tmax.NaN.f32 %0, t, 0fFF7FFFFF;\n\t}"
        : "=f"(r) : "f"(A * kLog2e));
    return r;
}
__device__ __forceinline__ F2 scaled_rate2(F2 A) {
    const float2 v = unpack2(A);
    return pack2(scaled_rate(v.x), scaled_rate(v.y));
}
__device__ __forceinline__ F2 decay2(F2 step, F2 rate) {
    const float2 v = unpack2(fma2(step, rate, pack2(kNudge, kNudge)));
    return pack2(ex2(v.x), ex2(v.y));
}

// ln(1 + e^v) = max(v, 0) + ln(1 + e), e = e^-|v|: ln(1 + e) / e on [0, 1] by a polynomial fitted
// for the least relative error (3e-8).  e is the step itself where that is small, so it must keep
// its relative precision: the exponent h = -|v| log2 e is off by half its last place, which for
// v = -7 is 3e-7 of e and grows with |v| (a step of 1e-3 was off by up to 5e-7, one of e^-70 by
// 3.5e-6).  What the rounding left out, r = -|v| - h ln 2 with ln 2 in two parts, goes back in as
// e (1 + r): the fused multiply-add forms it from the whole product (the error-free product of
// Ogita, Rump and Oishi).  Steps are within the exponential's 2^-22 and a few roundings.  Below
// 2^-126 they are 0; a NaN goes by the maximum.
constexpr int kLogTerms = 9;
__device__ __constant__ const float kLog1p[kLogTerms] = {
    9.999999404e-01f, -4.999949336e-01f, 3.331909776e-01f, -2.484298050e-01f, 1.910600215e-01f,
    -1.366323531e-01f, 7.822583616e-02f, -2.950516902e-02f, 5.232676864e-03f};
constexpr float kLn2Rest = -1.9046543e-09f;   // ln 2 - kLn2
__device__ __forceinline__ float positive_part(float v) {   // or NaN
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ F2 softplus2(F2 v) {
    const float2 u = unpack2(v);
    // (no further than where e is 0, so that r stays finite)
    const F2 w = pack2(fmaxf(-fabsf(u.x), -128.f), fmaxf(-fabsf(u.y), -128.f));
    const F2 h = mul2(w, both(kLog2e));
    const float2 hs = unpack2(h);
    F2 e = pack2(ex2(hs.x), ex2(hs.y));
    const F2 r = fma2(h, both(-kLn2Rest), fma2(h, both(-kLn2), w));
    e = fma2(e, r, e);
    F2 q = pack2(kLog1p[kLogTerms - 1], kLog1p[kLogTerms - 1]);
#pragma unroll
    for (int i = kLogTerms - 2; i >= 0; --i) q = fma2(q, e, pack2(kLog1p[i], kLog1p[i]));
    return fma2(q, e, pack2(positive_part(u.x), positive_part(u.y)));
}
__device__ __forceinline__ float softplus(float v) { return unpack2(softplus2(pack2(v, 0.f))).x; }

// How the work is cut: segments along the tokens (whole sequences when seg == 0) and blocks of
// channels, none of which spans two groups.
struct Cut {
    int64_t seg;        // tokens of a segment
    int64_t nseg;       // segments, or sequences
    int32_t per_group;  // channel blocks of a group
    int64_t items;      // nseg x blocks
};

// The sequence of `rank` in the order longest first (by number among equals): sequences of
// different lengths, each a CTA's, then end together, if none takes longer than its share.  All threads of the CTA call it; batches
// of more than kRanked sequences keep their order.
constexpr int kRanked = 128;
__device__ __forceinline__ int32_t ranked_sequence(const int32_t* cu, int32_t N, int32_t rank,
                                                   volatile int32_t* found) {
    if (N > kRanked || N < 2) return rank;
    for (int32_t i = threadIdx.x; i < N; i += blockDim.x) {
        const int32_t len = cu[i + 1] - cu[i];
        int32_t before = 0;
        for (int32_t j = 0; j < N; ++j) {
            const int32_t other = cu[j + 1] - cu[j];
            before += other > len || (other == len && j < i);
        }
        if (before == rank) *found = i;
    }
    __syncthreads();
    const int32_t n = *found;
    __syncthreads();
    return n;
}

// The maps of the segments, in the workspace.
struct Maps {
    float* sum;     // [nseg][D]      sum of the step sizes
    float* state;   // [nseg][D][n]   end state from zero; then, joined, the entry state
    int32_t* reset; // [nseg]         whether what comes before the segment stays in it
};

// Values k .. k + 7 of a state row of n.
__device__ __forceinline__ void load8(const float* p, int k, int n, float (&v)[kNs]) {
#pragma unroll
    for (int i = 0; i < kNs; ++i) v[i] = 0.f;
    if (!p) return;
    if (n % 4 == 0) {
#pragma unroll
        for (int i = 0; i < kNs; i += 4)
            if (k + i < n) {
                const float4 u = *reinterpret_cast<const float4*>(p + k + i);
                v[i] = u.x; v[i + 1] = u.y; v[i + 2] = u.z; v[i + 3] = u.w;
            }
    } else {
#pragma unroll
        for (int i = 0; i < kNs; ++i)
            if (k + i < n) v[i] = p[k + i];
    }
}
__device__ __forceinline__ void store8(float* p, int k, int n, const F2 (&h)[kNs / 2]) {
    float v[kNs];
#pragma unroll
    for (int i = 0; i < kNs / 2; ++i) {
        const float2 u = unpack2(h[i]);
        v[2 * i] = u.x;
        v[2 * i + 1] = u.y;
    }
    if (n % 4 == 0) {
#pragma unroll
        for (int i = 0; i < kNs; i += 4)
            if (k + i < n)
                *reinterpret_cast<float4*>(p + k + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < kNs; ++i)
            if (k + i < n) p[k + i] = v[i];
    }
}

// What a forward kernel does with the tokens: the outputs, the maps of the segments, or the
// maps of the gradients' recurrence (on reversed tokens).
enum { kOutputs = 0, kMaps = 1, kGradMaps = 2 };

// L lanes share a channel, 8 values each.  (Two channels a lane take fewer instructions, but leave
// too few warps to hide the latencies of a token: see the head of the file.)
template <int L>
struct Fwd {
    static constexpr int kThreads = L == 1 ? 64 : 128;
    static constexpr int kCh = kThreads / L;
    static constexpr int kNp = kNs * L;
    // Step size and what drives the state, of a pair of channels side by side: (D, u) of one, (D,
    // u) of the other; and their outputs.  Where a thread writes V channels at once, the pairs of
    // a row lie in the order of the threads (pair_slot), so that neither side meets bank conflicts.
    using Steps = float4[kTile][kCh / 2];
    using Outs = float2[kTile][kCh / 2];
    using Rows = float[kTile][kNp];      // of B or C
};
// Where the pair of channel c (even) lies in a row of CH channels written V at a time.
template <int CH, int V>
__device__ __forceinline__ int pair_slot(int c) {
    return V == 1 ? c / 2 : c % V / 2 * (CH / V) + c / V;
}
template <int CH, int V>
__device__ __forceinline__ int slot_channel(int s) {
    return V == 1 ? s * 2 : s % (CH / V) * V + s / (CH / V) * 2;
}

// One tile: tokens [a, a + cnt) of sequence n, whose first token is `start`; whether the walk
// goes on behind it, and whether the sequence ends with it.
struct Tile {
    int64_t a, start;
    int32_t cnt, n;
    bool ends;
};

template <typename T, int L, int V, int PASS>
__global__ void __launch_bounds__(Fwd<L>::kThreads, V == 1 ? 1 : 512 / Fwd<L>::kThreads)
scan_kernel(const ScanArgs p, const Cut cut, const Maps maps, int32_t* status) {
    using G = Fwd<L>;
    constexpr int CH = G::kCh, NP = G::kNp, TH = G::kThreads;
    constexpr int VR = CH / V;                          // vectors of a row
    constexpr int NI = (kTile * VR + TH - 1) / TH;      // of a tile, a thread
    constexpr int VB = 16 / sizeof(T);                  // values of B and C at once
    constexpr int NB = (2 * kTile * NP / VB + TH - 1) / TH;
    static_assert(TH % VR == 0, "a thread keeps its channels");
    // (objects of their own: a store to one does not hold up the loads from another)
    __shared__ __align__(16) typename G::Steps s_du[2];
    __shared__ __align__(16) typename G::Rows s_B[2], s_C[2];
    __shared__ __align__(16) typename G::Outs s_y[PASS == kOutputs ? 2 : 1];
    const int32_t* cu = p.cu_seqlens;
    if (!offsets_ok(cu, p.num_seqs, p.total_tokens, status)) return;
    const int tid = threadIdx.x, li = tid % L, slot = tid / L;
    const int ch = slot_channel<CH, V>(slot / 2) + slot % 2;   // my channel
    const int64_t D = (int64_t)p.H * p.d, last = cu[p.num_seqs];
    const T* const X = static_cast<const T*>(PASS == kGradMaps ? p.dy : p.in.x);
    const int64_t ldx = PASS == kGradMaps ? D : p.in.ldx;
    const T* const DT = static_cast<const T*>(p.in.dt);
    const T* const Z = static_cast<const T*>(PASS == kMaps ? nullptr : p.in.z);
    const bool packed = p.n % VB == 0 && p.in.ldB % VB == 0 && p.in.ldC % VB == 0 &&
                        ((uint64_t)p.in.B | (uint64_t)p.in.C) % 16 == 0;

    for (int64_t item = blockIdx.x; item < cut.items; item += gridDim.x) {
        const int64_t blocks = (int64_t)cut.per_group * p.H;
        const int64_t sg = item / blocks;
        const int32_t cb = (int32_t)(item - sg * blocks);
        const int32_t g = cb / cut.per_group;
        const int32_t c0 = (cb - g * cut.per_group) * CH;          // first channel in the group
        const int32_t width = p.d - c0 < CH ? p.d - c0 : CH;
        const int64_t base = (int64_t)g * p.d + c0;                // and of all

        int64_t t0, t1;   // tokens to walk
        int32_t n;
        bool reset = false;
        if (cut.seg == 0) {
            n = ranked_sequence(cu, p.num_seqs, (int32_t)sg, reinterpret_cast<int32_t*>(s_du));
            t0 = cu[n];
            t1 = cu[n + 1];
        } else {
            t0 = sg * cut.seg;
            t1 = t0 + cut.seg < last ? t0 + cut.seg : last;
            if (t0 >= t1) continue;
            if (PASS == kMaps) {
                n = sequence_of(cu, p.num_seqs, t1 - 1);
                reset = cu[n] >= t0;
                if (reset) t0 = cu[n];
            } else if (PASS == kGradMaps) {
                n = sequence_of(cu, p.num_seqs, t0);
                reset = cu[n + 1] <= t1;
                if (reset) t1 = cu[n + 1];
            } else {
                n = sequence_of(cu, p.num_seqs, t0);
            }
        }

        F2 A[kNs / 2], h[kNs / 2];
        const bool on = ch < width;
        const int64_t my_state = (base + ch) * p.n;
        auto load_state = [&](const float* from, F2 (&to)[kNs / 2]) {
            float v[kNs];
            load8(from && on ? from + my_state : nullptr, li * kNs, p.n, v);
#pragma unroll
            for (int i = 0; i < kNs / 2; ++i) to[i] = pack2(v[2 * i], v[2 * i + 1]);
        };
        auto store_state = [&](float* to) {
            if (on) store8(to + my_state, li * kNs, p.n, h);
        };
        auto first_state = [&](int32_t m) { load_state(p.S0 ? p.S0 + m * D * p.n : nullptr, h); };
        load_state(p.A, A);
#pragma unroll
        for (int i = 0; i < kNs / 2; ++i) A[i] = scaled_rate2(A[i]);
        if (PASS == kGradMaps)
            load_state(reset && p.dS_T ? p.dS_T + n * D * p.n : nullptr, h);
        else if (t0 == cu[n])
            first_state(n);
        else
            load_state(PASS == kOutputs ? maps.state + sg * D * p.n : nullptr, h);
        if (PASS == kOutputs && t0 >= t1) {   // an empty sequence
            if (p.S_T) store_state(p.S_T + n * D * p.n);
            continue;
        }
        float sum = 0.f;   // of the step sizes

        // the tile that holds token t (reversed: that ends before t) of sequence m
        auto tile_at = [&](int64_t t, int32_t m) {
            Tile k;
            k.n = m;
            k.start = cu[m];
            int64_t b;
            if (PASS == kGradMaps) {
                b = t;
                k.a = (t - 1) / kTile * kTile;
                if (k.a < t0) k.a = t0;
                k.ends = false;
            } else {
                const int64_t end = cu[m + 1];
                k.a = t;
                b = t / kTile * kTile + kTile;
                if (b > t1) b = t1;
                if (b > end) b = end;
                k.ends = b == end;
            }
            k.cnt = (int32_t)(b - k.a);
            return k;
        };
        auto has_next = [&](const Tile& k) {
            return PASS == kGradMaps ? k.a > t0 : k.a + k.cnt < t1;
        };
        auto next_of = [&](const Tile& k) {
            if (PASS == kGradMaps) return tile_at(k.a, k.n);
            int32_t m = k.n;
            const int64_t t = k.a + k.cnt;
            if (PASS == kOutputs && k.ends)
                while (cu[m + 1] <= t) ++m;
            return tile_at(t, m);
        };

        // my vectors of a tile: row row_of(i), V channels from my_c on
        const int my_c = tid % VR * V;
        const bool in_row = my_c < width;
        auto row_of = [&](int i) { return (tid + i * TH) / VR; };
        float bias[V], skip[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            bias[k] = in_row && p.dt_bias ? p.dt_bias[base + my_c + k] : 0.f;
            skip[k] = in_row && p.skip && PASS == kOutputs ? p.skip[base + my_c + k] : 0.f;
        }
        Pack<T, V> rx[NI], rd[NI], rz[NI], kx[NI], kz[NI];
        Pack<T, VB> rb[NB];
        auto fetch = [&](const Tile& k) {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int r = row_of(i);
                if (r < k.cnt && in_row) {
                    rx[i].load(X + (k.a + r) * ldx + base + my_c);
                    rd[i].load(DT + (k.a + r) * p.in.lddt + base + my_c);
                    if (Z) rz[i].load(Z + (k.a + r) * p.in.ldz + base + my_c);
                }
            }
        };
        // vector i of the tile's B and C: which of the two, its row and first value
        auto bc_of = [&](int i, int& row, int& at) {
            const int v = tid + i * TH;
            row = v % (kTile * NP / VB) / (NP / VB);
            at = v % (NP / VB) * VB;
            return v / (kTile * NP / VB);
        };
        auto fetch_bc = [&](const Tile& k) {
            if (!packed) return;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                int r, at;
                const int which = bc_of(i, r, at);
                rb[i].zero();
                if (which < 2 && r < k.cnt && at < p.n && !(PASS == kMaps && which == 1) &&
                    !(PASS == kGradMaps && which == 0))
                    rb[i].load(static_cast<const T*>(which ? p.in.C : p.in.B) +
                               (k.a + r) * (which ? p.in.ldC : p.in.ldB) + (int64_t)g * p.n + at);
            }
        };
        // what the tile's tokens drive the states with, into s
        auto convert = [&](const Tile& k, int side) {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int r = row_of(i);
                if (r >= k.cnt || !in_row) continue;
                if constexpr (V == 1) {
                    float v = rd[i].get(0) + bias[0];
                    if (p.softplus) v = softplus(v);
                    float u = rx[i].get(0);
                    if (PASS == kGradMaps) u = Z ? u * silu(rz[i].get(0)) : u;
                    else u *= v;
                    reinterpret_cast<float2*>(s_du[side][r])[my_c] = make_float2(v, u);
                } else {
#pragma unroll
                    for (int q = 0; q < V; q += 2) {
                        F2 v = pack2(rd[i].get(q) + bias[q], rd[i].get(q + 1) + bias[q + 1]);
                        if (p.softplus) v = softplus2(v);
                        float2 u = make_float2(rx[i].get(q), rx[i].get(q + 1));
                        if (PASS == kGradMaps) {
                            if (Z) {
                                u.x *= silu(rz[i].get(q));
                                u.y *= silu(rz[i].get(q + 1));
                            }
                        } else {
                            u = unpack2(mul2(v, pack2(u.x, u.y)));
                        }
                        const float2 w = unpack2(v);
                        s_du[side][r][q / 2 * VR + my_c / V] = make_float4(w.x, u.x, w.y, u.y);
                    }
                }
            }
            if (packed) {
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    int r, at;
                    const int which = bc_of(i, r, at);
                    if (which > 1) continue;
                    float* to = which ? &s_C[side][r][at] : &s_B[side][r][at];
#pragma unroll
                    for (int q = 0; q < VB; q += 4)
                        *reinterpret_cast<float4*>(to + q) = make_float4(
                            rb[i].get(q), rb[i].get(q + 1), rb[i].get(q + 2), rb[i].get(q + 3));
                }
            } else {
                for (int i = tid; i < kTile * NP; i += TH) {
                    const int r = i / NP, q = i % NP;
                    float bv = 0.f, cv = 0.f;
                    if (r < k.cnt && q < p.n) {
                        if (PASS != kGradMaps)
                            bv = Elem<T>::load(static_cast<const T*>(p.in.B) +
                                               (k.a + r) * p.in.ldB + (int64_t)g * p.n + q);
                        if (PASS != kMaps)
                            cv = Elem<T>::load(static_cast<const T*>(p.in.C) +
                                               (k.a + r) * p.in.ldC + (int64_t)g * p.n + q);
                    }
                    s_B[side][r][q] = bv;
                    s_C[side][r][q] = cv;
                }
            }
        };
        // The decays of a token are formed one token ahead: the special-function unit and the
        // multiply-adds then work on different tokens.
        struct Step {
            float2 du;
            F2 a[kNs / 2];
        };
        auto step_of = [&](int side, int r) {
            Step t;
            t.du = reinterpret_cast<const float2*>(s_du[side][r])[slot];
            const F2 dd = pack2(t.du.x, t.du.x);
#pragma unroll
            for (int k = 0; k < kNs / 2; ++k) t.a[k] = decay2(dd, A[k]);
            return t;
        };
        // one token: row r
        auto token = [&](const Step& t, int side, int r) {
            const ulonglong2* Bp = reinterpret_cast<const ulonglong2*>(&s_B[side][r][li * kNs]);
            const ulonglong2* Cp = reinterpret_cast<const ulonglong2*>(&s_C[side][r][li * kNs]);
            if (PASS != kOutputs) sum += t.du.x;
            F2 y = 0;
            const F2 uu = pack2(t.du.y, t.du.y);
#pragma unroll
            for (int i = 0; i < kNs / 4; ++i) {
                ulonglong2 bv = {}, cv = {};
                if (PASS != kGradMaps) bv = Bp[i];
                if (PASS != kMaps) cv = Cp[i];
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    const int k = 2 * i + o;
                    if (PASS == kGradMaps) {
                        h[k] = mul2(t.a[k], fma2(uu, o ? cv.y : cv.x, h[k]));
                    } else {
                        h[k] = fma2(t.a[k], h[k], mul2(uu, o ? bv.y : bv.x));
                        if (PASS == kOutputs) y = fma2(h[k], o ? cv.y : cv.x, y);
                    }
                }
            }
            if (PASS == kOutputs) {
                float v = sum2(y);
#pragma unroll
                for (int o = 1; o < L; o *= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (li == 0) reinterpret_cast<float*>(s_y[side][r])[slot] = v;
            }
        };
        // the outputs of a tile whose sums are there
        auto finish = [&](const Tile& k, int side) {
            if (!p.y) return;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int r = row_of(i);
                if (r >= k.cnt || !in_row) continue;
                float o[V];
                if constexpr (V == 1) {
                    o[0] = fmaf(skip[0], kx[i].get(0), reinterpret_cast<const float*>(s_y[side][r])[my_c]);
                    if (Z) o[0] *= silu(kz[i].get(0));
                } else {
#pragma unroll
                    for (int q = 0; q < V; q += 2) {
                        const float2 v = s_y[side][r][q / 2 * VR + my_c / V];
                        o[q] = fmaf(skip[q], kx[i].get(q), v.x);
                        o[q + 1] = fmaf(skip[q + 1], kx[i].get(q + 1), v.y);
                        if (Z) {
                            o[q] *= silu(kz[i].get(q));
                            o[q + 1] *= silu(kz[i].get(q + 1));
                        }
                    }
                }
                Pack<T, V> ky;
                ky.set(o);
                ky.store(static_cast<T*>(p.y) + (k.a + r) * D + base + my_c);
            }
        };

        Tile now = tile_at(PASS == kGradMaps ? t1 : t0, n), before = now;
        fetch(now);
        fetch_bc(now);
        convert(now, 0);
        int side = 0;
        bool first = true;
        while (true) {
            // One barrier a tile: behind it this tile's buffer is written, the other's sums are
            // done, and the next tile's may go where those have been read.
            __syncthreads();
            if constexpr (PASS == kOutputs)
                if (!first) finish(before, side ^ 1);
            first = false;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                kx[i] = rx[i];
                kz[i] = rz[i];
            }
            const bool more = has_next(now);
            Tile next = now;
            if (more) {
                next = next_of(now);
                fetch(next);
                fetch_bc(next);
            }
            if (PASS == kOutputs && p.states && now.a % SELSCAN_CHUNK == 0 && now.a > now.start)
                store_state(p.states + now.a / SELSCAN_CHUNK * D * p.n);
            if (now.cnt == kTile) {   // every place known at compile time
                Step t = step_of(side, PASS == kGradMaps ? kTile - 1 : 0);
#pragma unroll
                for (int j = 0; j < kTile; ++j) {
                    Step ahead = t;
                    if (j + 1 < kTile) ahead = step_of(side, PASS == kGradMaps ? kTile - 2 - j : j + 1);
                    token(t, side, PASS == kGradMaps ? kTile - 1 - j : j);
                    t = ahead;
                }
            } else {
#pragma unroll 1
                for (int j = 0; j < now.cnt; ++j) {
                    const int r = PASS == kGradMaps ? now.cnt - 1 - j : j;
                    token(step_of(side, r), side, r);
                }
            }
            if (PASS == kOutputs && now.ends) {
                if (p.S_T) store_state(p.S_T + now.n * D * p.n);
                if (more) first_state(next.n);
            }
            before = now;
            if (!more) break;
            convert(next, side ^ 1);
            now = next;
            side ^= 1;
        }
        __syncthreads();
        if constexpr (PASS == kOutputs) finish(before, side);
        if (PASS != kOutputs) {
            store_state(maps.state + sg * D * p.n);
            if (li == 0 && on) maps.sum[sg * D + base + ch] = sum;
            if (cb == 0 && tid == 0) maps.reset[sg] = reset;
        }
        __syncthreads();
    }
}

// Joins the segments' maps: state[s] becomes the state that enters segment s (reversed: that
// reaches it from behind).
constexpr int kJoin = 16;   // segments loaded at once
constexpr int kJoinEmpty = 64;   // sequences among which the join looks for empty ones
__global__ void __launch_bounds__(kThreads)
join_kernel(const ScanArgs p, const Cut cut, const Maps maps, bool reversed, const float* in,
            float* out, const int32_t* status) {
    if (*status != KDA_OK) return;
    const int64_t D = (int64_t)p.H * p.d, i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= D * p.n) return;
    // out[n] = in[n] (or zeros) for the empty sequences, which no segment holds
    for (int32_t n = 0; out && p.num_seqs <= kJoinEmpty && n < p.num_seqs; ++n)
        if (p.cu_seqlens[n] == p.cu_seqlens[n + 1])
            out[n * D * p.n + i] = in ? in[n * D * p.n + i] : 0.f;
    const int64_t last = p.cu_seqlens[p.num_seqs], segs = (last + cut.seg - 1) / cut.seg;
    const int64_t c = i / p.n;
    const float A = scaled_rate(p.A[i]);
    float h = 0.f;
    for (int64_t s0 = 0; s0 < segs; s0 += kJoin) {
        float e[kJoin], d[kJoin];
        bool r[kJoin];
#pragma unroll
        for (int k = 0; k < kJoin; ++k) {
            const int64_t s = reversed ? segs - 1 - (s0 + k) : s0 + k;
            if (s0 + k < segs) {
                e[k] = maps.state[s * D * p.n + i];
                d[k] = maps.sum[s * D + c];
                r[k] = maps.reset[s] != 0;
            }
        }
#pragma unroll
        for (int k = 0; k < kJoin; ++k) {
            const int64_t s = reversed ? segs - 1 - (s0 + k) : s0 + k;
            if (s0 + k < segs) {
                maps.state[s * D * p.n + i] = h;
                h = r[k] ? e[k] : fmaf(decay(d[k], A), h, e[k]);
            }
        }
    }
}

// The same for more sequences than that.
__global__ void __launch_bounds__(kThreads)
empty_kernel(const int32_t* cu, int32_t N, int64_t row, const float* in, float* out,
             const int32_t* status) {
    if (*status != KDA_OK) return;
    for (int64_t n = blockIdx.x; n < N; n += gridDim.x) {
        if (cu[n] != cu[n + 1]) continue;
        for (int64_t i = threadIdx.x; i < row; i += kThreads)
            out[n * row + i] = in ? in[n * row + i] : 0.f;
    }
}

// ---------------------------------------------------------------- backward

// A segment's sums for dA, dskip and ddt_bias, whole vectors long.
__host__ __device__ inline int64_t part_row(int64_t D, int32_t n) { return (D * (n + 2) + 3) / 4 * 4; }

// NL lanes share two channels, four values of each a lane.
template <int NL>
struct Back {
    static constexpr int kThreads = 128;
    static constexpr int kWarps = kThreads / 32;
    static constexpr int kCh = kThreads / NL * 2;
    static constexpr int kNp = 4 * NL;
    static constexpr int kPart = 2 * kNp * kSub > 256 ? 2 * kNp * kSub : 256;
    // Channels lie in the order of the threads that write them, V at a time; step and
    // u twice over, as the packed instructions take them.
    struct Shared {
        float4 du[kBack][kCh];               // D, D, D x, D x
        float dr[kBack][kCh];                // dy silu(z)
        F2 A[4][kThreads];                   // each thread's rates: they would not fit its registers
        float B[kBack][kNp], C[kBack][kNp];
        float y[kBack][kCh];                 // C . h
        float s[2][kBack][kCh];              // B . g and A . (g a h)
        // A warp's states before the tile's parts, a place a lane; and, where a part's have been
        // used, dB and dC of its tokens over the warp's channels.
        float part[kWarps][kParts][kPart];
        float acc[2][kWarps][kCh];           // sums for dskip and ddt_bias
    };
};
// The place of a slot in the rows of single values: turned by `by` (its low two bits) times eight
// places, by the row, so that lanes that hold four rows, and (by the value) four values of one
// row, meet four different quarters of the banks.  (Within a half of the row: the halves hold a
// thread's two channels, which are turned differently.)
template <int CH>
__device__ __forceinline__ int place_of(int by, int slot) {
    return slot ^ ((by & 3) * 8 & (CH / 2 - 1));
}

// U channels' values of a parameter that may be absent.
template <int U>
__device__ __forceinline__ Pack<float, U> channels(const float* p, int32_t at) {
    Pack<float, U> k;
    if (p) k.load(p + at);
    else k.zero();
    return k;
}

// Sums v[0..N) over the lanes that differ in the bits LO .. HI (powers of two): each exchange
// halves the values a lane carries, down to one, and adds it up from there on.  Returns the index of
// v[0] among the N; the others that are left follow it.
template <int N, int HI, int LO>
__device__ __forceinline__ int spread_sum(float (&v)[N], int lane) {
    int at = 0;
#pragma unroll
    for (int o = HI, nv = N; o >= LO; o >>= 1) {
        if (nv > 1) {
            nv /= 2;
            const bool upper = lane & o;
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                if (i < nv) {
                    const float give = upper ? v[i] : v[i + nv];
                    v[i] = (upper ? v[i + nv] : v[i]) + __shfl_xor_sync(0xffffffffu, give, o);
                }
            at += upper ? nv : 0;
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        }
    }
    return at;
}
// How many are left.
constexpr int spread_left(int n, int hi, int lo) {
    for (int o = hi; o >= lo && n > 1; o >>= 1) n /= 2;
    return n;
}

template <typename T, int NL, int V>
__global__ void __launch_bounds__(Back<NL>::kThreads, V == 1 ? 1 : 4)
scan_bwd_kernel(const ScanArgs p, const Cut cut, const Maps maps, float* part, float* part_BC,
                const int32_t* status) {
    using G = Back<NL>;
    constexpr int CH = G::kCh, TH = G::kThreads, NP = G::kNp;
    constexpr int VR = CH / V;                              // vectors of a row
    constexpr int NI = (kBack * VR + TH - 1) / TH;          // of a tile, a thread
    constexpr int VB = 16 / sizeof(T);                      // values of B and C at once
    extern __shared__ __align__(16) char raw[];
    typename G::Shared& s = *reinterpret_cast<typename G::Shared*>(raw);
    if (*status != KDA_OK) return;
    const int32_t* cu = p.cu_seqlens;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nl = lane % NL, slot = tid / NL;   // my values; my channels' slots: this and
    constexpr int kOther = CH / 2;               // that one behind it
    // (tokens and channels are counted in 32 bits, places in memory in 64)
    const int32_t D = p.H * p.d;
    const int64_t Dn = (int64_t)D * p.n;
    const T* const X = static_cast<const T*>(p.in.x);
    const T* const DT = static_cast<const T*>(p.in.dt);
    const T* const Z = static_cast<const T*>(p.in.z);
    const T* const DY = static_cast<const T*>(p.dy);
    const bool packed = p.n % VB == 0 && p.in.ldB % VB == 0 && p.in.ldC % VB == 0 &&
                        ((uint64_t)p.in.B | (uint64_t)p.in.C) % 16 == 0;
    const int my[2] = {slot % VR * V + slot / VR, (slot + kOther) % VR * V + (slot + kOther) / VR};

    for (int64_t item = blockIdx.x; item < cut.items; item += gridDim.x) {
        const int32_t blocks = cut.per_group * p.H;
        const int32_t sg = (int32_t)(item / blocks);
        const int32_t cb = (int32_t)(item - (int64_t)sg * blocks);
        const int32_t g = cb / cut.per_group, cg = cb - g * cut.per_group;
        const int32_t c0 = cg * CH;
        const int32_t width = p.d - c0 < CH ? p.d - c0 : CH;
        const int32_t base = g * p.d + c0;
        int32_t t0, t1;
        int32_t n;
        if (cut.seg == 0) {
            n = ranked_sequence(cu, p.num_seqs, sg, reinterpret_cast<int32_t*>(&s.part));
            t0 = cu[n];
            t1 = cu[n + 1];
        } else {
            const int32_t last = cu[p.num_seqs];
            const int64_t from = sg * cut.seg, to = from + cut.seg;
            t0 = (int32_t)(from < last ? from : last);
            t1 = (int32_t)(to < last ? to : last);
            n = t0 < t1 ? sequence_of(cu, p.num_seqs, t1 - 1) : 0;
        }
        // four values of my two channels in a [..][D][n] tensor
        auto load4 = [&](const float* from, F2 (&v)[2][2]) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float u[4] = {0.f, 0.f, 0.f, 0.f};
                if (from && my[q] < width) {
                    const float* r = from + ((base + my[q]) * p.n + nl * 4);
                    if (p.n % 4 == 0) {
                        if (nl * 4 < p.n) {
                            const float4 w = *reinterpret_cast<const float4*>(r);
                            u[0] = w.x; u[1] = w.y; u[2] = w.z; u[3] = w.w;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (nl * 4 + i < p.n) u[i] = r[i];
                    }
                }
                v[q][0] = pack2(u[0], u[1]);
                v[q][1] = pack2(u[2], u[3]);
            }
        };
        auto store4 = [&](float* to, const F2 (&v)[2][2]) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (my[q] >= width) continue;
                float* r = to + ((base + my[q]) * p.n + nl * 4);
                const float2 lo = unpack2(v[q][0]), hi = unpack2(v[q][1]);
                const float u[4] = {lo.x, lo.y, hi.x, hi.y};
                if (p.n % 4 == 0) {
                    if (nl * 4 < p.n)
                        *reinterpret_cast<float4*>(r) = make_float4(u[0], u[1], u[2], u[3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (nl * 4 + i < p.n) r[i] = u[i];
                }
            }
        };
        F2 dA[2][2], r[2][2];   // gradients of the rates, the gradient from behind
        load4(p.A, dA);
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                s.A[q * 2 + i][tid] = scaled_rate2(dA[q][i]);
                dA[q][i] = 0;
            }
        const float* behind = nullptr;
        if (t0 < t1 && t1 != cu[n + 1]) behind = maps.state + sg * Dn;
        else if (p.dS_T && (t0 < t1 || cut.seg == 0)) behind = p.dS_T + n * Dn;
        load4(behind, r);
        for (int i = tid; i < 2 * G::kWarps * CH; i += TH) (&s.acc[0][0][0])[i] = 0.f;
        // The sums for dA, dskip and ddt_bias of at most kSumTokens tokens lie in registers and s.acc,
        // those of the item in its row of `part`: a sequence of any length then loses no more to
        // roundings than kSumTokens of its tokens and as many sums do.
        float* const sums = part + sg * part_row(D, p.n);
        store4(sums, dA);
        auto each_acc = [&](auto&& f) {   // (a column is the same thread's each time)
            for (int i = tid; i < 2 * CH; i += TH) {
                const int which = i / CH, sl = i % CH, c = sl % VR * V + sl / VR;
                if (c < width) f(sums[Dn + (int64_t)which * D + base + c], which, sl);
            }
        };
        each_acc([&](float& to, int, int) { to = 0.f; });
        auto add_sums = [&]() {
            F2 at[2][2];
            load4(sums, at);
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    at[q][i] = add2(at[q][i], dA[q][i]);
                    dA[q][i] = 0;
                }
            store4(sums, at);
            __syncthreads();
            each_acc([&](float& to, int which, int sl) {   // the warps, in order
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < G::kWarps; ++w) {
                    sum += s.acc[which][w][sl];
                    s.acc[which][w][sl] = 0.f;
                }
                to += sum;
            });
        };
        if (cut.seg == 0 && t0 >= t1 && p.g.dS0) store4(p.g.dS0 + n * Dn, r);

        // my vectors of a tile: V channels of a row
        auto row_of = [&](int i) { return (tid + i * TH) / VR; };
        auto col_of = [&](int i) { return (tid + i * TH) % VR * V; };
        // Inputs of tokens [a, a + cnt), to shared memory, each to its row of the grid of tiles.  The
        // rows around them get steps and inputs of zero, which leave the state, the gradient from
        // behind and the rates' sums as they are.
        auto convert = [&](int32_t a0, int cnt0) {
            const int32_t a = a0 / kBack * kBack;
            const int first = a0 - a, cnt = first + cnt0;   // rows [first, cnt)
            // (single values all at once, vectors one after the other: more do not fit)
            constexpr int kOnce = V == 1 ? NI : 1;
            Pack<T, V> kx[kOnce], kd[kOnce], kg[kOnce], kz[kOnce];
            auto load = [&](int i, int j) {
                const int k = row_of(i), c = col_of(i);
                const int64_t t = a + k;
                if (k < first || k >= cnt || c >= width) return;
                kx[j].load(X + t * p.in.ldx + base + c);
                kd[j].load(DT + t * p.in.lddt + base + c);
                kg[j].load(DY + t * D + base + c);
                if (Z) kz[j].load(Z + t * p.in.ldz + base + c);
            };
            if constexpr (V == 1) {
#pragma unroll
                for (int i = 0; i < NI; ++i) load(i, i);
            }
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                constexpr bool kLoaded = V == 1;
                const int k = row_of(i), c = col_of(i), j = kLoaded ? i : 0;
                if (k >= kBack) continue;
                if (k < first || k >= cnt || c >= width) {
#pragma unroll
                    for (int q = 0; q < V; ++q) {
                        s.du[k][q * VR + c / V] = make_float4(0.f, 0.f, 0.f, 0.f);
                        s.dr[k][place_of<CH>(k, q * VR + c / V)] = 0.f;
                    }
                    continue;
                }
                if (!kLoaded) load(i, 0);
                constexpr int U = V < 4 ? V : 4;
#pragma unroll
                for (int q0 = 0; q0 < V; q0 += U) {
                    const Pack<float, U> bias = channels<U>(p.dt_bias, base + c + q0);
#pragma unroll
                    for (int q = q0; q < q0 + U; q += 2) {   // in pairs, single ones in the low half
                        constexpr int o = V > 1 ? 1 : 0;
                        F2 v = add2(pack2(kd[j].get(q), kd[j].get(q + o)),
                                    pack2(bias.get(q - q0), bias.get(q - q0 + o)));
                        if (p.softplus) v = softplus2(v);
                        const float2 u = unpack2(mul2(v, pack2(kx[j].get(q), kx[j].get(q + o))));
                        F2 d = pack2(kg[j].get(q), kg[j].get(q + o));
                        if (Z) d = mul2(d, silu2(pack2(kz[j].get(q), kz[j].get(q + o))));
                        const float2 st = unpack2(v), dr = unpack2(d);
                        s.du[k][q * VR + c / V] = make_float4(st.x, st.x, u.x, u.x);
                        s.dr[k][place_of<CH>(k, q * VR + c / V)] = dr.x;
                        if (V > 1) {
                            s.du[k][(q + o) * VR + c / V] = make_float4(st.y, st.y, u.y, u.y);
                            s.dr[k][place_of<CH>(k, (q + o) * VR + c / V)] = dr.y;
                        }
                    }
                }
            }
            if (packed) {
                for (int i = tid; i < 2 * kBack * NP / VB; i += TH) {
                    const int which = i / (kBack * NP / VB), j = i % (kBack * NP / VB);
                    const int k = j / (NP / VB), at = j % (NP / VB) * VB;
                    Pack<T, VB> b;
                    b.zero();
                    if (k >= first && k < cnt && at < p.n)
                        b.load(static_cast<const T*>(which ? p.in.C : p.in.B) +
                               (a + k) * (which ? p.in.ldC : p.in.ldB) + (int64_t)g * p.n + at);
                    float* to = which ? &s.C[k][at] : &s.B[k][at];
#pragma unroll
                    for (int q = 0; q < VB; q += 4)
                        *reinterpret_cast<float4*>(to + q) =
                            make_float4(b.get(q), b.get(q + 1), b.get(q + 2), b.get(q + 3));
                }
            } else {
                for (int i = tid; i < kBack * NP; i += TH) {
                    const int k = i / NP, j = i % NP;
                    const bool in = k >= first && k < cnt && j < p.n;
                    s.B[k][j] = in ? Elem<T>::load(static_cast<const T*>(p.in.B) +
                                                   (a + k) * p.in.ldB + (int64_t)g * p.n + j) : 0.f;
                    s.C[k][j] = in ? Elem<T>::load(static_cast<const T*>(p.in.C) +
                                                   (a + k) * p.in.ldC + (int64_t)g * p.n + j) : 0.f;
                }
            }
        };
        // the gradients of tokens [a, a + cnt), whose sums are in shared memory
        auto finish = [&](int32_t a0, int cnt0) {
            const int32_t a = a0 / kBack * kBack;
            const int from = a0 - a, cnt = from + cnt0;   // rows [from, cnt)
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int k = row_of(i), c = col_of(i);
                const bool in = k >= from && k < cnt && c < width;
                const int64_t t = a + k, at = t * D + base + c;
                Pack<T, V> kx, kd, kg, kz;
                if (in) {
                    kx.load(X + t * p.in.ldx + base + c);
                    kd.load(DT + t * p.in.lddt + base + c);
                    if (Z) {
                        kz.load(Z + t * p.in.ldz + base + c);
                        kg.load(DY + at);
                    }
                }
                constexpr int U = V < 4 ? V : 4, R = VR < 32 ? VR : 32;   // lanes of a row
#pragma unroll
                for (int q0 = 0; q0 < V; q0 += U) {
                    float acc[2 * U] = {};   // for dskip, for ddt_bias
                    if (in) {
                        const Pack<float, U> bias = channels<U>(p.dt_bias, base + c + q0);
                        const Pack<float, U> skips = channels<U>(p.skip, base + c + q0);
                        // slopes of the step and of the gate, in pairs
                        float slope[U], dz[U];
#pragma unroll
                        for (int j = 0; j < U; j += 2) {
                            constexpr int o = U > 1 ? 1 : 0;
                            const int q = q0 + j;
                            if (p.softplus) {
                                const float2 t = unpack2(sigmoid2(
                                    add2(pack2(kd.get(q), kd.get(q + o)),
                                         pack2(bias.get(j), bias.get(j + o)))));
                                slope[j] = t.x;
                                if (U > 1) slope[j + o] = t.y;
                            } else {
                                slope[j] = slope[j + o] = 1.f;
                            }
                            if (Z) {
                                const float2 t = unpack2(
                                    mul2(pack2(kg.get(q), kg.get(q + o)),
                                         silu_grad2(pack2(kz.get(q), kz.get(q + o)))));
                                dz[j] = t.x;
                                if (U > 1) dz[j + o] = t.y;
                            }
                        }
                        float dx[U];
#pragma unroll
                        for (int j = 0; j < U; ++j) {
                            const int q = q0 + j, sl = q * VR + c / V;
                            const float skip = skips.get(j);
                            const int at1 = place_of<CH>(k ^ sl / kOther, sl), at0 = place_of<CH>(k, sl);
                            const float x = kx.get(q), s1 = s.s[0][k][at1], dr = s.dr[k][at0];
                            acc[j] = dr * x;
                            acc[U + j] = slope[j] *
                                fmaf(x, s1, s.s[1][k][place_of<CH>(k ^ (2 + sl / kOther), sl)] * kLn2);
                            dx[j] = fmaf(s.du[k][sl].x, s1, skip * dr);
                            if (Z) dz[j] *= fmaf(skip, x, s.y[k][at1]);
                        }
                        Pack<float, U> o;
                        o.set(dx);
                        o.store(p.g.dx + at + q0);
#pragma unroll
                        for (int j = 0; j < U; ++j) dx[j] = acc[U + j];
                        o.set(dx);
                        o.store(p.g.ddt + at + q0);
                        if (Z) {
                            o.set(dz);
                            o.store(p.g.dz + at + q0);
                        }
                    }
                    // the rows of my warp, then the tiles before
                    const int first = spread_sum<2 * U, 16, R>(acc, lane);
                    constexpr int kLeftU = spread_left(2 * U, 16, R);
                    constexpr int kSame = 32 / R / (2 * U / kLeftU);   // lanes with the same sum
                    if (kSame <= 1 || lane / R % (kSame > 0 ? kSame : 1) == 0) {
#pragma unroll
                        for (int q = 0; q < kLeftU; ++q) {
                            const int j = first + q;
                            s.acc[j / U][warp][(q0 + j % U) * VR + c / V] += acc[q];
                        }
                    }
                }
            }
            // sums over the CTA's channels: to the outputs if it has the whole group
            for (int i = from * NP / 2 + tid; i < cnt * NP / 2; i += TH) {
                const int k = i / (NP / 2), j = i % (NP / 2) * 4, st = j % NP;
                if (st >= p.n) continue;
                const int at = k % kSub * 2 * NP + j;
                float4 v = *reinterpret_cast<const float4*>(&s.part[0][k / kSub][at]);
#pragma unroll
                for (int w = 1; w < G::kWarps; ++w) {
                    const float4 u = *reinterpret_cast<const float4*>(&s.part[w][k / kSub][at]);
                    v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
                }
                const int64_t row = (int64_t)(a + k) * p.H + g;
                float* to = cut.per_group == 1
                                ? (j < NP ? p.g.dB : p.g.dC) + row * p.n + st
                                : part_BC + ((int64_t)cg * p.total_tokens * p.H + row) * 2 * p.n +
                                      (j < NP ? 0 : p.n) + st;
                if (p.n % 4 == 0) {
                    *reinterpret_cast<float4*>(to) = v;
                } else {
                    const float u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (st + q < p.n) to[q] = u[q];
                }
            }
        };

        struct Inputs {
            F2 dd[2], uu[2];
        };
        auto inputs = [&](int k) {
            Inputs v;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const ulonglong2 u =
                    *reinterpret_cast<const ulonglong2*>(&s.du[k][slot + q * kOther]);
                v.dd[q] = u.x;
                v.uu[q] = u.y;
            }
            return v;
        };
        auto row4 = [&](const float (&m)[kBack][NP], int k) {
            return *reinterpret_cast<const ulonglong2*>(&m[k][nl * 4]);
        };
        struct Rates {
            F2 v[2][2];
        };
        auto rates = [&]() {
            Rates A;
#pragma unroll
            for (int i = 0; i < 4; ++i) A.v[i / 2][i % 2] = s.A[i][tid];
            return A;
        };
        auto advance = [&](const Rates& A, int k, F2 (&h)[2][2]) {
            const Inputs v = inputs(k);
            const ulonglong2 b = row4(s.B, k);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                h[q][0] = fma2(decay2(v.dd[q], A.v[q][0]), h[q][0], mul2(v.uu[q], b.x));
                h[q][1] = fma2(decay2(v.dd[q], A.v[q][1]), h[q][1], mul2(v.uu[q], b.y));
            }
        };
        // A part, rows from `from` on, from state h: rebuilt, then backward.
        auto sub = [&](int from, F2 (&h)[2][2], float* sums) {
            asm volatile("" ::: "memory");
            const Rates A = rates();
            F2 before[kSub][2][2];
#pragma unroll
            for (int j = 0; j < kSub; ++j) {
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int i = 0; i < 2; ++i) before[j][q][i] = h[q][i];
                advance(A, from + j, h);
                if (Z) {
                    const ulonglong2 c = row4(s.C, from + j);
                    float y[2];
#pragma unroll
                    for (int q = 0; q < 2; ++q) y[q] = sum2(fma2(h[q][0], c.x, mul2(h[q][1], c.y)));
                    const int at = spread_sum<2, NL / 2, 1>(y, lane);
                    if (nl % (NL / 2) == 0)
                        s.y[from + j][place_of<CH>(j ^ at, slot + at * kOther)] = y[0];
                }
            }
#pragma unroll
            for (int j = kSub - 1; j >= 0; --j) {
                const int k = from + j;
                asm volatile("" ::: "memory");   // (tokens further ahead would not fit the registers)
                const Inputs v = inputs(k);
                const ulonglong2 b = row4(s.B, k), c = row4(s.C, k);
                F2 vB[2] = {0, 0}, vC[2] = {0, 0}, t1[2] = {0, 0}, t2[2] = {0, 0};
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float rv = s.dr[k][place_of<CH>(j, slot + q * kOther)];
                    const F2 rr = pack2(rv, rv);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const F2 a = decay2(v.dd[q], A.v[q][i]);
                        const F2 gr = fma2(i ? c.y : c.x, rr, r[q][i]);   // gradient of h
                        vC[i] = fma2(h[q][i], rr, vC[i]);
                        vB[i] = fma2(gr, v.uu[q], vB[i]);
                        t1[q] = fma2(gr, i ? b.y : b.x, t1[q]);
                        const F2 ag = mul2(a, gr), w = mul2(ag, before[j][q][i]);
                        dA[q][i] = fma2(w, v.dd[q], dA[q][i]);
                        t2[q] = fma2(w, A.v[q][i], t2[q]);
                        r[q][i] = ag;
                        h[q][i] = before[j][q][i];
                    }
                }
                float sv[4] = {sum2(t1[0]), sum2(t1[1]), sum2(t2[0]), sum2(t2[1])};
                const int sat = spread_sum<4, NL / 2, 1>(sv, lane);
                constexpr int kLeftS = spread_left(4, NL / 2, 1);
                if (NL <= 4 || nl % (NL > 4 ? NL / 4 : 1) == 0) {
#pragma unroll
                    for (int i = 0; i < kLeftS; ++i) {
                        const int v = sat + i;
                        s.s[v / 2][k][place_of<CH>(j ^ v, slot + v % 2 * kOther)] = sv[i];
                    }
                }
                const float2 b0 = unpack2(vB[0]), b1 = unpack2(vB[1]);
                const float2 e0 = unpack2(vC[0]), e1 = unpack2(vC[1]);
                float bv[8] = {b0.x, b0.y, b1.x, b1.y, e0.x, e0.y, e1.x, e1.y};
                const int at = spread_sum<8, 16, NL>(bv, lane);
#pragma unroll
                for (int i = 0; i < spread_left(8, 16, NL); ++i)
                    sums[j * 2 * NP + (at + i) / 4 * NP + nl * 4 + (at + i) % 4] = bv[i];
            }
        };

        // the tile that ends before token e of a sequence that starts at `start`
        auto tile_start = [&](int32_t e, int32_t start) {
            int32_t a = (e - 1) / kBack * kBack;
            if (a < start) a = start;
            return a < t0 ? t0 : a;
        };
        int32_t te = t1, ta = t0 < t1 ? tile_start(t1, cu[n]) : t0;
        __syncthreads();
        if (te > t0) convert(ta, te - ta);
        while (te > t0) {
            const int32_t start = cu[n];
            const int cnt = te - ta;
            // The tile in parts of kSub tokens: the states before them are formed on one walk,
            // then the parts are taken from the last one on.
            const int off = ta % kBack, p0 = off / kSub, p1 = (off + cnt - 1) / kSub;
            F2 h[2][2];
            load4(ta == start ? (p.S0 ? p.S0 + n * Dn : nullptr) : p.states + ta / kBack * Dn, h);
            __syncthreads();
            auto place = [&](int part) { return reinterpret_cast<F2*>(s.part[warp][part]) + lane; };
            auto keep = [&](int part) {
#pragma unroll
                for (int i = 0; i < 4; ++i) place(part)[i * 32] = h[i / 2][i % 2];
            };
            auto back_to = [&](int part) {
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i / 2][i % 2] = place(part)[i * 32];
                __syncwarp();   // the place takes the part's sums from here on
            };
            keep(p0);
            {
                const Rates A = rates();
#pragma unroll 1
                for (int part = p0; part < p1; ++part) {
#pragma unroll
                    for (int j = 0; j < kSub; ++j) advance(A, part * kSub + j, h);
                    keep(part + 1);
                }
            }
#pragma unroll 1
            for (int part = p1; part >= p0; --part) {
                back_to(part);
                sub(part * kSub, h, s.part[warp][part]);
            }
            __syncthreads();
            finish(ta, cnt);
            te = ta;
            if (te == start) {
                if (p.g.dS0) store4(p.g.dS0 + n * Dn, r);
                if (te > t0) {
                    do --n; while (cu[n] == cu[n + 1]);
                    load4(p.dS_T ? p.dS_T + n * Dn : nullptr, r);
                }
            }
            if (te <= t0 || te % kSumTokens == 0) add_sums();
            if (te > t0) {
                ta = tile_start(te, cu[n]);
                // (what finish reads of the inputs' places, the same threads write now; the
                // sums' places are written behind the barrier)
                convert(ta, te - ta);
            }
        }
        __syncthreads();   // (the next item's sums)
    }
}

// dB, dC: the sums over the groups' channel blocks, in order.
__global__ void __launch_bounds__(256)
sum_blocks_kernel(const ScanArgs p, int32_t blocks, const float* __restrict__ part,
                  const int32_t* status) {
    if (*status != KDA_OK) return;
    const int64_t rows = (int64_t)p.cu_seqlens[p.num_seqs] * p.H, w = 2 * p.n;
    const int64_t stride = p.total_tokens * p.H * w;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * w;
         i += (int64_t)gridDim.x * 256) {
        float sum = 0.f;
        int32_t b = 0;
        for (; b + 4 <= blocks; b += 4) {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = part[(b + k) * stride + i];
            sum += (v[0] + v[1]) + (v[2] + v[3]);
        }
        for (; b < blocks; ++b) sum += part[b * stride + i];
        const int64_t row = i / w;
        const int k = (int)(i - row * w);
        (k < p.n ? p.g.dB : p.g.dC)[row * p.n + (k < p.n ? k : k - p.n)] = sum;
    }
}

// ---------------------------------------------------------------- decode step

// One token for each of `rows` sequences a warp, 32 channels of a group.  A lane forms one
// channel's step, skip and gate; the states go by NL lanes a channel, four values each, so that the
// warp reads and writes whole lines of them, 32 / NL channels at a time, with the steps passed on
// by exchanges.  The rates are read once for all the rows.
// Bound: loads in flight (96 registers leave 17 warps an SM).  Measured: 256 x 4096 x 16 from parents
// 31 us (122 MB, 3.9 TB/s); a thread for four values of one channel by itself took 40, the next row's
// loads ahead 37 (121 registers).
constexpr int kStepThreads = 128;
template <typename T, int NL>
__global__ void __launch_bounds__(kStepThreads)
scan_step_kernel(const ScanStepArgs p, int32_t per_group, int32_t rows) {
    constexpr int kAt = 32 / NL;                // channels at a time
    constexpr int kHold = NL <= 4 ? NL : 4;     // times whose states are loaded at once
    const int32_t warps = per_group * p.H;
    const int64_t item = (int64_t)blockIdx.x * (kStepThreads / 32) + threadIdx.x / 32;
    const int32_t rb = (int32_t)(item / warps), wb = (int32_t)(item - (int64_t)rb * warps);
    const int32_t g = wb / per_group, c0 = (wb - g * per_group) * 32;
    if ((int64_t)rb * rows >= p.B) return;
    const int lane = threadIdx.x & 31, k = lane % NL * 4, mine = lane / NL;
    const int32_t width = p.d - c0 < 32 ? p.d - c0 : 32, base = g * p.d + c0;
    const int32_t D = p.H * p.d;
    const bool on = lane < width, whole = p.n % 4 == 0;
    const float bias = on && p.dt_bias ? p.dt_bias[base + lane] : 0.f;
    const float skip = on && p.skip ? p.skip[base + lane] : 0.f;
    // four values from k on of a channel's row
    auto load = [&](const float* at, bool live, float (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = 0.f;
        if (!live) return;
        if (whole) {
            if (k < p.n) {
                const float4 u = *reinterpret_cast<const float4*>(at);
                v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (k + i < p.n) v[i] = at[i];
        }
    };
    float A[kHold][4];
    auto rates = [&](int from) {
#pragma unroll
        for (int j = 0; j < kHold; ++j) {
            const int ch = (from + j) * kAt + mine;
            load(p.A + (int64_t)(base + ch) * p.n + k, ch < width, A[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) A[j][i] = scaled_rate(A[j][i]);
        }
    };
    if (NL <= 4) rates(0);
    const int32_t stop = (rb + 1) * (int64_t)rows < p.B ? (rb + 1) * rows : p.B;
    for (int64_t b = (int64_t)rb * rows; b < stop; ++b) {
        const int32_t row = p.parents ? p.parents[b] : (int32_t)b;
        const bool live = row >= 0 && row < p.num_rows;
        float x = 0.f, step = 0.f, gate = 1.f;
        if (on) {
            x = Elem<T>::load(static_cast<const T*>(p.in.x) + b * p.in.ldx + base + lane);
            step = Elem<T>::load(static_cast<const T*>(p.in.dt) + b * p.in.lddt + base + lane) + bias;
            if (p.in.z)
                gate = Elem<T>::load(static_cast<const T*>(p.in.z) + b * p.in.ldz + base + lane);
        }
        float bv[4], cv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = k + i < p.n;
            bv[i] = in ? Elem<T>::load(static_cast<const T*>(p.in.B) + b * p.in.ldB +
                                       (int64_t)g * p.n + k + i) : 0.f;
            cv[i] = in ? Elem<T>::load(static_cast<const T*>(p.in.C) + b * p.in.ldC +
                                       (int64_t)g * p.n + k + i) : 0.f;
        }
        if (p.softplus) step = softplus(step);
        const float u = step * x;
        float y = 0.f;
#pragma unroll 1
        for (int from = 0; from < NL; from += kHold) {
            float h[kHold][4];
#pragma unroll
            for (int j = 0; j < kHold; ++j) {
                const int ch = (from + j) * kAt + mine;
                load(p.S + ((int64_t)row * D + base + ch) * p.n + k, live && ch < width, h[j]);
            }
            if (NL > 4) rates(from);
#pragma unroll
            for (int j = 0; j < kHold; ++j) {
                const int ch = (from + j) * kAt + mine;
                const float st = __shfl_sync(0xffffffffu, step, ch);
                const float uc = __shfl_sync(0xffffffffu, u, ch);
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    h[j][i] = fmaf(decay(st, A[j][i]), h[j][i], uc * bv[i]);
                    sum = fmaf(h[j][i], cv[i], sum);
                }
                if (ch < width) {
                    float* out = p.S_out + ((int64_t)b * D + base + ch) * p.n + k;
                    if (whole) {
                        if (k < p.n)
                            *reinterpret_cast<float4*>(out) =
                                make_float4(h[j][0], h[j][1], h[j][2], h[j][3]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (k + i < p.n) out[i] = h[j][i];
                    }
                }
#pragma unroll
                for (int o = 1; o < NL; o *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                // to the lane whose channel it is
                const float there = __shfl_sync(0xffffffffu, sum, lane % kAt * NL);
                if (lane / kAt == from + j) y = there;
            }
        }
        if (on) {
            y = fmaf(skip, x, y);
            if (p.in.z) y *= silu(gate);
            Elem<T>::store(static_cast<T*>(p.y) + b * D + base + lane, y);
        }
    }
}

// ---------------------------------------------------------------- host

size_t pad(size_t b) { return (b + 255) & ~(size_t)255; }
constexpr size_t kHead = 256;   // the status word's part of the workspace
int64_t sms() { return sm_count() > 0 ? sm_count() : 1; }

int lanes_of(int n) { return n <= 8 ? 1 : n <= 16 ? 2 : n <= 32 ? 4 : 8; }
int forward_channels(int n) {
    switch (lanes_of(n)) {
        case 1: return Fwd<1>::kCh;
        case 2: return Fwd<2>::kCh;
        case 4: return Fwd<4>::kCh;
        default: return Fwd<8>::kCh;
    }
}
int back_lanes_of(int n) { return n <= 8 ? 2 : n <= 16 ? 4 : n <= 32 ? 8 : 16; }
int back_channels(int n) {
    switch (back_lanes_of(n)) {
        case 2: return Back<2>::kCh;
        case 4: return Back<4>::kCh;
        case 8: return Back<8>::kCh;
        default: return Back<16>::kCh;
    }
}

// Whole sequences where they and the channel blocks of `ch` make `fill` CTAs an SM, or are short
// (a walk takes 130 ns a token, cutting 20 us: 64 tokens of 64 channels 14 us whole and 31 cut);
// else segments of at least `least` tokens, as many as take the GPU's places (`each` CTAs an SM)
// twice.  (A last round that fills them in part costs as much as a whole one: 131072 x 4096 in 960
// pieces on 608 places took 5.25 ms, in 1216 4.6.)  The lengths are on the device: the choice is made
// by N and T alone.
Cut make_cut(int32_t N, int64_t T, int32_t H, int32_t d, int ch, int each, int fill,
             int least) {
    Cut c = {};
    c.per_group = (d + ch - 1) / ch;
    const int64_t blocks = (int64_t)c.per_group * H;
    if (N == 0 || N * blocks >= fill * sms() || T < (int64_t)N * 64 || T < 256) {
        c.nseg = N;
    } else {
        int64_t most = 2 * each * sms() / blocks;
        if (most < 1) most = 1;
        c.seg = ((T + most - 1) / most + kTile - 1) / kTile * kTile;
        if (c.seg < least) c.seg = least;
        c.nseg = (T + c.seg - 1) / c.seg;
    }
    c.items = c.nseg * blocks;
    return c;
}
Cut forward_cut(int32_t N, int64_t T, int32_t H, int32_t d, int32_t n) {
    return make_cut(N, T, H, d, forward_channels(n), n <= 8 ? 8 : 4, 3, 64);
}
Cut backward_cut(int32_t N, int64_t T, int32_t H, int32_t d, int32_t n) {
    return make_cut(N, T, H, d, back_channels(n), n <= 8 ? 2 : 4, 1, 128);
}
// The maps of the gradients' recurrence are formed by the forward kernel: the same segments, but
// its own channel blocks.
Cut grad_map_cut(const Cut& back, int32_t H, int32_t d, int32_t n) {
    Cut c = back;
    const int ch = forward_channels(n);
    c.per_group = (d + ch - 1) / ch;
    c.items = c.nseg * c.per_group * H;
    return c;
}

size_t maps_bytes(const Cut& c, int64_t D, int32_t n) {
    if (c.seg == 0) return 0;
    return pad((size_t)c.nseg * D * 4) + pad((size_t)c.nseg * D * n * 4) + pad((size_t)c.nseg * 4);
}
Maps place_maps(const Cut& c, int64_t D, int32_t n, char* ws) {
    Maps m = {};
    if (c.seg == 0) return m;
    m.sum = reinterpret_cast<float*>(ws);
    m.state = reinterpret_cast<float*>(ws + pad((size_t)c.nseg * D * 4));
    m.reset = reinterpret_cast<int32_t*>(ws + pad((size_t)c.nseg * D * 4) +
                                         pad((size_t)c.nseg * D * n * 4));
    return m;
}

template <int N>
using Int = std::integral_constant<int, N>;
template <typename F>
cudaError_t by_type(kda_dtype dtype, F&& f) {
    return dtype == KDA_BF16 ? f((__nv_bfloat16*)nullptr) : f((float*)nullptr);
}
template <typename F>
cudaError_t by_lanes(int n, F&& f) {
    switch (lanes_of(n)) {
        case 1: return f(Int<1>());
        case 2: return f(Int<2>());
        case 4: return f(Int<4>());
        default: return f(Int<8>());
    }
}
template <typename F>
cudaError_t by_back_lanes(int n, F&& f) {
    switch (back_lanes_of(n)) {
        case 2: return f(Int<2>());
        case 4: return f(Int<4>());
        case 8: return f(Int<8>());
        default: return f(Int<16>());
    }
}

template <int PASS>
cudaError_t run_scan(const ScanArgs& a, const Cut& cut, const Maps& maps, int32_t* status,
                     cudaStream_t stream) {
    const int64_t D = (int64_t)a.H * a.d;
    return by_type(a.dtype, [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int V = 16 / sizeof(T);
        const bool wide =
            a.d % V == 0 && rows_fit(a.in.dt, a.in.lddt, D, sizeof(T), V) &&
            (PASS == kGradMaps || rows_fit(a.in.x, a.in.ldx, D, sizeof(T), V)) &&
            (PASS == kMaps || !a.in.z || rows_fit(a.in.z, a.in.ldz, D, sizeof(T), V));
        return by_lanes(a.n, [&](auto l) {
            constexpr int L = decltype(l)::value;
            const int64_t most = (int64_t)1 << 30;
            const unsigned grid = (unsigned)(cut.items < 1 ? 1 : cut.items < most ? cut.items : most);
            auto kernel = wide ? scan_kernel<T, L, V, PASS> : scan_kernel<T, L, 1, PASS>;
            kernel<<<grid, Fwd<L>::kThreads, 0, stream>>>(a, cut, maps, status);
            return cudaGetLastError();
        });
    });
}

// (in, out: of the empty sequences)
cudaError_t run_join(const ScanArgs& a, const Cut& cut, const Maps& maps, bool reversed,
                     const float* in, float* out, const int32_t* status, cudaStream_t stream) {
    const int64_t D = (int64_t)a.H * a.d;
    join_kernel<<<(unsigned)((D * a.n + kThreads - 1) / kThreads), kThreads, 0, stream>>>(
        a, cut, maps, reversed, in, out, status);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess || a.num_seqs <= kJoinEmpty || !out) return err;
    const int64_t row = (int64_t)a.H * a.d * a.n;
    empty_kernel<<<(unsigned)(a.num_seqs < 1024 ? a.num_seqs : 1024), kThreads, 0, stream>>>(
        a.cu_seqlens, a.num_seqs, row, in, out, status);
    return cudaGetLastError();
}

// The forward scan in a workspace of forward_bytes behind the status word.
size_t forward_bytes(int32_t N, int64_t T, int32_t H, int32_t d, int32_t n) {
    const Cut c = forward_cut(N, T, H, d, n);
    const int64_t D = (int64_t)H * d;
    return maps_bytes(c, D, n) + (c.seg ? pad((size_t)N * D * n * 4) : 0);
}
cudaError_t run_forward(const ScanArgs& args, char* ws, int32_t* status, cudaStream_t stream) {
    ScanArgs a = args;
    const Cut cut = forward_cut(a.num_seqs, a.total_tokens, a.H, a.d, a.n);
    const int64_t D = (int64_t)a.H * a.d;
    const Maps maps = place_maps(cut, D, a.n, ws);
    if (cut.seg) {
        if (a.S0 && a.S0 == a.S_T) {   // in place: segments read S0 while others write S_T
            float* copy = reinterpret_cast<float*>(ws + maps_bytes(cut, D, a.n));
            const cudaError_t err = cudaMemcpyAsync(copy, a.S0, (size_t)a.num_seqs * D * a.n * 4,
                                                    cudaMemcpyDeviceToDevice, stream);
            if (err != cudaSuccess) return err;
            a.S0 = copy;
        }
        cudaError_t err = run_scan<kMaps>(a, cut, maps, status, stream);
        if (err == cudaSuccess) err = run_join(a, cut, maps, false, a.S0, a.S_T, status, stream);
        if (err != cudaSuccess) return err;
    }
    return run_scan<kOutputs>(a, cut, maps, status, stream);
}

struct BackLayout {
    size_t maps, part, part_BC, states, forward, end;
};
BackLayout back_layout(const Cut& cut, int32_t N, int64_t T, int32_t H, int32_t d, int32_t n,
                       bool with_states) {
    BackLayout L;
    const size_t D = (size_t)H * d;
    size_t at = kHead;
    L.maps = at;
    at += maps_bytes(cut, D, n);
    L.part = at;   // [segment][dA, dskip, ddt_bias]
    at += pad((size_t)cut.nseg * part_row(D, n) * 4);
    L.part_BC = at;
    if (cut.per_group > 1) at += pad((size_t)cut.per_group * T * H * 2 * n * 4);
    L.states = at;
    if (!with_states) at += pad((size_t)(T + SELSCAN_CHUNK - 1) / SELSCAN_CHUNK * D * n * 4);
    L.forward = at;
    if (!with_states) at += forward_bytes(N, T, H, d, n);
    L.end = at;
    return L;
}

}  // namespace

size_t scan_prefill_bytes(int32_t N, int64_t T, int32_t H, int32_t d, int32_t n) {
    return kHead + forward_bytes(N, T, H, d, n);
}
size_t scan_backward_bytes(int32_t N, int64_t T, int32_t H, int32_t d, int32_t n,
                           bool with_states) {
    return back_layout(backward_cut(N, T, H, d, n), N, T, H, d, n, with_states).end;
}

cudaError_t launch_scan_prefill(const ScanArgs& a, char* ws, cudaStream_t stream) {
    int32_t* status = reinterpret_cast<int32_t*>(ws);
    const cudaError_t err = launch_offsets_check(a.cu_seqlens, a.num_seqs, a.total_tokens, status,
                                                 stream);
    if (err != cudaSuccess) return err;
    return run_forward(a, ws + kHead, status, stream);
}

cudaError_t launch_scan_backward(const ScanArgs& args, char* ws, cudaStream_t stream) {
    ScanArgs a = args;
    int32_t* status = reinterpret_cast<int32_t*>(ws);
    const int64_t D = (int64_t)a.H * a.d;
    const Cut cut = backward_cut(a.num_seqs, a.total_tokens, a.H, a.d, a.n);
    const BackLayout L = back_layout(cut, a.num_seqs, a.total_tokens, a.H, a.d, a.n,
                                     a.states != nullptr);
    const Maps maps = place_maps(cut, D, a.n, ws + L.maps);
    float* part = reinterpret_cast<float*>(ws + L.part);
    float* part_BC = reinterpret_cast<float*>(ws + L.part_BC);
    // (the backward kernel reads the outcome; the forward kernel leaves it there if it runs before)
    cudaError_t err = launch_offsets_check(a.cu_seqlens, a.num_seqs, a.total_tokens, status, stream,
                                           a.states && cut.seg == 0);
    if (err != cudaSuccess) return err;
    if (!a.states) {   // the forward scan once more, for the states alone
        ScanArgs f = a;
        f.y = nullptr;
        f.S_T = nullptr;
        f.states = reinterpret_cast<float*>(ws + L.states);
        err = run_forward(f, ws + L.forward, status, stream);
        if (err != cudaSuccess) return err;
        a.states = f.states;
    }
    if (cut.seg) {
        err = run_scan<kGradMaps>(a, grad_map_cut(cut, a.H, a.d, a.n), maps, status, stream);
        if (err == cudaSuccess) err = run_join(a, cut, maps, true, a.dS_T, a.g.dS0, status, stream);
        if (err != cudaSuccess) return err;
    }
    err = by_type(a.dtype, [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int V = 16 / sizeof(T);
        const bool wide = a.d % V == 0 && rows_fit(a.in.x, a.in.ldx, D, sizeof(T), V) &&
                          rows_fit(a.in.dt, a.in.lddt, D, sizeof(T), V) &&
                          (!a.in.z || rows_fit(a.in.z, a.in.ldz, D, sizeof(T), V));
        return by_back_lanes(a.n, [&](auto l) {
            constexpr int NL = decltype(l)::value;
            auto kernel = wide ? scan_bwd_kernel<T, NL, V> : scan_bwd_kernel<T, NL, 1>;
            constexpr int smem = sizeof(typename Back<NL>::Shared);
            const cudaError_t e = cudaFuncSetAttribute(
                kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            const int64_t most = (int64_t)1 << 30;
            const unsigned grid = (unsigned)(cut.items < 1 ? 1 : cut.items < most ? cut.items : most);
            kernel<<<grid, Back<NL>::kThreads, smem, stream>>>(a, cut, maps, part, part_BC, status);
            return cudaGetLastError();
        });
    });
    if (err != cudaSuccess) return err;
    if (cut.per_group > 1 && a.total_tokens > 0) {
        const int64_t n = a.total_tokens * a.H * 2 * a.n, most = 32 * sms();
        const int64_t blocks = (n + 255) / 256;
        sum_blocks_kernel<<<(unsigned)(blocks < most ? blocks : most), 256, 0, stream>>>(
            a, cut.per_group, part_BC, status);
        err = cudaGetLastError();
        if (err != cudaSuccess) return err;
    }
    return launch_column_sums(part, cut.nseg, {D * a.n, D, D}, {a.g.dA, a.g.dskip, a.g.ddt_bias},
                              status, stream);
}

int64_t scan_step_blocks(int32_t B, int32_t H, int32_t d, int32_t* rows) {
    const int64_t warps = (int64_t)((d + 31) / 32) * H;
    // as many rows a warp, up to four, as leave each SM 16 warps
    int32_t r = 4;
    while (r > 1 && (B + (int64_t)r - 1) / r * warps < 16 * sms()) r /= 2;
    *rows = r;
    static_assert(kStepThreads == 128, "four warps a CTA");
    return ((B + (int64_t)r - 1) / r * warps + 3) / 4;
}

cudaError_t launch_scan_step(const ScanStepArgs& a, cudaStream_t stream) {
    int32_t rows;
    const int64_t blocks = scan_step_blocks(a.B, a.H, a.d, &rows);
    const int32_t per_group = (a.d + 31) / 32;
    return by_type(a.dtype, [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        return by_back_lanes(a.n, [&](auto l) {   // (four values a lane, as in the backward pass)
            scan_step_kernel<T, decltype(l)::value>
                <<<(unsigned)blocks, kStepThreads, 0, stream>>>(a, per_group, rows);
            return cudaGetLastError();
        });
    });
}

}  // namespace kda
