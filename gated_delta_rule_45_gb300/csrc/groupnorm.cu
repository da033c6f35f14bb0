// Gated group norm of the heads (include/groupnorm.h): forward and backward.
//
// Mathematics.  Per (token, head): m = mean(x), r = 1 / sqrt(mean((x - m)^2) + eps), xh = (x - m)
// r, v = w xh + b, y = v act(z) or act(v).  Backward, with dv = dL/dv and g = w dv,
//
//     dx = r (g - xh mean(g xh) - mean(g)),   dw = sum_t dv xh,   db = sum_t dv
//
// (without the mean's term for the RMS form).  A row lies in the registers of 1 to 32 lanes, so
// x is read once and the deviations are formed from the mean itself; rows too wide for that
// take a CTA that reads them again.  A lane keeps its head and channels over all its tokens:
// the parameters are read once, and their gradients are summed in registers and joined by a
// second kernel in a fixed order.
//
// Bound: HBM.  Measured, bf16 with a gate, 32768 x 32 x 128: forward 131 us (0.8 GB, 6.1 TB/s; 150
// with divisions and a square root instead of reciprocals, 208 without the next row's loads
// ahead), backward 321 us (1.9 GB, 5.9) with weights of each head's own.  Weights that all heads
// share leave the join of the sums few columns: 410 us, and 97 instead of 37 at 2048 tokens.  Widths
// that are no whole 16 bytes take single values: 8192 x 16 x 201 322 us forward (0.16 GB) and 451
// backward, 200 wide 40 and 87.
#include "layer_ops.h"

#include <type_traits>

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxVec = 4;        // vectors of a row that a lane holds, at most
constexpr int64_t kMaxParts = 1024;   // rows of partial sums of a head, at most

// How the rows are laid over the threads: a group of `lanes` lanes a row, `hpb` heads side by
// side in a CTA, `tpb` tokens, and CTAs over the heads and the tokens.
struct NormGrid {
    int32_t lanes, nv;       // lanes a row, vectors a lane (0: a CTA a row, which reads it again)
    int32_t hpb, tpb, hblocks;
    int64_t tblocks;
};

__device__ __forceinline__ float group_sum(float v, int lanes) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < lanes) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float activate(float v, int act) {
    return act == GROUPNORM_SILU ? silu(v) : act == GROUPNORM_SIGMOID ? sigmoid(v) : v;
}
__device__ __forceinline__ float activate_grad(float v, int act) {
    if (act == GROUPNORM_SILU) return silu_grad(v);
    if (act == GROUPNORM_SIGMOID) {
        const float s = sigmoid(v);
        return s * (1.f - s);
    }
    return 1.f;
}

// act(v) of a pair, and its slope.
__device__ __forceinline__ F2 activate2(F2 v, int act) {
    return act == GROUPNORM_SILU ? silu2(v) : act == GROUPNORM_SIGMOID ? sigmoid2(v) : v;
}
__device__ __forceinline__ F2 activate_grad2(F2 v, int act) {
    if (act == GROUPNORM_SILU) return silu_grad2(v);
    if (act == GROUPNORM_SIGMOID) {
        const F2 s = sigmoid2(v);
        return mul2(s, fma2(s, both(-1.f), both(1.f)));
    }
    return both(1.f);
}

// A row as stored: the vectors lane, lane + lanes, ..
template <typename T, int V, int NV>
struct Row {
    Pack<T, V> k[NV];
    __device__ __forceinline__ void load(const T* p, int lane, int lanes, int nvec, bool on) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = lane + j * lanes;
            if (on && v < nvec) k[j].load(p + v * V);
            else k[j].zero();
        }
    }
};

// xh of one row, and its r.
template <typename T, int V, int NV>
__device__ __forceinline__ float normalise(const Row<T, V, NV>& x, Lane<V> (&xh)[NV], int lane,
                                           int lanes, int nvec, float inv_d, bool center,
                                           float eps) {
#pragma unroll
    for (int j = 0; j < NV; ++j) xh[j].from(x.k[j]);
    if (center) {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) m += xh[j].sum();
        const F2 mean = both(-group_sum(m, lanes) * inv_d);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < Lane<V>::kPairs; ++i)
                xh[j].v[i] = lane + j * lanes < nvec ? add2(xh[j].v[i], mean) : 0;
    }
    Lane<V> q;
    q.zero();
#pragma unroll
    for (int j = 0; j < NV; ++j) q.fma(xh[j], xh[j]);
    const float r = rsqrtf(group_sum(q.sum(), lanes) * inv_d + eps);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < Lane<V>::kPairs; ++i) xh[j].v[i] = mul2(xh[j].v[i], both(r));
    return r;
}

// A lane group's head, first token and stride over the tokens.
struct NormPlace {
    int lane, h;
    int64_t t, step;
    bool on;
};
__device__ __forceinline__ NormPlace norm_place(const NormArgs& p, const NormGrid& g) {
    NormPlace a;
    const int group = threadIdx.x / g.lanes;
    a.lane = threadIdx.x & (g.lanes - 1);
    const int tl = group / g.hpb, hl = group - tl * g.hpb;
    const int64_t tb = blockIdx.x / g.hblocks;
    a.h = (int)(blockIdx.x - tb * g.hblocks) * g.hpb + hl;
    a.on = tl < g.tpb && a.h < p.H;
    a.t = tb * g.tpb + tl;
    a.step = g.tblocks * g.tpb;
    return a;
}

// The parameters of a lane's channels.
template <int V, int NV>
__device__ __forceinline__ void load_params(const NormArgs& p, const NormPlace& a, int lanes,
                                            int nvec, Lane<V> (&w)[NV], Lane<V> (&b)[NV]) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < Lane<V>::kPairs; ++i) {
            const int v = a.lane + j * lanes;
            const bool in = a.on && v < nvec;
            const int64_t at = (p.param_heads == 1 ? 0 : (int64_t)a.h * p.d) + v * V + 2 * i;
            constexpr int o = V > 1 ? 1 : 0;
            w[j].v[i] = in && p.w ? pack2(p.w[at], p.w[at + o]) : both(1.f);
            b[j].v[i] = in && p.b ? pack2(p.b[at], p.b[at + o]) : 0;
        }
}

// The rows of the next token are loaded while this one's are worked on.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(kThreads)
norm_fwd_kernel(const NormArgs p, const NormGrid g) {
    const NormPlace a = norm_place(p, g);
    const int nvec = p.d / V;
    const float inv_d = 1.f / p.d;
    Lane<V> w[NV], b[NV];
    load_params(p, a, g.lanes, nvec, w, b);
    const T* px = static_cast<const T*>(p.x) + a.t * p.ldx + (int64_t)a.h * p.d;
    const T* pz = static_cast<const T*>(p.z) + a.t * p.ldz + (int64_t)a.h * p.d;
    T* y = static_cast<T*>(p.y) + (a.t * p.H + a.h) * p.d;
    Row<T, V, NV> x, z, nx, nz;
    bool on = a.on && a.t < p.T;
    x.load(px, a.lane, g.lanes, nvec, on);
    if (p.z) z.load(pz, a.lane, g.lanes, nvec, on);
    // (all lanes of a warp take part in its sums, so they leave the loop together)
    for (int64_t t = a.t; __any_sync(0xffffffffu, on); t += a.step) {
        const bool next = a.on && t + a.step < p.T;
        px += a.step * p.ldx;
        nx.load(px, a.lane, g.lanes, nvec, next);
        if (p.z) {
            pz += a.step * p.ldz;
            nz.load(pz, a.lane, g.lanes, nvec, next);
        }
        Lane<V> xh[NV];
        normalise(x, xh, a.lane, g.lanes, nvec, inv_d, p.center, p.eps);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = a.lane + j * g.lanes;
            Lane<V> o, zv;
            if (p.z) zv.from(z.k[j]);
#pragma unroll
            for (int i = 0; i < Lane<V>::kPairs; ++i) {
                const F2 n = fma2(xh[j].v[i], w[j].v[i], b[j].v[i]);
                o.v[i] = p.z ? mul2(n, activate2(zv.v[i], p.act)) : activate2(n, p.act);
            }
            if (on && v < nvec) o.template to<T>().store(y + v * V);
        }
        y += a.step * p.H * p.d;
        x = nx;
        z = nz;
        on = next;
    }
}

template <int V>
__device__ __forceinline__ void store_f32(float* p, const Lane<V>& l) {
    constexpr int U = V < 4 ? V : 4;
#pragma unroll
    for (int i = 0; i < V; i += U) {
        float f[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float2 t = unpack2(l.v[(i + u) / 2]);
            f[u] = u % 2 ? t.y : t.x;
        }
        Pack<float, U> k;
        k.set(f);
        k.store(p + i);
    }
}

template <typename T, int V, int NV>
__global__ void __launch_bounds__(kThreads)
norm_bwd_kernel(const NormArgs p, const NormGrid g, float* part) {
    const NormPlace a = norm_place(p, g);
    const int nvec = p.d / V;
    const float inv_d = 1.f / p.d;
    Lane<V> w[NV], b[NV], dw[NV], db[NV];
    load_params(p, a, g.lanes, nvec, w, b);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        dw[j].zero();
        db[j].zero();
    }
    const T* px = static_cast<const T*>(p.x) + a.t * p.ldx + (int64_t)a.h * p.d;
    const T* pz = static_cast<const T*>(p.z) + a.t * p.ldz + (int64_t)a.h * p.d;
    int64_t out = (a.t * p.H + a.h) * p.d;
    const int64_t stride = a.step * p.H * p.d;
    constexpr bool kAhead = NV <= 2;   // (wider rows leave no registers for the next)
    Row<T, V, NV> x, z, dy, nx, nz, ndy;
    bool on = a.on && a.t < p.T;
    auto load = [&](Row<T, V, NV>& rx, Row<T, V, NV>& rz, Row<T, V, NV>& rd, const T* x_,
                    const T* z_, int64_t at, bool live) {
        rx.load(x_, a.lane, g.lanes, nvec, live);
        rd.load(static_cast<const T*>(p.dy) + at, a.lane, g.lanes, nvec, live);
        if (p.z) rz.load(z_, a.lane, g.lanes, nvec, live);
    };
    if (kAhead) load(x, z, dy, px, pz, out, on);
    for (int64_t t = a.t; __any_sync(0xffffffffu, on); t += a.step) {
        const bool next = a.on && t + a.step < p.T;
        if (kAhead)
            load(nx, nz, ndy, px + a.step * p.ldx, pz + a.step * p.ldz, out + stride, next);
        else
            load(x, z, dy, px, pz, out, on);
        Lane<V> xh[NV], gv[NV];
        // (a group behind the last token has a row of zeros: without an eps 0 / 0, which would
        // reach its sums over the tokens)
        const float r = normalise(x, xh, a.lane, g.lanes, nvec, inv_d, p.center, on ? p.eps : 1.f);
        Lane<V> q1, q2;   // g xh and g
        q1.zero();
        q2.zero();
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = a.lane + j * g.lanes;
            Lane<V> zv, dv, dz;
            dv.from(dy.k[j]);
            if (p.z) zv.from(z.k[j]);
#pragma unroll
            for (int i = 0; i < Lane<V>::kPairs; ++i) {
                const F2 n = fma2(xh[j].v[i], w[j].v[i], b[j].v[i]);
                if (p.z) {
                    dz.v[i] = mul2(mul2(dv.v[i], n), activate_grad2(zv.v[i], p.act));
                    dv.v[i] = mul2(dv.v[i], activate2(zv.v[i], p.act));
                } else {
                    dv.v[i] = mul2(dv.v[i], activate_grad2(n, p.act));
                }
                gv[j].v[i] = mul2(dv.v[i], w[j].v[i]);
            }
            dw[j].fma(dv, xh[j]);
            db[j].add(dv);
            q1.fma(gv[j], xh[j]);
            q2.add(gv[j]);
            if (p.dz && on && v < nvec) store_f32(p.dz + out + v * V, dz);
        }
        const float s1 = group_sum(q1.sum(), g.lanes) * inv_d;
        const float s2 = p.center ? group_sum(q2.sum(), g.lanes) * inv_d : 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = a.lane + j * g.lanes;
            Lane<V> dx;
#pragma unroll
            for (int i = 0; i < Lane<V>::kPairs; ++i) {   // r (g - (xh s1 + s2))
                const F2 off = fma2(xh[j].v[i], both(s1), both(s2));
                dx.v[i] = mul2(fma2(off, both(-1.f), gv[j].v[i]), both(r));
            }
            if (on && v < nvec) store_f32(p.dx + out + v * V, dx);
        }
        px += a.step * p.ldx;
        pz += a.step * p.ldz;
        out += stride;
        if (kAhead) {
            x = nx;
            z = nz;
            dy = ndy;
        }
        on = next;
    }
    if (!part || !a.on) return;
    // part[token part][head][dw, db][d]
    float* row = part + (a.t * p.H + a.h) * 2 * p.d;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = a.lane + j * g.lanes;
        if (v >= nvec) continue;
        store_f32(row + v * V, dw[j]);
        store_f32(row + p.d + v * V, db[j]);
    }
}

// ---- rows wider than the registers of a warp: a CTA a row

__device__ __forceinline__ float block_sum(float v, float* s) {
    v = group_sum(v, 32);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) sum += s[k];
    return sum;
}

template <typename T, int V, typename F>
__device__ __forceinline__ void over_row(const T* p, int d, F&& f) {
    for (int c = threadIdx.x * V; c < d; c += kThreads * V) {
        Pack<T, V> k;
        k.load(p + c);
        f(c, k);
    }
}

template <typename T, int V>
__device__ __forceinline__ void wide_stats(const NormArgs& p, const T* x, float* s, float& m,
                                           float& r) {
    m = 0.f;
    if (p.center) {
        over_row<T, V>(x, p.d, [&](int, const Pack<T, V>& k) {
#pragma unroll
            for (int i = 0; i < V; ++i) m += k.get(i);
        });
        m = block_sum(m, s) / p.d;
    }
    float q = 0.f;
    over_row<T, V>(x, p.d, [&](int, const Pack<T, V>& k) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float u = k.get(i) - m;
            q = fmaf(u, u, q);
        }
    });
    r = rsqrtf(block_sum(q, s) / p.d + p.eps);
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads)
norm_fwd_wide_kernel(const NormArgs p, const NormGrid g) {
    __shared__ float s[kThreads / 32];
    const int64_t tb = blockIdx.x / p.H;
    const int h = (int)(blockIdx.x - tb * p.H);
    const float* w = p.w ? p.w + (p.param_heads == 1 ? 0 : (int64_t)h * p.d) : nullptr;
    const float* b = p.b ? p.b + (p.param_heads == 1 ? 0 : (int64_t)h * p.d) : nullptr;
    for (int64_t t = tb; t < p.T; t += g.tblocks) {
        const T* x = static_cast<const T*>(p.x) + t * p.ldx + (int64_t)h * p.d;
        const T* z = static_cast<const T*>(p.z) + t * p.ldz + (int64_t)h * p.d;
        T* y = static_cast<T*>(p.y) + (t * p.H + h) * p.d;
        float m, r;
        wide_stats<T, V>(p, x, s, m, r);
        over_row<T, V>(x, p.d, [&](int c, const Pack<T, V>& k) {
            Pack<T, V> kz;
            if (p.z) kz.load(z + c);
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float n = fmaf((k.get(i) - m) * r, w ? w[c + i] : 1.f, b ? b[c + i] : 0.f);
                o[i] = p.z ? n * activate(kz.get(i), p.act) : activate(n, p.act);
            }
            Pack<T, V> ky;
            ky.set(o);
            ky.store(y + c);
        });
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads)
norm_bwd_wide_kernel(const NormArgs p, const NormGrid g, float* part) {
    __shared__ float s[kThreads / 32];
    const int64_t tb = blockIdx.x / p.H;
    const int h = (int)(blockIdx.x - tb * p.H);
    const float* w = p.w ? p.w + (p.param_heads == 1 ? 0 : (int64_t)h * p.d) : nullptr;
    const float* b = p.b ? p.b + (p.param_heads == 1 ? 0 : (int64_t)h * p.d) : nullptr;
    float* row = part ? part + (tb * p.H + h) * 2 * p.d : nullptr;
    if (row)
        for (int c = threadIdx.x; c < 2 * p.d; c += kThreads) row[c] = 0.f;
    __syncthreads();
    for (int64_t t = tb; t < p.T; t += g.tblocks) {
        const T* x = static_cast<const T*>(p.x) + t * p.ldx + (int64_t)h * p.d;
        const T* z = static_cast<const T*>(p.z) + t * p.ldz + (int64_t)h * p.d;
        const int64_t out = (t * p.H + h) * p.d;
        const T* dy = static_cast<const T*>(p.dy) + out;
        float m, r;
        wide_stats<T, V>(p, x, s, m, r);
        // f(channel, xh, dv, dz) for every channel of this thread
        auto each = [&](auto&& f) {
            over_row<T, V>(x, p.d, [&](int c, const Pack<T, V>& k) {
                Pack<T, V> kz, kd;
                if (p.z) kz.load(z + c);
                kd.load(dy + c);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float xh = (k.get(i) - m) * r;
                    const float n = fmaf(xh, w ? w[c + i] : 1.f, b ? b[c + i] : 0.f);
                    const float d = kd.get(i);
                    if (p.z) f(c + i, xh, d * activate(kz.get(i), p.act),
                               d * n * activate_grad(kz.get(i), p.act));
                    else f(c + i, xh, d * activate_grad(n, p.act), 0.f);
                }
            });
        };
        float s1 = 0.f, s2 = 0.f;
        each([&](int c, float xh, float dv, float dz) {
            const float gv = dv * (w ? w[c] : 1.f);
            s1 = fmaf(gv, xh, s1);
            s2 += gv;
            if (p.dz) p.dz[out + c] = dz;
            if (row) {   // a channel is the same thread's for every token
                row[c] = fmaf(dv, xh, row[c]);
                row[p.d + c] += dv;
            }
        });
        s1 = block_sum(s1, s) / p.d;
        s2 = block_sum(s2, s) / p.d;
        if (!p.center) s2 = 0.f;
        each([&](int c, float xh, float dv, float) {
            p.dx[out + c] = r * (dv * (w ? w[c] : 1.f) - fmaf(xh, s1, s2));
        });
    }
}

// Sums part's rows [parts][heads joined by a parameter][2 d] to dw and db.
__global__ void __launch_bounds__(kThreads)
norm_param_sum_kernel(const float* __restrict__ part, int64_t parts, int32_t H, int32_t d,
                      int32_t param_heads, float* dw, float* db) {
    __shared__ float s[8][32];
    const int cl = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.x * 32 + cl;   // of param_heads x 2 d
    const int32_t ph = (int32_t)(col / (2 * d)), c = (int32_t)(col - (int64_t)ph * 2 * d);
    const bool on = ph < param_heads;
    // row r of the column: part r / joined, head ph or (shared) r mod H
    const int64_t joined = param_heads == 1 ? H : 1, rows = parts * joined;
    const int64_t first = (int64_t)ph * 2 * d + c;
    const int64_t stride = (param_heads == 1 ? 1 : (int64_t)H) * 2 * d;
    float sum = 0.f;
    if (on) {
        int64_t r = rl;
        for (; r + 24 < rows; r += 32) {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = part[first + (r + 8 * k) * stride];
            sum += (v[0] + v[1]) + (v[2] + v[3]);
        }
        for (; r < rows; r += 8) sum += part[first + r * stride];
    }
    s[rl][cl] = sum;
    __syncthreads();
    if (rl != 0 || !on) return;
#pragma unroll
    for (int k = 1; k < 8; ++k) sum += s[k][cl];
    float* out = c < d ? dw : db;
    if (out) out[(int64_t)ph * d + (c < d ? c : c - d)] = sum;
}

// `parts`: most rows of partial sums of a head (0: as many as there are tokens).
NormGrid norm_grid(int64_t T, int32_t H, int32_t d, int V, int64_t parts) {
    NormGrid g = {};
    const int nvec = d / V;
    const int64_t sms = sm_count() > 0 ? sm_count() : 1;
    if (nvec > 32 * kMaxVec) {
        g.tblocks = (8 * sms + H - 1) / H;
        if (parts > 0 && g.tblocks > parts) g.tblocks = parts;
        if (g.tblocks > T) g.tblocks = T;
        return g;
    }
    g.lanes = 1;
    while (g.lanes < 32 && g.lanes < nvec) g.lanes *= 2;
    g.nv = (nvec + g.lanes - 1) / g.lanes;
    const int groups = kThreads / g.lanes;
    g.hpb = H < groups ? H : groups;
    g.tpb = groups / g.hpb;
    g.hblocks = (H + g.hpb - 1) / g.hpb;
    g.tblocks = (T + g.tpb - 1) / g.tpb;
    const int64_t most = (4 * sms + g.hblocks - 1) / g.hblocks;
    if (g.tblocks > most) g.tblocks = most;
    if (parts > 0 && g.tblocks * g.tpb > parts) g.tblocks = parts / g.tpb > 0 ? parts / g.tpb : 1;
    return g;
}
NormGrid backward_grid(int64_t T, int32_t H, int32_t d, int V) {
    return norm_grid(T, H, d, V, T < kMaxParts ? T : kMaxParts);
}
int64_t norm_parts(const NormGrid& g) { return g.nv == 0 ? g.tblocks : g.tblocks * g.tpb; }

int norm_vec(const NormArgs& a) {
    const size_t esz = a.dtype == KDA_BF16 ? 2 : 4;
    const int V = (int)(16 / esz);
    if (a.d % V != 0 || !rows_fit(a.x, a.ldx, a.d, esz, V)) return 1;
    if (a.z && !rows_fit(a.z, a.ldz, a.d, esz, V)) return 1;
    return V;
}

template <typename F>
cudaError_t by_layout(const NormArgs& a, int V, int nv, F&& f) {
    auto pick_nv = [&](auto* t, auto v) {
        switch (nv) {
            case 0: return f(t, v, std::integral_constant<int, 0>());
            case 1: return f(t, v, std::integral_constant<int, 1>());
            case 2: return f(t, v, std::integral_constant<int, 2>());
            default: return f(t, v, std::integral_constant<int, kMaxVec>());
        }
    };
    if (a.dtype == KDA_BF16) {
        __nv_bfloat16* t = nullptr;
        return V == 1 ? pick_nv(t, std::integral_constant<int, 1>())
                      : pick_nv(t, std::integral_constant<int, 8>());
    }
    float* t = nullptr;
    return V == 1 ? pick_nv(t, std::integral_constant<int, 1>())
                  : pick_nv(t, std::integral_constant<int, 4>());
}

}  // namespace

size_t norm_backward_bytes(int64_t T, int32_t H, int32_t d) {
    int64_t most = 1;   // over the layouts that a call's strides can lead to
    for (int V : {1, 4, 8}) {
        if (d % V != 0) continue;
        const int64_t n = norm_parts(backward_grid(T, H, d, V));
        if (n > most) most = n;
    }
    return (size_t)most * H * 2 * d * sizeof(float);
}

cudaError_t launch_norm_forward(const NormArgs& a, cudaStream_t stream) {
    const int V = norm_vec(a);
    const NormGrid g = norm_grid(a.T, a.H, a.d, V, 0);
    return by_layout(a, V, g.nv, [&](auto* t, auto v, auto nv) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int V = decltype(v)::value, NV = decltype(nv)::value;
        if constexpr (NV == 0)
            norm_fwd_wide_kernel<T, V><<<(unsigned)(g.tblocks * a.H), kThreads, 0, stream>>>(a, g);
        else
            norm_fwd_kernel<T, V, NV><<<(unsigned)(g.tblocks * g.hblocks), kThreads, 0, stream>>>(a, g);
        return cudaGetLastError();
    });
}

cudaError_t launch_norm_backward(const NormArgs& a, char* ws, cudaStream_t stream) {
    const int V = norm_vec(a);
    const NormGrid g = backward_grid(a.T, a.H, a.d, V);
    float* part = a.dw || a.db ? reinterpret_cast<float*>(ws) : nullptr;
    if (a.T > 0) {
        const cudaError_t err = by_layout(a, V, g.nv, [&](auto* t, auto v, auto nv) {
            using T = std::remove_pointer_t<decltype(t)>;
            constexpr int V = decltype(v)::value, NV = decltype(nv)::value;
            if constexpr (NV == 0)
                norm_bwd_wide_kernel<T, V><<<(unsigned)(g.tblocks * a.H), kThreads, 0, stream>>>(
                    a, g, part);
            else
                norm_bwd_kernel<T, V, NV><<<(unsigned)(g.tblocks * g.hblocks), kThreads, 0, stream>>>(
                    a, g, part);
            return cudaGetLastError();
        });
        if (err != cudaSuccess) return err;
    }
    if (!part) return cudaSuccess;
    const int64_t cols = (int64_t)a.param_heads * 2 * a.d;
    norm_param_sum_kernel<<<(unsigned)((cols + 31) / 32), kThreads, 0, stream>>>(
        part, a.T > 0 ? norm_parts(g) : 0, a.H, a.d, a.param_heads, a.dw, a.db);
    return cudaGetLastError();
}

}  // namespace kda
