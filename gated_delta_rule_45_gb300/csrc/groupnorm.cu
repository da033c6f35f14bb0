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
// Bound: HBM.
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

template <typename T, int V, int NV>
struct Row {
    Pack<T, V> k[NV];
    __device__ __forceinline__ void load(const T* p, int lane, int lanes, int nvec, bool on) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = lane + j * lanes;
            if (on && v < nvec) k[j].load(p + (int64_t)v * V);
            else k[j].zero();
        }
    }
    __device__ __forceinline__ float get(int j, int i) const { return k[j].get(i); }
};

// xh of one row, and its r.
template <typename T, int V, int NV>
__device__ __forceinline__ float normalise(const Row<T, V, NV>& x, float (&xh)[NV][V], int lane,
                                           int lanes, int nvec, int d, bool center, float eps) {
    float m = 0.f;
    if (center) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) m += x.get(j, i);
        m = group_sum(m, lanes) / d;
    }
    float q = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            xh[j][i] = lane + j * lanes < nvec ? x.get(j, i) - m : 0.f;
            q = fmaf(xh[j][i], xh[j][i], q);
        }
    const float r = 1.f / sqrtf(group_sum(q, lanes) / d + eps);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) xh[j][i] *= r;
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

template <typename T, int V, int NV>
__global__ void __launch_bounds__(kThreads)
norm_fwd_kernel(const NormArgs p, const NormGrid g) {
    const NormPlace a = norm_place(p, g);
    const int nvec = p.d / V;
    float w[NV][V], b[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = a.lane + j * g.lanes;
            const bool in = a.on && v < nvec;
            const int64_t at = (p.param_heads == 1 ? 0 : (int64_t)a.h * p.d) + v * V + i;
            w[j][i] = in && p.w ? p.w[at] : 1.f;
            b[j][i] = in && p.b ? p.b[at] : 0.f;
        }
    // (all lanes of a warp take part in its sums, so they leave the loop together)
    for (int64_t t = a.t; __any_sync(0xffffffffu, a.on && t < p.T); t += a.step) {
        const bool on = a.on && t < p.T;
        Row<T, V, NV> x, z;
        x.load(static_cast<const T*>(p.x) + t * p.ldx + (int64_t)a.h * p.d, a.lane, g.lanes, nvec,
               on);
        if (p.z)
            z.load(static_cast<const T*>(p.z) + t * p.ldz + (int64_t)a.h * p.d, a.lane, g.lanes,
                   nvec, on);
        float xh[NV][V];
        normalise(x, xh, a.lane, g.lanes, nvec, p.d, p.center, p.eps);
        T* y = static_cast<T*>(p.y) + (t * p.H + a.h) * p.d;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = a.lane + j * g.lanes;
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float n = fmaf(xh[j][i], w[j][i], b[j][i]);
                o[i] = p.z ? n * activate(z.get(j, i), p.act) : activate(n, p.act);
            }
            Pack<T, V> k;
            k.set(o);
            if (on && v < nvec) k.store(y + (int64_t)v * V);
        }
    }
}

template <typename T, int V, int NV>
__global__ void __launch_bounds__(kThreads)
norm_bwd_kernel(const NormArgs p, const NormGrid g, float* part) {
    const NormPlace a = norm_place(p, g);
    const int nvec = p.d / V;
    float w[NV][V], b[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = a.lane + j * g.lanes;
            const bool in = a.on && v < nvec;
            const int64_t at = (p.param_heads == 1 ? 0 : (int64_t)a.h * p.d) + v * V + i;
            w[j][i] = in && p.w ? p.w[at] : 1.f;
            b[j][i] = in && p.b ? p.b[at] : 0.f;
            dw[j][i] = db[j][i] = 0.f;
        }
    for (int64_t t = a.t; __any_sync(0xffffffffu, a.on && t < p.T); t += a.step) {
        const bool on = a.on && t < p.T;
        const int64_t out = (t * p.H + a.h) * p.d;
        Row<T, V, NV> x, z, dy;
        x.load(static_cast<const T*>(p.x) + t * p.ldx + (int64_t)a.h * p.d, a.lane, g.lanes, nvec,
               on);
        dy.load(static_cast<const T*>(p.dy) + out, a.lane, g.lanes, nvec, on);
        if (p.z)
            z.load(static_cast<const T*>(p.z) + t * p.ldz + (int64_t)a.h * p.d, a.lane, g.lanes,
                   nvec, on);
        float xh[NV][V], gv[NV][V];
        const float r = normalise(x, xh, a.lane, g.lanes, nvec, p.d, p.center, p.eps);
        float s1 = 0.f, s2 = 0.f;   // sums of g xh and of g
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = a.lane + j * g.lanes;
            float dz[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float n = fmaf(xh[j][i], w[j][i], b[j][i]);
                float dv;
                if (p.z) {
                    const float zv = z.get(j, i);
                    dv = dy.get(j, i) * activate(zv, p.act);
                    dz[i] = dy.get(j, i) * n * activate_grad(zv, p.act);
                } else {
                    dv = dy.get(j, i) * activate_grad(n, p.act);
                    dz[i] = 0.f;
                }
                dw[j][i] = fmaf(dv, xh[j][i], dw[j][i]);
                db[j][i] += dv;
                gv[j][i] = dv * w[j][i];
                s1 = fmaf(gv[j][i], xh[j][i], s1);
                s2 += gv[j][i];
            }
            if (p.dz && on && v < nvec) {
#pragma unroll
                for (int i = 0; i < V; i += V < 4 ? V : 4) {
                    constexpr int U = V < 4 ? V : 4;
                    Pack<float, U> k;
                    float o[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) o[u] = dz[i + u];
                    k.set(o);
                    k.store(p.dz + out + (int64_t)v * V + i);
                }
            }
        }
        s1 = group_sum(s1, g.lanes) / p.d;
        s2 = p.center ? group_sum(s2, g.lanes) / p.d : 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int v = a.lane + j * g.lanes;
            if (!on || v >= nvec) continue;
#pragma unroll
            for (int i = 0; i < V; i += V < 4 ? V : 4) {
                constexpr int U = V < 4 ? V : 4;
                Pack<float, U> k;
                float o[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    o[u] = r * (gv[j][i + u] - fmaf(xh[j][i + u], s1, s2));
                k.set(o);
                k.store(p.dx + out + (int64_t)v * V + i);
            }
        }
    }
    if (!part || !a.on) return;
    // part[token part][head][dw, db][d]
    float* row = part + (a.t * p.H + a.h) * 2 * p.d;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = a.lane + j * g.lanes;
        if (v >= nvec) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            row[v * V + i] = dw[j][i];
            row[p.d + v * V + i] = db[j][i];
        }
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
    r = 1.f / sqrtf(block_sum(q, s) / p.d + p.eps);
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
    const int64_t most = (8 * sms + g.hblocks - 1) / g.hblocks;
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
