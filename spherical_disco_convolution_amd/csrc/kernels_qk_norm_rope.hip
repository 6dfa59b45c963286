// Root-mean-square norm of each head of queries and keys, and the rotation of
// its pairs by the token's position, in one pass; and its gradient.
//
//   r = 1/sqrt(1/D sum_d x_d^2 + eps),  n_d = x_d r w_d
//   (y_a, y_b) = (n_a cos f - n_b sin f, n_a sin f + n_b cos f),  f = position * frequency
// and, with gn = gy turned back and t = gn w,
//   gx = r (t - x r^2 1/D sum_d t_d x_d),   gw_d = sum over tokens and heads of gn_d x_d r.
//
// HBM bounds both: each element is read and written once.  A group of lanes
// takes a token and walks over its heads, so that an angle is taken once for all
// heads (in float64: a float32 product has lost the angle of position 10^6).  A
// lane holds V pairs of a head in registers, between the sum and the output, and
// the next heads are on their way meanwhile (without: 73 and 148 us).  33024 tokens of
// 16 heads of 128, bf16: forward 66 us, 4.1 TB/s; gradient 99 us, 4.1 TB/s, and 4 us
// for the weights' sums.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "disco_internal.h"
#include "vector_io.h"

namespace disco {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 1024;    // workgroups of the gradient, and rows of partial sums

// Where a lane's V pairs of slot p lie: elements a .. a + V - 1 and b .. b + V - 1.
// Pairs of the half layout are (i, i + R/2); side by side they are 2 V elements
// in a row, as are the elements behind the R that turn.
struct Place {
    int a, b;
    bool turns, has_a, has_b;
};
template <int V, bool INTER>
__device__ __forceinline__ Place place(int p, int D, int R) {
    Place s;
    const int i = p * V;
    s.turns = i < R / 2;
    if (s.turns && !INTER) {
        s.a = i;
        s.b = i + R / 2;
    } else {
        s.a = s.turns ? 2 * i : R + 2 * (i - R / 2);
        s.b = s.a + V;
    }
    s.has_a = s.a < D;
    s.has_b = s.b < D;
    return s;
}

// a lane's elements of a row as they lie in memory
template <typename T, int V>
struct Raw {
    struct __attribute__((packed, aligned(sizeof(T)))) U { T e[V]; };
    U a, b;
    __device__ __forceinline__ void load(const T* row, const Place& s) {
        if (s.has_a) a = *reinterpret_cast<const U*>(row + s.a);
        if (s.has_b) b = *reinterpret_cast<const U*>(row + s.b);
    }
    __device__ __forceinline__ void get(const Place& s, float* f) const {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            f[i] = s.has_a ? load_f(a.e, i) : 0.0f;
            f[V + i] = s.has_b ? load_f(b.e, i) : 0.0f;
        }
    }
};
template <typename T, int V>
__device__ __forceinline__ void load_pairs(const T* row, const Place& s, float* f) {
    Raw<T, V> r = {};
    r.load(row, s);
    r.get(s, f);
}
template <typename T, int V>
__device__ __forceinline__ void store_pairs(T* row, const Place& s, const float* f) {
    if (s.has_a) store_v<T, V>(row + s.a, f);
    if (s.has_b) store_v<T, V>(row + s.b, f + V);
}

template <int V, bool INTER>
__device__ __forceinline__ void turn(float* f, const float* cs, const float* sn) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float& x = f[INTER ? 2 * i : i];
        float& y = f[INTER ? 2 * i + 1 : V + i];
        const float a = x, b = y;
        x = a * cs[i] - b * sn[i];
        y = a * sn[i] + b * cs[i];
    }
}

// Sum over groups of L lanes: neighbours, pairs, fours and eights by the lane
// crossings of vector instructions
template <int CTRL>
__device__ __forceinline__ float crossed(float v) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
    v += crossed<0xB1>(v);                            // lane ^ 1
    if constexpr (L >= 4) v += crossed<0x4E>(v);      // lane ^ 2
    if constexpr (L >= 8) v += crossed<0x141>(v);     // the other four of eight
    if constexpr (L >= 16) v += crossed<0x140>(v);    // the other eight of sixteen
    if constexpr (L >= 32) v += __shfl_xor(v, 16, 64);
    if constexpr (L >= 64) v += __shfl_xor(v, 32, 64);
    return v;
}

// 1/sqrt(v) to one unit in the last place
__device__ __forceinline__ float inverse_root(float v) {
    if (v < 1e-30f) return 1.0f / sqrtf(v);   // the instruction takes no subnormal numbers
    return __builtin_amdgcn_rsqf(v);
}

template <int V>
__device__ __forceinline__ void angles(const QkCall& c, int64_t tok, int p, bool turns, float sign, float* cs, float* sn) {
    const int pairs = c.rot / 2;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        cs[i] = 1.0f;
        sn[i] = 0.0f;
        if (!turns) continue;
        const int k = p * V + i;
        const int64_t at = tok * c.axes + (int64_t)k * c.axes / pairs;
        const double pos = c.pos_is_int ? (double)((const int32_t*)c.positions)[at] : (double)((const float*)c.positions)[at];
        const double rev = pos * (double)c.inv_freq[k] * 0.15915494309189533577;   // turns
        float s, q;
        sincospif(2.0f * (float)(rev - rint(rev)), &s, &q);
        cs[i] = q;
        sn[i] = sign * s;
    }
}

// The rows of one tensor that a token's lanes walk over
template <typename T>
struct HeadsOf {
    const T* x;
    const T* g;      // gradient of the result, or NULL
    T* y;
    int64_t xs, gs, ys;   // from head to head
    const float* weight;
};

template <typename T>
__device__ __forceinline__ HeadsOf<T> heads_of(const QkCall& c, bool isq, int64_t tok, int h0) {
    if (isq)
        return {(const T*)c.q + tok * c.q_ts + (int64_t)h0 * c.q_hs, c.gq ? (const T*)c.gq + tok * c.gq_ts + (int64_t)h0 * c.gq_hs : nullptr,
                (T*)c.q_out + tok * c.qo_ts + (int64_t)h0 * c.qo_hs, c.q_hs, c.gq_hs, c.qo_hs, c.q_weight};
    return {(const T*)c.k + tok * c.k_ts + (int64_t)h0 * c.k_hs, c.gk ? (const T*)c.gk + tok * c.gk_ts + (int64_t)h0 * c.gk_hs : nullptr,
            (T*)c.k_out + tok * c.ko_ts + (int64_t)h0 * c.ko_hs, c.k_hs, c.gk_hs, c.ko_hs, c.k_weight};
}

template <int V>
__device__ __forceinline__ void load_weight(const float* w, const Place& s, float* f) {
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) f[i] = 1.0f;
    if (w) load_pairs<float, V>(w, s, f);
}

// V pairs a lane and slot, L lanes a token, N slots a lane; U heads are in flight
template <typename T, int V, int L, int N, bool INTER>
__global__ __launch_bounds__(kThreads) void qk_fwd(QkCall c) {
    constexpr int U = V * N >= 8 ? 2 : 4;
    const int lane = threadIdx.x % L;
    const int64_t tok = (int64_t)blockIdx.x * (kThreads / L) + threadIdx.x / L;
    if (tok >= c.tokens) return;
    const int h0 = blockIdx.y * c.heads_each, h1 = min(h0 + c.heads_each, c.hq + c.hkv);
    Place s[N];
    float cs[N][V], sn[N][V];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        s[n] = place<V, INTER>(lane + n * L, c.d, c.rot);
        angles<V>(c, tok, lane + n * L, s[n].turns, 1.0f, cs[n], sn[n]);
    }
    const float inv_d = 1.0f / (float)c.d;
    auto walk = [&](const HeadsOf<T>& t, int heads) {
        float w[N][2 * V];
#pragma unroll
        for (int n = 0; n < N; ++n) load_weight<V>(t.weight, s[n], w[n]);
        Raw<T, V> in[U][N] = {}, next[U][N] = {};
        const T* x = t.x;
        T* y = t.y;
        auto fetch = [&](Raw<T, V> (*r)[N], int h) {   // the last head again behind the end
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const T* row = x;
                if (h + u < heads - 1) x += t.xs;
#pragma unroll
                for (int n = 0; n < N; ++n) r[u][n].load(row, s[n]);
            }
        };
        fetch(in, 0);
        for (int h = 0; h < heads; h += U) {
            if (h + U < heads) fetch(next, h + U);
            float f[U][N][2 * V], sq[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                sq[u] = 0.0f;
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    in[u][n].get(s[n], f[u][n]);
#pragma unroll
                    for (int i = 0; i < 2 * V; ++i) sq[u] = fmaf(f[u][n][i], f[u][n][i], sq[u]);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) sq[u] = group_sum<L>(sq[u]);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float r = inverse_root(sq[u] * inv_d + c.eps);
#pragma unroll
                for (int n = 0; n < N; ++n) {
#pragma unroll
                    for (int i = 0; i < 2 * V; ++i) f[u][n][i] *= r * w[n][i];
                    if (s[n].turns) turn<V, INTER>(f[u][n], cs[n], sn[n]);
                    if (h + u < heads) store_pairs<T, V>(y, s[n], f[u][n]);
                }
                y += t.ys;
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int n = 0; n < N; ++n) in[u][n] = next[u][n];
        }
    };
    if (h0 < c.hq) walk(heads_of<T>(c, true, tok, h0), min(h1, c.hq) - h0);
    if (h1 > c.hq) walk(heads_of<T>(c, false, tok, max(h0 - c.hq, 0)), h1 - max(h0, c.hq));
}

template <typename T, int V, int L, int N, bool INTER>
__global__ __launch_bounds__(kThreads) void qk_bwd(QkCall c) {
    constexpr int TOK = kThreads / L;
    const int lane = threadIdx.x % L;
    const int heads = c.hq + c.hkv;
    Place s[N];
    float gwq[N][2 * V], gwk[N][2 * V];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        s[n] = place<V, INTER>(lane + n * L, c.d, c.rot);
#pragma unroll
        for (int i = 0; i < 2 * V; ++i) gwq[n][i] = gwk[n][i] = 0.0f;
    }
    const float inv_d = 1.0f / (float)c.d;
    // a unit is a token and a share of its heads
    const int64_t units = c.tokens * c.head_parts;
    for (int64_t u0 = (int64_t)blockIdx.x * TOK; u0 < units; u0 += (int64_t)gridDim.x * TOK) {
        const int64_t unit = u0 + threadIdx.x / L;
        if (unit >= units) continue;
        const int64_t tok = c.head_parts == 1 ? unit : unit / c.head_parts;
        const int h0 = (int)(unit - tok * c.head_parts) * c.heads_each, h1 = min(h0 + c.heads_each, heads);
        float cs[N][V], sn[N][V];
#pragma unroll
        for (int n = 0; n < N; ++n) angles<V>(c, tok, lane + n * L, s[n].turns, -1.0f, cs[n], sn[n]);
        auto walk = [&](const HeadsOf<T>& t, int nh, float (*gw)[2 * V]) {
            float w[N][2 * V];
#pragma unroll
            for (int n = 0; n < N; ++n) load_weight<V>(t.weight, s[n], w[n]);
            Raw<T, V> x[N] = {}, g[N] = {}, xn[N] = {}, gn[N] = {};
            const T *xr = t.x, *gr = t.g;
            T* y = t.y;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                x[n].load(xr, s[n]);
                g[n].load(gr, s[n]);
            }
            for (int h = 0; h < nh; ++h) {
                if (h + 1 < nh) {   // the next head is under way
                    xr += t.xs;
                    gr += t.gs;
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        xn[n].load(xr, s[n]);
                        gn[n].load(gr, s[n]);
                    }
                }
                float f[N][2 * V], v[N][2 * V], sq = 0.0f, dot = 0.0f;
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    x[n].get(s[n], f[n]);
                    g[n].get(s[n], v[n]);
                    if (s[n].turns) turn<V, INTER>(v[n], cs[n], sn[n]);
#pragma unroll
                    for (int i = 0; i < 2 * V; ++i) {
                        sq = fmaf(f[n][i], f[n][i], sq);
                        dot = fmaf(f[n][i], v[n][i] * w[n][i], dot);
                    }
                }
                sq = group_sum<L>(sq);
                dot = group_sum<L>(dot);
                const float r = inverse_root(sq * inv_d + c.eps);
                const float back = r * r * inv_d * dot;
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    float o[2 * V];
#pragma unroll
                    for (int i = 0; i < 2 * V; ++i) {
                        o[i] = r * (v[n][i] * w[n][i] - f[n][i] * back);
                        gw[n][i] += v[n][i] * (f[n][i] * r);
                    }
                    store_pairs<T, V>(y, s[n], o);
                    x[n] = xn[n];
                    g[n] = gn[n];
                }
                y += t.ys;
            }
        };
        if (h0 < c.hq) walk(heads_of<T>(c, true, tok, h0), min(h1, c.hq) - h0, gwq);
        if (h1 > c.hq) walk(heads_of<T>(c, false, tok, max(h0 - c.hq, 0)), h1 - max(h0, c.hq), gwk);
    }
    if (!c.partial) return;
    // sums of the workgroup's units: lanes of the same place meet in LDS
    __shared__ float red[kThreads / 64][2][2 * V * N * L];
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 2 * V; ++i) {
            float q = gwq[n][i], k = gwk[n][i];
#pragma unroll
            for (int d = L; d < 64; d *= 2) {
                q += __shfl_xor(q, d, 64);
                k += __shfl_xor(k, d, 64);
            }
            if ((threadIdx.x & 63) < L) {
                const int at = (n * L + lane) * 2 * V + i;
                red[wave][0][at] = q;
                red[wave][1][at] = k;
            }
        }
    __syncthreads();
    if (threadIdx.x >= L) return;
    float* row = c.partial + (int64_t)blockIdx.x * 2 * c.d;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 2 * V; ++i) {
            const int d = i < V ? s[n].a + i : s[n].b + i - V;
            if (!(i < V ? s[n].has_a : s[n].has_b)) continue;
            float q = 0.0f, k = 0.0f;
#pragma unroll
            for (int w = 0; w < kThreads / 64; ++w) {
                q += red[w][0][(n * L + lane) * 2 * V + i];
                k += red[w][1][(n * L + lane) * 2 * V + i];
            }
            row[d] = q;
            row[c.d + d] = k;
        }
}

// Column sums of the partial rows [rows][2 d]: sixteen columns and 64 shares of the
// rows a workgroup, in a fixed order
__global__ __launch_bounds__(1024) void qk_reduce(const float* __restrict__ partial, float* gqw, float* gkw, int rows, int d) {
    __shared__ float red[64][17];
    const int col = blockIdx.x * 16 + (threadIdx.x & 15), part = threadIdx.x >> 4, at = min(col, 2 * d - 1);
    float v = 0.0f;
#pragma unroll 8
    for (int r = part; r < rows; r += 64) v += partial[(int64_t)r * 2 * d + at];
    red[part][threadIdx.x & 15] = v;
    __syncthreads();
    if (threadIdx.x >= 64) return;   // one wave: four lanes a column
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += red[16 * part + i][threadIdx.x & 15];
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
    if (part != 0 || col >= 2 * d) return;
    float* out = col < d ? gqw : gkw;
    if (out) out[col < d ? col : col - d] = v;
}

int bwd_blocks(int64_t units, int L) {
    return (int)std::min<int64_t>((units * L + kThreads - 1) / kThreads, kMaxBlocks);
}

// Pairs a lane holds: whole vectors fall on one side of every border.  33024 tokens
// of 16 heads of 128, bf16: forward eight 66 us, four 69; gradient four 105 us (four
// waves a SIMD), eight 118 (two).
int pairs_a_lane(const QkCall& c) {
    if (c.dtype == DISCO_BF16 && !c.backward && c.rot % 16 == 0 && c.d % 16 == 0) return 8;
    return c.rot % 8 == 0 && c.d % 8 == 0 ? 4 : 1;
}

// Shares of a token's heads: all in one where the tokens alone fill the chip.
// 33024 tokens of 16 heads go in one share each; 8 tokens of 18 heads in 18.
int head_parts(int64_t tokens, int heads, int L) {
    const int64_t waves = (tokens * L + 63) / 64;
    if (waves >= 2048) return 1;
    return (int)std::min<int64_t>(heads, 2048 / std::max<int64_t>(waves, 1));
}

int lanes_of(int d, int V) {
    const int slots = ((d + 1) / 2 + V - 1) / V;
    int L = 4;
    while (L < slots && L < 64) L *= 2;
    return L;
}

template <typename T, int V, int L, int N>
int go(QkCall c, hipStream_t st) {
    const int heads = c.hq + c.hkv;
    c.head_parts = head_parts(c.tokens, heads, L);
    c.heads_each = (heads + c.head_parts - 1) / c.head_parts;
    c.head_parts = (heads + c.heads_each - 1) / c.heads_each;
    if (!c.backward) {   // one launch
        KernelTimer timer("qk_fwd", st);
        const dim3 grid((unsigned)((c.tokens + kThreads / L - 1) / (kThreads / L)), (unsigned)c.head_parts);
        if (c.interleaved) qk_fwd<T, V, L, N, true><<<grid, kThreads, 0, st>>>(c);
        else qk_fwd<T, V, L, N, false><<<grid, kThreads, 0, st>>>(c);
    } else if constexpr (V <= 4) {
        const int blocks = bwd_blocks(c.tokens * c.head_parts, L);
        {
            KernelTimer timer("qk_bwd", st);
            if (c.interleaved) qk_bwd<T, V, L, N, true><<<blocks, kThreads, 0, st>>>(c);
            else qk_bwd<T, V, L, N, false><<<blocks, kThreads, 0, st>>>(c);
        }
        if (c.partial) {
            KernelTimer timer("qk_reduce", st);
            qk_reduce<<<(2 * c.d + 15) / 16, 1024, 0, st>>>(c.partial, c.gq_weight, c.gk_weight, blocks, c.d);
        }
    }
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess) return DISCO_OK;
    return set_error(DISCO_EHIP, "qk_norm_rope: launch failed: %s", hipGetErrorString(e));
}

template <typename T>
int typed(const QkCall& c, hipStream_t st) {
    const int V = pairs_a_lane(c);
    if constexpr (sizeof(T) == 2) {
        if (V == 8) switch (lanes_of(c.d, 8)) {
            case 4: return go<T, 8, 4, 1>(c, st);
            case 8: return go<T, 8, 8, 1>(c, st);
            default: return go<T, 8, 16, 1>(c, st);
        }
    }
    if (V == 4) {
        switch (lanes_of(c.d, 4)) {
            case 4: return go<T, 4, 4, 1>(c, st);
            case 8: return go<T, 4, 8, 1>(c, st);
            case 16: return go<T, 4, 16, 1>(c, st);
            default: return go<T, 4, 32, 1>(c, st);
        }
    }
    if (lanes_of(c.d, 1) <= 16) return go<T, 1, 16, 1>(c, st);
    return go<T, 1, 64, 2>(c, st);
}

}  // namespace

size_t qk_norm_rope_bwd_workspace(int d) { return (size_t)kMaxBlocks * 2 * d * sizeof(float); }

int launch_qk_norm_rope(const QkCall& c, void* stream) {
    hipStream_t st = static_cast<hipStream_t>(stream);
    return c.dtype == DISCO_F32 ? typed<float>(c, st) : typed<bf16_t>(c, st);
}

}  // namespace disco
