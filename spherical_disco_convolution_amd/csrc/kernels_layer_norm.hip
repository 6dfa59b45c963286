// Layer norm over the channels of a tensor seen as [outer, C, inner], and its
// gradient.
//
//   s = x (+ residual, rounded to x's type)
//   mu = 1/C sum_c s,  var = 1/C sum_c (s - mu)^2,  r = 1/sqrt(var + eps)
//   y = (s - mu) r gamma_c + beta_c
// and, with h = (s - mu) r and t = gy gamma_c,
//   gx = r (t - 1/C sum_c t - h 1/C sum_c t h) (+ gsum)
//   ggamma_c = sum_points gy h,   gbeta_c = sum_points gy.
//
// Both directions do about ten operations on an element, so HBM bounds them; the
// kernels hold a point's channels in registers between the statistics and the
// output so that nothing is read twice.  Only the walk kernels, for what registers
// do not hold, read everything two or three times (backward of 181 x 360 points
// float32: 256 channels in registers 56 us, 300 by walks 104 us, 512 186 us; the
// bytes take 40, 47 and 80 us at 5 TB/s).  Forward,
// 721 x 1440 x 128 bf16 with a residual (1.07 GB): 228 us, 4.7 TB/s, where a
// large copy reaches 4.9 to 5.2.
// inner > 1 ("field" kernels): a lane owns V neighbouring points, the waves of
// a workgroup split the channels, and the partial statistics meet in LDS.
// inner == 1 ("row" kernels): a row's channels are spread over 1 to 1024 lanes.
// Statistics are float32 at least: the mean first, then the centred squares (no
// E[x^2] - mu^2), merged across waves as (mean, sum of squares) pairs.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "disco_internal.h"
#include "kernels_common.h"

namespace disco {

namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    bf16x2_t v;
    v[0] = (__bf16)a;
    v[1] = (__bf16)b;
    return __builtin_bit_cast(uint32_t, v);
}

// V consecutive elements of T in 32-bit words, moved with the widest accesses
// that element alignment allows (gfx950 global memory takes dword and wider
// accesses at any element alignment, so rows of odd length need no other path).
template <typename T, int V>
struct Pack;

template <int V>
struct Pack<float, V> {
    float w[V];
    __device__ __forceinline__ float get(int i) const { return w[i]; }
    // nothing to keep unpacked: see the bf16 form
    __device__ __forceinline__ void keep_packed() {}
    __device__ __forceinline__ void load(const float* p) {
        struct __attribute__((packed, aligned(4))) U { float e[V]; };
        const U u = *reinterpret_cast<const U*>(p);
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] = u.e[i];
    }
    __device__ __forceinline__ void load_part(const float* p, int n) {
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] = i < n ? p[i] : 0.0f;
    }
    __device__ __forceinline__ void set(const float* f) {
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] = f[i];
    }
    __device__ __forceinline__ void store(float* p) const {
        struct __attribute__((packed, aligned(4))) U { float e[V]; };
        U u;
#pragma unroll
        for (int i = 0; i < V; ++i) u.e[i] = w[i];
        *reinterpret_cast<U*>(p) = u;
    }
    __device__ __forceinline__ void store_part(float* p, int n) const {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < n) p[i] = w[i];
    }
};

template <int V>
struct Pack<bf16_t, V> {
    static constexpr int W = (V + 1) / 2;
    uint32_t w[W];
    __device__ __forceinline__ float get(int i) const {
        return __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
    }
    // hides the words' values from the compiler, so that it unpacks them again
    // in the next pass instead of holding twice the registers across it
    __device__ __forceinline__ void keep_packed() {
#pragma unroll
        for (int i = 0; i < W; ++i) asm volatile("" : "+v"(w[i]));
    }
    __device__ __forceinline__ void load(const bf16_t* p) {
        if constexpr (V == 1) {
            w[0] = p[0];
        } else {
            struct __attribute__((packed, aligned(2))) U { uint32_t e[W]; };
            const U u = *reinterpret_cast<const U*>(p);
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = u.e[i];
        }
    }
    __device__ __forceinline__ void load_part(const bf16_t* p, int n) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const uint32_t lo = 2 * i < n ? p[2 * i] : 0u;
            const uint32_t hi = 2 * i + 1 < n ? p[2 * i + 1] : 0u;
            w[i] = lo | (hi << 16);
        }
    }
    __device__ __forceinline__ void set(const float* f) {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = pack_bf16(f[2 * i], 2 * i + 1 < V ? f[2 * i + 1] : 0.0f);
    }
    __device__ __forceinline__ void store(bf16_t* p) const {
        if constexpr (V == 1) {
            p[0] = (bf16_t)w[0];
        } else {
            struct __attribute__((packed, aligned(2))) U { uint32_t e[W]; };
            U u;
#pragma unroll
            for (int i = 0; i < W; ++i) u.e[i] = w[i];
            *reinterpret_cast<U*>(p) = u;
        }
    }
    __device__ __forceinline__ void store_part(bf16_t* p, int n) const {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < n) p[i] = (bf16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
};

template <typename T, int V>
__device__ __forceinline__ void load_n(Pack<T, V>& k, const T* p, int n) {
    if (n == V) k.load(p);
    else k.load_part(p, n);
}

template <typename T, int V>
__device__ __forceinline__ void store_n(const Pack<T, V>& k, T* p, int n) {
    if (n == V) k.store(p);
    else k.store_part(p, n);
}

// g / d for a uniform d; the 64-bit division only where the count needs it
__device__ __forceinline__ int64_t split_index(int64_t g, int64_t d, int64_t total) {
    if (total <= d) return 0;
    if (total <= 0x7fffffffLL) return (int64_t)((uint32_t)g / (uint32_t)d);
    return g / d;
}

// ---------------------------------------------------------------------------
// fields: inner > 1
// ---------------------------------------------------------------------------
// blockDim (64, WC, WP): wave (wc, wp) holds channels [wc CPW, wc CPW + CPW) of
// 64 groups of V points; WP independent groups of waves share a workgroup.
// `groups` = ceil(inner / V) per outer index, `total` = outer * groups.
template <typename TX, typename TY, int V, int CPW, bool RES>
__global__ __launch_bounds__(CPW > 16 ? 1024 : 512, 4) void ln_fwd_field(
    const TX* __restrict__ x, const TX* __restrict__ res, const float* __restrict__ gamma,
    const float* __restrict__ beta, TY* __restrict__ y, TX* __restrict__ s,
    float* __restrict__ mean_out, float* __restrict__ rstd_out, int C, int64_t inner,
    int64_t groups, int64_t total, float eps) {
    extern __shared__ __attribute__((aligned(16))) float red[];
    const int lane = threadIdx.x, WC = blockDim.y;
    const int wc = uniform(threadIdx.y), wp = uniform(threadIdx.z);
    // lanes past the end repeat the last group, and a row's last group starts V
    // points before its end (inner >= V): every access is whole, and a point that
    // two lanes hold gets the same value from both
    const int64_t g0 = ((int64_t)blockIdx.x * blockDim.z + wp) * 64 + lane;
    const int64_t g = min(g0, total - 1);
    const int64_t b = split_index(g, groups, total);
    const int64_t n0 = min((g - b * groups) * V, inner - V);
    const int c0 = wc * CPW, nc = min(CPW, C - c0);
    const int64_t o = (b * C + c0) * inner + n0;

    Pack<TX, V> v[CPW];
#pragma unroll
    for (int i = 0; i < CPW; ++i) v[i].load(x + o + (int64_t)min(i, nc - 1) * inner);
    if constexpr (RES) {
#pragma unroll
        for (int i = 0; i < CPW; ++i) {
            Pack<TX, V> r;
            r.load(res + o + (int64_t)min(i, nc - 1) * inner);
            float f[V];
#pragma unroll
            for (int e = 0; e < V; ++e) f[e] = v[i].get(e) + r.get(e);
            v[i].set(f);   // the sum as it is stored: the gradient reads it back
            if (i < nc) v[i].store(s + o + (int64_t)i * inner);
        }
    }

    float mu[V], m2[V];
    const float rn = 1.0f / (float)nc;
#pragma unroll
    for (int e = 0; e < V; ++e) mu[e] = m2[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < CPW; ++i)
        if (i < nc)
#pragma unroll
            for (int e = 0; e < V; ++e) mu[e] += v[i].get(e);
#pragma unroll
    for (int e = 0; e < V; ++e) mu[e] *= rn;
#pragma unroll
    for (int i = 0; i < CPW; ++i) v[i].keep_packed();
#pragma unroll
    for (int i = 0; i < CPW; ++i)
        if (i < nc)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = v[i].get(e) - mu[e];
                m2[e] += d * d;
            }
#pragma unroll
    for (int i = 0; i < CPW; ++i) v[i].keep_packed();
    if (WC > 1) {
        // [wp][wc][mean | squares][64 V]
        float* base = red + (size_t)wp * WC * 128 * V;
        float* mine = base + (size_t)wc * 128 * V + lane * V;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            mine[e] = mu[e];
            mine[64 * V + e] = m2[e];
        }
        __syncthreads();
        const float rc = 1.0f / (float)C;
#pragma unroll
        for (int e = 0; e < V; ++e) mu[e] = m2[e] = 0.0f;
        for (int k = 0; k < WC; ++k) {
            const float w = (float)min(CPW, C - k * CPW) * rc;
            const float* q = base + (size_t)k * 128 * V + lane * V;
#pragma unroll
            for (int e = 0; e < V; ++e) mu[e] += w * q[e];
        }
        for (int k = 0; k < WC; ++k) {
            const float w = (float)min(CPW, C - k * CPW);
            const float* q = base + (size_t)k * 128 * V + lane * V;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = q[e] - mu[e];
                m2[e] += q[64 * V + e] + w * d * d;
            }
        }
    }
    float r[V];
#pragma unroll
    for (int e = 0; e < V; ++e) r[e] = rsqrtf(m2[e] / (float)C + eps);
    if (wc == 0 && mean_out != nullptr) {
        Pack<float, V> k;
        k.set(mu);
        k.store(mean_out + b * inner + n0);
        k.set(r);
        k.store(rstd_out + b * inner + n0);
    }
#pragma unroll
    for (int i = 0; i < CPW; ++i)
        if (i < nc) {
            const float ga = gamma ? gamma[c0 + i] : 1.0f, be = beta ? beta[c0 + i] : 0.0f;
            float f[V];
#pragma unroll
            for (int e = 0; e < V; ++e) f[e] = (v[i].get(e) - mu[e]) * r[e] * ga + be;
            Pack<TY, V> k;
            k.set(f);
            k.store(y + o + (int64_t)i * inner);
        }
}

// More channels than the registers of a workgroup hold: the waves walk the
// channels three times (mean, centred squares, output), a point per lane; the
// second and third walk find the tile in the caches.  Runs of kRun terms of the walk
// kernels' sums are added in float64: in float32 chains of C / 16 (rows: C / 1024)
// terms rstd is 1e-4 off at 2^24 channels.
constexpr int kRun = 64;

template <typename TX, typename TY, bool RES>
__global__ __launch_bounds__(1024) void ln_fwd_field_walk(
    const TX* __restrict__ x, const TX* __restrict__ res, const float* __restrict__ gamma,
    const float* __restrict__ beta, TY* __restrict__ y, TX* __restrict__ s,
    float* __restrict__ mean_out, float* __restrict__ rstd_out, int C, int64_t inner,
    int64_t total, float eps) {
    __shared__ float red[2][16][64];
    const int lane = threadIdx.x;
    const int wc = uniform(threadIdx.y);
    const int64_t g = (int64_t)blockIdx.x * 64 + lane;
    const bool active = g < total;
    const int64_t b = active ? split_index(g, inner, total) : 0;
    const int64_t o = b * C * inner + (active ? g - b * inner : 0);
    double acc = 0.0;
    for (int first = wc; first < C; first += 16 * kRun) {
        const int end = min(C, first + 16 * kRun);
        float run = 0.0f;
        for (int c = first; c < end; c += 16) {
            const int64_t at = o + (int64_t)c * inner;
            float f = active ? load_f(x, at) : 0.0f;
            if constexpr (RES) {
                if (active) {
                    store_f(s, at, f + load_f(res, at));
                    f = load_f(s, at);
                }
            }
            run += f;
        }
        acc += run;
    }
    red[0][wc][lane] = (float)acc;
    __syncthreads();
    float mu = 0.0f;
    for (int k = 0; k < 16; ++k) mu += red[0][k][lane];
    mu /= (float)C;
    const TX* src = RES ? s : x;
    acc = 0.0;
    for (int first = wc; first < C; first += 16 * kRun) {
        const int end = min(C, first + 16 * kRun);
        float run = 0.0f;
        for (int c = first; c < end; c += 16) {
            const float d = active ? load_f(src, o + (int64_t)c * inner) - mu : 0.0f;
            run += d * d;
        }
        acc += run;
    }
    red[1][wc][lane] = (float)acc;
    __syncthreads();
    float m2 = 0.0f;
    for (int k = 0; k < 16; ++k) m2 += red[1][k][lane];
    const float r = rsqrtf(m2 / (float)C + eps);
    if (!active) return;
    if (wc == 0 && mean_out != nullptr) {
        mean_out[g] = mu;
        rstd_out[g] = r;
    }
    for (int c = wc; c < C; c += 16) {
        const int64_t at = o + (int64_t)c * inner;
        store_f(y, at, (load_f(src, at) - mu) * r * (gamma ? gamma[c] : 1.0f) +
                           (beta ? beta[c] : 0.0f));
    }
}

__device__ __forceinline__ float lane_of(float v, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// Sums of N values over a wave's lanes.  Each step a lane passes on the half of
// its values that the lane across keeps, N - 1 exchanges and then one a step for
// the last value instead of 6 N: at the end of a workgroup of 16 waves those
// take longer than a tile (four fields of 256 channels and 65 x 128 points, bf16:
// 29 us in all against 43).  Both halves are read before the choice, which keeps
// them in registers (chosen first: 80 us).  Returns which value's sum v[0] is; lanes that differ in
// the last 6 - log2(N) bits hold the same.
template <int N>
__device__ __forceinline__ int spread_sums(float* v, int lane) {
    int which = 0, m = 32;
#pragma unroll
    for (int half = N / 2; half > 0; half /= 2, m /= 2) {
        const bool upper = (lane & m) != 0;
        which += upper ? half : 0;
#pragma unroll
        for (int k = 0; k < half; ++k) {
            const float low = v[k], high = v[k + half];
            v[k] = (upper ? high : low) + __shfl_xor(upper ? low : high, m);
        }
    }
#pragma unroll
    for (m = 32 / N; m > 0; m /= 2) v[0] += __shfl_xor(v[0], m);
    return which;
}

// Backward of a field.  Persistent workgroups walk tiles of 64 V points; each
// lane keeps its channels' ggamma and gbeta in registers over all its tiles,
// and a workgroup's sums go to partial[block * WP + wp][2][C] at the end.
//
// At C = 128 bf16 with gsum (721 x 1440, 1.07 GB) the tile is two points a lane:
// 110 registers, so that two workgroups of 8 waves share a compute unit and one
// loads while the other waits for its sums: 236 us, 4.5 TB/s.  Four points a
// lane spill (367 us), and loading the next tile ahead with 244 registers and
// one workgroup a unit comes to 281 us.
template <typename TX, typename TG, typename TO, int V, int CPW, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 4) void ln_bwd_field(
    const TX* __restrict__ x, const TG* __restrict__ gy, const float* __restrict__ mean_in,
    const float* __restrict__ rstd_in, const float* __restrict__ gamma,
    const TG* __restrict__ gsum, TO* __restrict__ gx, float* __restrict__ partial, int C,
    int64_t inner, int64_t groups, int64_t total, int64_t tiles) {
    extern __shared__ __attribute__((aligned(16))) float red[];
    const int lane = threadIdx.x, WC = blockDim.y, WP = blockDim.z;
    const int wc = uniform(threadIdx.y), wp = uniform(threadIdx.z);
    const int c0 = wc * CPW, nc = min(CPW, C - c0);
    // read once and kept by a lane each: loads among the products would wait one by one
    const float mine_of_gamma = gamma ? gamma[c0 + min(lane, nc - 1)] : 1.0f;
    float dg[CPW], db[CPW];
#pragma unroll
    for (int i = 0; i < CPW; ++i) dg[i] = db[i] = 0.0f;
    const float rc = 1.0f / (float)C;
    int parity = 0;

    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        // whole accesses only, as in the forward kernel; a lane's first `skip`
        // points are another lane's and stay out of the parameter sums
        const int64_t g0 = (tile * WP + wp) * 64 + lane;
        const int64_t g = min(g0, total - 1);
        const int64_t b = split_index(g, groups, total);
        const int64_t at0 = (g - b * groups) * V, n0 = min(at0, inner - V);
        const int skip = g0 < total ? (int)(at0 - n0) : V;
        const int64_t o = (b * C + c0) * inner + n0;
        Pack<TX, V> vx[CPW];
        Pack<TG, V> vg[CPW], vs[CPW];
        Pack<float, V> mu, r;
        mu.load(mean_in + b * inner + n0);
        r.load(rstd_in + b * inner + n0);
#pragma unroll
        for (int i = 0; i < CPW; ++i) {
            const int64_t at = o + (int64_t)min(i, nc - 1) * inner;
            vx[i].load(x + at);
            vg[i].load(gy + at);
        }
        if (gsum != nullptr)
#pragma unroll
            for (int i = 0; i < CPW; ++i)
                vs[i].load(gsum + o + (int64_t)min(i, nc - 1) * inner);
        float s1[V], s2[V];
#pragma unroll
        for (int e = 0; e < V; ++e) s1[e] = s2[e] = 0.0f;
#pragma unroll
        for (int i = 0; i < CPW; ++i)
            if (i < nc) {
                const float ga = lane_of(mine_of_gamma, i);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float gr = vg[i].get(e);
                    const float h = (vx[i].get(e) - mu.get(e)) * r.get(e);
                    const float t = gr * ga;
                    s1[e] += t;
                    s2[e] += t * h;
                    dg[i] += e >= skip ? gr * h : 0.0f;
                    db[i] += e >= skip ? gr : 0.0f;
                }
            }
#pragma unroll
        for (int i = 0; i < CPW; ++i) {
            vx[i].keep_packed();
            vg[i].keep_packed();
        }
        if (WC > 1) {
            float* base = red + ((size_t)parity * WP + wp) * WC * 128 * V;
            float* mine = base + (size_t)wc * 128 * V + lane * V;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                mine[e] = s1[e];
                mine[64 * V + e] = s2[e];
            }
            // two buffers in turn: the next tile's writes cannot reach a
            // wave that still reads this tile's sums
            __syncthreads();
            parity ^= 1;
#pragma unroll
            for (int e = 0; e < V; ++e) s1[e] = s2[e] = 0.0f;
            for (int k = 0; k < WC; ++k) {
                const float* q = base + (size_t)k * 128 * V + lane * V;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    s1[e] += q[e];
                    s2[e] += q[64 * V + e];
                }
            }
        }
        if (gx != nullptr) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                s1[e] *= rc;
                s2[e] *= rc;
            }
#pragma unroll
            for (int i = 0; i < CPW; ++i)
                if (i < nc) {
                    const float ga = lane_of(mine_of_gamma, i);
                    float f[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float h = (vx[i].get(e) - mu.get(e)) * r.get(e);
                        f[e] = r.get(e) * (vg[i].get(e) * ga - s1[e] - h * s2[e]);
                        if (gsum != nullptr) f[e] += vs[i].get(e);
                    }
                    Pack<TO, V> k;
                    k.set(f);
                    k.store(gx + o + (int64_t)i * inner);
                }
        }
    }
    if (partial != nullptr) {
        float* row = partial + ((size_t)blockIdx.x * WP + wp) * 2 * C;
        float v[2 * CPW];
#pragma unroll
        for (int i = 0; i < CPW; ++i) {
            v[i] = dg[i];
            v[CPW + i] = db[i];
        }
        const int i = spread_sums<2 * CPW>(v, lane), c = i % CPW;
        if ((lane & (32 / CPW - 1)) == 0 && c < nc) row[(i / CPW) * C + c0 + c] = v[0];
    }
}

// gx of a field with more channels than the register kernel holds: two walks.
template <typename TX, typename TG, typename TO>
__global__ __launch_bounds__(1024) void ln_bwd_field_walk(
    const TX* __restrict__ x, const TG* __restrict__ gy, const float* __restrict__ mean_in,
    const float* __restrict__ rstd_in, const float* __restrict__ gamma,
    const TG* __restrict__ gsum, TO* __restrict__ gx, int C, int64_t inner, int64_t total) {
    __shared__ float red[2][16][64];
    const int lane = threadIdx.x;
    const int wc = uniform(threadIdx.y);
    const int64_t g = (int64_t)blockIdx.x * 64 + lane;
    const bool active = g < total;
    const int64_t b = active ? split_index(g, inner, total) : 0;
    const int64_t o = b * C * inner + (active ? g - b * inner : 0);
    const float mu = active ? mean_in[g] : 0.0f, r = active ? rstd_in[g] : 0.0f;
    double a1 = 0.0, a2 = 0.0;
    if (active)
        for (int first = wc; first < C; first += 16 * kRun) {
            const int end = min(C, first + 16 * kRun);
            float run1 = 0.0f, run2 = 0.0f;
            for (int c = first; c < end; c += 16) {
                const int64_t at = o + (int64_t)c * inner;
                const float t = load_f(gy, at) * (gamma ? gamma[c] : 1.0f);
                run1 += t;
                run2 += t * ((load_f(x, at) - mu) * r);
            }
            a1 += run1;
            a2 += run2;
        }
    red[0][wc][lane] = (float)a1;
    red[1][wc][lane] = (float)a2;
    __syncthreads();
    float s1 = 0.0f, s2 = 0.0f;
    for (int k = 0; k < 16; ++k) {
        s1 += red[0][k][lane];
        s2 += red[1][k][lane];
    }
    if (!active) return;
    s1 /= (float)C;
    s2 /= (float)C;
    for (int c = wc; c < C; c += 16) {
        const int64_t at = o + (int64_t)c * inner;
        const float h = (load_f(x, at) - mu) * r;
        float f = r * (load_f(gy, at) * (gamma ? gamma[c] : 1.0f) - s1 - h * s2);
        if (gsum != nullptr) f += load_f(gsum, at);
        store_f(gx, at, f);
    }
}

// ggamma and gbeta partial sums of one channel over one slice of the points:
// grid (C, slices), its first channel `first`; partial[slice][2][C].  For shapes the
// other kernels do not hold in registers.
template <typename TX, typename TG>
__global__ __launch_bounds__(256) void ln_bwd_params_walk(
    const TX* __restrict__ x, const TG* __restrict__ gy, const float* __restrict__ mean_in,
    const float* __restrict__ rstd_in, float* __restrict__ partial, int C, int64_t inner,
    int64_t points, int first) {
    __shared__ float red[2][4];
    const int c = first + (int)blockIdx.x;
    float a = 0.0f, q = 0.0f;
    for (int64_t p = (int64_t)blockIdx.y * 256 + threadIdx.x; p < points;
         p += (int64_t)gridDim.y * 256) {
        const int64_t b = split_index(p, inner, points);
        const int64_t at = (b * C + c) * inner + (p - b * inner);
        const float gr = load_f(gy, at);
        a += gr * ((load_f(x, at) - mean_in[p]) * rstd_in[p]);
        q += gr;
    }
    for (int m = 32; m > 0; m >>= 1) {
        a += __shfl_xor(a, m);
        q += __shfl_xor(q, m);
    }
    if ((threadIdx.x & 63) == 0) {
        red[0][threadIdx.x >> 6] = a;
        red[1][threadIdx.x >> 6] = q;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        float* row = partial + (size_t)blockIdx.y * 2 * C;
        row[c] = red[0][0] + red[0][1] + red[0][2] + red[0][3];
        row[(int64_t)C + c] = red[1][0] + red[1][1] + red[1][2] + red[1][3];
    }
}

// ---------------------------------------------------------------------------
// rows: inner == 1
// ---------------------------------------------------------------------------
// Sum over the `tpr` threads of a row; tpr <= 64: lanes of one wave, else
// tpr / 64 waves through LDS (red: 16 floats; the whole workgroup takes part and
// red is free again at the end).
__device__ __forceinline__ float row_sum(float v, int tpr, float* red) {
    if (tpr <= 64) {
        for (int m = tpr >> 1; m > 0; m >>= 1) v += __shfl_xor(v, m);
        return v;
    }
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
    const int wave = threadIdx.x >> 6, n = tpr >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    const float* mine = red + wave / n * n;
    float t = 0.0f;
    for (int k = 0; k < n; ++k) t += mine[k];
    __syncthreads();
    return t;
}

// Two sums at once in a loop over rows: one barrier, the caller alternating
// between two places of 32 floats from one row to the next.
__device__ __forceinline__ void row_sums(float& a, float& b, int tpr, float* red) {
    for (int m = min(tpr, 64) >> 1; m > 0; m >>= 1) {
        a += __shfl_xor(a, m);
        b += __shfl_xor(b, m);
    }
    if (tpr <= 64) return;
    const int wave = threadIdx.x >> 6, n = tpr >> 6;
    if ((threadIdx.x & 63) == 0) {
        red[2 * wave] = a;
        red[2 * wave + 1] = b;
    }
    __syncthreads();
    const float* mine = red + 2 * (wave / n * n);
    a = b = 0.0f;
    for (int k = 0; k < n; ++k) {
        a += mine[2 * k];
        b += mine[2 * k + 1];
    }
}

// A row's C channels over tpr threads, thread t holding vectors t, t + tpr, ...
template <typename TX, typename TY, int V, int NV, bool RES>
__global__ __launch_bounds__(1024) void ln_fwd_row(
    const TX* __restrict__ x, const TX* __restrict__ res, const float* __restrict__ gamma,
    const float* __restrict__ beta, TY* __restrict__ y, TX* __restrict__ s,
    float* __restrict__ mean_out, float* __restrict__ rstd_out, int C, int64_t rows, int tpr,
    float eps) {
    __shared__ float red[16];
    const int t = threadIdx.x & (tpr - 1);
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
    const bool active = row < rows;
    const int64_t o = active ? row * C : 0;
    Pack<TX, V> v[NV];
    int nv[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * tpr + t) * V;
        nv[j] = active ? max(0, min(V, C - c)) : 0;
        if (nv[j] > 0) load_n(v[j], x + o + c, nv[j]);
        else v[j].load_part(x, 0);
    }
    if constexpr (RES) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (nv[j] > 0) {
                const int c = (j * tpr + t) * V;
                Pack<TX, V> k;
                load_n(k, res + o + c, nv[j]);
                float f[V];
#pragma unroll
                for (int e = 0; e < V; ++e) f[e] = v[j].get(e) + k.get(e);
                v[j].set(f);
                store_n(v[j], s + o + c, nv[j]);
            }
    }
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) a += v[j].get(e);
    const float mu = row_sum(a, tpr, red) / (float)C;
    a = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < nv[j]) {
                const float d = v[j].get(e) - mu;
                a += d * d;
            }
    const float r = rsqrtf(row_sum(a, tpr, red) / (float)C + eps);
    if (!active) return;
    if (t == 0 && mean_out != nullptr) {
        mean_out[row] = mu;
        rstd_out[row] = r;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (nv[j] > 0) {
            const int c = (j * tpr + t) * V;
            Pack<float, V> ga, be;
            if (gamma) load_n(ga, gamma + c, nv[j]);
            if (beta) load_n(be, beta + c, nv[j]);
            float f[V];
#pragma unroll
            for (int e = 0; e < V; ++e)
                f[e] = (v[j].get(e) - mu) * r * (gamma ? ga.get(e) : 1.0f) +
                       (beta ? be.get(e) : 0.0f);
            Pack<TY, V> k;
            k.set(f);
            store_n(k, y + o + c, nv[j]);
        }
}

// Rows too long for the registers of a workgroup: three walks, a workgroup a row.
template <typename TX, typename TY, bool RES>
__global__ __launch_bounds__(1024) void ln_fwd_row_walk(
    const TX* __restrict__ x, const TX* __restrict__ res, const float* __restrict__ gamma,
    const float* __restrict__ beta, TY* __restrict__ y, TX* __restrict__ s,
    float* __restrict__ mean_out, float* __restrict__ rstd_out, int C, float eps) {
    __shared__ float red[16];
    const int64_t row = blockIdx.x, o = row * C;
    double a = 0.0;
    for (int first = threadIdx.x; first < C; first += 1024 * kRun) {
        const int end = min(C, first + 1024 * kRun);
        float run = 0.0f;
        for (int c = first; c < end; c += 1024) {
            float f = load_f(x, o + c);
            if constexpr (RES) {
                store_f(s, o + c, f + load_f(res, o + c));
                f = load_f(s, o + c);
            }
            run += f;
        }
        a += run;
    }
    const float mu = row_sum((float)a, 1024, red) / (float)C;
    const TX* src = RES ? s : x;
    a = 0.0;
    for (int first = threadIdx.x; first < C; first += 1024 * kRun) {
        const int end = min(C, first + 1024 * kRun);
        float run = 0.0f;
        for (int c = first; c < end; c += 1024) {
            const float d = load_f(src, o + c) - mu;
            run += d * d;
        }
        a += run;
    }
    const float r = rsqrtf(row_sum((float)a, 1024, red) / (float)C + eps);
    if (threadIdx.x == 0 && mean_out != nullptr) {
        mean_out[row] = mu;
        rstd_out[row] = r;
    }
    for (int c = threadIdx.x; c < C; c += 1024)
        store_f(y, o + c, (load_f(src, o + c) - mu) * r * (gamma ? gamma[c] : 1.0f) +
                              (beta ? beta[c] : 0.0f));
}

// Backward of rows.  Persistent workgroups of blockDim / tpr row slots; each
// thread keeps the parameter sums of its channels in registers over all its
// rows, and the slots are added in LDS, in slot order, at the end, so that a
// workgroup leaves one row of partial sums.  gamma waits in LDS.  HBM bounds it:
// 16384 rows of 2048 bf16 (201 MB) take 51 us, 3.9 TB/s, the second launch 4 us
// of them (46 us repeated on the same tensors, whose 201 MB the last cache partly
// keeps); the same in float32 85 us, 4.7 TB/s.
template <typename TX, typename TG, typename TO, int V, int NV>
__global__ __launch_bounds__(1024) void ln_bwd_row(
    const TX* __restrict__ x, const TG* __restrict__ gy, const float* __restrict__ mean_in,
    const float* __restrict__ rstd_in, const float* __restrict__ gamma,
    const TG* __restrict__ gsum, TO* __restrict__ gx, float* __restrict__ partial, int C,
    int64_t rows, int tpr) {
    extern __shared__ __attribute__((aligned(16))) float lds[];   // 64 floats, then gamma or the sums
    float* red = lds;
    float* vec = lds + 64;
    int odd = 0;
    const int t = threadIdx.x & (tpr - 1);
    const int slots = blockDim.x / tpr, slot = threadIdx.x / tpr;
    float dg[NV][V], db[NV][V];
    int nc[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        nc[j] = max(0, min(V, C - (j * tpr + t) * V));
#pragma unroll
        for (int e = 0; e < V; ++e) dg[j][e] = db[j][e] = 0.0f;
    }
    // padded to whole vectors with zeros: channels past C add nothing
    for (int c = threadIdx.x; c < NV * tpr * V; c += blockDim.x)
        vec[c] = c < C ? (gamma ? gamma[c] : 1.0f) : 0.0f;
    __syncthreads();
    const float rc = 1.0f / (float)C;
    // every thread takes part in each step's sums, with zeros past the last row
    for (int64_t row0 = (int64_t)blockIdx.x * slots; row0 < rows;
         row0 += (int64_t)gridDim.x * slots) {
        const int64_t row = row0 + slot;
        const bool active = row < rows;
        const int64_t o = active ? row * C : 0;
        Pack<TX, V> vx[NV];
        Pack<TG, V> vg[NV];
        const float mu = active ? mean_in[row] : 0.0f, r = active ? rstd_in[row] : 0.0f;
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * tpr + t) * V, n = active ? nc[j] : 0;
            if (n > 0) {
                load_n(vx[j], x + o + c, n);
                load_n(vg[j], gy + o + c, n);
            } else {
                vx[j].load_part(x, 0);
                vg[j].load_part(gy, 0);
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const float* ga = vec + (j * tpr + t) * V;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float gr = vg[j].get(e);   // zero past C
                const float h = (vx[j].get(e) - mu) * r;
                const float q = gr * ga[e];
                s1 += q;
                s2 += q * h;
                dg[j][e] += gr * h;
                db[j][e] += gr;
            }
            vx[j].keep_packed();
            vg[j].keep_packed();
        }
        row_sums(s1, s2, tpr, red + odd);
        odd ^= 32;
        s1 *= rc;
        s2 *= rc;
        if (gx != nullptr && active) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (nc[j] > 0) {
                    const int c = (j * tpr + t) * V;
                    const float* ga = vec + c;
                    float f[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float h = (vx[j].get(e) - mu) * r;
                        f[e] = r * (vg[j].get(e) * ga[e] - s1 - h * s2);
                    }
                    if (gsum != nullptr) {
                        Pack<TG, V> k;
                        load_n(k, gsum + o + c, nc[j]);
#pragma unroll
                        for (int e = 0; e < V; ++e) f[e] += k.get(e);
                    }
                    Pack<TO, V> k;
                    k.set(f);
                    store_n(k, gx + o + c, nc[j]);
                }
        }
    }
    if (partial == nullptr) return;
    float* row = partial + (size_t)blockIdx.x * 2 * C;
    if (slots == 1) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * tpr + t) * V;
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (e < nc[j]) {
                    row[c + e] = dg[j][e];
                    row[C + c + e] = db[j][e];
                }
        }
        return;
    }
    // lanes of one wave that hold the same channels (tpr < 64) first
    for (int m = 32; m >= tpr; m >>= 1)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                dg[j][e] += __shfl_xor(dg[j][e], m);
                db[j][e] += __shfl_xor(db[j][e], m);
            }
    __syncthreads();   // gamma has been read
    // then the waves (or groups of tpr / 64 waves) one after another
    const int turn = tpr < 64 ? threadIdx.x >> 6 : slot;
    const int turns = tpr < 64 ? blockDim.x >> 6 : slots;
    const bool holds = tpr >= 64 || (threadIdx.x & 63) < tpr;
    for (int w = 0; w < turns; ++w) {
        if (w == turn && holds)
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * tpr + t) * V;
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (e < nc[j]) {
                        vec[c + e] = dg[j][e] + (w ? vec[c + e] : 0.0f);
                        vec[C + c + e] = db[j][e] + (w ? vec[C + c + e] : 0.0f);
                    }
            }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < 2 * C; i += blockDim.x) row[i] = vec[i];
}

// gx of rows too long for the registers: two walks, a workgroup a row.
template <typename TX, typename TG, typename TO>
__global__ __launch_bounds__(1024) void ln_bwd_row_walk(
    const TX* __restrict__ x, const TG* __restrict__ gy, const float* __restrict__ mean_in,
    const float* __restrict__ rstd_in, const float* __restrict__ gamma,
    const TG* __restrict__ gsum, TO* __restrict__ gx, int C) {
    __shared__ float red[16];
    const int64_t row = blockIdx.x, o = row * C;
    const float mu = mean_in[row], r = rstd_in[row];
    double a1 = 0.0, a2 = 0.0;
    for (int first = threadIdx.x; first < C; first += 1024 * kRun) {
        const int end = min(C, first + 1024 * kRun);
        float run1 = 0.0f, run2 = 0.0f;
        for (int c = first; c < end; c += 1024) {
            const float q = load_f(gy, o + c) * (gamma ? gamma[c] : 1.0f);
            run1 += q;
            run2 += q * ((load_f(x, o + c) - mu) * r);
        }
        a1 += run1;
        a2 += run2;
    }
    const float s1 = row_sum((float)a1, 1024, red) / (float)C;
    const float s2 = row_sum((float)a2, 1024, red) / (float)C;
    for (int c = threadIdx.x; c < C; c += 1024) {
        const float h = (load_f(x, o + c) - mu) * r;
        float f = r * (load_f(gy, o + c) * (gamma ? gamma[c] : 1.0f) - s1 - h * s2);
        if (gsum != nullptr) f += load_f(gsum, o + c);
        store_f(gx, o + c, f);
    }
}

// ggamma, gbeta partials of a slice of rows, a channel per thread:
// grid (ceil(C / 256), slices).
template <typename TX, typename TG>
__global__ __launch_bounds__(256) void ln_bwd_row_params_walk(
    const TX* __restrict__ x, const TG* __restrict__ gy, const float* __restrict__ mean_in,
    const float* __restrict__ rstd_in, float* __restrict__ partial, int C, int64_t rows) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= C) return;
    float a = 0.0f, q = 0.0f;
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        const float gr = load_f(gy, row * C + c);
        a += gr * ((load_f(x, row * C + c) - mean_in[row]) * rstd_in[row]);
        q += gr;
    }
    partial[(size_t)blockIdx.y * 2 * C + c] = a;
    partial[(size_t)blockIdx.y * 2 * C + C + c] = q;
}

// ggamma and gbeta from partial[n][2][C]: 16 columns a workgroup, the rows in 64
// interleaved slices, added in a fixed order; a launch starts at column `first`.
__global__ __launch_bounds__(1024) void ln_reduce_params(const float* __restrict__ partial, int n,
                                                         int C, int64_t first,
                                                         float* __restrict__ ggamma,
                                                         float* __restrict__ gbeta) {
    __shared__ float red[64][17];
    const int col = threadIdx.x & 15, slice = threadIdx.x >> 4;
    const int64_t i = first + (int64_t)blockIdx.x * 16 + col;
    float a = 0.0f;
    if (i < 2 * (int64_t)C) {
#pragma unroll 8
        for (int k = slice; k < n; k += 64) a += partial[(size_t)k * 2 * C + i];
    }
    red[slice][col] = a;
    __syncthreads();
    if (slice == 0 && i < 2 * (int64_t)C) {
        a = 0.0f;
#pragma unroll
        for (int k = 0; k < 64; ++k) a += red[k][col];
        if (i < C) {
            if (ggamma) ggamma[i] = a;
        } else if (gbeta) {
            gbeta[i - C] = a;
        }
    }
}

// ---------------------------------------------------------------------------
// launch shapes
// ---------------------------------------------------------------------------
constexpr int kMaxWaves = 16;
constexpr int kFwdMaxCpw = 32, kBwdMaxCpw = 16;

// Channels a wave holds and the waves over the channels.
struct FieldShape {
    int cpw = 0, wc = 0, wp = 0;
};

FieldShape field_shape(int C, int max_cpw) {
    FieldShape f;
    if (C > max_cpw * kMaxWaves) return f;   // walk kernels
    f.cpw = 4;
    while (f.cpw < max_cpw && (C + f.cpw - 1) / f.cpw > 8) f.cpw *= 2;
    if (f.cpw == 4 && C > 4) f.cpw = 8;
    f.wc = (C + f.cpw - 1) / f.cpw;
    f.wp = f.wc >= 4 ? 1 : 4 / f.wc;
    return f;
}

struct RowShape {
    int nv = 0, tpr = 0, threads = 0;
};

// Vectors a thread holds and threads a row: one vector a thread for few rows
// (the shortest chain), up to four when there are rows enough to fill the chip.
RowShape row_shape(int C, int64_t rows, int v) {
    RowShape r;
    const int64_t vecs = ((int64_t)C + v - 1) / v;
    if (vecs > 4 * 1024) return r;
    const int want = rows >= 2048 ? 4 : 1;
    r.nv = 1;
    r.tpr = 1;
    while ((int64_t)r.tpr * want < vecs && r.tpr < 1024) r.tpr *= 2;
    if (r.tpr < 64 && want > 1) {   // short rows: one vector a lane while a wave holds the row
        r.tpr = 1;
        while (r.tpr < vecs && r.tpr < 64) r.tpr *= 2;
    }
    while ((int64_t)r.tpr * r.nv < vecs) r.nv *= 2;
    r.threads = r.tpr <= 64 ? 256 : r.tpr;   // longer rows: a workgroup each
    return r;
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A launch may have at most 2^32 - 1 threads (more are cut off without an error): the
// sums of more channels than that take several launches of up to 2^31.
constexpr int64_t kLaunchThreads = (int64_t)1 << 31;
bool fits(int64_t grid, int threads) { return grid <= 0xffffffffLL / threads && grid <= 0x7fffffff; }

int done(const char* what) {
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return set_error(DISCO_EHIP, "%s launch failed: %s", what, hipGetErrorString(e));
    return DISCO_OK;
}

template <typename K>
int allow_lds(K* kernel, size_t bytes) {
    if (bytes <= 65536) return DISCO_OK;
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == hipSuccess) return DISCO_OK;
    (void)hipGetLastError();
    return set_error(DISCO_EHIP, "layer norm: %zu bytes of LDS refused: %s", bytes,
                     hipGetErrorString(e));
}

template <typename TX, typename TY, bool RES>
int fwd_typed(const TX* x, const TX* res, const float* gamma, const float* beta, TY* y, TX* s,
              float* mean, float* rstd, int64_t outer, int C, int64_t inner, float eps,
              hipStream_t st) {
    constexpr int V16 = 16 / sizeof(TX);
    if (inner == 1) {
        const RowShape r = row_shape(C, outer, V16);
        if (r.nv == 0) {
            if (!fits(outer, 1024)) return set_error(DISCO_EUNSUPPORTED, "too many rows");
            KernelTimer timer("ln_fwd_row_walk", st);
            hipLaunchKernelGGL((ln_fwd_row_walk<TX, TY, RES>), dim3((unsigned)outer), dim3(1024), 0,
                               st, x, res, gamma, beta, y, s, mean, rstd, C, eps);
            return done("ln_fwd_row_walk");
        }
        const int64_t grid = cdiv(outer, r.threads / r.tpr);
        if (!fits(grid, r.threads)) return set_error(DISCO_EUNSUPPORTED, "too many rows");
        KernelTimer timer("ln_fwd_row", st);
#define DISCO_LN(NV)                                                                             \
    hipLaunchKernelGGL((ln_fwd_row<TX, TY, V16, NV, RES>), dim3((unsigned)grid), dim3(r.threads), 0, \
                       st, x, res, gamma, beta, y, s, mean, rstd, C, outer, r.tpr, eps)
        if (r.nv == 1) DISCO_LN(1);
        else if (r.nv == 2) DISCO_LN(2);
        else DISCO_LN(4);
#undef DISCO_LN
        return done("ln_fwd_row");
    }
    const FieldShape f = field_shape(C, kFwdMaxCpw);
    if (f.cpw == 0) {
        const int64_t total = outer * inner, grid = cdiv(total, 64);
        if (!fits(grid, 1024)) return set_error(DISCO_EUNSUPPORTED, "too many points");
        KernelTimer timer("ln_fwd_field_walk", st);
        hipLaunchKernelGGL((ln_fwd_field_walk<TX, TY, RES>), dim3((unsigned)grid), dim3(64, 16), 0,
                           st, x, res, gamma, beta, y, s, mean, rstd, C, inner, total, eps);
        return done("ln_fwd_field_walk");
    }
    // 16 bytes a lane (8 where a wave holds 32 channels: 64 registers of data
    // either way) where that leaves 512 workgroups, else a point a lane; the step is
    // felt by bf16 fields just below it (128 x 361 x 720: 41 us, the bytes take 27)
    const int vw = f.cpw > 16 ? V16 / 2 : V16;
    const bool wide = inner >= vw && outer * cdiv(inner, vw) >= (int64_t)512 * 64 * f.wp;
    const int V = wide ? vw : 1;
    const int64_t groups = cdiv(inner, V), total = outer * groups, grid = cdiv(total, 64 * f.wp);
    if (!fits(grid, 64 * f.wc * f.wp)) return set_error(DISCO_EUNSUPPORTED, "too many points");
    const size_t lds = f.wc > 1 ? (size_t)f.wc * f.wp * 128 * V * sizeof(float) : 0;
    KernelTimer timer("ln_fwd_field", st);
#define DISCO_LN(VV, CPW)                                                                        \
    hipLaunchKernelGGL((ln_fwd_field<TX, TY, VV, CPW, RES>), dim3((unsigned)grid),               \
                       dim3(64, f.wc, f.wp), lds, st, x, res, gamma, beta, y, s, mean, rstd, C,  \
                       inner, groups, total, eps)
#define DISCO_LN_V(VW, CPW)         \
    do {                            \
        if (wide) DISCO_LN(VW, CPW); \
        else DISCO_LN(1, CPW);      \
    } while (0)
    switch (f.cpw) {
        case 4: DISCO_LN_V(V16, 4); break;
        case 8: DISCO_LN_V(V16, 8); break;
        case 16: DISCO_LN_V(V16, 16); break;
        default: DISCO_LN_V(V16 / 2, 32); break;
    }
#undef DISCO_LN_V
#undef DISCO_LN
    return done("ln_fwd_field");
}

// The backward kernel's.  One vector a thread and 512 threads a workgroup, two of
// them a compute unit: 16384 rows of 2048 bf16 take 46 us, with four vectors (64
// sums a thread, one workgroup a unit) 62 us, repeated on the same tensors.  Fewer than
// 8192 rows over 512 threads and more get workgroups of 1024, one a unit: half as
// many rows of partial sums (1024 rows of 4096 bf16: 21 us against 29; 16384 of
// 2048 float32: 103 us against 85), and up to 16 channels a thread to leave room
// for two rows (4096 rows of 8192 bf16: 52 us against 62).
struct BwdRowShape : RowShape {
    int slots = 0;
    int grid = 0;
};

BwdRowShape bwd_row_shape(int C, int64_t rows, int v) {
    BwdRowShape r;
    const int vecs = (int)(((int64_t)C + v - 1) / v);
    if (C > 16384) return r;   // walk kernels
    r.tpr = 1;
    while (r.tpr < vecs && r.tpr < 512) r.tpr *= 2;
    if (16 * r.tpr < C) r.tpr = 1024;
    r.nv = 1;
    while (r.tpr * r.nv < vecs) r.nv *= 2;
    const int most = r.tpr >= 512 && rows < 8192 ? 1024 : 512;
    r.slots = std::max(1, 256 / r.tpr);
    while (r.slots * 2 * r.tpr <= most && rows >= (int64_t)256 * 2 * r.slots) r.slots *= 2;
    r.threads = r.slots * r.tpr;
    r.grid = (int)std::min<int64_t>(r.threads > 512 ? 256 : 512, cdiv(rows, r.slots));
    return r;
}

constexpr int kBwdFieldGrid = 512;

// at most this many rows of partial parameter sums
int bwd_partial_rows(int64_t outer, int C, int64_t inner) {
    if (inner == 1) {
        int n = 0;
        for (int v : {4, 8}) {   // whichever vector length the types give
            const BwdRowShape r = bwd_row_shape(C, outer, v);
            n = std::max(n, r.nv == 0 ? (int)std::min<int64_t>(64, outer) : r.grid);
        }
        return n;
    }
    const FieldShape f = field_shape(C, kBwdMaxCpw);
    if (f.cpw == 0) return (int)std::min<int64_t>(64, cdiv(outer * inner, 256));
    return (int)std::min<int64_t>(kBwdFieldGrid, cdiv(outer * inner, 64 * f.wp)) * f.wp;
}

template <typename TX, typename TG, typename TO>
int bwd_typed(const TX* x, const TG* gy, const float* mean, const float* rstd, const float* gamma,
              const TG* gsum, TO* gx, float* ggamma, float* gbeta, float* partial, int64_t outer,
              int C, int64_t inner, hipStream_t st) {
    // points a lane: 4 bytes of each tensor at 16 channels a wave, else 8
    constexpr int V = sizeof(TX) + sizeof(TG) == 4 ? 4 : 2;
    constexpr int VR = sizeof(TX) + sizeof(TG) == 4 ? 8 : 4;   // row kernel
    const bool params = ggamma != nullptr || gbeta != nullptr;
    float* part = params ? partial : nullptr;
    int n = 0;
    if (inner == 1) {
        const BwdRowShape r = bwd_row_shape(C, outer, VR);
        if (r.nv == 0) {
            if (!fits(outer, 1024)) return set_error(DISCO_EUNSUPPORTED, "too many rows");
            if (gx != nullptr) {
                KernelTimer timer("ln_bwd_row_walk", st);
                hipLaunchKernelGGL((ln_bwd_row_walk<TX, TG, TO>), dim3((unsigned)outer), dim3(1024),
                                   0, st, x, gy, mean, rstd, gamma, gsum, gx, C);
                if (int rc = done("ln_bwd_row_walk")) return rc;
            }
            if (params) {
                n = (int)std::min<int64_t>(64, outer);
                KernelTimer timer("ln_bwd_row_params_walk", st);
                hipLaunchKernelGGL((ln_bwd_row_params_walk<TX, TG>),
                                   dim3((unsigned)cdiv(C, 256), n), dim3(256), 0, st, x, gy, mean,
                                   rstd, part, C, outer);
                if (int rc = done("ln_bwd_row_params_walk")) return rc;
            }
        } else {
            n = r.grid;
            const size_t lds =
                (64 + std::max<size_t>((size_t)r.nv * r.tpr * VR, r.slots > 1 ? 2 * (size_t)C : 0)) *
                sizeof(float);   // up to 64.25 KB
            KernelTimer timer("ln_bwd_row", st);
#define DISCO_LN(NV)                                                                               \
    do {                                                                                           \
        if (int rc = allow_lds(&ln_bwd_row<TX, TG, TO, VR, NV>, lds)) return rc;                   \
        hipLaunchKernelGGL((ln_bwd_row<TX, TG, TO, VR, NV>), dim3(n), dim3(r.threads), lds, st, x, \
                           gy, mean, rstd, gamma, gsum, gx, part, C, outer, r.tpr);                \
    } while (0)
            if (r.nv == 1) DISCO_LN(1);
            else if (r.nv == 2) DISCO_LN(2);
            else if constexpr (VR == 4) DISCO_LN(4);   // 16 channels at most
#undef DISCO_LN
            if (int rc = done("ln_bwd_row")) return rc;
        }
    } else {
        const FieldShape f = field_shape(C, kBwdMaxCpw);
        if (f.cpw == 0) {
            const int64_t total = outer * inner, grid = cdiv(total, 64);
            if (!fits(grid, 1024)) return set_error(DISCO_EUNSUPPORTED, "too many points");
            if (gx != nullptr) {
                KernelTimer timer("ln_bwd_field_walk", st);
                hipLaunchKernelGGL((ln_bwd_field_walk<TX, TG, TO>), dim3((unsigned)grid),
                                   dim3(64, 16), 0, st, x, gy, mean, rstd, gamma, gsum, gx, C,
                                   inner, total);
                if (int rc = done("ln_bwd_field_walk")) return rc;
            }
            if (params) {
                n = (int)std::min<int64_t>(64, cdiv(total, 256));
                constexpr int64_t kChannels = kLaunchThreads / 256;
                for (int64_t c = 0; c < C; c += kChannels) {
                    KernelTimer timer("ln_bwd_params_walk", st);
                    hipLaunchKernelGGL((ln_bwd_params_walk<TX, TG>),
                                       dim3((unsigned)std::min(C - c, kChannels), n), dim3(256), 0, st, x,
                                       gy, mean, rstd, part, C, inner, total, (int)c);
                    if (int rc = done("ln_bwd_params_walk")) return rc;
                }
            }
        } else {
            const int vw = f.cpw == 16 ? V / 2 : V;
            const bool wide = inner >= vw && outer * cdiv(inner, vw) >= (int64_t)512 * 64 * f.wp;
            const int VV = wide ? vw : 1;
            const int64_t groups = cdiv(inner, VV), total = outer * groups;
            const int64_t tiles = cdiv(total, 64 * f.wp);
            const int grid = (int)std::min<int64_t>(kBwdFieldGrid, tiles);
            n = grid * f.wp;
            const size_t lds = f.wc > 1 ? (size_t)2 * f.wc * f.wp * 128 * VV * sizeof(float) : 0;
            KernelTimer timer("ln_bwd_field", st);
#define DISCO_LN(VW, CPW, WAVES)                                                                \
    hipLaunchKernelGGL((ln_bwd_field<TX, TG, TO, VW, CPW, WAVES>), dim3(grid),           \
                       dim3(64, f.wc, f.wp), lds, st, x, gy, mean, rstd, gamma, gsum, gx, part, C, \
                       inner, groups, total, tiles)
#define DISCO_LN_V(VW, CPW, WAVES)             \
    do {                                       \
        if (wide) DISCO_LN(VW, CPW, WAVES);    \
        else DISCO_LN(1, CPW, WAVES);          \
    } while (0)
            if (f.cpw == 4) DISCO_LN_V(V, 4, 8);
            else if (f.cpw == 8) DISCO_LN_V(V, 8, 8);
            else if (f.wc <= 8) DISCO_LN_V(V / 2, 16, 8);
            else DISCO_LN_V(V / 2, 16, 16);
#undef DISCO_LN_V
#undef DISCO_LN
            if (int rc = done("ln_bwd_field")) return rc;
        }
    }
    if (!params) return DISCO_OK;
    constexpr int64_t kColumns = kLaunchThreads / 1024 * 16;
    for (int64_t i = 0; i < 2 * (int64_t)C; i += kColumns) {
        KernelTimer timer("ln_reduce_params", st);
        hipLaunchKernelGGL(ln_reduce_params, dim3((unsigned)cdiv(std::min(2 * (int64_t)C - i, kColumns), 16)),
                           dim3(1024), 0, st, partial, n, C, i, ggamma, gbeta);
        if (int rc = done("ln_reduce_params")) return rc;
    }
    return DISCO_OK;
}

}  // namespace

size_t layer_norm_bwd_workspace(int64_t outer, int C, int64_t inner) {
    return (size_t)bwd_partial_rows(outer, C, inner) * 2 * C * sizeof(float);
}

int launch_layer_norm_fwd(const void* x, int x_dtype, const void* res, const float* gamma,
                          const float* beta, void* y, int y_dtype, void* s, float* mean,
                          float* rstd, int64_t outer, int C, int64_t inner, float eps,
                          void* stream) {
    hipStream_t st = static_cast<hipStream_t>(stream);
#define DISCO_LN(TX, TY, R)                                                                      \
    return fwd_typed<TX, TY, R>((const TX*)x, (const TX*)res, gamma, beta, (TY*)y, (TX*)s, mean, \
                                rstd, outer, C, inner, eps, st)
#define DISCO_LN_R(TX, TY)                 \
    do {                                   \
        if (res) DISCO_LN(TX, TY, true);   \
        else DISCO_LN(TX, TY, false);      \
    } while (0)
    if (x_dtype == DISCO_F32) {
        if (y_dtype == DISCO_F32) DISCO_LN_R(float, float);
        else DISCO_LN_R(float, bf16_t);
    } else {
        if (y_dtype == DISCO_F32) DISCO_LN_R(bf16_t, float);
        else DISCO_LN_R(bf16_t, bf16_t);
    }
#undef DISCO_LN_R
#undef DISCO_LN
    return DISCO_OK;
}

int launch_layer_norm_bwd(const void* x, int x_dtype, const void* gy, int gy_dtype,
                          const float* mean, const float* rstd, const float* gamma,
                          const void* gsum, void* gx, int gx_dtype, float* ggamma, float* gbeta,
                          float* partial, int64_t outer, int C, int64_t inner, void* stream) {
    hipStream_t st = static_cast<hipStream_t>(stream);
#define DISCO_LN(TX, TG, TO)                                                                   \
    return bwd_typed<TX, TG, TO>((const TX*)x, (const TG*)gy, mean, rstd, gamma, (const TG*)gsum, \
                                 (TO*)gx, ggamma, gbeta, partial, outer, C, inner, st)
#define DISCO_LN_O(TX, TG)                              \
    do {                                                \
        if (gx_dtype == DISCO_F32) DISCO_LN(TX, TG, float); \
        else DISCO_LN(TX, TG, bf16_t);                  \
    } while (0)
    if (x_dtype == DISCO_F32) {
        if (gy_dtype == DISCO_F32) DISCO_LN_O(float, float);
        else DISCO_LN_O(float, bf16_t);
    } else {
        if (gy_dtype == DISCO_F32) DISCO_LN_O(bf16_t, float);
        else DISCO_LN_O(bf16_t, bf16_t);
    }
#undef DISCO_LN_O
#undef DISCO_LN
    return DISCO_OK;
}

}  // namespace disco
