// Orthogonalised matrix updates by Newton-Schulz products, and the weight
// update built on them.
//
//   X_0 = M / (|M|_F + eps), transposed where rows > cols so that X is m x n, m <= n
//   steps times:  A = X X^T,  P = b A + c A^2,  X <- a X + P X
//
// Number format.  X, A and P live as pairs of float16 (hi + lo, 22 bits)
// scaled by powers of two, and products run on the matrix cores with float32
// accumulation: three products hi hi + hi lo + lo hi keep float32 accuracy at
// a third of the float16 rate, five times that of the float32 matrix
// instructions.  bfloat16 operands would lose too much: the map f(s) = a s +
// b s^3 + c s^5 amplifies small singular values by up to a^steps, and 8-bit
// operands leave results 1 to 10 percent off.  Singular values stay below 16
// (checked by the caller), so the scales below keep every entry inside float16's
// range and the lo parts' granularity below 2^-36.
//
// X is kept in both orders, [m][n] for X X^T and [n][m] for P X, so that both
// operands of every product are contiguous along the summed index; the matrix
// core's output layout holds four neighbouring rows of a column in a lane and
// writes either order.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "disco_internal.h"
#include "kernels_common.h"

namespace disco {

namespace {

typedef _Float16 half_t;
typedef _Float16 halfx4 __attribute__((ext_vector_type(4)));
typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) halfx8 lds_halfx8;

// powers of two that X, A and P are stored times
constexpr float kSX = 4096.0f, kSA = 4096.0f, kSP = 2048.0f;

struct Pair {
    half_t h, l;
};

__device__ __forceinline__ Pair split(float v) {
    Pair p;
    p.h = (half_t)v;
    p.l = (half_t)(v - (float)p.h);
    return p;
}

// The matrix to orthogonalise, element i of one batch entry: a matrix as it
// is, or the momentum update (buf already advanced).
struct Source {
    const void* m;        // matrix or gradient
    const float* buf;     // advanced momentum, or NULL
    float beta;
    int nesterov;
};

template <typename T>
__device__ __forceinline__ float source_at(const Source& s, int64_t i) {
    if (s.buf == nullptr) return load_f(static_cast<const T*>(s.m), i);
    if (!s.nesterov) return s.buf[i];
    return load_f(static_cast<const T*>(s.m), i) + s.beta * s.buf[i];
}

// What becomes of the orthogonalised matrix.
struct Sink {
    void* o;              // result, or NULL
    int bf16;             // type of o / w_out
    const void* w;        // weights, or NULL
    void* w_out;
    bf16_t* w16;          // bf16 copy of the new weights, or NULL
    float keep, rate;     // w_out = keep * w - rate * o
};

__device__ __forceinline__ void sink_store(const Sink& s, int64_t i, float o) {
    if (s.o != nullptr) {
        if (s.bf16) store_f(static_cast<bf16_t*>(s.o), i, o);
        else static_cast<float*>(s.o)[i] = o;
        return;
    }
    if (s.bf16) {
        const float w = load_f(static_cast<const bf16_t*>(s.w), i);
        store_f(static_cast<bf16_t*>(s.w_out), i, s.keep * w - s.rate * o);
    } else {
        const float v = s.keep * static_cast<const float*>(s.w)[i] - s.rate * o;
        static_cast<float*>(s.w_out)[i] = v;
        if (s.w16 != nullptr) store_f(s.w16, i, v);
    }
}

// Advances the momentum (where there is one) and sums the squares of the
// update in float64: no overflow for any float32 matrix.  partial[batch][gridDim.x].
template <typename T>
__global__ __launch_bounds__(256) void ns_norm(Source src, const float* buf_in,
                                               float* buf_out, int64_t n,
                                               double* __restrict__ partial) {
    __shared__ double red[4];
    const int64_t base = (int64_t)blockIdx.y * n;
    double acc = 0.0;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        float v;
        if (buf_out != nullptr) {
            const float g = load_f(static_cast<const T*>(src.m), base + i);
            const float b = src.beta * buf_in[base + i] + g;
            buf_out[base + i] = b;
            v = src.nesterov ? g + src.beta * b : b;
        } else {
            v = load_f(static_cast<const T*>(src.m), base + i);
        }
        acc += (double)v * (double)v;
    }
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) acc += __shfl_xor(acc, m);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = acc;
    __syncthreads();
    if (threadIdx.x == 0)
        partial[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = red[0] + red[1] + red[2] + red[3];
}

// 1 / (|M|_F + eps) of this batch entry, on every thread of a 256-thread group.
__device__ __forceinline__ double inv_norm(const double* partial, int nparts, float eps,
                                           double* red) {
    double acc = 0.0;
    for (int k = threadIdx.x; k < nparts; k += 256) acc += partial[k];
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) acc += __shfl_xor(acc, m);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = acc;
    __syncthreads();
    return 1.0 / (sqrt(red[0] + red[1] + red[2] + red[3]) + (double)eps);
}

// X_0 in both orders, zero padded to mp x np: a 64 x 64 tile a workgroup,
// through LDS.  tall: the source is [n][m].
template <typename T>
__global__ __launch_bounds__(256) void ns_load(Source src, const double* __restrict__ partial,
                                               int nparts, float eps, int m, int n, int mp, int np,
                                               int tall, half_t* __restrict__ X,
                                               half_t* __restrict__ XT, size_t xplane) {
    __shared__ double red[4];
    __shared__ float tile[64][65];   // [i][j] of X
    const int b = blockIdx.z;
    const double inv = inv_norm(partial + (size_t)b * nparts, nparts, eps, red);
    const int64_t base = (int64_t)b * m * n;
    const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;
    const int lo = threadIdx.x & 63, hi = threadIdx.x >> 6;
    for (int k = hi; k < 64; k += 4) {
        const int i = tall ? lo : k, j = tall ? k : lo;
        float v = 0.0f;
        if (i0 + i < m && j0 + j < n) {
            const int64_t at = tall ? (int64_t)(j0 + j) * m + i0 + i : (int64_t)(i0 + i) * n + j0 + j;
            v = (float)((double)source_at<T>(src, base + at) * inv) * kSX;
        }
        tile[i][j] = v;
    }
    __syncthreads();
    half_t* x = X + (size_t)b * 2 * xplane;
    half_t* xt = XT + (size_t)b * 2 * xplane;
    for (int k = hi; k < 64; k += 4) {
        const Pair p = split(tile[k][lo]);
        const size_t at = (size_t)(i0 + k) * np + j0 + lo;
        x[at] = p.h;
        x[xplane + at] = p.l;
        const Pair q = split(tile[lo][k]);
        const size_t att = (size_t)(j0 + k) * mp + i0 + lo;
        xt[att] = q.h;
        xt[xplane + att] = q.l;
    }
}

enum Epilogue { kGram, kPoly, kStep, kLast };

// One product of the iteration, U V^T with both operands [rows][K], as hi and
// lo planes.
struct Product {
    const half_t *u, *v;      // hi planes of batch entry 0; lo planes at + plane
    size_t u_plane, v_plane;  // elements of a plane; a batch entry has two
    int K;                    // summed length, a multiple of 64; also the row stride
    int tiles_j;              // tiles along j (kStep, kLast)
    // results and other operands
    half_t *out, *out_t;      // [i][j] and [j][i] (hi, lo); kGram / kPoly: one symmetric matrix
    const half_t* add;        // kPoly: A; kStep, kLast: X^T as [j][i]
    size_t o_plane, add_plane;
    int ld_out, ld_t;         // row strides of out and out_t (and add)
    int lo_out, lo_t;         // whether the lo planes of out, out_t are wanted
    float ca, cb;             // factors of `add` and of the accumulated product
    int m, n, tall;           // kLast: true sizes and orientation
    Sink sink;
};

// BM x BN tile of a product, WM x WN waves, NS stages of 64-deep slices in LDS.
// Slices arrive by direct-to-LDS loads; 16-byte slot s of a 128-byte row r
// holds chunk s ^ (r & 7), so the 16-byte fragment reads of eight neighbouring
// rows fall on distinct banks.
template <int BM, int BN, int WM, int WN, int NP, int NS, Epilogue E>
__global__ __launch_bounds__(64 * WM * WN) void ns_product(Product p) {
    constexpr int W = WM * WN;
    constexpr int PL = NP == 3 ? 2 : 1;                      // planes of an operand
    constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
    constexpr int UNITS = (BM + BN) * PL / 8, OPS = UNITS / W;
    constexpr int STAGE = (BM + BN) * PL * 128;
    static_assert(UNITS % W == 0, "whole loads per wave");
    __shared__ __attribute__((aligned(1024))) uint8_t ring[NS * STAGE];

    const int lane = threadIdx.x & 63;
    const int wave = uniform(threadIdx.x >> 6);
    const int b = blockIdx.y;
    int ti, tj;
    if constexpr (E == kGram || E == kPoly) {
        // lower triangle, row by row
        const int t = blockIdx.x;
        ti = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
        while ((ti + 1) * (ti + 2) / 2 <= t) ++ti;
        while (ti * (ti + 1) / 2 > t) --ti;
        tj = t - ti * (ti + 1) / 2;
    } else {
        ti = blockIdx.x / p.tiles_j;
        tj = blockIdx.x % p.tiles_j;
    }
    const int i0 = ti * BM, j0 = tj * BN;
    const half_t* u = p.u + (size_t)b * 2 * p.u_plane;
    const half_t* v = p.v + (size_t)b * 2 * p.v_plane;

    const half_t* src[OPS];
#pragma unroll
    for (int o = 0; o < OPS; ++o) {
        const int unit = o * W + wave;
        const int plane_units_u = BM / 8, plane_units_v = BN / 8;
        const half_t* q;
        int row;
        if (unit < PL * plane_units_u) {
            const int pl = unit / plane_units_u;
            row = i0 + (unit - pl * plane_units_u) * 8;
            q = u + (size_t)pl * p.u_plane;
        } else {
            const int uv = unit - PL * plane_units_u, pl = uv / plane_units_v;
            row = j0 + (uv - pl * plane_units_v) * 8;
            q = v + (size_t)pl * p.v_plane;
        }
        src[o] = q + (size_t)(row + (lane >> 3)) * p.K + 8 * ((lane & 7) ^ (lane >> 3));
    }
    const uint32_t ring_at = (uint32_t)(uintptr_t)(lds_u8*)&ring[0];
    const int nk = p.K / 64;
    auto issue = [&](int k) {
        const uint32_t st = ring_at + (uint32_t)((k % NS) * STAGE);
#pragma unroll
        for (int o = 0; o < OPS; ++o)
            dma_lds16(src[o] + (size_t)k * 64, st + (uint32_t)((o * W + wave) * 1024));
    };

    floatx16 acc[TM][TN];
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
        for (int c = 0; c < TN; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[a][c][e] = 0.0f;

    const int wm = wave / WN, wn = wave % WN, l32 = lane & 31, lg = lane >> 5;
    const lds_u8* base = (const lds_u8*)&ring[0];
    const uint32_t row_u = (uint32_t)((wm * TM * 32 + l32) * 128);
    const uint32_t row_v = (uint32_t)(BM * PL * 128 + (wn * TN * 32 + l32) * 128);

    const int pre = min(NS - 1, nk);
    for (int k = 0; k < pre; ++k) issue(k);
    for (int k = 0; k < nk; ++k) {
        // slice k has landed when at most the later slices' loads are out
        if (k + NS - 1 <= nk) wait_vmcnt<OPS*(NS - 2)>();
        else wait_vmcnt<0>();
        __syncthreads();
        if (k + NS - 1 < nk) issue(k + NS - 1);   // into the stage read at slice k - 1
        const lds_u8* st = base + (k % NS) * STAGE;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            const uint32_t ch = (uint32_t)(16 * ((2 * ks + lg) ^ (l32 & 7)));
            halfx8 fu[TM][PL], fv[TN][PL];
#pragma unroll
            for (int a = 0; a < TM; ++a)
#pragma unroll
                for (int q = 0; q < PL; ++q)
                    fu[a][q] = *(const lds_halfx8*)(st + row_u + ch + q * BM * 128 + a * 4096);
#pragma unroll
            for (int c = 0; c < TN; ++c)
#pragma unroll
                for (int q = 0; q < PL; ++q)
                    fv[c][q] = *(const lds_halfx8*)(st + row_v + ch + q * BN * 128 + c * 4096);
#pragma unroll
            for (int a = 0; a < TM; ++a)
#pragma unroll
                for (int c = 0; c < TN; ++c) {
                    if constexpr (NP == 3) {
                        acc[a][c] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fu[a][1], fv[c][0],
                                                                          acc[a][c], 0, 0, 0);
                        acc[a][c] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fu[a][0], fv[c][1],
                                                                          acc[a][c], 0, 0, 0);
                    }
                    acc[a][c] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fu[a][0], fv[c][0],
                                                                      acc[a][c], 0, 0, 0);
                }
        }
    }

    // lane: column j = lane % 32, rows i = 8 (e / 4) + 4 (lane / 32) + e % 4
    half_t* out = p.out + (size_t)b * 2 * p.o_plane;
    half_t* out_t = p.out_t + (size_t)b * 2 * p.o_plane;
    const half_t* add = p.add + (size_t)b * 2 * p.add_plane;
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
        for (int c = 0; c < TN; ++c)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = i0 + (wm * TM + a) * 32 + 8 * q + 4 * lg;
                const int j = j0 + (wn * TN + c) * 32 + l32;
                const size_t at_t = (size_t)j * p.ld_t + i;
                float f[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = p.cb * acc[a][c][4 * q + e];
                if constexpr (E != kGram) {
                    const halfx4 xh = *reinterpret_cast<const halfx4*>(add + at_t);
                    const halfx4 xl = *reinterpret_cast<const halfx4*>(add + p.add_plane + at_t);
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[e] += p.ca * ((float)xh[e] + (float)xl[e]);
                }
                if constexpr (E == kLast) {
                    if (j < p.n) {
                        const int64_t at0 = (int64_t)b * p.m * p.n;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (i + e < p.m)
                                sink_store(p.sink, at0 + (p.tall ? (int64_t)j * p.m + i + e
                                                                : (int64_t)(i + e) * p.n + j),
                                           f[e]);
                    }
                } else {
                    halfx4 h, l;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const Pair s = split(f[e]);
                        h[e] = s.h;
                        l[e] = s.l;
                    }
                    *reinterpret_cast<halfx4*>(out_t + at_t) = h;
                    if (p.lo_t) *reinterpret_cast<halfx4*>(out_t + p.o_plane + at_t) = l;
                    // a symmetric result's diagonal tiles are whole already
                    if ((E == kStep) || ti != tj) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const size_t at = (size_t)(i + e) * p.ld_out + j;
                            out[at] = h[e];
                            if (p.lo_out) out[p.o_plane + at] = l[e];
                        }
                    }
                }
            }
}

size_t up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// Where everything of a call lies in its workspace.
struct Layout {
    int m, n, mp, np, tall, nparts;
    size_t xplane, aplane;                 // elements of one plane
    size_t partial, X, XT0, XT1, A, P;     // byte offsets
    size_t bytes;
};

Layout layout(int batch, int rows, int cols) {
    Layout l;
    l.tall = rows > cols;
    l.m = std::min(rows, cols);
    l.n = std::max(rows, cols);
    l.mp = (int)up(l.m, 64);
    l.np = (int)up(l.n, 64);
    const int64_t elems = (int64_t)rows * cols;
    l.nparts = (int)std::max<int64_t>(1, std::min<int64_t>(1024, elems / 4096));
    l.xplane = (size_t)l.mp * l.np;
    l.aplane = (size_t)l.mp * l.mp;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at = up(at + bytes, 1024);
        return here;
    };
    l.partial = take((size_t)batch * l.nparts * sizeof(double));
    l.X = take((size_t)batch * 2 * l.xplane * sizeof(half_t));
    l.XT0 = take((size_t)batch * 2 * l.xplane * sizeof(half_t));
    l.XT1 = take((size_t)batch * 2 * l.xplane * sizeof(half_t));
    l.A = take((size_t)batch * 2 * l.aplane * sizeof(half_t));
    l.P = take((size_t)batch * 2 * l.aplane * sizeof(half_t));
    l.bytes = at;
    return l;
}

int done(const char* what) {
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return set_error(DISCO_EHIP, "%s launch failed: %s", what, hipGetErrorString(e));
    return DISCO_OK;
}

template <int NP, Epilogue E>
int launch_product(const Product& p, int tiles, int batch, hipStream_t st) {
    constexpr const char* names[] = {"ns_gram", "ns_poly", "ns_step", "ns_last"};
    KernelTimer timer(names[E], st);
    hipLaunchKernelGGL((ns_product<64, 64, 2, 2, NP, 2, E>), dim3((unsigned)tiles, batch), dim3(256),
                       0, st, p);
    return done(names[E]);
}

template <Epilogue E>
int launch_product(bool three, const Product& p, int tiles, int batch, hipStream_t st) {
    return three ? launch_product<3, E>(p, tiles, batch, st) : launch_product<1, E>(p, tiles, batch, st);
}

}  // namespace

size_t orthogonalize_workspace(int batch, int rows, int cols) {
    return layout(batch, rows, cols).bytes;
}

int launch_orthogonalize(const OrthoCall& c, void* stream) {
    hipStream_t st = static_cast<hipStream_t>(stream);
    const Layout l = layout(c.batch, c.rows, c.cols);
    char* ws = static_cast<char*>(c.workspace);
    double* partial = reinterpret_cast<double*>(ws + l.partial);
    half_t* X = reinterpret_cast<half_t*>(ws + l.X);
    half_t* XT[2] = {reinterpret_cast<half_t*>(ws + l.XT0), reinterpret_cast<half_t*>(ws + l.XT1)};
    half_t* A = reinterpret_cast<half_t*>(ws + l.A);
    half_t* P = reinterpret_cast<half_t*>(ws + l.P);

    Source src{c.m, c.momentum_out, c.beta, c.nesterov};
    {
        KernelTimer timer("ns_norm", st);
        const dim3 grid(l.nparts, c.batch);
        const int64_t n = (int64_t)c.rows * c.cols;
        if (c.m_dtype == DISCO_F32)
            hipLaunchKernelGGL(ns_norm<float>, grid, dim3(256), 0, st, src, c.momentum,
                               c.momentum_out, n, partial);
        else
            hipLaunchKernelGGL(ns_norm<bf16_t>, grid, dim3(256), 0, st, src, c.momentum,
                               c.momentum_out, n, partial);
        if (int rc = done("ns_norm")) return rc;
    }
    {
        KernelTimer timer("ns_load", st);
        const dim3 grid(l.np / 64, l.mp / 64, c.batch);
        if (c.m_dtype == DISCO_F32)
            hipLaunchKernelGGL(ns_load<float>, grid, dim3(256), 0, st, src, partial, l.nparts, c.eps,
                               l.m, l.n, l.mp, l.np, l.tall, X, XT[0], l.xplane);
        else
            hipLaunchKernelGGL(ns_load<bf16_t>, grid, dim3(256), 0, st, src, partial, l.nparts,
                               c.eps, l.m, l.n, l.mp, l.np, l.tall, X, XT[0], l.xplane);
        if (int rc = done("ns_load")) return rc;
    }
    Sink sink{};
    sink.o = c.o;
    sink.bf16 = c.out_dtype == DISCO_BF16;
    sink.w = c.w;
    sink.w_out = c.w_out;
    sink.w16 = static_cast<bf16_t*>(c.w16);
    sink.keep = c.keep;
    sink.rate = c.rate;

    const int tm = l.mp / 64, tn = l.np / 64;
    // A bfloat16 result takes single float16 products in all but the last two
    // steps: 2e-4 to 1e-3 off before its own rounding of 1.7e-3 (three products
    // in the last two steps matter most: there A's entries are of order one and
    // their rounding enters X unscaled).
    const int exact_from = sink.bf16 ? std::max(0, c.steps - 2) : 0;
    for (int t = 0; t < c.steps; ++t) {
        const bool three = t >= exact_from, last = t + 1 == c.steps;
        half_t* xt = XT[t & 1];
        Product g{};
        g.u = g.v = X;
        g.u_plane = g.v_plane = l.xplane;
        g.K = l.np;
        g.out = g.out_t = A;
        g.o_plane = l.aplane;
        g.add = X;   // not read
        g.ld_out = g.ld_t = l.mp;
        g.lo_out = g.lo_t = 1;
        g.cb = kSA / (kSX * kSX);
        if (int rc = launch_product<kGram>(three, g, tm * (tm + 1) / 2, c.batch, st)) return rc;

        Product q{};
        q.u = q.v = A;
        q.u_plane = q.v_plane = l.aplane;
        q.K = l.mp;
        q.out = q.out_t = P;
        q.add = A;
        q.o_plane = q.add_plane = l.aplane;
        q.ld_out = q.ld_t = l.mp;
        q.lo_out = q.lo_t = three;
        q.ca = c.coeffs[1] * kSP / kSA;
        q.cb = c.coeffs[2] * kSP / (kSA * kSA);
        if (int rc = launch_product<kPoly>(three, q, tm * (tm + 1) / 2, c.batch, st)) return rc;

        Product s{};
        s.u = P;
        s.v = xt;
        s.u_plane = l.aplane;
        s.v_plane = s.add_plane = s.o_plane = l.xplane;
        s.K = l.mp;
        s.tiles_j = tn;
        s.out = X;
        s.out_t = XT[(t + 1) & 1];
        s.add = xt;
        s.ld_out = l.np;
        s.ld_t = l.mp;
        s.lo_out = t + 1 >= exact_from;   // the next X X^T reads it
        s.lo_t = 1;
        s.ca = c.coeffs[0];
        s.cb = 1.0f / kSP;
        if (last) {
            s.ca /= kSX;
            s.cb /= kSX;
            s.m = l.m;
            s.n = l.n;
            s.tall = l.tall;
            s.sink = sink;
        }
        const int rc = last ? launch_product<kLast>(three, s, tm * tn, c.batch, st)
                            : launch_product<kStep>(three, s, tm * tn, c.batch, st);
        if (rc) return rc;
    }
    return DISCO_OK;
}

}  // namespace disco
