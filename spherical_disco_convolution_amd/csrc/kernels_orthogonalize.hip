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

// The sink of one batch entry, whose first element is `base`.
__device__ __forceinline__ Sink sink_from(Sink s, int64_t base) {
    const int64_t bytes = base * (s.bf16 ? 2 : 4);
    if (s.o != nullptr) {
        s.o = static_cast<char*>(s.o) + bytes;
    } else {
        s.w = static_cast<const char*>(s.w) + bytes;
        s.w_out = static_cast<char*>(s.w_out) + bytes;
        if (s.w16 != nullptr) s.w16 += base;
    }
    return s;
}

template <typename I>
__device__ __forceinline__ void sink_store(const Sink& s, I i, float o) {
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

// ---------------------------------------------------------------------------
// Small matrices: the whole iteration in one workgroup per matrix
// ---------------------------------------------------------------------------
// X stays in registers.  A wave owns CB blocks of 32 columns with all 32 MT rows
// in the matrix core's output layout (lane: column lane % 32; element 4 q + r:
// row 8 q + 4 (lane / 32) + r).  Eight consecutive elements of that layout are
// a valid operand of P X when P is read with the same permutation of the summed
// rows, so the products chain without moving X.  X X^T sums over columns, which
// lie across lanes: each wave turns its block over in its own piece of LDS
// (transposing reads), the waves' partial sums meet in LDS, and A and P live
// there too.  Always three products: a step is a few hundred matrix
// instructions and the barriers and LDS round trips around them cost as much.
typedef __attribute__((address_space(3))) halfx4 lds_halfx4;
typedef int16_t v4i16_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16_t lds_v4i16;

__device__ __forceinline__ floatx16 mfma3(halfx8 uh, halfx8 ul, halfx8 vh, halfx8 vl, floatx16 acc) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(ul, vh, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(uh, vl, acc, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(uh, vh, acc, 0, 0, 0);
}

// Fragment of a 32-wide block from LDS rows [k][i] (i contiguous): lane gets
// i = lane % 32, k = 8 (lane / 32) .. + 7.  `at`: address of k = 0, i = 0.
__device__ __forceinline__ halfx8 read_turned(uint32_t at, int stride, int lane) {
    const int s = lane & 15, g = lane >> 4;
    const uint32_t p = at + (uint32_t)((8 * (g >> 1) + (s >> 2)) * stride +
                                       2 * (16 * (g & 1) + 4 * (s & 3)));
    const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(uintptr_t)p);
    const v4i16_t hi =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(uintptr_t)(p + 4 * stride));
    return __builtin_bit_cast(halfx8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Elements at .. at + 3 of a `total`-element tensor, at any element alignment;
// what lies past the end reads as zero and is not written.
__device__ __forceinline__ void load4(const float* p, int at, int total, float* v) {
    struct __attribute__((packed, aligned(4))) U { float e[4]; };
    if (at + 4 <= total) {
        const U u = *reinterpret_cast<const U*>(p + at);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = u.e[e];
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = at + e < total ? p[at + e] : 0.0f;
    }
}

__device__ __forceinline__ void load4(const bf16_t* p, int at, int total, float* v) {
    struct __attribute__((packed, aligned(2))) U { uint32_t e[2]; };
    if (at + 4 <= total) {
        const U u = *reinterpret_cast<const U*>(p + at);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            v[2 * e] = __uint_as_float(u.e[e] << 16);
            v[2 * e + 1] = __uint_as_float(u.e[e] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = at + e < total ? bf16_to_f32(p[at + e]) : 0.0f;
    }
}

__device__ __forceinline__ void store4(float* p, int at, int total, const float* v) {
    struct __attribute__((packed, aligned(4))) U { float e[4]; };
    if (at + 4 <= total) {
        *reinterpret_cast<U*>(p + at) = U{{v[0], v[1], v[2], v[3]}};
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (at + e < total) p[at + e] = v[e];
    }
}

__device__ __forceinline__ void store4(bf16_t* p, int at, int total, const float* v) {
    struct __attribute__((packed, aligned(2))) U { uint32_t e[2]; };
    if (at + 4 <= total) {
        U u;
#pragma unroll
        for (int e = 0; e < 2; ++e)
            u.e[e] = (uint32_t)f32_to_bf16(v[2 * e]) | ((uint32_t)f32_to_bf16(v[2 * e + 1]) << 16);
        *reinterpret_cast<U*>(p + at) = u;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (at + e < total) store_f(p, at + e, v[e]);
    }
}

template <int MT>
struct SmallCfg {
    static constexpr int M = 32 * MT;
    static constexpr int NT = MT * (MT + 1) / 2;     // lower-triangle tiles
    static constexpr int TURN = 2 * M + 8;           // bytes of a column while turned over
    static constexpr int ROW_A = 2 * M + 16;         // bytes of a row of A: 16-byte reads
    static constexpr int ROW_P = 2 * M + 8;          // of P: 8-byte reads
    // a wave's piece: its columns (hi, lo), then its partial sums
    static constexpr int PIECE = (2 * 32 * TURN > NT * 4096 ? 2 * 32 * TURN : NT * 4096);
    static constexpr int A_BYTES = 2 * M * ROW_A, P_BYTES = 2 * M * ROW_P;
    // A, P and the pieces; X in float32 before and after them
    static size_t lds(int waves, int m, int n) {
        return 256 + std::max((size_t)A_BYTES + P_BYTES + (size_t)waves * PIECE, (size_t)m * (n | 1) * 4);
    }
};

template <typename T, int MT, int CB>
__global__ __launch_bounds__(512) void ns_small(Source src, const float* buf_in, float* buf_out,
                                                Sink sink, int m, int n, int tall, int steps,
                                                float ca, float cb, float cc, float eps) {
    using C = SmallCfg<MT>;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds_raw[];
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_u8*)&lds_raw[0];
    double* red = reinterpret_cast<double*>(lds_raw);
    const uint32_t A_at = lds0 + 256, P_at = A_at + C::A_BYTES;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), W = blockDim.x >> 6;
    const int l32 = lane & 31, lg = lane >> 5;
    const uint32_t piece = P_at + C::P_BYTES + (uint32_t)(wave * C::PIECE);
    // 32-bit offsets from here on: at most 64 x 1024 elements
    const int64_t base = (int64_t)blockIdx.x * m * n;
    const T* in = static_cast<const T*>(src.m) + base;
    const float* old = buf_out ? buf_in + base : nullptr;
    float* fresh = buf_out ? buf_out + base : nullptr;
    const Sink to = sink_from(sink, base);

    // ---- X_0: through LDS as rows of X, in a short loop of whole reads (the
    // unrolled alternative, each lane reading its own elements, costs 15 us more
    // at 64 x 448, most of it fetching instructions that run once) ----
    typedef __attribute__((address_space(3))) float lds_float;
    const int ld = n | 1;   // odd: both orders of access spread over the banks
    const uint32_t x_at = lds0 + 256;
    double acc2 = 0.0;
    const int total = m * n, width = tall ? m : n;   // of a row in memory
    const float rwidth = 1.0f / (float)width;
    // LDS place of element `at` and of the ones after it in its row
    auto place = [&](int at, int& q, int& r) {
        q = (int)(((float)at + 0.5f) * rwidth);   // at < 2^16: exact
        r = at - q * width;
    };
    auto slot = [&](int q, int r) {
        return (lds_float*)(uintptr_t)(x_at + 4u * (uint32_t)(tall ? r * ld + q : q * ld + r));
    };
    constexpr int K = 8;   // reads of four elements in flight
    for (int at0 = 4 * threadIdx.x; at0 < total; at0 += 4 * K * blockDim.x) {
        float v[K][4], o[K][4];
#pragma unroll
        for (int k = 0; k < K; ++k) load4(in, at0 + 4 * k * (int)blockDim.x, total, v[k]);
        if (fresh != nullptr) {
#pragma unroll
            for (int k = 0; k < K; ++k) load4(old, at0 + 4 * k * (int)blockDim.x, total, o[k]);
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int at = at0 + 4 * k * (int)blockDim.x;
            if (at >= total) break;
            int q, r;
            place(at, q, r);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (at + e >= total) break;
                float u = v[k][e];
                if (fresh != nullptr) {
                    const float b = src.beta * o[k][e] + u;
                    fresh[at + e] = b;
                    u = src.nesterov ? u + src.beta * b : b;
                }
                acc2 += (double)u * (double)u;
                *slot(q, r) = u;
                if (++r == width) {
                    r = 0;
                    ++q;
                }
            }
        }
    }
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) acc2 += __shfl_xor(acc2, k);
    if (lane == 0) red[wave] = acc2;
    __syncthreads();
    acc2 = 0.0;
    for (int w = 0; w < W; ++w) acc2 += red[w];
    const double inv = 1.0 / (sqrt(acc2) + (double)eps) * (double)kSX;

    // hi and lo parts: [column block][row tile][half of 16 rows]
    halfx8 xh[CB][MT][2], xl[CB][MT][2];
#pragma unroll
    for (int c = 0; c < CB; ++c)
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int i = 32 * a + 8 * (e >> 2) + 4 * lg + (e & 3);
                const int j = 32 * (wave + W * c) + l32;
                const bool ok = i < m && j < n;
                const float v = *(const lds_float*)(uintptr_t)(x_at + 4u * (uint32_t)(ok ? i * ld + j : 0));
                const Pair p = split(ok ? (float)((double)v * inv) : 0.0f);
                xh[c][a][e >> 3][e & 7] = p.h;
                xl[c][a][e >> 3][e & 7] = p.l;
            }
    __syncthreads();   // the pieces lie where X_0 lay

    for (int t = 0; t < steps; ++t) {
        // ---- this wave's part of X X^T, lower tiles ----
        floatx16 g[C::NT];
#pragma unroll
        for (int k = 0; k < C::NT; ++k)
#pragma unroll
            for (int e = 0; e < 16; ++e) g[k][e] = 0.0f;
#pragma unroll
        for (int c = 0; c < CB; ++c) {
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t at = piece + (uint32_t)(l32 * C::TURN + 2 * (32 * a + 8 * q + 4 * lg));
                    const halfx8 h = xh[c][a][q >> 1], l = xl[c][a][q >> 1];
                    halfx4 h4, l4;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        h4[r] = h[4 * (q & 1) + r];
                        l4[r] = l[4 * (q & 1) + r];
                    }
                    *(lds_halfx4*)(uintptr_t)at = h4;
                    *(lds_halfx4*)(uintptr_t)(at + 32 * C::TURN) = l4;
                }
            // one wave's LDS accesses are carried out in order; the fence keeps
            // the compiler from moving the reads up
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int kc = 0; kc < 2; ++kc) {
                halfx8 fh[MT], fl[MT];
#pragma unroll
                for (int a = 0; a < MT; ++a) {
                    const uint32_t at = piece + (uint32_t)(16 * kc * C::TURN + 64 * a);
                    fh[a] = read_turned(at, C::TURN, lane);
                    fl[a] = read_turned(at + 32 * C::TURN, C::TURN, lane);
                }
                int k = 0;
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int b = 0; b <= a; ++b, ++k) g[k] = mfma3(fh[a], fl[a], fh[b], fl[b], g[k]);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
        typedef float floatx4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) floatx4 lds_floatx4;
#pragma unroll
        for (int k = 0; k < C::NT; ++k)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const floatx4 v = {g[k][4 * q], g[k][4 * q + 1], g[k][4 * q + 2], g[k][4 * q + 3]};
                *(lds_floatx4*)(uintptr_t)(piece + (uint32_t)(k * 4096 + q * 1024 + lane * 16)) = v;
            }
        __syncthreads();
        // ---- A: the waves' parts added, both triangles, hi and lo ----
        const uint32_t piece0 = P_at + C::P_BYTES;
        for (int pos = threadIdx.x; pos < C::NT * 256; pos += blockDim.x) {
            floatx4 v = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int w = 0; w < W; ++w)
                v += *(const lds_floatx4*)(uintptr_t)(piece0 + (uint32_t)(w * C::PIECE + pos * 16));
            const int k = pos >> 8, q = (pos >> 6) & 3, pl = pos & 63;
            const int a = k == 0 ? 0 : 1, b = k == 2 ? 1 : 0;   // (0,0) (1,0) (1,1)
            const int i = 32 * a + 8 * q + 4 * (pl >> 5), j = 32 * b + (pl & 31);
            halfx4 h, l;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const Pair p = split(v[r] * (kSA / (kSX * kSX)));
                h[r] = p.h;
                l[r] = p.l;
            }
            // [j][i]: four neighbours; [i][j] too where the tile is not diagonal
            const uint32_t at = A_at + (uint32_t)(j * C::ROW_A + 2 * i);
            *(lds_halfx4*)(uintptr_t)at = h;
            *(lds_halfx4*)(uintptr_t)(at + C::M * C::ROW_A) = l;
            if (a != b) {
                typedef __attribute__((address_space(3))) half_t lds_half;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint32_t at2 = A_at + (uint32_t)((i + r) * C::ROW_A + 2 * j);
                    *(lds_half*)(uintptr_t)at2 = h[r];
                    *(lds_half*)(uintptr_t)(at2 + C::M * C::ROW_A) = l[r];
                }
            }
        }
        __syncthreads();
        // ---- P = b A + c A^2, a tile per wave ----
        for (int tile = wave; tile < MT * MT; tile += W) {
            const int a = tile / MT, b = tile % MT;
            floatx16 acc;
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
#pragma unroll
            for (int kc = 0; kc < 2 * MT; ++kc) {
                const uint32_t u = A_at + (uint32_t)((32 * a + l32) * C::ROW_A + 32 * kc + 16 * lg);
                const uint32_t v = A_at + (uint32_t)((32 * b + l32) * C::ROW_A + 32 * kc + 16 * lg);
                const halfx8 uh = *(const lds_halfx8*)(uintptr_t)u;
                const halfx8 ul = *(const lds_halfx8*)(uintptr_t)(u + C::M * C::ROW_A);
                const halfx8 vh = *(const lds_halfx8*)(uintptr_t)v;
                const halfx8 vl = *(const lds_halfx8*)(uintptr_t)(v + C::M * C::ROW_A);
                acc = mfma3(uh, ul, vh, vl, acc);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = 32 * a + 8 * q + 4 * lg, j = 32 * b + l32;
                const uint32_t at = A_at + (uint32_t)(j * C::ROW_A + 2 * i);
                const halfx4 ah = *(const lds_halfx4*)(uintptr_t)at;
                const halfx4 al = *(const lds_halfx4*)(uintptr_t)(at + C::M * C::ROW_A);
                halfx4 h, l;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const Pair p = split(cb * (kSP / kSA) * ((float)ah[r] + (float)al[r]) +
                                         cc * (kSP / (kSA * kSA)) * acc[4 * q + r]);
                    h[r] = p.h;
                    l[r] = p.l;
                }
                const uint32_t pt = P_at + (uint32_t)(j * C::ROW_P + 2 * i);
                *(lds_halfx4*)(uintptr_t)pt = h;
                *(lds_halfx4*)(uintptr_t)(pt + C::M * C::ROW_P) = l;
            }
        }
        __syncthreads();
        // ---- X <- a X + P X ----
        floatx16 y[CB][MT];
#pragma unroll
        for (int c = 0; c < CB; ++c)
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int e = 0; e < 16; ++e) y[c][a][e] = 0.0f;
#pragma unroll
        for (int kc = 0; kc < 2 * MT; ++kc)
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                // rows 16 kc + 4 lg .. + 3 and + 8: the order X's elements have
                const uint32_t at = P_at + (uint32_t)((32 * a + l32) * C::ROW_P + 32 * kc + 8 * lg);
                const halfx4 h0 = *(const lds_halfx4*)(uintptr_t)at;
                const halfx4 h1 = *(const lds_halfx4*)(uintptr_t)(at + 16);
                const halfx4 l0 = *(const lds_halfx4*)(uintptr_t)(at + C::M * C::ROW_P);
                const halfx4 l1 = *(const lds_halfx4*)(uintptr_t)(at + C::M * C::ROW_P + 16);
                const halfx8 ph = __builtin_shufflevector(h0, h1, 0, 1, 2, 3, 4, 5, 6, 7);
                const halfx8 pl = __builtin_shufflevector(l0, l1, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
                for (int c = 0; c < CB; ++c)
                    y[c][a] = mfma3(ph, pl, xh[c][kc >> 1][kc & 1], xl[c][kc >> 1][kc & 1], y[c][a]);
            }
#pragma unroll
        for (int c = 0; c < CB; ++c)
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const Pair p = split(
                        ca * ((float)xh[c][a][e >> 3][e & 7] + (float)xl[c][a][e >> 3][e & 7]) +
                        y[c][a][e] * (1.0f / kSP));
                    xh[c][a][e >> 3][e & 7] = p.h;
                    xl[c][a][e >> 3][e & 7] = p.l;
                }
    }
    // ---- result: back through LDS, written as it lies in memory ----
    __syncthreads();
#pragma unroll
    for (int c = 0; c < CB; ++c)
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int i = 32 * a + 8 * (e >> 2) + 4 * lg + (e & 3);
                const int j = 32 * (wave + W * c) + l32;
                if (i < m && j < n)
                    *(lds_float*)(uintptr_t)(x_at + 4u * (uint32_t)(i * ld + j)) =
                        ((float)xh[c][a][e >> 3][e & 7] + (float)xl[c][a][e >> 3][e & 7]) * (1.0f / kSX);
            }
    __syncthreads();
    for (int at0 = 4 * threadIdx.x; at0 < total; at0 += 4 * K * blockDim.x) {
        float w[K][4];
        if (to.o == nullptr) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int at = at0 + 4 * k * (int)blockDim.x;
                if (to.bf16) load4(static_cast<const bf16_t*>(to.w), at, total, w[k]);
                else load4(static_cast<const float*>(to.w), at, total, w[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int at = at0 + 4 * k * (int)blockDim.x;
            if (at >= total) break;
            int q, r;
            place(at, q, r);
            float f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[e] = at + e < total ? *slot(q, r) : 0.0f;
                if (++r == width) {
                    r = 0;
                    ++q;
                }
            }
            if (to.o == nullptr) {
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = to.keep * w[k][e] - to.rate * f[e];
            }
            void* out = to.o ? to.o : to.w_out;
            if (to.bf16) store4(static_cast<bf16_t*>(out), at, total, f);
            else store4(static_cast<float*>(out), at, total, f);
            if (to.o == nullptr && to.w16 != nullptr) store4(to.w16, at, total, f);
        }
    }
}

// Column blocks a wave takes (0: the matrix is not small) and the waves.
struct SmallShape {
    int mt = 0, cb = 0, waves = 0;
};

SmallShape small_shape(int m, int n) {
    SmallShape s;
    const int blocks = (n + 31) / 32, mt = (m + 31) / 32;
    if (mt > 2 || blocks > (mt == 1 ? 32 : 16)) return s;
    s.mt = mt;
    s.cb = 1;
    while (s.cb * 8 < blocks) s.cb *= 2;
    // at least a wave for each tile of A, also where there are fewer columns
    s.waves = std::max(mt * mt, (blocks + s.cb - 1) / s.cb);
    return s;
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
    if (small_shape(std::min(rows, cols), std::max(rows, cols)).cb != 0) return 0;
    return layout(batch, rows, cols).bytes;
}

namespace {

template <typename T, int MT, int CB>
int launch_small(const OrthoCall& c, const Sink& sink, int waves, hipStream_t st) {
    const size_t lds =
        SmallCfg<MT>::lds(waves, std::min(c.rows, c.cols), std::max(c.rows, c.cols));
    if (lds > 65536) {
        hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&ns_small<T, MT, CB>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) {
            (void)hipGetLastError();
            return set_error(DISCO_EHIP, "ns_small: %zu bytes of LDS refused: %s", lds,
                             hipGetErrorString(e));
        }
    }
    const Source src{c.m, c.momentum_out, c.beta, c.nesterov};
    const int tall = c.rows > c.cols;
    KernelTimer timer("ns_small", st);
    hipLaunchKernelGGL((ns_small<T, MT, CB>), dim3(c.batch), dim3(64 * waves), lds, st, src,
                       c.momentum, c.momentum_out, sink, std::min(c.rows, c.cols),
                       std::max(c.rows, c.cols), tall, c.steps, c.coeffs[0], c.coeffs[1],
                       c.coeffs[2], c.eps);
    return done("ns_small");
}

template <typename T>
int launch_small(const OrthoCall& c, const Sink& sink, const SmallShape& s, hipStream_t st) {
    if (s.mt == 1) {
        if (s.cb == 1) return launch_small<T, 1, 1>(c, sink, s.waves, st);
        if (s.cb == 2) return launch_small<T, 1, 2>(c, sink, s.waves, st);
        return launch_small<T, 1, 4>(c, sink, s.waves, st);
    }
    if (s.cb == 1) return launch_small<T, 2, 1>(c, sink, s.waves, st);
    return launch_small<T, 2, 2>(c, sink, s.waves, st);
}

}  // namespace

int launch_orthogonalize(const OrthoCall& c, void* stream) {
    hipStream_t st = static_cast<hipStream_t>(stream);
    Sink sink{};
    sink.o = c.o;
    sink.bf16 = c.out_dtype == DISCO_BF16;
    sink.w = c.w;
    sink.w_out = c.w_out;
    sink.w16 = static_cast<bf16_t*>(c.w16);
    sink.keep = c.keep;
    sink.rate = c.rate;
    const SmallShape small = small_shape(std::min(c.rows, c.cols), std::max(c.rows, c.cols));
    if (small.cb != 0)
        return c.m_dtype == DISCO_F32 ? launch_small<float>(c, sink, small, st)
                                      : launch_small<bf16_t>(c, sink, small, st);

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
