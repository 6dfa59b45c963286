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
// operands leave results 1 to 10 percent off.  Single float16 products in the
// first steps of a bfloat16 result were no way either: 2e-3 off after five steps
// with one strong direction over equal ones a fifth as large, 1e-1 after sixteen,
// where the result's own rounding is 1.7e-3.  So every result is computed the
// same way and rounded once, to its type.  The caller has checked that
// singular values stay below 3.5 in what goes into a step, and the polynomial below
// 24, so the scales below keep every operand inside float16's range, and the lo
// parts' granularity is 2^-36.  The last step's result goes out in float32.
//
// X is kept in both orders, [m][n] for X X^T and [n][m] for P X, so that both
// operands of every product are contiguous along the summed index; the matrix
// core's output layout holds four neighbouring rows of a column in a lane and
// writes either order.
//
// Three ways, by size: ns_small does everything in one workgroup per matrix,
// ns_panel a step per launch, ns_product a tiled product per launch.  What
// bounds them: the first two their chain of barriers and LDS round trips (2 to 8
// us a step), the third launches of 5 us each up to about 512 x 512 and the
// matrix cores above: at 4096 x 4096 they do 0.84 to 0.97 PFLOP/s of float16 work,
// where a large float16 library product reaches 1.3 to 1.5 (4.3 to 4.6 ms for five steps).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "disco_internal.h"
#include "kernels_common.h"

namespace disco {

namespace {

typedef _Float16 half_t;
typedef _Float16 halfx4 __attribute__((ext_vector_type(4)));
typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) halfx8 lds_halfx8;
typedef __attribute__((address_space(3))) halfx4 lds_halfx4;

// powers of two that X, A and P are stored times
constexpr float kSX = 4096.0f, kSA = 4096.0f, kSP = 2048.0f;

struct Pair {
    half_t h, l;
};

// v as hi + lo.  The empty asm pins v to its float32 value: without it the
// compiler may round hi from the unrounded product that v comes from and lo
// from v, and near a tie the two then belong to different neighbours (single
// entries 2^-11 off).
__device__ __forceinline__ Pair split(float v) {
    Pair p;
    asm volatile("" : "+v"(v));
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

// The new weight.  The fused multiply-add is written out, here and where P is
// formed: left to the compiler, which of the two products is the rounded one could
// change from one kernel to the next.
__device__ __forceinline__ float new_weight(const Sink& s, float w, float o) {
    return fmaf(-s.rate, o, s.keep * w);
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
        store_f(static_cast<bf16_t*>(s.w_out), i, new_weight(s, w, o));
    } else {
        const float v = new_weight(s, static_cast<const float*>(s.w)[i], o);
        static_cast<float*>(s.w_out)[i] = v;
        if (s.w16 != nullptr) store_f(s.w16, i, v);
    }
}

// Elements at .. at + 3 of a `total`-element tensor, at any element alignment;
// what lies past the end reads as zero and is not written.
__device__ __forceinline__ void load4(const float* p, int64_t at, int64_t total, float* v) {
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

__device__ __forceinline__ void load4(const bf16_t* p, int64_t at, int64_t total, float* v) {
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

__device__ __forceinline__ void store4(float* p, int64_t at, int64_t total, const float* v) {
    struct __attribute__((packed, aligned(4))) U { float e[4]; };
    if (at + 4 <= total) {
        *reinterpret_cast<U*>(p + at) = U{{v[0], v[1], v[2], v[3]}};
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (at + e < total) p[at + e] = v[e];
    }
}

__device__ __forceinline__ void store4(bf16_t* p, int64_t at, int64_t total, const float* v) {
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

// Advances the momentum (where there is one) and sums the squares of the
// update in float64: no overflow for any float32 matrix.  partial[batch][gridDim.x].
template <typename T>
__global__ __launch_bounds__(1024) void ns_norm(Source src, const float* buf_in, float* buf_out,
                                                int64_t n, double* __restrict__ partial) {
    __shared__ double red[16];
    const int64_t base = (int64_t)blockIdx.y * n;
    const T* m = static_cast<const T*>(src.m) + base;
    const float* old = buf_out ? buf_in + base : nullptr;
    float* fresh = buf_out ? buf_out + base : nullptr;
    double acc = 0.0;
    constexpr int K = 4;
    const int64_t stride = (int64_t)gridDim.x * 4096;
    for (int64_t at0 = (int64_t)blockIdx.x * 4096 + 4 * threadIdx.x; at0 < n; at0 += K * stride) {
        float v[K][4], o[K][4];
#pragma unroll
        for (int k = 0; k < K; ++k) load4(m, min(at0 + k * stride, n), n, v[k]);
        if (fresh != nullptr) {
#pragma unroll
            for (int k = 0; k < K; ++k) load4(old, min(at0 + k * stride, n), n, o[k]);
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (fresh != nullptr) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    o[k][e] = src.beta * o[k][e] + v[k][e];
                    v[k][e] = src.nesterov ? v[k][e] + src.beta * o[k][e] : o[k][e];
                }
                store4(fresh, min(at0 + k * stride, n), n, o[k]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) acc += (double)v[k][e] * (double)v[k][e];   // zero past the end
        }
    }
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) acc += __shfl_xor(acc, k);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = acc;
    __syncthreads();
    if (threadIdx.x == 0) {
        acc = 0.0;
        for (int k = 0; k < 16; ++k) acc += red[k];
        partial[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = acc;
    }
}

// 1 / (|M|_F + eps) of this batch entry, on every thread of a 256-thread group.
__device__ __forceinline__ double inv_norm(const double* partial, int nparts, float eps,
                                           double* red) {
    double acc = (int)threadIdx.x < nparts ? partial[threadIdx.x] : 0.0;
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) acc += __shfl_xor(acc, m);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = acc;
    __syncthreads();
    return 1.0 / (sqrt(red[0] + red[1] + red[2] + red[3]) + (double)eps);
}

// X_0 in both orders, zero padded to multiples of 64: a 64 x 64 tile a workgroup,
// through LDS.  tall: the source is [n][m].
template <typename T>
__global__ __launch_bounds__(256) void ns_load(Source src, const double* __restrict__ partial,
                                               int nparts, float eps, int m, int n, int mp, int np,
                                               int tall, half_t* __restrict__ X,
                                               half_t* __restrict__ XT, size_t xplane) {
    __shared__ double red[4];
    __shared__ float tile[64][65];   // rows and columns as in memory
    const int b = blockIdx.z;
    const int64_t base = (int64_t)b * m * n;
    const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;
    // rows of `width` elements in memory; this tile starts at (r0, c0) of them
    const int rows = tall ? n : m, width = tall ? m : n, r0 = tall ? j0 : i0, c0 = tall ? i0 : j0;
    float v[4][4], g[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int r = r0 + 16 * k + (threadIdx.x >> 4), c = c0 + 4 * (threadIdx.x & 15);
        const int64_t row = base + (int64_t)min(r, rows - 1) * width;
        const int len = r < rows ? width : 0;
        if (src.buf != nullptr) {
            load4(src.buf + row, min(c, len), len, v[k]);
            if (src.nesterov) load4(static_cast<const T*>(src.m) + row, min(c, len), len, g[k]);
        } else {
            load4(static_cast<const T*>(src.m) + row, min(c, len), len, v[k]);
        }
    }
    const double inv = inv_norm(partial + (size_t)b * nparts, nparts, eps, red) * (double)kSX;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float f = v[k][e];
            if (src.buf != nullptr && src.nesterov) f = g[k][e] + src.beta * f;
            tile[16 * k + (threadIdx.x >> 4)][4 * (threadIdx.x & 15) + e] = (float)((double)f * inv);
        }
    __syncthreads();
    // eight neighbours a thread, along the rows in memory and across them
    half_t* along = (tall ? XT : X) + (size_t)b * 2 * xplane;
    half_t* across = (tall ? X : XT) + (size_t)b * 2 * xplane;
    const int ld_along = tall ? mp : np, ld_across = tall ? np : mp;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int r = 32 * k + (threadIdx.x >> 3), c = 8 * (threadIdx.x & 7);
        halfx8 h, l;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const Pair p = split(tile[r][c + e]);
            h[e] = p.h;
            l[e] = p.l;
        }
        half_t* q = along + (size_t)(r0 + r) * ld_along + c0 + c;
        *reinterpret_cast<halfx8*>(q) = h;
        *reinterpret_cast<halfx8*>(q + xplane) = l;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const Pair p = split(tile[c + e][r]);
            h[e] = p.h;
            l[e] = p.l;
        }
        q = across + (size_t)(c0 + r) * ld_across + r0 + c;
        *reinterpret_cast<halfx8*>(q) = h;
        *reinterpret_cast<halfx8*>(q + xplane) = l;
    }
}

enum Epilogue { kGram, kPoly, kStep, kLast };

// One product of the iteration, U V^T with both operands [rows][K], as hi and
// lo planes.  Row counts and K are multiples of 64.
struct Product {
    const half_t *u, *v;      // hi planes of batch entry 0; lo planes at + plane
    size_t u_plane, v_plane;  // elements of a plane; a batch entry has two
    int K;                    // summed length, also the row stride of u and v
    int rows_u, rows_v;
    int tiles_i, tiles_j;     // tiles along i and j
    int splits;               // workgroups that share a tile's sum
    float* part;              // [batch][tile][split][BM * BN] where splits > 1
    // results and other operands
    half_t *out, *out_t;      // [i][j] and [j][i] (hi, lo); kGram / kPoly: one symmetric matrix
    const half_t* add;        // kPoly: A
    size_t o_plane, add_plane;
    int ld_out, ld_t;         // row strides of out and out_t (and add)
    float ca, cb;             // factors of `add` and of the accumulated product
    float diagonal;           // added where i == j (kPoly)
    int m, n, tall;           // kLast: true sizes and orientation
    Sink sink;
};

// A wave's TM x TN block of 32 x 32 tiles, one plane, between the matrix core's
// layout and rows in memory, through the wave's own piece of LDS at `at`.  One
// wave's LDS accesses are carried out in order; the fences keep the compiler
// from reordering them.
enum Keep { kAll, kFromDiagonal, kLeft };

template <int TM, int TN>
struct BlockIO {
    static constexpr int ROW_T = TM * 64 + 16, ROW = TN * 64 + 16;   // bytes of a padded row
    static constexpr int BYTES = TN * 32 * ROW_T > TM * 32 * ROW ? TN * 32 * ROW_T : TM * 32 * ROW;

    // 16-byte pieces of R rows of 8 C elements, row r at g + r * ld.  K: only those
    // whose 32 x 32 tile, `right` tiles right of the diagonal at the first row and
    // column, lies on the diagonal or right of it, or left of it.
    template <int R, int C, bool LOAD, Keep K = kAll>
    static __device__ __forceinline__ void move(half_t* g, size_t ld, int rows, int cols,
                                                uint32_t at, int row_bytes, int lane, int right = 0) {
#pragma unroll 4
        for (int it = 0; it < (R * C + 63) / 64; ++it) {
            const int idx = it * 64 + lane, r = idx / C, c = idx % C;
            const int over = right + (c >> 2) - (r >> 5);
            if (K == kFromDiagonal && over < 0) continue;
            if (K == kLeft && over >= 0) continue;
            if ((R * C % 64 == 0 || idx < R * C) && r < rows && 8 * c < cols) {
                half_t* q = g + (size_t)r * ld + 8 * c;
                lds_halfx8* l = (lds_halfx8*)(uintptr_t)(at + (uint32_t)(r * row_bytes + 16 * c));
                if constexpr (LOAD) *l = *reinterpret_cast<const halfx8*>(q);
                else *reinterpret_cast<halfx8*>(q) = *l;
            }
        }
    }

    // where rows 8 q + 4 lg .. + 3 of tile row a, column l32 of tile column c lie
    static __device__ __forceinline__ uint32_t cell_t(uint32_t at, int a, int c, int q, int lane) {
        return at + (uint32_t)((c * 32 + (lane & 31)) * ROW_T + 2 * (a * 32 + 8 * q + 4 * (lane >> 5)));
    }
};

__device__ __forceinline__ void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// What becomes of a wave's block of sums whose first row and column are ib and jb.
template <int TM, int TN, Epilogue E>
__device__ __forceinline__ void finish(const Product& p, floatx16 (&acc)[TM][TN], int b, int ib, int jb,
                                       uint32_t piece, int lane) {
    using IO = BlockIO<TM, TN>;
    const int l32 = lane & 31, lg = lane >> 5;
    // lane: column j = lane % 32, rows i = 8 (e / 4) + 4 (lane / 32) + e % 4
    const int rows_i = p.rows_u - ib, rows_j = p.rows_v - jb;   // of it inside the matrix
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
        for (int c = 0; c < TN; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[a][c][e] *= p.cb;
    if constexpr (E == kPoly) {
        half_t* add = const_cast<half_t*>(p.add) + (size_t)b * 2 * p.add_plane + (size_t)jb * p.ld_t + ib;
#pragma unroll
        for (int pl = 0; pl < 2; ++pl) {
            IO::template move<TN * 32, TM * 4, true>(add + (size_t)pl * p.add_plane, p.ld_t, rows_j,
                                                     rows_i, piece, IO::ROW_T, lane);
            wave_fence();
#pragma unroll
            for (int a = 0; a < TM; ++a)
#pragma unroll
                for (int c = 0; c < TN; ++c)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const halfx4 x = *(const lds_halfx4*)(uintptr_t)IO::cell_t(piece, a, c, q, lane);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[a][c][4 * q + e] = fmaf(p.ca, (float)x[e], acc[a][c][4 * q + e]);
                    }
            wave_fence();
        }
#pragma unroll
        for (int a = 0; a < TM; ++a)
#pragma unroll
            for (int c = 0; c < TN; ++c)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (ib + 32 * a + 8 * (e >> 2) + 4 * lg + (e & 3) == jb + 32 * c + l32)
                        acc[a][c][e] += p.diagonal;
    }
    if constexpr (E == kLast) {
        const int64_t at0 = (int64_t)b * p.m * p.n;
#pragma unroll
        for (int a = 0; a < TM; ++a)
#pragma unroll
            for (int c = 0; c < TN; ++c)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int i = ib + 32 * a + 8 * (e >> 2) + 4 * lg + (e & 3), j = jb + 32 * c + l32;
                    if (i < p.m && j < p.n)
                        sink_store(p.sink, at0 + (p.tall ? (int64_t)j * p.m + i : (int64_t)i * p.n + j),
                                   acc[a][c][e]);
                }
    } else {
        half_t* out = p.out + (size_t)b * 2 * p.o_plane + (size_t)ib * p.ld_out + jb;
        half_t* out_t = p.out_t + (size_t)b * 2 * p.o_plane + (size_t)jb * p.ld_t + ib;
        // Of a symmetric result what is right of the diagonal (in 32 x 32 tiles) is the
        // mirror image of what is left of it, also inside a workgroup's tile: the two
        // sums add lo hi and hi lo in another order, and which of them counts must
        // not depend on the tile's size.
        constexpr bool kMirrored = E != kStep;
        const int right = (ib - jb) / 32;
#pragma unroll
        for (int pl = 0; pl < 2; ++pl) {
#pragma unroll
            for (int a = 0; a < TM; ++a)
#pragma unroll
                for (int c = 0; c < TN; ++c)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        halfx4 h;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const Pair s = split(acc[a][c][4 * q + e]);
                            h[e] = pl ? s.l : s.h;
                        }
                        *(lds_halfx4*)(uintptr_t)IO::cell_t(piece, a, c, q, lane) = h;
                    }
            wave_fence();
            IO::template move<TN * 32, TM * 4, false, kMirrored ? kFromDiagonal : kAll>(
                out_t + (size_t)pl * p.o_plane, p.ld_t, rows_j, rows_i, piece, IO::ROW_T, lane, right);
            wave_fence();
            typedef __attribute__((address_space(3))) half_t lds_half;
#pragma unroll
            for (int a = 0; a < TM; ++a)
#pragma unroll
                for (int c = 0; c < TN; ++c)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const Pair s = split(acc[a][c][e]);
                        const int i = 32 * a + 8 * (e >> 2) + 4 * lg + (e & 3);
                        *(lds_half*)(uintptr_t)(piece + (uint32_t)(i * IO::ROW + 2 * (32 * c + l32))) =
                            pl ? s.l : s.h;
                    }
            wave_fence();
            IO::template move<TM * 32, TN * 4, false, kMirrored ? kLeft : kAll>(
                out + (size_t)pl * p.o_plane, p.ld_out, rows_i, rows_j, piece, IO::ROW, lane, -right);
            wave_fence();
        }
    }
}

// Workgroups go to the eight dies in turn; this gives each die a run of
// neighbouring numbers, so that the tiles it holds share operands in its L2.
__device__ __forceinline__ uint32_t die_order(uint32_t id, uint32_t total) {
    const uint32_t die = id & 7, q = total >> 3, r = total & 7;
    return die * q + min(die, r) + (id >> 3);
}

// Tile number -> tile row and column, by bands of kBand tile rows, column by
// column within a band, so that neighbouring numbers form squares and a die's tiles share
// operands in its L2: in all 419 us at 1024 x 4096, without die_order 447 us, with
// neither it nor bands 449 us.  Symmetric results have the lower triangle only.
constexpr int kBand = 8;

template <Epilogue E>
__device__ __forceinline__ void tile_of(int tile, int tiles_i, int tiles_j, int& ti, int& tj) {
    if constexpr (E == kGram || E == kPoly) {
        int row = (int)((sqrtf(8.0f * (float)tile + 1.0f) - 1.0f) * 0.5f);
        while ((row + 1) * (row + 2) / 2 <= tile) ++row;
        while (row * (row + 1) / 2 > tile) --row;
        const int first = row / kBand * kBand, rows = min(kBand, tiles_i - first);
        int rest = tile - first * (first + 1) / 2;
        if (rest < (first + 1) * rows) {   // columns that cross the whole band
            tj = rest / rows;
            ti = first + rest - tj * rows;
            return;
        }
        rest -= (first + 1) * rows;
        tj = first + 1;
        int height = rows - 1;
        while (rest >= height) {
            rest -= height;
            ++tj;
            --height;
        }
        ti = tj + rest;
    } else {
        const int band = tile / (kBand * tiles_j), first = band * kBand;
        const int rows = min(kBand, tiles_i - first), rest = tile - first * tiles_j;
        tj = rest / rows;
        ti = first + rest - tj * rows;
    }
}

// BM x BN tile of a product, WM x WN waves, NS stages of BK-deep slices in LDS.
// Slices arrive by direct-to-LDS loads, 1 KB each.  A row of a slice is CH = BK / 8
// chunks of 16 bytes, and its slot s holds chunk s ^ (r / (16 / CH)) % CH: the
// 16-byte fragment reads of 16 neighbouring rows fall on all 64 banks once.
// Fragments are read one 16-deep step ahead of the products that use them, and
// the barrier between two slices stands before the last step's products, so
// that they cover the first reads of the next slice.
//
// `splits` workgroups may share a tile along K: each leaves its sum in `part` for
// ns_join.  (The last of them could add the parts itself, but the fence that
// makes them visible writes back a die's whole L2: 65 us against 24 with the
// second launch at 1024 x 4096.)
template <int BM, int BN, int WM, int WN, int BK, int NS, Epilogue E>
__global__ __launch_bounds__(64 * WM * WN, NS * (BM + BN) * 4 * BK > 81920 ? 1 : 2) void ns_product(
    Product p) {
    constexpr int W = WM * WN;
    constexpr int PL = 2;                                    // planes of an operand
    constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
    constexpr int CH = BK / 8, RPU = 64 / CH;                // chunks a row, rows a load
    constexpr int ROWB = 2 * BK, KS = BK / 16;
    constexpr int UNITS = (BM + BN) * PL / RPU, OPS = UNITS / W;
    constexpr int STAGE = (BM + BN) * PL * ROWB;
    using IO = BlockIO<TM, TN>;
    constexpr int PIECE = (IO::BYTES + 15) / 16 * 16;
    static_assert(UNITS % W == 0 && BM % RPU == 0 && BN % RPU == 0, "whole loads per wave");
    static_assert(TM * WM * 32 == BM && TN * WN * 32 == BN, "whole tiles per wave");
    __shared__ __attribute__((aligned(1024))) uint8_t ring[NS * STAGE > W * PIECE ? NS * STAGE : W * PIECE];

    const int lane = threadIdx.x & 63;
    const int wave = uniform(threadIdx.x >> 6);
    const uint32_t id = die_order(blockIdx.y * gridDim.x + blockIdx.x, gridDim.x * gridDim.y);
    const int b = (int)(id / gridDim.x), shared = (int)(id - b * gridDim.x);
    const int tile = shared / p.splits, part = shared - tile * p.splits;
    int ti, tj;
    tile_of<E>(tile, p.tiles_i, p.tiles_j, ti, tj);
    const int i0 = ti * BM, j0 = tj * BN;
    const half_t* u = p.u + (size_t)b * 2 * p.u_plane;
    const half_t* v = p.v + (size_t)b * 2 * p.v_plane;

    // this workgroup's slices: shares are whole 64-deep slices for every tile
    const int nk_all = p.K / 64;
    const int k_lo = (int)((int64_t)nk_all * part / p.splits) * (64 / BK);
    const int nk = (int)((int64_t)nk_all * (part + 1) / p.splits) * (64 / BK) - k_lo;

    const half_t* src[OPS];
#pragma unroll
    for (int o = 0; o < OPS; ++o) {
        const int unit = o * W + wave;
        constexpr int UU = BM / RPU, UV = BN / RPU;
        const half_t* q;
        int row;   // within the tile; rows past the matrix repeat its last one
        if (unit < PL * UU) {
            const int pl = unit / UU;
            row = (unit - pl * UU) * RPU + lane / CH;
            q = u + (size_t)pl * p.u_plane + (size_t)min(i0 + row, p.rows_u - 1) * p.K;
        } else {
            const int pl = (unit - PL * UU) / UV;
            row = (unit - PL * UU - pl * UV) * RPU + lane / CH;
            q = v + (size_t)pl * p.v_plane + (size_t)min(j0 + row, p.rows_v - 1) * p.K;
        }
        src[o] = q + 8 * ((lane % CH) ^ ((row / (16 / CH)) % CH)) + (size_t)k_lo * BK;
    }
    const uint32_t ring_at = (uint32_t)(uintptr_t)(lds_u8*)&ring[0];
    // load o of slice k
    auto issue_one = [&](int k, int o) {
        dma_lds16(src[o] + (size_t)k * BK,
                  ring_at + (uint32_t)((k % NS) * STAGE) + (uint32_t)((o * W + wave) * 1024));
    };
    auto issue = [&](int k) {
#pragma unroll
        for (int o = 0; o < OPS; ++o) issue_one(k, o);
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
    const uint32_t row_u = (uint32_t)((wm * TM * 32 + l32) * ROWB);
    const uint32_t row_v = (uint32_t)(BM * PL * ROWB + (wn * TN * 32 + l32) * ROWB);
    halfx8 fu[2][TM][PL], fv[2][TN][PL];
    auto fetch = [&](int set, int k, int ks) {
        const lds_u8* st = base + (k % NS) * STAGE;
        // the tiles' rows differ by multiples of 32: one swizzle for all
        const uint32_t ch = (uint32_t)(16 * ((2 * ks + lg) ^ ((l32 / (16 / CH)) % CH)));
#pragma unroll
        for (int a = 0; a < TM; ++a)
#pragma unroll
            for (int q = 0; q < PL; ++q)
                fu[set][a][q] = *(const lds_halfx8*)(st + row_u + ch + (q * BM + a * 32) * ROWB);
#pragma unroll
        for (int c = 0; c < TN; ++c)
#pragma unroll
            for (int q = 0; q < PL; ++q)
                fv[set][c][q] = *(const lds_halfx8*)(st + row_v + ch + (q * BN + c * 32) * ROWB);
    };
    // One 16-deep step's products.  The next slice's loads go out between them,
    // evenly over the slice: issued in a row they hold up the wave, and with it
    // the matrix core, for as long as the products take.
    constexpr int PRODUCTS = TM * TN * 3;   // of one step
    // two stages: before the last step, which waits for them
    constexpr int SPREAD = PRODUCTS * (NS == 2 ? KS - 1 : KS);
    auto multiply = [&](int set, int ks, int load_k, bool load) {
        int n = ks * PRODUCTS;   // products of the slice so far
#pragma unroll
        for (int part = 0; part < 3; ++part)   // lo hi, hi lo, hi hi
#pragma unroll
            for (int a = 0; a < TM; ++a)
#pragma unroll
                for (int c = 0; c < TN; ++c) {
                    acc[a][c] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                        fu[set][a][part == 0], fv[set][c][part == 1], acc[a][c], 0, 0, 0);
                    const int o0 = min(n * OPS / SPREAD, OPS), o1 = min((n + 1) * OPS / SPREAD, OPS);
                    ++n;
                    if (load && o1 > o0) {
                        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                        for (int o = o0; o < o1; ++o) issue_one(load_k, o);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
    };

    const int ahead = min(NS - 1, nk);
    for (int k = 0; k < ahead; ++k) issue(k);
    // slice k has landed when at most the loads of the NS - 2 after it are out
    if (ahead == NS - 1) wait_vmcnt<OPS*(NS - 2)>();
    else wait_vmcnt<0>();
    __syncthreads();
    fetch(0, 0, 0);
    for (int k = 0; k < nk; ++k) {
        const bool more = k + 1 < nk;
        const bool issued = k + NS - 1 < nk;   // into the stage that everyone has left
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            if (ks + 1 < KS) {
                fetch((ks + 1) & 1, k, ks + 1);
            } else if (more) {
                // the loads of this slice's products so far are the youngest
                if (issued) wait_vmcnt<NS == 2 ? 0 : OPS*(NS - 3) + OPS*(KS - 1) / KS>();
                else wait_vmcnt<0>();
                __syncthreads();
                fetch(KS & 1, k + 1, 0);
            }
            multiply(ks & 1, ks, k + NS - 1, issued);
        }
        static_assert(KS % 2 == 0, "the next slice starts on set 0");
    }

    if (p.splits > 1) {
        // in the accumulators' own order: every access is whole
        float* mine = p.part + ((size_t)b * gridDim.x + shared) * (BM * BN);
#pragma unroll
        for (int a = 0; a < TM; ++a)
#pragma unroll
            for (int c = 0; c < TN; ++c)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    reinterpret_cast<floatx4*>(mine)[((wave * TM + a) * TN + c) * 256 + q * 64 + lane] =
                        floatx4{acc[a][c][4 * q], acc[a][c][4 * q + 1], acc[a][c][4 * q + 2],
                                acc[a][c][4 * q + 3]};
        return;
    }
    __syncthreads();   // the ring is free
    finish<TM, TN, E>(p, acc, b, i0 + wm * TM * 32, j0 + wn * TN * 32,
                      ring_at + (uint32_t)(wave * PIECE), lane);
}

// Adds the parts of a tile that `splits` workgroups computed, in order, and
// finishes it: a wave for each wave's block of the tile.
template <int BM, int BN, int WM, int WN, Epilogue E>
__global__ __launch_bounds__(64) void ns_join(Product p) {
    constexpr int W = WM * WN, TM = BM / WM / 32, TN = BN / WN / 32;
    __shared__ __attribute__((aligned(16))) uint8_t lds[(BlockIO<TM, TN>::BYTES + 15) / 16 * 16];
    const int lane = threadIdx.x, b = blockIdx.y;
    const int tile = blockIdx.x / W, wave = blockIdx.x - tile * W;
    int ti, tj;
    tile_of<E>(tile, p.tiles_i, p.tiles_j, ti, tj);
    const size_t first = ((size_t)b * (gridDim.x / W) + tile) * p.splits;
    floatx16 acc[TM][TN];
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
        for (int c = 0; c < TN; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[a][c][e] = 0.0f;
    for (int t = 0; t < p.splits; ++t) {
        const floatx4* from = reinterpret_cast<const floatx4*>(p.part + (first + t) * (BM * BN));
#pragma unroll
        for (int a = 0; a < TM; ++a)
#pragma unroll
            for (int c = 0; c < TN; ++c)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const floatx4 f = from[((wave * TM + a) * TN + c) * 256 + q * 64 + lane];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[a][c][4 * q + e] += f[e];
                }
    }
    const int wm = wave / WN, wn = wave % WN;
    finish<TM, TN, E>(p, acc, b, ti * BM + wm * TM * 32, tj * BN + wn * TN * 32,
                      (uint32_t)(uintptr_t)(lds_u8*)&lds[0], lane);
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
// there too.
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
    // 32-bit offsets from here on: at most 2^14 elements
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
        q = (int)(((float)at + 0.5f) * rwidth);   // at <= 2^14: exact
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

    floatx16 y[CB][MT];
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
            wave_fence();
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
            wave_fence();
        }
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
                    y[c][a][e] = ca * ((float)xh[c][a][e >> 3][e & 7] + (float)xl[c][a][e >> 3][e & 7]) +
                                 y[c][a][e] * (1.0f / kSP);
                    const Pair p = split(y[c][a][e]);
                    xh[c][a][e >> 3][e & 7] = p.h;
                    xl[c][a][e >> 3][e & 7] = p.l;
                }
    }
    // ---- result: the last step's float32 values, back through LDS and written as
    // they lie in memory.  No step reads them: they may exceed float16's range (16
    // times kSX), as the caller's check allows them to ----
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
                    *(lds_float*)(uintptr_t)(x_at + 4u * (uint32_t)(i * ld + j)) = y[c][a][e] * (1.0f / kSX);
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
                for (int e = 0; e < 4; ++e) f[e] = new_weight(to, w[k][e], f[e]);
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
    // 32 x 512 and 64 x 256; past that a step on one compute unit takes longer
    // than a launch over several (64 x 448: 42 us here, 38 us by ns_panel)
    if (mt > 2 || blocks > (mt == 1 ? 16 : 8)) return s;
    s.mt = mt;
    s.cb = 1;
    while (s.cb * 8 < blocks) s.cb *= 2;
    // at least a wave for each tile of A, also where there are fewer columns
    s.waves = std::max(mt * mt, (blocks + s.cb - 1) / s.cb);
    return s;
}

// ---------------------------------------------------------------------------
// Flat matrices: one launch a step
// ---------------------------------------------------------------------------
// Up to 64 rows by 8192 columns, or 128 by 1536.  A workgroup owns a panel of 128 columns and
// does a whole step on it: it adds the panels' parts of X X^T, forms P (every
// workgroup the same one: 128^3 products cost less than a launch), advances its
// panel and leaves its part of the new X X^T.  At 128 x 896 the tiled products'
// three launches a step, each 5 us long with next to no work in it, become one.
//
// LDS: the panel's X^T as rows of a column's M entries, hi then lo, whose
// 16-byte chunk c lies in slot c ^ (column % chunks); A and then P as padded rows.
template <int MT>
struct PanelCfg {
    static constexpr int M = 32 * MT, NT = MT * (MT + 1) / 2, CH = M / 8;
    static constexpr int COLS = 128, WAVES = 4 * MT;        // a 32 x 32 block of the panel each
    static constexpr int X_PLANE = COLS * 2 * M;            // bytes
    static constexpr int ROW_A = 2 * M + 16, A_PLANE = M * ROW_A;
    static constexpr int LDS = 2 * X_PLANE + 2 * A_PLANE;
    static __device__ __forceinline__ uint32_t x_cell(int col, int row) {
        return (uint32_t)(col * 2 * M + 16 * ((row >> 3) ^ (col & (CH - 1))) + 2 * (row & 7));
    }
};

struct PanelArgs {
    half_t* XT;                // [batch][hi, lo][np][M], advanced in place
    size_t xplane;
    const float* part_in;      // [batch][panel][tile][1024]
    float* part_out;
    int* exponents;            // [batch][panel]: X as loaded is the matrix times 2^-exponent
    int panels, np;
    int m, n, tall;
    float ca, cb, cc, eps;
    int raw, last;             // the step on X as loaded; only the result
    Sink sink;
};

// A panel's part of X X^T: a lower tile a wave.
template <int MT>
__device__ __forceinline__ void panel_gram(uint32_t x_at, int cols, float* out, int wave, int lane) {
    using C = PanelCfg<MT>;
    if (wave >= C::NT) return;
    int ta = 0;
    while ((ta + 1) * (ta + 2) / 2 <= wave) ++ta;
    const int tb = wave - ta * (ta + 1) / 2;
    floatx16 g;
#pragma unroll
    for (int e = 0; e < 16; ++e) g[e] = 0.0f;
    // this lane's cells of the first 16 columns, for the two halves of a read
    const int s16 = lane & 15, q16 = lane >> 4;
    const int col = 8 * (q16 >> 1) + (s16 >> 2), row = 16 * (q16 & 1) + 4 * (s16 & 3);
    const uint32_t ca[2] = {x_at + C::x_cell(col, 32 * ta + row), x_at + C::x_cell(col + 4, 32 * ta + row)};
    const uint32_t cb[2] = {x_at + C::x_cell(col, 32 * tb + row), x_at + C::x_cell(col + 4, 32 * tb + row)};
    for (int kc0 = 0; kc0 < cols / 16; kc0 += 4)   // 64 or 128 columns
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            // 16 columns on, the slots are the same
            auto turned = [&](const uint32_t (&cell)[2], int pl) {
                const uint32_t at = (uint32_t)(pl * C::X_PLANE + (kc0 + u) * 32 * C::M);
                const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(uintptr_t)(cell[0] + at));
                const v4i16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(uintptr_t)(cell[1] + at));
                return __builtin_bit_cast(halfx8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            };
            g = mfma3(turned(ca, 0), turned(ca, 1), turned(cb, 0), turned(cb, 1), g);
        }
#pragma unroll
    for (int q = 0; q < 4; ++q)
        reinterpret_cast<floatx4*>(out)[wave * 256 + q * 64 + lane] =
            floatx4{g[4 * q], g[4 * q + 1], g[4 * q + 2], g[4 * q + 3]};
}

// Loads a panel (advancing the momentum where there is one), as the matrix times
// the power of two that brings the panel's largest entry into [1, 2), and leaves
// its part of X X^T.  The Frobenius norm is that product's trace: the first
// ns_panel divides by it, which saves the two launches that a norm of its own
// and the division take.
template <typename T, int MT>
__global__ __launch_bounds__(256 * MT) void ns_panel_load(Source src, const float* buf_in, float* buf_out,
                                                          PanelArgs p) {
    using C = PanelCfg<MT>;
    constexpr int THREADS = 64 * C::WAVES;
    __shared__ __attribute__((aligned(1024))) uint8_t lds_raw[2 * C::X_PLANE];
    __shared__ float stage[C::COLS * (C::M + 1) > C::M * (C::COLS + 1) ? C::COLS * (C::M + 1) : C::M * (C::COLS + 1)];
    __shared__ float red[C::WAVES];
    const uint32_t x_at = (uint32_t)(uintptr_t)(lds_u8*)&lds_raw[0];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int panel = blockIdx.x, b = blockIdx.y, col0 = panel * C::COLS;
    const int cols = min(C::COLS, p.np - col0);
    const int64_t base = (int64_t)b * p.m * p.n;
    const T* in = static_cast<const T*>(src.m) + base;
    const float* old = buf_out ? buf_in + base : nullptr;
    float* fresh = buf_out ? buf_out + base : nullptr;

    // rows of memory that cross the panel, four elements a thread and pass
    const int real = min(C::COLS, p.n - col0);                     // columns of the matrix, at least 1
    const int rows = p.tall ? real : p.m, width = p.tall ? p.m : real;
    const int ld = (p.tall ? C::M : C::COLS) + 1;
    constexpr int ROWS_MOST = C::COLS > C::M ? C::COLS : C::M, QUADS = ROWS_MOST / 4;
    constexpr int PASSES = ROWS_MOST * QUADS / THREADS;
    float v[PASSES][4], o[PASSES][4];
    auto where = [&](int k, int& r, int& c, int64_t& at) {
        const int idx = k * THREADS + threadIdx.x;
        r = idx / QUADS;
        c = idx % QUADS * 4;
        at = p.tall ? (int64_t)(col0 + r) * p.m : (int64_t)r * p.n + col0;
        return r < rows && c < width;
    };
#pragma unroll
    for (int k = 0; k < PASSES; ++k) {
        int r, c;
        int64_t at;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k][e] = o[k][e] = 0.0f;
        if (where(k, r, c, at)) {
            load4(in + at, c, width, v[k]);
            if (fresh != nullptr) load4(old + at, c, width, o[k]);
        }
    }
    float most = 0.0f;
#pragma unroll
    for (int k = 0; k < PASSES; ++k) {
        int r, c;
        int64_t at;
        if (!where(k, r, c, at)) continue;
        if (fresh != nullptr) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                o[k][e] = src.beta * o[k][e] + v[k][e];
                v[k][e] = src.nesterov ? v[k][e] + src.beta * o[k][e] : o[k][e];
            }
            store4(fresh + at, c, width, o[k]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c + e < width) {
                most = fmaxf(most, fabsf(v[k][e]));   // passes over a NaN, which poisons the sums later
                stage[r * ld + c + e] = v[k][e];
            }
    }
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) most = fmaxf(most, __shfl_xor(most, k));
    if (lane == 0) red[wave] = most;
    __syncthreads();
    for (int w = 0; w < C::WAVES; ++w) most = fmaxf(most, red[w]);
    // -200: a panel of zeros counts for nothing beside any other
    const int exponent = most > 0.0f ? (most < INFINITY ? ilogbf(most) : 127) : -200;
    if (threadIdx.x == 0) p.exponents[b * p.panels + panel] = exponent;

    half_t* xt = p.XT + (size_t)b * 2 * p.xplane + (size_t)col0 * C::M;
#pragma unroll
    for (int k = 0; k < C::X_PLANE / 16 / THREADS; ++k) {
        const int chunk = k * THREADS + threadIdx.x, col = chunk / C::CH, c = chunk % C::CH;
        halfx8 h, l;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = 8 * c + e;
            const float f = col < real && i < p.m ? stage[p.tall ? col * ld + i : i * ld + col] : 0.0f;
            const Pair q = split(ldexpf(f, -exponent) * kSX);
            h[e] = q.h;
            l[e] = q.l;
        }
        const uint32_t at = x_at + C::x_cell(col, 8 * c);
        *(lds_halfx8*)(uintptr_t)at = h;
        *(lds_halfx8*)(uintptr_t)(at + C::X_PLANE) = l;
        if (col < cols) {
            *reinterpret_cast<halfx8*>(xt + (size_t)col * C::M + 8 * c) = h;
            *reinterpret_cast<halfx8*>(xt + p.xplane + (size_t)col * C::M + 8 * c) = l;
        }
    }
    __syncthreads();
    panel_gram<MT>(x_at, cols, p.part_out + ((size_t)b * p.panels + panel) * C::NT * 1024, wave, lane);
}

template <int MT>
__global__ __launch_bounds__(256 * MT) void ns_panel(PanelArgs p) {
    using C = PanelCfg<MT>;
    constexpr int THREADS = 64 * C::WAVES;
    __shared__ __attribute__((aligned(1024))) uint8_t lds_raw[C::LDS];
    __shared__ float red[C::WAVES];
    const uint32_t x_at = (uint32_t)(uintptr_t)(lds_u8*)&lds_raw[0];
    const uint32_t a_at = x_at + 2 * C::X_PLANE;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int l32 = lane & 31, lg = lane >> 5;
    const int panel = blockIdx.x, b = blockIdx.y, col0 = panel * C::COLS;
    const int cols = min(C::COLS, p.np - col0);   // 64 or 128
    half_t* xt = p.XT + (size_t)b * 2 * p.xplane + (size_t)col0 * C::M;

    // the panel's X^T: 1 KB a load, 16 bytes a lane
    constexpr int PER = C::X_PLANE / 1024 / C::WAVES;   // loads of a wave and plane
#pragma unroll
    for (int pl = 0; pl < 2; ++pl)
#pragma unroll
        for (int o = 0; o < PER; ++o) {
            const int unit = o * C::WAVES + wave, chunk = unit * 64 + lane;
            const int col = min(chunk / C::CH, cols - 1);   // past a half panel: its last column
            const int slot = chunk % C::CH;
            dma_lds16(xt + (size_t)pl * p.xplane + (size_t)col * C::M + 8 * (slot ^ ((chunk / C::CH) & (C::CH - 1))),
                      x_at + (uint32_t)(pl * C::X_PLANE + unit * 1024));
        }

    typedef __attribute__((address_space(3))) half_t lds_half;
    float x_scale = 1.0f;   // of the panel: the matrix's norm, once
    {
        // ---- A from the panels' parts, in order ----
        const floatx4* in = reinterpret_cast<const floatx4*>(p.part_in) + (size_t)b * p.panels * C::NT * 256;
        constexpr int POS = (C::NT * 256 + THREADS - 1) / THREADS;
        floatx4 v[POS];
#pragma unroll
        for (int k = 0; k < POS; ++k) v[k] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
        int top = -200;   // the panels' largest exponent
        if (p.raw)
            for (int q = 0; q < p.panels; ++q) top = max(top, p.exponents[b * p.panels + q]);
        // four panels' reads in flight; past the last panel it is read again and dropped
        for (int q0 = 0; q0 < p.panels; q0 += 4) {
            floatx4 f[4][POS];
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int k = 0; k < POS; ++k)
                    f[u][k] = in[(size_t)min(q0 + u, p.panels - 1) * C::NT * 256 +
                                 min(k * THREADS + (int)threadIdx.x, C::NT * 256 - 1)];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (q0 + u < p.panels) {
                    const float weight =
                        p.raw ? ldexpf(1.0f, 2 * (p.exponents[b * p.panels + q0 + u] - top)) : 1.0f;
#pragma unroll
                    for (int k = 0; k < POS; ++k) v[k] += weight * f[u][k];
                }
        }
        float a_scale = kSA / (kSX * kSX);
        if (p.raw) {
            // |M|_F^2 = trace(M M^T), in units of 2^(2 top) / kSX^2
            float trace = 0.0f;
#pragma unroll
            for (int k = 0; k < POS; ++k) {
                const int group = uniform(C::WAVES * k + wave);
                if (group >= C::NT * 4) break;
                int ta = 0;
                while ((ta + 1) * (ta + 2) / 2 <= group >> 2) ++ta;
                if ((group >> 2) != ta * (ta + 3) / 2) continue;   // not a diagonal tile
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (8 * (group & 3) + 4 * lg + r == l32) trace += v[k][r];
            }
#pragma unroll
            for (int k = 32; k > 0; k >>= 1) trace += __shfl_xor(trace, k);
            if (lane == 0) red[wave] = trace;
            __syncthreads();
            double sum = 0.0;
            for (int w = 0; w < C::WAVES; ++w) sum += (double)red[w];
            const double unit = ldexp(1.0, top);
            const double r = unit / (sqrt(sum) * (1.0 / kSX) * unit + (double)p.eps);
            a_scale *= (float)(r * r);
            x_scale = (float)(r * ldexp(1.0, p.exponents[b * p.panels + panel] - top));
        }
#pragma unroll
        for (int k = 0; k < POS; ++k) {
            const int group = uniform(C::WAVES * k + wave);   // of 64 places: a quarter of a tile
            if (group >= C::NT * 4) break;
            const int tile = group >> 2, q = group & 3, pl = lane;
            int ta = 0;
            while ((ta + 1) * (ta + 2) / 2 <= tile) ++ta;
            const int tb = tile - ta * (ta + 1) / 2;
            const int i = 32 * ta + 8 * q + 4 * (pl >> 5), j = 32 * tb + (pl & 31);
            halfx4 h, l;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const Pair s = split(v[k][r] * a_scale);
                h[r] = s.h;
                l[r] = s.l;
            }
            const uint32_t at = a_at + (uint32_t)(j * C::ROW_A + 2 * i);
            *(lds_halfx4*)(uintptr_t)at = h;
            *(lds_halfx4*)(uintptr_t)(at + C::A_PLANE) = l;
            if (ta != tb) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint32_t at2 = a_at + (uint32_t)((i + r) * C::ROW_A + 2 * j);
                    *(lds_half*)(uintptr_t)at2 = h[r];
                    *(lds_half*)(uintptr_t)(at2 + C::A_PLANE) = l[r];
                }
            }
        }
        __syncthreads();
        // ---- P = a I + b A + c A^2: a lower tile a wave ----
        static_assert(C::NT <= C::WAVES, "a wave for each tile");
        int ta = 0;
        while ((ta + 1) * (ta + 2) / 2 <= wave) ++ta;
        const int tb = wave - ta * (ta + 1) / 2;
        floatx16 g;
#pragma unroll
        for (int e = 0; e < 16; ++e) g[e] = 0.0f;
        if (wave < C::NT) {
#pragma unroll
            for (int kc = 0; kc < 2 * MT; ++kc) {
                const uint32_t u = a_at + (uint32_t)((32 * ta + l32) * C::ROW_A + 32 * kc + 16 * lg);
                const uint32_t w = a_at + (uint32_t)((32 * tb + l32) * C::ROW_A + 32 * kc + 16 * lg);
                g = mfma3(*(const lds_halfx8*)(uintptr_t)u, *(const lds_halfx8*)(uintptr_t)(u + C::A_PLANE),
                          *(const lds_halfx8*)(uintptr_t)w, *(const lds_halfx8*)(uintptr_t)(w + C::A_PLANE), g);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = 32 * ta + 8 * q + 4 * lg, j = 32 * tb + l32;
                const uint32_t at = a_at + (uint32_t)(j * C::ROW_A + 2 * i);
                const halfx4 h = *(const lds_halfx4*)(uintptr_t)at;
                const halfx4 l = *(const lds_halfx4*)(uintptr_t)(at + C::A_PLANE);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    g[4 * q + r] = p.cb * (kSP / kSA) * ((float)h[r] + (float)l[r]) +
                                   p.cc * (kSP / (kSA * kSA)) * g[4 * q + r] + (i + r == j ? p.ca * kSP : 0.0f);
            }
        }
        __syncthreads();   // A has been read: P takes its place
        if (wave < C::NT)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = 32 * ta + 8 * q + 4 * lg, j = 32 * tb + l32;
                halfx4 h, l;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const Pair s = split(g[4 * q + r]);
                    h[r] = s.h;
                    l[r] = s.l;
                }
                const uint32_t at = a_at + (uint32_t)(j * C::ROW_A + 2 * i);
                *(lds_halfx4*)(uintptr_t)at = h;
                *(lds_halfx4*)(uintptr_t)(at + C::A_PLANE) = l;
                if (ta != tb) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const uint32_t at2 = a_at + (uint32_t)((i + r) * C::ROW_A + 2 * j);
                        *(lds_half*)(uintptr_t)at2 = h[r];
                        *(lds_half*)(uintptr_t)(at2 + C::A_PLANE) = l[r];
                    }
                }
            }
        wait_vmcnt<0>();   // the panel has landed
        __syncthreads();
        // ---- X <- (a I + P) X: a 32 x 32 block a wave ----
        const int rt = wave % MT, cb = wave / MT;
        floatx16 y;
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = 0.0f;
#pragma unroll
        for (int kc = 0; kc < 2 * MT; ++kc) {
            const uint32_t v = x_at + C::x_cell(32 * cb + l32, 16 * kc + 8 * lg);
            const uint32_t u = a_at + (uint32_t)((32 * rt + l32) * C::ROW_A + 32 * kc + 16 * lg);
            y = mfma3(*(const lds_halfx8*)(uintptr_t)u, *(const lds_halfx8*)(uintptr_t)(u + C::A_PLANE),
                      *(const lds_halfx8*)(uintptr_t)v, *(const lds_halfx8*)(uintptr_t)(v + C::X_PLANE), y);
        }
        if (p.last) {
            const int64_t at0 = (int64_t)b * p.m * p.n;
            const int j = col0 + 32 * cb + l32;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int i = 32 * rt + 8 * (e >> 2) + 4 * lg + (e & 3);
                if (i < p.m && j < p.n)
                    sink_store(p.sink, at0 + (p.tall ? (int64_t)j * p.m + i : (int64_t)i * p.n + j),
                               y[e] * (x_scale / (kSP * kSX)));
            }
            return;
        }
        __syncthreads();   // the old panel has been read
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            halfx4 h, l;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const Pair s = split(y[4 * q + r] * (x_scale / kSP));
                h[r] = s.h;
                l[r] = s.l;
            }
            const uint32_t at = x_at + C::x_cell(32 * cb + l32, 32 * rt + 8 * q + 4 * lg);
            *(lds_halfx4*)(uintptr_t)at = h;
            *(lds_halfx4*)(uintptr_t)(at + C::X_PLANE) = l;
        }
        __syncthreads();
        // whole rows back to memory
#pragma unroll
        for (int pl = 0; pl < 2; ++pl)
#pragma unroll
            for (int o = 0; o < PER; ++o) {
                const int chunk = (o * C::WAVES + wave) * 64 + lane, col = chunk / C::CH, c = chunk % C::CH;
                if (col < cols)
                    *reinterpret_cast<halfx8*>(xt + (size_t)pl * p.xplane + (size_t)col * C::M + 8 * c) =
                        *(const lds_halfx8*)(uintptr_t)(x_at + pl * C::X_PLANE + C::x_cell(col, 8 * c));
            }
    }
    panel_gram<MT>(x_at, cols, p.part_out + ((size_t)b * p.panels + panel) * C::NT * 1024, wave, lane);
}

// Whether a matrix takes ns_panel, and its parts of X X^T.  Every panel reads
// all parts: 0.1 us a part and step for 64 rows, 0.4 us for 128, which the tiled
// products' two further launches a step are worth up to about here (in all 38 us
// at 64 x 448 and 84 us at 128 x 896, against 80 and 119 us tiled).
bool panel_shape(int m, int n) { return (m <= 64 && n <= 8192) || (m <= 128 && n <= 1536); }
int panels_of(int np) { return (np + 127) / 128; }
size_t panel_part_bytes(int mp, int np) {
    const int mt = mp / 32;
    return (size_t)panels_of(np) * (mt * (mt + 1) / 2) * 4096;
}

size_t up(size_t v, size_t a) { return (v + a - 1) / a * a; }

int done(const char* what) {
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return set_error(DISCO_EHIP, "%s launch failed: %s", what, hipGetErrorString(e));
    return DISCO_OK;
}

// Tile of a product: kinds 0 and 1 are 64 x 64 with a deep ring (one workgroup a
// compute unit) and with a shallow one (two), 2 is 128 x 128, 3 is 192 x 192;
// `splits` workgroups share a tile along K.
struct TileChoice {
    int kind = 0, splits = 1;
};

constexpr int kSides[4] = {64, 64, 128, 192};

// The choice with the least estimated time.  Times in microseconds as measured
// from 256 x 256 to 4096 x 4096: a 64-deep slice of one tile, and a tile's start
// and end.  For instance 1024 x 4096: X X^T on 136 tiles of 64 takes 32 us, on 36 of
// 128 73 us, on 128-tiles shared by seven 23 us and 7 us more for their joining; P X
// on 1024 tiles of 64 41 to 45 us, on 256 of 128 35 us, on 132 of 192 57 us.  4096 x
// 4096: P X on 1024 tiles of 128 417 us, on 484 of 192 411 us.
// The shares decide the order of the float32 sums and are those of one matrix, so
// that its bits do not depend on how many others share the call; the tile does not
// change them, and goes by the whole batch.  (Shares by the batch as well would be
// worth up to an eighth: four matrices of 640 x 4096 take 679 us, and took 605; two of
// 1024 x 4096 750 and 689.)
TileChoice choose_tile(int batch, int ni, int nj, int K, bool can_split, bool symmetric) {
    static const double slice_us[4] = {0.39, 0.65, 1.0, 2.5};
    static const double ends_us[4] = {2.0, 2.0, 3.5, 8.0};
    constexpr double kNever = 1e300;
    auto tiles_of = [&](int kind) {
        const int64_t side = kSides[kind], ti = (ni + side - 1) / side, tj = (nj + side - 1) / side;
        return symmetric ? ti * (ti + 1) / 2 : ti * tj;
    };
    auto at_once = [](int kind) { return kind == 1 ? 512 : 256; };
    auto estimate = [&](int kind, int splits, int matrices) {
        if (splits > 1 && kind == 3) return kNever;
        const int64_t rounds = (matrices * tiles_of(kind) * splits + at_once(kind) - 1) / at_once(kind);
        const double us = rounds * (K / 64.0 / splits * slice_us[kind] + ends_us[kind]);
        return splits > 1 ? us + 4.0 + 0.2 * splits * kSides[kind] / 64 : us;
    };
    TileChoice best;
    double best_us = kNever;
    auto consider = [&](int kind, int splits, int matrices) {
        const double us = estimate(kind, splits, matrices);
        if (us < best_us) {
            best_us = us;
            best.kind = kind;
            best.splits = splits;
        }
    };
    for (int kind = 0; kind < 4; ++kind) {
        const int64_t tiles = tiles_of(kind);
        // also as many as fill the compute units once
        for (int splits : {1, 2, 4, 8, 16, (int)std::min<int64_t>(16, std::max<int64_t>(1, at_once(kind) / tiles))})
            if (splits == 1 || (can_split && K / 64 >= 4 * splits && tiles * splits <= 2048))
                consider(kind, splits, 1);
    }
    if (batch > 1) {
        best_us = kNever;
        for (int kind = 0; kind < 4; ++kind) consider(kind, best.splits, batch);
    }
    return best;
}

// Where everything of a call lies in its workspace.
struct Layout {
    int m, n, mp, np, tall, nparts;
    size_t xplane, aplane;                 // elements of one plane
    size_t partial, X, XT0, XT1, A, P, part;     // byte offsets
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
    l.nparts = (int)std::max<int64_t>(1, std::min<int64_t>(256, elems / 16384));   // ns_load adds 256
    l.xplane = (size_t)l.mp * l.np;
    l.aplane = (size_t)l.mp * l.mp;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at = up(at + bytes, 1024);
        return here;
    };
    if (panel_shape(l.m, l.n)) {   // two sets of parts: one read, one written
        l.partial = take((size_t)batch * panels_of(l.np) * sizeof(int));
        l.XT0 = take((size_t)batch * 2 * l.xplane * sizeof(half_t));
        l.part = take(2 * batch * panel_part_bytes(l.mp, l.np));
        l.bytes = at;
        return l;
    }
    l.partial = take((size_t)batch * l.nparts * sizeof(double));
    l.X = take((size_t)batch * 2 * l.xplane * sizeof(half_t));
    l.XT0 = take((size_t)batch * 2 * l.xplane * sizeof(half_t));
    l.XT1 = take((size_t)batch * 2 * l.xplane * sizeof(half_t));
    l.A = take((size_t)batch * 2 * l.aplane * sizeof(half_t));
    l.P = take((size_t)batch * 2 * l.aplane * sizeof(half_t));
    // the parts of X X^T where workgroups share its tiles
    const TileChoice t = choose_tile(batch, l.mp, l.mp, l.np, true, true);
    const size_t side = kSides[t.kind], ti = (l.mp + side - 1) / side;
    l.part = take(t.splits > 1 ? (size_t)batch * (ti * (ti + 1) / 2) * t.splits * side * side * sizeof(float) : 0);
    l.bytes = at;
    return l;
}

template <int SIDE, int WM, int WN, int BK, int NS, Epilogue E>
int launch_tiles(Product p, int splits, int batch, hipStream_t st) {
    constexpr const char* names[] = {"ns_gram", "ns_poly", "ns_step", "ns_last"};
    const int64_t ti = (p.rows_u + SIDE - 1) / SIDE, tj = (p.rows_v + SIDE - 1) / SIDE;
    const int64_t tiles = E == kGram || E == kPoly ? ti * (ti + 1) / 2 : ti * tj;
    if (tiles * splits * batch > 0x7fffffff / 8) return set_error(DISCO_EUNSUPPORTED, "matrix too large");
    p.tiles_i = (int)ti;
    p.tiles_j = (int)tj;
    p.splits = splits;
    {
        KernelTimer timer(names[E], st);
        hipLaunchKernelGGL((ns_product<SIDE, SIDE, WM, WN, BK, NS, E>), dim3((unsigned)(tiles * splits), batch),
                           dim3(64 * WM * WN), 0, st, p);
    }
    if (int rc = done(names[E])) return rc;
    if constexpr (E == kGram && SIDE < 192) {
        if (splits > 1) {
            KernelTimer timer("ns_join", st);
            hipLaunchKernelGGL((ns_join<SIDE, SIDE, WM, WN, E>), dim3((unsigned)(tiles * WM * WN), batch),
                               dim3(64), 0, st, p);
            return done("ns_join");
        }
    }
    return DISCO_OK;
}

template <Epilogue E>
int launch_product(const Product& p, int batch, hipStream_t st) {
    const TileChoice t = choose_tile(batch, p.rows_u, p.rows_v, p.K, E == kGram, E == kGram || E == kPoly);
    // rings of 128, 64, 128 and 144 KB
    switch (t.kind) {
        case 0: return launch_tiles<64, 2, 2, 64, 4, E>(p, t.splits, batch, st);
        case 1: return launch_tiles<64, 2, 2, 64, 2, E>(p, t.splits, batch, st);
        case 2: return launch_tiles<128, 2, 4, 32, 4, E>(p, t.splits, batch, st);
        default: return launch_tiles<192, 2, 2, 32, 3, E>(p, t.splits, batch, st);
    }
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
        return launch_small<T, 1, 2>(c, sink, s.waves, st);
    }
    return launch_small<T, 2, 1>(c, sink, s.waves, st);
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
    if (panel_shape(l.m, l.n)) {
        PanelArgs a{};
        a.XT = reinterpret_cast<half_t*>(ws + l.XT0);
        a.xplane = l.xplane;
        a.exponents = reinterpret_cast<int*>(ws + l.partial);
        a.np = l.np;
        a.panels = panels_of(l.np);
        a.m = l.m;
        a.n = l.n;
        a.tall = l.tall;
        a.ca = c.coeffs[0];
        a.cb = c.coeffs[1];
        a.cc = c.coeffs[2];
        a.eps = c.eps;
        a.sink = sink;
        char* parts[2] = {ws + l.part, ws + l.part + c.batch * panel_part_bytes(l.mp, l.np)};
        const dim3 grid(a.panels, c.batch), block(l.mp == 64 ? 512 : 1024);
        const Source from{c.m, c.momentum_out, c.beta, c.nesterov};
        a.part_out = reinterpret_cast<float*>(parts[0]);
        {
            KernelTimer timer("ns_panel_load", st);
            const bool f32 = c.m_dtype == DISCO_F32;
#define DISCO_NS(T, MT) \
    hipLaunchKernelGGL((ns_panel_load<T, MT>), grid, block, 0, st, from, c.momentum, c.momentum_out, a)
            if (l.mp == 64) {
                if (f32) DISCO_NS(float, 2);
                else DISCO_NS(bf16_t, 2);
            } else {
                if (f32) DISCO_NS(float, 4);
                else DISCO_NS(bf16_t, 4);
            }
#undef DISCO_NS
        }
        if (int rc = done("ns_panel_load")) return rc;
        for (int t = 0; t < c.steps; ++t) {
            a.raw = t == 0;
            a.last = t + 1 == c.steps;
            a.part_in = reinterpret_cast<const float*>(parts[t & 1]);
            a.part_out = reinterpret_cast<float*>(parts[(t + 1) & 1]);
            KernelTimer timer("ns_panel", st);
            if (l.mp == 64) hipLaunchKernelGGL(ns_panel<2>, grid, block, 0, st, a);
            else hipLaunchKernelGGL(ns_panel<4>, grid, block, 0, st, a);
            if (int rc = done("ns_panel")) return rc;
        }
        return DISCO_OK;
    }

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
            hipLaunchKernelGGL(ns_norm<float>, grid, dim3(1024), 0, st, src, c.momentum,
                               c.momentum_out, n, partial);
        else
            hipLaunchKernelGGL(ns_norm<bf16_t>, grid, dim3(1024), 0, st, src, c.momentum,
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
    for (int t = 0; t < c.steps; ++t) {
        const bool last = t + 1 == c.steps;
        half_t* xt = XT[t & 1];
        Product g{};
        g.part = reinterpret_cast<float*>(ws + l.part);
        Product q = g, s = g;
        g.u = g.v = X;
        g.u_plane = g.v_plane = l.xplane;
        g.K = l.np;
        g.rows_u = g.rows_v = l.mp;
        g.out = g.out_t = A;
        g.o_plane = l.aplane;
        g.ld_out = g.ld_t = l.mp;
        g.cb = kSA / (kSX * kSX);
        if (int rc = launch_product<kGram>(g, c.batch, st)) return rc;

        q.u = q.v = A;
        q.u_plane = q.v_plane = l.aplane;
        q.K = l.mp;
        q.rows_u = q.rows_v = l.mp;
        q.out = q.out_t = P;
        q.add = A;
        q.o_plane = q.add_plane = l.aplane;
        q.ld_out = q.ld_t = l.mp;
        q.ca = c.coeffs[1] * kSP / kSA;
        q.cb = c.coeffs[2] * kSP / (kSA * kSA);
        q.diagonal = c.coeffs[0] * kSP;   // a I + P: no separate a X
        if (int rc = launch_product<kPoly>(q, c.batch, st)) return rc;

        s.u = P;
        s.v = xt;
        s.u_plane = l.aplane;
        s.v_plane = s.o_plane = l.xplane;
        s.K = l.mp;
        s.rows_u = l.mp;
        s.rows_v = l.np;
        s.out = X;
        s.out_t = XT[(t + 1) & 1];
        s.ld_out = l.np;
        s.ld_t = l.mp;
        s.cb = 1.0f / kSP;
        int rc;
        if (last) {
            s.cb /= kSX;
            s.m = l.m;
            s.n = l.n;
            s.tall = l.tall;
            s.sink = sink;
            rc = launch_product<kLast>(s, c.batch, st);
        } else {
            rc = launch_product<kStep>(s, c.batch, st);
        }
        if (rc) return rc;
    }
    return DISCO_OK;
}

}  // namespace disco
