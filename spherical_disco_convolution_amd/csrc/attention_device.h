// Device parts shared by the attention kernels, forward and backward.
//
// For a sequence of Lq queries and Lk keys, query head h reading key head
// h / G (G = hq / hkv):
//   x_ij = scale q_i . k_j + b_j        (-inf where j is left out)
//   l_i = log sum_j exp x_ij,  p_ij = exp(x_ij - l_i),  o_i = sum_j p_ij v_j
// The G heads of a group are rows of one tile: row r of a sequence and key head
// is query r / G of head r % G, so their keys and values are read once, and the
// sums over a group in the gradients of k and v need no second pass.
//
// Every product runs on the matrix cores as (rows from LDS) x (columns in
// registers).  The 32 x 32 result leaves lane L with column L % 32 and rows
// 8 (e / 4) + 4 (L / 32) + e % 4, e = 0..15: eight (bf16) or four (float32)
// consecutive e are themselves an operand of the next product, whose other
// operand is read with the same order of the summed rows.  So scores, weights
// and their gradients never leave registers.
#pragma once

#include <hip/hip_runtime.h>

#include "disco_internal.h"
#include "kernels_common.h"

namespace disco {
namespace attn {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int16_t v4i16_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) float lds_f32;
typedef __attribute__((address_space(3))) int32_t lds_i32;
typedef __attribute__((address_space(3))) floatx4 lds_f32x4;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) v4i16_t lds_v4i16;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kInf = __builtin_inff();
// biases below this leave a key out, as -inf does: masks made of a type's
// lowest value, which no sum could tell from each other
constexpr float kLowest = -1e30f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    bf16x2_t v;
    v[0] = (__bf16)a;
    v[1] = (__bf16)b;
    return __builtin_bit_cast(uint32_t, v);
}

// The value of lane ^ 32 joined with this lane's
__device__ __forceinline__ float other_half(float x, float* mine) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    *mine = __uint_as_float(r[0]);
    return __uint_as_float(r[1]);
}
__device__ __forceinline__ float half_max(float x) {
    float a;
    const float b = other_half(x, &a);
    return fmaxf(a, b);
}
__device__ __forceinline__ float half_sum(float x) {
    float a;
    const float b = other_half(x, &a);
    return a + b;
}

// One operand of a product: 16 bytes a lane, KE summed elements in a wave's
// fragment (lane L: row or column L % 32, elements (L / 32) KE/2 .. + KE/2 - 1).
template <typename T>
struct Op;

template <>
struct Op<bf16_t> {
    typedef bf16x8_t Frag;
    static constexpr int KE = 16;
    static __device__ __forceinline__ floatx16 mma(Frag a, Frag b, floatx16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    // elements e0 .. e0 + 7 of a product's result, rounded to bfloat16: the
    // weights are at most 1 (2^24 while a maximum lags); this costs each at most 2^-8 of itself
    static __device__ __forceinline__ Frag from(const floatx16& s, int e0) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack_bf16(s[e0 + 2 * i], s[e0 + 2 * i + 1]);
        return __builtin_bit_cast(Frag, w);
    }
    // what that rounding left behind
    static __device__ __forceinline__ Frag rest(const floatx16& s, int e0, Frag rounded) {
        const u32x4 r = __builtin_bit_cast(u32x4, rounded);
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = pack_bf16(s[e0 + 2 * i] - __uint_as_float(r[i] << 16), s[e0 + 2 * i + 1] - __uint_as_float(r[i] & 0xffff0000u));
        return __builtin_bit_cast(Frag, w);
    }
};

template <>
struct Op<float> {
    typedef floatx4 Frag;
    static constexpr int KE = 8;
    static __device__ __forceinline__ floatx16 mma(Frag a, Frag b, floatx16 c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ Frag from(const floatx16& s, int e0) {
        Frag f;
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = s[e0 + i];
        return f;
    }
};

// A tile of rows in LDS: RB bytes a row, 16-byte chunks at chunk ^ turn(row).
// The turn spreads over the banks both the 16-byte reads of 16 rows (one chunk)
// and the transposing reads of four rows (four chunks).
template <typename T, int DP>
struct Tile {
    static constexpr int EPC = 16 / (int)sizeof(T);     // elements of a chunk
    static constexpr int USED = DP / EPC;               // chunks that products read
    static constexpr int NCH = USED <= 4 ? 4 : USED <= 8 ? 8 : USED <= 16 ? 16 : 32;
    static constexpr int RB = 16 * NCH;
    static __device__ __forceinline__ int turn(int row) {
        // float32 products are too slow for banks to matter: whole groups of eight
        // chunks change places, so that few addresses need registers
        if constexpr (sizeof(T) == 4) return NCH == 8 ? 0 : ((((row & 3) ^ ((row >> 2) & 1)) << 3) & (NCH - 1));
        if constexpr (NCH == 4) return (row >> 2) & 3;
        if constexpr (NCH == 8) return (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
        return ((row & 3) << 2) | ((row >> 2) & 3);
    }
    static __device__ __forceinline__ uint32_t at(int row, int chunk) {
        return (uint32_t)(row * RB + ((chunk ^ turn(row)) << 4));
    }
};

// Where a lane reads the operands of a tile whose place in LDS is known when
// compiled: addresses are taken once, what changes goes into the instructions.
// rows(): rows 32 k .. + 31 of the tile `off` bytes from base, summed elements of
// chunks 2 c and 2 c + 1.  columns(): columns 32 d .. + 31, summed over rows KE b ..
// in the order of a product's result.
template <typename T, int DP>
struct Reader;

template <int DP>
struct Reader<bf16_t, DP> {
    typedef Tile<bf16_t, DP> L;
    typedef bf16x8_t Frag;
    static constexpr int NT = DP / 32;
    uint32_t row[DP / 16], col[NT][2];
    __device__ __forceinline__ void init(uint32_t base, int lane) {
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) row[c] = base + L::at(lane & 31, 2 * c + (lane >> 5));
        const int s = lane & 15, r = 4 * (lane >> 5) + (s >> 2);
#pragma unroll
        for (int d = 0; d < NT; ++d)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int e = 32 * d + 16 * ((lane >> 4) & 1) + 4 * (s & 3);
                col[d][j] = base + L::at(r + 8 * j, e >> 3) + (e & 7) * 2;
            }
    }
    __device__ __forceinline__ Frag rows(uint32_t off, int k, int c) const {
        return __builtin_bit_cast(Frag, *(const lds_u32x4*)(uintptr_t)(row[c] + (off + k * 32 * L::RB)));
    }
    __device__ __forceinline__ Frag columns(uint32_t off, int b, int d) const {
        const uint32_t o = off + b * 16 * L::RB;
        const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(uintptr_t)(col[d][0] + o));
        const v4i16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(uintptr_t)(col[d][1] + o));
        return __builtin_bit_cast(Frag, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

template <int DP>
struct Reader<float, DP> {
    typedef Tile<float, DP> L;
    typedef floatx4 Frag;
    static constexpr int NT = DP / 32;
    uint32_t row[NT];   // of eight chunks each
    uint32_t col[2];    // where the lane's half of the rows moves a group of chunks up, or down
    __device__ __forceinline__ void init(uint32_t base, int lane) {
        const int h = lane >> 5;
#pragma unroll
        for (int g = 0; g < NT; ++g) row[g] = base + L::at(lane & 31, 8 * g + h);
        const uint32_t at = base + 4 * h * L::RB + (lane & 31) * 4;
        col[0] = at + (NT > 1 ? 128 * h : 0);
        col[1] = at - (NT > 1 ? 128 * h : 0);
    }
    __device__ __forceinline__ Frag rows(uint32_t off, int k, int c) const {
        return *(const lds_f32x4*)(uintptr_t)(row[c / 4] + (off + k * 32 * L::RB + (c % 4) * 32));
    }
    __device__ __forceinline__ Frag columns(uint32_t off, int b, int d) const {
        Frag f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // row 8 b + 4 h + i has group d at d ^ i ^ h
            const int g = (d ^ i) & (NT - 1);
            f[i] = *(const lds_f32*)(uintptr_t)(col[g & 1] + (off + (8 * b + i) * L::RB + 128 * g));
        }
        return f;
    }
};

// Asks the scheduler to lay out what stands before it in this order: AHEAD reads
// of LDS, then M times a matrix instruction with the reads and the vector
// instructions that fit beside it.
template <int M, int AHEAD, int READS, int VALU, int TRANS>
__device__ __forceinline__ void mix() {
    __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
#pragma unroll
    for (int i = 0; i < M; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);
        __builtin_amdgcn_sched_group_barrier(0x400, TRANS, 0);
    }
}

// A value of a row (a key's bias, say) as the first summand of its products: one
// of its own, of the value in three bfloat16 parts (24 bits) with ones.  -inf stays
// -inf.  The upper half of the lanes gives zeros.
template <typename T>
struct Addend;

template <>
struct Addend<bf16_t> {
    typedef uint32_t Word __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ Word pack(float b) {
        const bf16_t hi = f32_to_bf16(b);
        const float r = b == -kInf ? 0.0f : b - bf16_to_f32(hi);
        const bf16_t mid = f32_to_bf16(r);
        return Word{hi | (uint32_t)mid << 16, f32_to_bf16(r - bf16_to_f32(mid))};
    }
    static __device__ __forceinline__ floatx16 spread(Word w) {
        const bf16x8_t a = __builtin_bit_cast(bf16x8_t, u32x4{w[0], w[1], 0, 0});
        const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, u32x4{0x3f803f80u, 0x3f80u, 0, 0});
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, ones, floatx16{}, 0, 0, 0);
    }
};

template <>
struct Addend<float> {
    typedef float Word;
    static __device__ __forceinline__ Word pack(float b) { return b; }
    static __device__ __forceinline__ floatx16 spread(Word w) {
        return __builtin_amdgcn_mfma_f32_32x32x2f32(w, 1.0f, floatx16{}, 0, 0, 0);
    }
};

// 16 bytes of a row from element d0, zeros past D.  FAST: D, strides and
// addresses are multiples of 16 bytes.
template <typename T, bool FAST>
__device__ __forceinline__ u32x4 load_chunk(const T* row, int d0, int D, bool valid) {
    u32x4 w = {0, 0, 0, 0};
    if (!valid || d0 >= D) return w;
    if constexpr (FAST) return *reinterpret_cast<const u32x4*>(row + d0);
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t v = d0 + i < D ? (uint32_t)row[d0 + i] : 0u;
            w[i / 2] |= v << (16 * (i & 1));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = d0 + i < D ? __float_as_uint(row[d0 + i]) : 0u;
    }
    return w;
}

// A row that a lane keeps in registers, as an operand
template <typename T, int DP, bool FAST>
__device__ __forceinline__ void load_columns(typename Op<T>::Frag* f, const T* row, int D, bool valid, int lane) {
    constexpr int EPC = 16 / (int)sizeof(T);
#pragma unroll
    for (int c = 0; c < DP / Op<T>::KE; ++c)
        f[c] = __builtin_bit_cast(typename Op<T>::Frag,
                                  load_chunk<T, FAST>(row, (2 * c + (lane >> 5)) * EPC, D, valid));
}

// Four elements d0 .. d0 + 3 of a row, past D left alone
template <typename T, bool FAST>
__device__ __forceinline__ void store4(T* row, int d0, int D, const float* v) {
    if (d0 >= D) return;
    if constexpr (FAST) {
        if constexpr (sizeof(T) == 2) {
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
            *reinterpret_cast<u32x2*>(row + d0) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        } else {
            *reinterpret_cast<floatx4*>(row + d0) = floatx4{v[0], v[1], v[2], v[3]};
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (d0 + i < D) store_f(row, d0 + i, v[i]);
    }
}

// ---------------------------------------------------------------------------
// Tiles from global memory straight into LDS
// ---------------------------------------------------------------------------
constexpr uint32_t kNowhere = 0x80000000u;   // past every buffer: the copy writes zeros

// 16 bytes a lane from base + off (zeros for kNowhere) to LDS at + 16 lane; no
// registers are written, and completion counts as a vector memory operation.  The
// compiler does not see into the block: a scalar register written by a vector
// instruction (readfirstlane of the descriptor, a spilled one read back) needs five
// wait states before a memory instruction reads it, which the s_nop gives.
// off reaches 2^31 bytes: the caller checks that a tile's rows lie that near.
__device__ __forceinline__ void copy16(u32x4 buffer, uint32_t off, uint32_t at) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 :
                 : "v"(off), "s"(buffer), "s"(__builtin_amdgcn_readfirstlane(at))
                 : "memory", "m0");
}

// 4 bytes a lane in the same way
__device__ __forceinline__ void copy4(u32x4 buffer, uint32_t off, uint32_t at) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tbuffer_load_dword %0, %1, 0 offen lds"
                 :
                 : "v"(off), "s"(buffer), "s"(__builtin_amdgcn_readfirstlane(at))
                 : "memory", "m0");
}

__device__ __forceinline__ u32x4 buffer_of(const void* p) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    u32x4 b;
    b[0] = __builtin_amdgcn_readfirstlane((uint32_t)a);
    b[1] = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
    b[2] = 0x7fffffffu;   // bytes
    b[3] = 0x00027000u;   // raw, 32-bit elements
    return b;
}

// All of the workgroup's reads and writes of LDS so far are done, and its copies
// but for the last N of each wave
template <int N = 0>
__device__ __forceinline__ void all_arrived() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// A tile of R rows, NW waves: instruction j of a wave moves 1 KiB of it, and its
// rows lie R / N further on than those of instruction j - 1
template <typename T, int DP, int R, int NW>
struct Copy {
    typedef Tile<T, DP> L;
    static constexpr int ALL = R * L::RB / 1024, N = ALL < NW ? 1 : ALL / NW;
    static_assert(ALL * 1024 == R * L::RB && (ALL < NW || N * NW == ALL) && R <= 64, "whole instructions");
    // a small tile leaves waves without a share
    static __device__ __forceinline__ bool shares(int wave) { return ALL >= NW || wave < ALL; }
    int row;             // of instruction 0
    __device__ __forceinline__ void init(int wave, int lane) { row = (wave * 64 + lane) / L::NCH; }
    // offsets of rows ts elements apart, d elements long
    __device__ __forceinline__ void offsets(uint32_t* off, int64_t ts, int d, int lane) const {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int r = row + j * (R / N), src = ((lane % L::NCH) ^ L::turn(r)) * L::EPC;
            off[j] = src < d ? (uint32_t)((r * ts + src) * (int64_t)sizeof(T)) : kNowhere;
        }
    }
    // rows whose bit in `out` is set become zeros
    __device__ __forceinline__ void start(const T* p, const uint32_t* off, uint32_t at, uint64_t out, int wave) const {
        if (!shares(wave)) return;
        const u32x4 b = buffer_of(p);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            uint32_t drop;   // all ones if this lane's row is left out
            if constexpr (R <= 32 || N > 1) drop = (uint32_t)__builtin_amdgcn_sbfe((int)(uint32_t)(out >> (j * (R / N))), row, 1);
            else drop = (out >> row) & 1 ? ~0u : 0u;
            copy16(b, off[j] | (drop & kNowhere), at + (uint32_t)(j * NW + wave) * 1024u);
        }
    }
};

// Whether elements from e on of a head of d take part.  float32 products are worth
// skipping; bfloat16 ones are not worth a branch between them.
template <typename T>
__device__ __forceinline__ bool worth(int e, int d) {
    return sizeof(T) == 2 || e < d;
}

// bits n .. 63
__device__ __forceinline__ uint64_t from_bit(int n) { return n >= 64 ? 0 : ~(uint64_t)0 << max(n, 0); }

// ---------------------------------------------------------------------------
// Which sequence, head and part a workgroup works on
// ---------------------------------------------------------------------------
struct Span {
    int64_t first;   // of the packed tokens
    int len;
};

// Boundaries out of order or out of range are cut to what the tensors hold.
// Without boundaries every sequence has `each` tokens.
__device__ __forceinline__ Span span_of(const int32_t* cu, int s, int each, int total) {
    if (cu == nullptr) return {(int64_t)s * each, each};
    const int a = min(max(uniform(cu[s]), 0), total), b = min(max(uniform(cu[s + 1]), a), total);
    return {a, b - a};
}

// Tiles of T rows (a power of two), `per` rows a token.  Without boundaries the
// sequences have equal counts.  With them first(s) per / T + s tiles lie before
// sequence s, which leaves every sequence the tiles it needs and at most one that
// it does not: the launch needs no list and no lengths.  Tokens times heads stay
// below 2^30 - 4096.
inline int64_t tile_slots(bool packed, int64_t total, int n_seq, int per, int T) {
    if (!packed) return n_seq * ((total / n_seq * per + T - 1) / T);
    return total * per / T + n_seq;
}

// Up to 64 sequences each workgroup counts the tiles before its own, a sequence a
// lane, and those too many stand behind the last.  More are searched with the tiles
// too many between the others, in groups of eight that are turned: at even distances
// they would all meet the same compute units (256 sequences of 128 tokens, 8 heads
// of 64: not turned 63 us, turned 41, counted 48, a dense batch 35).
//
// GROWS, SHRINKS: a causal call's later tiles have more steps, or fewer.  Those with
// the most go first, of all sequences: workgroups are dealt to the groups of a die's
// compute units in turn, whatever room these have, and sequence by sequence the same
// group would get the longest of each (gk and gv of 16 sequences of 1024 tokens, 12
// heads of 128 over 4: sequence by sequence 301 us, longest first 204).  Tiles of
// equal steps stay together, for the L2 cache.
enum Order { GROWS, SHRINKS };

__device__ __forceinline__ int wave_sum(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xf, 0xf, true);    // lane ^ 1
    v += __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xf, 0xf, true);    // lane ^ 2
    v += __builtin_amdgcn_update_dpp(0, v, 0x141, 0xf, 0xf, true);   // the other four of eight
    v += __builtin_amdgcn_update_dpp(0, v, 0x140, 0xf, 0xf, true);   // the other eight of sixteen
    return __builtin_amdgcn_readlane(v, 0) + __builtin_amdgcn_readlane(v, 16) + __builtin_amdgcn_readlane(v, 32) +
           __builtin_amdgcn_readlane(v, 48);
}

template <Order O>
__device__ __forceinline__ bool locate(bool causal, const int32_t* cu, int n_seq, int total, int each, int per, int T, int slot, int slots,
                                       int* seq, int* tile, int* tiles) {
    if (cu == nullptr) {
        const int nt = (each * per + T - 1) / T;
        *tiles = nt;
        if (n_seq == 1) {
            *seq = 0;
            *tile = slot;
        } else if (!causal) {
            *seq = slot / nt;
            *tile = slot - *seq * nt;
        } else {
            *tile = slot / n_seq;
            *seq = slot - *tile * n_seq;
        }
        if (O == GROWS && causal) *tile = nt - 1 - *tile;
        return *seq < n_seq && *tile >= 0 && *tile < nt;
    }
    const int lane = threadIdx.x & 63;
    if (n_seq <= 64) {
        int n = 0;
        if (lane < n_seq) {
            const int a = min(max(cu[lane], 0), total), b = min(max(cu[lane + 1], a), total);
            n = ((b - a) * per + T - 1) / T;
        }
        if (causal) {
            // a tile's rank: how many of its sequence have as many steps or fewer.  The
            // highest rank v that leaves more than `slot` tiles of v or above
            int v = 0, above = 0;
            for (int bit = 1 << 25; bit; bit >>= 1) {
                if (!__any(n >= v + bit)) continue;
                const int c = wave_sum(max(n - (v + bit) + 1, 0));
                if (c > slot) v += bit;
                else above = c;
            }
            if (v == 0) return false;
            const uint64_t with = __ballot(n >= v);
            const uint64_t here = __ballot(n >= v && __popcll(with & (((uint64_t)1 << lane) - 1)) == slot - above);
            if (!here) return false;   // boundaries out of order
            const int w = __builtin_ctzll(here);
            *seq = w;
            *tiles = __builtin_amdgcn_readlane(n, w);
            *tile = O == GROWS ? v - 1 : *tiles - v;
            return true;
        }
        int sum = n;   // of the lanes up to this one
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int below = __shfl_up(sum, d, 64);
            if (lane >= d) sum += below;
        }
        const uint64_t here = __ballot(slot < sum);
        if (!here) return false;
        const int w = __builtin_ctzll(here);
        *seq = w;
        *tiles = __builtin_amdgcn_readlane(n, w);
        *tile = slot - (__builtin_amdgcn_readlane(sum, w) - *tiles);
        return *tile >= 0 && *tile < *tiles;   // boundaries out of order
    }
    if (slot < (slots & ~7)) slot = (slot & ~7) | ((slot + (((uint32_t)slot >> 3) * 0x9E3779B1u >> 29)) & 7);
    // the lanes look at 64 sequences at a time: first(lo) <= slot < first(hi), if the
    // boundaries are in order
    auto first = [&](int at) { return min(max(at, 0), total) * per / T; };
    int lo = 0, hi = n_seq;
    while (hi - lo > 1) {
        const int each_lane = (hi - lo + 63) >> 6, s = min(lo + lane * each_lane, hi - 1);
        const uint64_t before = __ballot(lane == 0 || (lo + lane * each_lane < hi && first(cu[s]) + s <= slot));
        const int n = before == ~(uint64_t)0 ? 64 : __builtin_ctzll(~before);
        lo += (n - 1) * each_lane;
        hi = min(hi, lo + each_lane);
    }
    const Span sp = span_of(cu, lo, 0, total);
    *seq = lo;
    *tile = slot - first(uniform(cu[lo])) - lo;
    *tiles = (sp.len * per + T - 1) / T;
    if (*tile < 0 || *tile >= *tiles) return false;
    if (O == GROWS && causal) *tile = *tiles - 1 - *tile;
    return true;
}

// Workgroups go round the eight dies by their index; each die gets whole key
// heads (or an even share of one), so that its L2 holds their keys and values.
__host__ __device__ inline int64_t grid_size(int64_t per_head, int hkv) {
    if (hkv < 8 && 8 % hkv == 0) {
        const int share = 8 / hkv;
        return (per_head + share - 1) / share * 8;
    }
    return per_head * hkv;
}

__device__ __forceinline__ bool head_of(int id, int per_head, int hkv, bool causal, int* head, int* idx) {
    if (hkv % 8 == 0) {
        const int j = id >> 3;
        if (causal) {   // the longest tiles of all heads first
            *idx = j / (hkv >> 3);
            *head = (id & 7) + 8 * (j - *idx * (hkv >> 3));
            return true;
        }
        *head = (id & 7) + 8 * (j / per_head);
        *idx = j % per_head;
        return true;
    }
    if (8 % hkv == 0) {
        const int share = 8 / hkv, x = id & 7;
        *head = x % hkv;
        const int j = id >> 3, y = x / hkv;   // there and back: tiles of falling sizes are shared evenly
        *idx = j * share + (j & 1 ? share - 1 - y : y);
        return *idx < per_head;
    }
    *head = id % hkv;
    *idx = id / hkv;
    return true;
}

// Row r of a sequence's tile rows: token r / G, head r % G
__device__ __forceinline__ void row_of(int r, int G, int* token, int* head) {
    *token = G == 1 ? r : r / G;
    *head = r - *token * G;
}

// What the exponents of a row are taken from, in units of log 2: weights are
// exp2(fma(x - raw, scale2, -two)).  `two` is m * scale2 rounded, whose error all of a
// row's weights share, 2^-4 at most below kFarTwo.  Above, where the error passes the
// range of an exponential (2^9 at a bias of -1e10), m itself is subtracted: the
// largest score's exponent is then exactly 0.
constexpr float kFarTwo = 1048576.0f;
struct Reference {
    float raw, two;
};
__device__ __forceinline__ Reference reference_of(float m, float scale2, float far) {   // far: kFarTwo / scale2
    if (fabsf(m) < far) return {0.0f, m * scale2};
    return {m == -kInf ? 0.0f : m, 0.0f};
}
// what weights under `from` are multiplied with to stand under `to`
__device__ __forceinline__ float change_of(Reference from, Reference to, float scale2) {
    return exp2_fast(fmaf(from.raw - to.raw, scale2, from.two - to.two));
}
// the logarithm of a sum of weights
__device__ __forceinline__ float log_of(Reference r, float scale, float sum) {
    return sum == 0.0f ? -kInf : fmaf(r.raw, scale, r.two * kLn2 + logf(sum));
}

// Rows whose l has lost what a gradient's weights exp(x - l) need: its rounding alone is
// 2^-9 of each from here on, and at -1e9 (every key of the row behind such a mask) more
// than the weights' range.  Gradients take the maximum and the sum of these rows' scores
// anew.
constexpr float kFarLse = 65536.0f * kLn2;
__device__ __forceinline__ bool lse_is_far(float lse) { return fabsf(lse) >= kFarLse && fabsf(lse) < kInf; }

__device__ __forceinline__ float bias2(float b) {   // in units of log 2
    return b < kLowest ? -kInf : b * kLog2e;
}

}  // namespace attn
}  // namespace disco
