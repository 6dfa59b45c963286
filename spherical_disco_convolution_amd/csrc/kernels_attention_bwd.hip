// Gradients of the attention over points or tokens.
//
//   delta_i = go_i . o_i,  dp_ij = go_i . v_j,  ds_ij = p_ij (dp_ij - delta_i)
//   gq_i = scale sum_j ds_ij k_j,  gk_j = scale sum_i ds_ij q_i,  gv_j = sum_i p_ij go_i
// with p_ij = exp(x_ij - l_i) from the forward's l.  Two kernels, one that walks
// over the keys for tiles of rows (gq) and one that walks over the rows for tiles
// of keys (gk, gv): seven products where one kernel would do with five, but no
// sum is taken in an order that changes from run to run, and no atomics.
#include "attention_device.h"

#include <algorithm>

namespace disco {

using namespace attn;

namespace {

constexpr int kStep = 64;   // keys (gq) or rows (gk, gv) of a step

template <typename T, int DP, int NW, int NC, bool BIAS, bool FAST>
__global__ __launch_bounds__(64 * NW) void attn_bwd_q(AttnArgs a) {
    typedef Tile<T, DP> L;
    typedef typename Op<T>::Frag Frag;
    constexpr int KE = Op<T>::KE, NT = DP / 32, TR = 32 * NC * NW, KB = 32 / KE;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kStep * L::RB];
    __shared__ __attribute__((aligned(16))) float bias_s[kStep];
    const uint32_t kbase = (uint32_t)(uintptr_t)(lds_u8*)&smem[0];
    const uint32_t vbase = kbase + kStep * L::RB;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), h = lane >> 5;

    int hk, idx, seq, tile, tiles;
    if (!head_of(blockIdx.x, a.slots * a.splits, a.hkv, &hk, &idx)) return;
    const int split = idx % a.splits;
    if (!locate(a.cu_q, a.n_seq, (int)a.total_q, a.each_q, a.G, TR, idx / a.splits, &seq, &tile, &tiles)) return;
    if (a.causal) tile = tiles - 1 - tile;
    const Span sq = span_of(a.cu_q, seq, a.each_q, (int)a.total_q);
    const Span sk = span_of(a.cu_k, seq, a.each_k, (int)a.total_k);
    const int rows = sq.len * a.G, lk = sk.len, ahead = sk.len - sq.len;

    Frag qf[NC][DP / KE], gf[NC][DP / KE];
    int lim[NC];
    float lse2[NC], delta[NC];
    const int row0 = tile * TR + wave * 32 * NC;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
        int token, g;
        const int r = row0 + 32 * n + (lane & 31);
        const bool ok = r < rows;
        row_of(r, a.G, &token, &g);
        const int64_t tok = sq.first + token;
        const int head = hk * a.G + g;
        load_columns<T, DP, FAST>(qf[n], (const T*)a.q + tok * a.q_ts + (int64_t)head * a.q_hs, a.dk, ok, lane);
        load_columns<T, DP, FAST>(gf[n], (const T*)a.go + tok * a.go_ts + (int64_t)head * a.go_hs, a.dv, ok, lane);
        lim[n] = a.causal ? min(max(token + ahead + 1, 0), lk) : lk;
        // rows that see nothing have no gradient: their l is -inf
        const float lse = ok ? a.lse_in[tok * a.hq + head] : -kInf;
        lse2[n] = lse == -kInf ? kInf : lse * kLog2e;
        float d = 0.0f;
        const T* orow = (const T*)a.o + tok * a.o_ts + (int64_t)head * a.o_hs;
#pragma unroll
        for (int c = 0; c < DP / KE; ++c) {
            const u32x4 ow = load_chunk<T, FAST>(orow, (2 * c + h) * L::EPC, a.dv, ok);
            const u32x4 gw = __builtin_bit_cast(u32x4, gf[n][c]);
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    d = fmaf(__uint_as_float(ow[i] << 16), __uint_as_float(gw[i] << 16), d);
                    d = fmaf(__uint_as_float(ow[i] & 0xffff0000u), __uint_as_float(gw[i] & 0xffff0000u), d);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) d = fmaf(__uint_as_float(ow[i]), __uint_as_float(gw[i]), d);
            }
        }
        delta[n] = half_sum(d);
        if (split == 0 && h == 0 && ok) a.delta[tok * a.hq + head] = delta[n];
    }
    if (!a.gq) return;   // only delta is wanted
    int t_first, t_last, unused;
    row_of(tile * TR, a.G, &t_first, &unused);
    row_of(min(tile * TR + TR, rows) - 1, a.G, &t_last, &unused);
    const int most = a.causal ? min(max(t_last + ahead + 1, 0), lk) : lk;
    const int least = a.causal ? min(max(t_first + ahead + 1, 0), lk) : lk;
    const int all = (most + kStep - 1) / kStep;
    const int t0 = (int)((int64_t)all * split / a.splits), t1 = (int)((int64_t)all * (split + 1) / a.splits);

    const T* K = (const T*)a.k + sk.first * a.k_ts + (int64_t)hk * a.k_hs;
    const T* V = (const T*)a.v + sk.first * a.v_ts + (int64_t)hk * a.v_hs;
    const float* B = BIAS ? a.bias + sk.first : nullptr;
    const float scale2 = a.scale * kLog2e;

    floatx16 gq[NC][NT];
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int d = 0; d < NT; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) gq[n][d][e] = 0.0f;

    for (int t = t0; t < t1; ++t) {
        const int k0 = t * kStep;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kStep * L::NCH / (64 * NW); ++i) {
            const int id = tid + i * 64 * NW, row = id / L::NCH, c = id % L::NCH;
            bool ok = k0 + row < lk;
            if constexpr (BIAS) ok = ok && !(B[min(k0 + row, lk - 1)] < kLowest);
            const int64_t key = k0 + row;
            const u32x4 kw = load_chunk<T, FAST>(K + key * a.k_ts, c * L::EPC, a.dk, ok);
            const u32x4 vw = load_chunk<T, FAST>(V + key * a.v_ts, c * L::EPC, a.dv, ok);
            *(lds_u32x4*)(uintptr_t)(kbase + L::at(row, c)) = kw;
            *(lds_u32x4*)(uintptr_t)(vbase + L::at(row, c)) = vw;
        }
        if constexpr (BIAS)
            if (tid < kStep) bias_s[tid] = k0 + tid < lk ? bias2(B[k0 + tid]) : -kInf;
        __syncthreads();
        const bool cut = k0 + kStep > least;
#pragma unroll
        for (int kt = 0; kt < kStep / 32; ++kt) {
            floatx16 s[NC], dp[NC];
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int e = 0; e < 16; ++e) s[n][e] = dp[n][e] = 0.0f;
#pragma unroll
            for (int c = 0; c < DP / KE; ++c) {
                const Frag f = L::rows(kbase, 32 * kt, c, lane);
#pragma unroll
                for (int n = 0; n < NC; ++n) s[n] = Op<T>::mma(f, qf[n][c], s[n]);
            }
#pragma unroll
            for (int c = 0; c < DP / KE; ++c) {
                const Frag f = L::rows(vbase, 32 * kt, c, lane);
#pragma unroll
                for (int n = 0; n < NC; ++n) dp[n] = Op<T>::mma(f, gf[n][c], dp[n]);
            }
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int e4 = 0; e4 < 4; ++e4) {
                    const int key = 32 * kt + 8 * e4 + 4 * h;
                    floatx4 b = {0, 0, 0, 0};
                    if constexpr (BIAS) b = *(const lds_f32x4*)(uintptr_t)((uint32_t)(uintptr_t)(lds_f32*)&bias_s[0] + 4 * key);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = fmaf(s[n][4 * e4 + e], scale2, b[e] - lse2[n]);
                        if (cut && k0 + key + e >= lim[n]) x = -kInf;
                        s[n][4 * e4 + e] = exp2_fast(x) * (dp[n][4 * e4 + e] - delta[n]);
                    }
                }
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                Frag sf[NC];
#pragma unroll
                for (int n = 0; n < NC; ++n) sf[n] = Op<T>::from(s[n], b * KE / 2);
#pragma unroll
                for (int d = 0; d < NT; ++d) {
                    const Frag f = L::columns(kbase, 32 * kt + b * KE, d, lane);
#pragma unroll
                    for (int n = 0; n < NC; ++n) gq[n][d] = Op<T>::mma(f, sf[n], gq[n][d]);
                }
            }
        }
    }

#pragma unroll
    for (int n = 0; n < NC; ++n) {
        const int r = row0 + 32 * n + (lane & 31);
        if (r >= rows) continue;
        int token, g;
        row_of(r, a.G, &token, &g);
        const int64_t tok = sq.first + token;
        const int head = hk * a.G + g;
        float* part = a.part + (((int64_t)split * a.total_q + tok) * a.hq + head) * a.dk;
        T* out = (T*)a.gq + tok * a.gq_ts + (int64_t)head * a.gq_hs;
#pragma unroll
        for (int d = 0; d < NT; ++d)
#pragma unroll
            for (int e4 = 0; e4 < 4; ++e4) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = gq[n][d][4 * e4 + e] * a.scale;
                if (a.splits > 1) store4<float, FAST>(part, 32 * d + 8 * e4 + 4 * h, a.dk, v);
                else store4<T, FAST>(out, 32 * d + 8 * e4 + 4 * h, a.dk, v);
            }
    }
}

// A workgroup has 32 NC keys a wave and walks over the rows of all heads that
// read its key head.
template <typename T, int DP, int NW, int NC, bool FAST>
__global__ __launch_bounds__(64 * NW) void attn_bwd_kv(AttnArgs a) {
    typedef Tile<T, DP> L;
    typedef typename Op<T>::Frag Frag;
    constexpr int KE = Op<T>::KE, NT = DP / 32, TK = 32 * NC * NW, KB = 32 / KE;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kStep * L::RB];
    __shared__ __attribute__((aligned(16))) float lse_s[kStep], delta_s[kStep];
    __shared__ __attribute__((aligned(16))) int32_t lim_s[kStep];
    const uint32_t qbase = (uint32_t)(uintptr_t)(lds_u8*)&smem[0];
    const uint32_t gbase = qbase + kStep * L::RB;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), h = lane >> 5;

    int hk, idx, seq, tile, tiles;
    if (!head_of(blockIdx.x, a.slots * a.splits, a.hkv, &hk, &idx)) return;
    const int split = idx % a.splits;
    if (!locate(a.cu_k, a.n_seq, (int)a.total_k, a.each_k, 1, TK, idx / a.splits, &seq, &tile, &tiles)) return;
    const Span sq = span_of(a.cu_q, seq, a.each_q, (int)a.total_q);
    const Span sk = span_of(a.cu_k, seq, a.each_k, (int)a.total_k);
    const int rows = sq.len * a.G, lk = sk.len, ahead = sk.len - sq.len;

    Frag kf[NC][DP / KE], vf[NC][DP / KE];
    float bias[NC];
    const int key0 = tile * TK + wave * 32 * NC;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
        const int key = key0 + 32 * n + (lane & 31);
        bool ok = key < lk;
        const int64_t tok = sk.first + key;
        bias[n] = 0.0f;
        if (a.bias && ok) bias[n] = bias2(a.bias[tok]);
        ok = ok && bias[n] != -kInf;
        if (!ok) bias[n] = -kInf;
        load_columns<T, DP, FAST>(kf[n], (const T*)a.k + tok * a.k_ts + (int64_t)hk * a.k_hs, a.dk, ok, lane);
        load_columns<T, DP, FAST>(vf[n], (const T*)a.v + tok * a.v_ts + (int64_t)hk * a.v_hs, a.dv, ok, lane);
    }
    // the first row that sees the tile's first key, and the rows from which all see all of it
    const int r_first = a.causal ? min(max(tile * TK - ahead, 0), sq.len) * a.G : 0;
    const int r_all = a.causal ? min(max(min(tile * TK + TK, lk) - 1 - ahead, 0), sq.len) * a.G : 0;
    const int b0 = r_first / kStep, all = (rows + kStep - 1) / kStep - b0;
    const int t0 = b0 + (int)((int64_t)all * split / a.splits), t1 = b0 + (int)((int64_t)all * (split + 1) / a.splits);
    const float scale2 = a.scale * kLog2e;

    floatx16 gk[NC][NT], gv[NC][NT];
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int d = 0; d < NT; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) gk[n][d][e] = gv[n][d][e] = 0.0f;

    for (int t = t0; t < t1; ++t) {
        const int r0 = t * kStep;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kStep * L::NCH / (64 * NW); ++i) {
            const int id = tid + i * 64 * NW, row = id / L::NCH, c = id % L::NCH;
            int token, g;
            row_of(r0 + row, a.G, &token, &g);
            const int64_t tok = sq.first + token, head = hk * a.G + g;
            const bool ok = r0 + row < rows;
            const u32x4 qw = load_chunk<T, FAST>((const T*)a.q + tok * a.q_ts + head * a.q_hs, c * L::EPC, a.dk, ok);
            const u32x4 gw = load_chunk<T, FAST>((const T*)a.go + tok * a.go_ts + head * a.go_hs, c * L::EPC, a.dv, ok);
            *(lds_u32x4*)(uintptr_t)(qbase + L::at(row, c)) = qw;
            *(lds_u32x4*)(uintptr_t)(gbase + L::at(row, c)) = gw;
        }
        if (tid < kStep) {
            int token, g;
            row_of(r0 + tid, a.G, &token, &g);
            const bool ok = r0 + tid < rows;
            const int64_t cell = (sq.first + token) * a.hq + hk * a.G + g;
            const float lse = ok ? a.lse_in[cell] : -kInf;
            lse_s[tid] = lse == -kInf ? kInf : lse * kLog2e;
            delta_s[tid] = ok ? a.delta[cell] : 0.0f;
            lim_s[tid] = a.causal ? token + ahead : 0x7fffffff;
        }
        __syncthreads();
        const bool cut = r0 < r_all;
#pragma unroll
        for (int rt = 0; rt < kStep / 32; ++rt) {
            floatx16 s[NC], dp[NC];
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int e = 0; e < 16; ++e) s[n][e] = dp[n][e] = 0.0f;
#pragma unroll
            for (int c = 0; c < DP / KE; ++c) {
                const Frag f = L::rows(qbase, 32 * rt, c, lane);
#pragma unroll
                for (int n = 0; n < NC; ++n) s[n] = Op<T>::mma(f, kf[n][c], s[n]);
            }
#pragma unroll
            for (int c = 0; c < DP / KE; ++c) {
                const Frag f = L::rows(gbase, 32 * rt, c, lane);
#pragma unroll
                for (int n = 0; n < NC; ++n) dp[n] = Op<T>::mma(f, vf[n][c], dp[n]);
            }
#pragma unroll
            for (int e4 = 0; e4 < 4; ++e4) {
                const int row = 32 * rt + 8 * e4 + 4 * h;
                const floatx4 l4 = *(const lds_f32x4*)(uintptr_t)((uint32_t)(uintptr_t)(lds_f32*)&lse_s[0] + 4 * row);
                const floatx4 d4 = *(const lds_f32x4*)(uintptr_t)((uint32_t)(uintptr_t)(lds_f32*)&delta_s[0] + 4 * row);
#pragma unroll
                for (int n = 0; n < NC; ++n) {
                    const int key = key0 + 32 * n + (lane & 31);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = fmaf(s[n][4 * e4 + e], scale2, bias[n] - l4[e]);
                        if (cut && key > lim_s[row + e]) x = -kInf;
                        const float p = exp2_fast(x);
                        s[n][4 * e4 + e] = p;
                        dp[n][4 * e4 + e] = p * (dp[n][4 * e4 + e] - d4[e]);
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                Frag pf[NC], sf[NC];
#pragma unroll
                for (int n = 0; n < NC; ++n) {
                    pf[n] = Op<T>::from(s[n], b * KE / 2);
                    sf[n] = Op<T>::from(dp[n], b * KE / 2);
                }
#pragma unroll
                for (int d = 0; d < NT; ++d) {
                    const Frag f = L::columns(gbase, 32 * rt + b * KE, d, lane);
#pragma unroll
                    for (int n = 0; n < NC; ++n) gv[n][d] = Op<T>::mma(f, pf[n], gv[n][d]);
                    const Frag e = L::columns(qbase, 32 * rt + b * KE, d, lane);
#pragma unroll
                    for (int n = 0; n < NC; ++n) gk[n][d] = Op<T>::mma(e, sf[n], gk[n][d]);
                }
            }
        }
    }

#pragma unroll
    for (int n = 0; n < NC; ++n) {
        const int key = key0 + 32 * n + (lane & 31);
        if (key >= lk) continue;
        const int64_t tok = sk.first + key;
        const int64_t cell = ((int64_t)split * a.total_k + tok) * a.hkv + hk;
        float* pk = a.part + cell * a.dk;
        float* pv = a.part2 + cell * a.dv;
        T* ok = (T*)a.gk + tok * a.gk_ts + (int64_t)hk * a.gk_hs;
        T* ov = (T*)a.gv + tok * a.gv_ts + (int64_t)hk * a.gv_hs;
#pragma unroll
        for (int d = 0; d < NT; ++d)
#pragma unroll
            for (int e4 = 0; e4 < 4; ++e4) {
                const int d0 = 32 * d + 8 * e4 + 4 * h;
                float x[4], y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = gk[n][d][4 * e4 + e] * a.scale;
                    y[e] = gv[n][d][4 * e4 + e];
                }
                if (a.splits > 1) {
                    store4<float, FAST>(pk, d0, a.dk, x);
                    store4<float, FAST>(pv, d0, a.dv, y);
                } else {
                    store4<T, FAST>(ok, d0, a.dk, x);
                    store4<T, FAST>(ov, d0, a.dv, y);
                }
            }
    }
}

// Sum of the parts of [tokens, heads, d], a wave a row; tokens of no sequence
// stay as they are.
template <typename T>
__global__ __launch_bounds__(256) void attn_sum(const float* __restrict__ part, T* __restrict__ out, int64_t ts, int64_t hs,
                                                int64_t total, int heads, int d, int splits, const int32_t* cu, int n_seq) {
    const int lane = threadIdx.x & 63;
    const int64_t cell = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t tok = cell / heads;
    const int head = (int)(cell - tok * heads);
    if (tok >= total) return;
    if (cu && (tok < cu[0] || tok >= cu[n_seq])) return;
    for (int i = lane; i < d; i += 64) {
        float v = 0.0f;
        for (int s = 0; s < splits; ++s) v += part[(s * total * heads + cell) * d + i];
        store_f(out + tok * ts + (int64_t)head * hs, i, v);
    }
}

template <typename T>
void sum_parts(const float* part, void* out, int64_t ts, int64_t hs, int64_t total, int heads, int d, int splits,
               const int32_t* cu, int n_seq, hipStream_t st) {
    KernelTimer timer("attn_sum", st);
    attn_sum<T><<<(unsigned)((total * heads + 3) / 4), 256, 0, st>>>(part, (T*)out, ts, hs, total, heads, d, splits, cu, n_seq);
}

template <typename T, int DP, bool FAST>
int bwd_go(AttnArgs a, const AttnPlan& pq, const AttnPlan& pk, hipStream_t st) {
    constexpr int NW = 4;
    a.slots = (int)tile_slots(a.cu_q != nullptr, a.total_q, a.n_seq, a.G, 32 * NW);
    a.splits = a.gq ? pq.splits : 1;
    if (a.total_q > 0) {   // delta, which gk and gv need too
        KernelTimer timer("attn_bwd_q", st);
        const unsigned grid = (unsigned)grid_size((int64_t)a.slots * a.splits, a.hkv);
        if (a.bias) attn_bwd_q<T, DP, NW, 1, true, FAST><<<grid, 64 * NW, 0, st>>>(a);
        else attn_bwd_q<T, DP, NW, 1, false, FAST><<<grid, 64 * NW, 0, st>>>(a);
    }
    if (a.splits > 1)
        sum_parts<T>(a.part, a.gq, a.gq_ts, a.gq_hs, a.total_q, a.hq, a.dk, a.splits, a.cu_q, a.n_seq, st);
    if (a.gk && a.total_k > 0) {
        a.slots = (int)tile_slots(a.cu_k != nullptr, a.total_k, a.n_seq, 1, 32 * NW);
        a.splits = pk.splits;
        a.part2 = a.part + (size_t)a.splits * a.total_k * a.hkv * a.dk;
        const unsigned grid = (unsigned)grid_size((int64_t)a.slots * a.splits, a.hkv);
        {
            KernelTimer timer("attn_bwd_kv", st);
            attn_bwd_kv<T, DP, NW, 1, FAST><<<grid, 64 * NW, 0, st>>>(a);
        }
        if (a.splits > 1) {
            sum_parts<T>(a.part, a.gk, a.gk_ts, a.gk_hs, a.total_k, a.hkv, a.dk, a.splits, a.cu_k, a.n_seq, st);
            sum_parts<T>(a.part2, a.gv, a.gv_ts, a.gv_hs, a.total_k, a.hkv, a.dv, a.splits, a.cu_k, a.n_seq, st);
        }
    }
    return attn_launched("attention_bwd");
}

template <typename T>
int bwd_typed(const AttnArgs& a, hipStream_t st) {
    const AttnPlan pq = attn_plan_bwd_q(a), pk = attn_plan_bwd_kv(a);
    if (!pq.fast) return bwd_go<T, 128, false>(a, pq, pk, st);
    const int d = std::max(a.dk, a.dv);
    if (d <= 32) return bwd_go<T, 32, true>(a, pq, pk, st);
    if (d <= 64) return bwd_go<T, 64, true>(a, pq, pk, st);
    return bwd_go<T, 128, true>(a, pq, pk, st);
}

}  // namespace

int launch_attention_bwd(const AttnArgs& a, void* stream) {
    hipStream_t st = static_cast<hipStream_t>(stream);
    return a.dtype == DISCO_F32 ? bwd_typed<float>(a, st) : bwd_typed<bf16_t>(a, st);
}

}  // namespace disco
