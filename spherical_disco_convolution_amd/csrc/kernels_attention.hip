// Attention over points or tokens, forward.
#include "attention_device.h"

#include <algorithm>

namespace disco {

using namespace attn;

namespace {

constexpr int kKeys = 64;   // keys of a tile

// A workgroup of NW waves has 32 NC rows a wave and walks over the keys of its
// part in tiles of 64: one pass with the running maximum and sum.
template <typename T, int DP, int NW, int NC, bool BIAS, bool FAST>
__global__ __launch_bounds__(64 * NW) void attn_fwd(AttnArgs a) {
    typedef Tile<T, DP> L;
    typedef typename Op<T>::Frag Frag;
    constexpr int KE = Op<T>::KE, NT = DP / 32, TR = 32 * NC * NW, KB = 32 / KE;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kKeys * L::RB];
    __shared__ __attribute__((aligned(16))) float bias_s[kKeys];
    const uint32_t kbase = (uint32_t)(uintptr_t)(lds_u8*)&smem[0];
    const uint32_t vbase = kbase + kKeys * L::RB;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), h = lane >> 5;

    int hk, idx, seq, tile, tiles;
    if (!head_of(blockIdx.x, a.slots * a.splits, a.hkv, &hk, &idx)) return;
    const int split = idx % a.splits;
    if (!locate(a.cu_q, a.n_seq, a.total_q, a.G, TR, idx / a.splits, &seq, &tile, &tiles)) return;
    if (a.causal) tile = tiles - 1 - tile;   // the longest rows first
    const Span sq = span_of(a.cu_q, seq, a.n_seq, a.total_q);
    const Span sk = span_of(a.cu_k, seq, a.n_seq, a.total_k);
    const int rows = sq.len * a.G, lk = sk.len, ahead = sk.len - sq.len;

    // queries, and how many keys each sees
    Frag qf[NC][DP / KE];
    int lim[NC];
    const int row0 = tile * TR + wave * 32 * NC;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
        int token, g;
        const int r = row0 + 32 * n + (lane & 31);
        row_of(r, a.G, &token, &g);
        const T* p = (const T*)a.q + (sq.first + token) * a.q_ts + (int64_t)(hk * a.G + g) * a.q_hs;
        load_columns<T, DP, FAST>(qf[n], p, a.dk, r < rows, lane);
        lim[n] = a.causal ? min(max(token + ahead + 1, 0), lk) : lk;
    }
    // keys of the tile's first and last row
    int t_first, t_last, unused;
    row_of(tile * TR, a.G, &t_first, &unused);
    row_of(min(tile * TR + TR, rows) - 1, a.G, &t_last, &unused);
    const int most = a.causal ? min(max(t_last + ahead + 1, 0), lk) : lk;
    const int least = a.causal ? min(max(t_first + ahead + 1, 0), lk) : lk;
    // this part's tiles of keys
    const int all = (most + kKeys - 1) / kKeys;
    const int t0 = (int)((int64_t)all * split / a.splits), t1 = (int)((int64_t)all * (split + 1) / a.splits);

    const T* K = (const T*)a.k + sk.first * a.k_ts + (int64_t)hk * a.k_hs;
    const T* V = (const T*)a.v + sk.first * a.v_ts + (int64_t)hk * a.v_hs;
    const float* B = BIAS ? a.bias + sk.first : nullptr;
    const float scale2 = a.scale * kLog2e;

    floatx16 o[NC][NT];
    float m[NC], l[NC];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
        m[n] = -kInf;
        l[n] = 0.0f;
#pragma unroll
        for (int d = 0; d < NT; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[n][d][e] = 0.0f;
    }

    for (int t = t0; t < t1; ++t) {
        const int k0 = t * kKeys;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kKeys * L::NCH / (64 * NW); ++i) {
            const int id = tid + i * 64 * NW, row = id / L::NCH, c = id % L::NCH;
            bool ok = k0 + row < lk;
            // what lies at a key that is left out stays out of every product
            if constexpr (BIAS) ok = ok && !(B[min(k0 + row, lk - 1)] < kLowest);
            const int64_t key = k0 + row;
            const u32x4 kw = load_chunk<T, FAST>(K + key * a.k_ts, c * L::EPC, a.dk, ok);
            const u32x4 vw = load_chunk<T, FAST>(V + key * a.v_ts, c * L::EPC, a.dv, ok);
            *(lds_u32x4*)(uintptr_t)(kbase + L::at(row, c)) = kw;
            *(lds_u32x4*)(uintptr_t)(vbase + L::at(row, c)) = vw;
        }
        if constexpr (BIAS)
            if (tid < kKeys) bias_s[tid] = k0 + tid < lk ? bias2(B[k0 + tid]) : -kInf;
        __syncthreads();

        floatx16 s[NC][kKeys / 32];
#pragma unroll
        for (int kt = 0; kt < kKeys / 32; ++kt) {
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int e = 0; e < 16; ++e) s[n][kt][e] = 0.0f;
#pragma unroll
            for (int c = 0; c < DP / KE; ++c) {
                const Frag f = L::rows(kbase, 32 * kt, c, lane);
#pragma unroll
                for (int n = 0; n < NC; ++n) s[n][kt] = Op<T>::mma(f, qf[n][c], s[n][kt]);
            }
        }
        const bool cut = k0 + kKeys > least;
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            float mx = -kInf;
#pragma unroll
            for (int kt = 0; kt < kKeys / 32; ++kt)
#pragma unroll
                for (int e4 = 0; e4 < 4; ++e4) {
                    const int key = 32 * kt + 8 * e4 + 4 * h;
                    floatx4 b = {0, 0, 0, 0};
                    if constexpr (BIAS) b = *(const lds_f32x4*)(uintptr_t)((uint32_t)(uintptr_t)(lds_f32*)&bias_s[0] + 4 * key);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = s[n][kt][4 * e4 + e];
                        if constexpr (BIAS) x = fmaf(x, scale2, b[e]);
                        if (cut && k0 + key + e >= lim[n]) x = -kInf;
                        s[n][kt][4 * e4 + e] = x;
                        mx = fmaxf(mx, x);
                    }
                }
            mx = half_max(mx);
            const float mnew = fmaxf(m[n], BIAS ? mx : mx * scale2);
            const float use = mnew == -kInf ? 0.0f : mnew;
            const float shrink = exp2_fast(m[n] - use);
            m[n] = mnew;
            float sum = 0.0f;
#pragma unroll
            for (int kt = 0; kt < kKeys / 32; ++kt)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float x = s[n][kt][e], p = exp2_fast(BIAS ? x - use : fmaf(x, scale2, -use));
                    s[n][kt][e] = p;
                    sum += p;
                }
            l[n] = l[n] * shrink + sum;
#pragma unroll
            for (int d = 0; d < NT; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[n][d][e] *= shrink;
        }
#pragma unroll
        for (int kt = 0; kt < kKeys / 32; ++kt)
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                Frag pf[NC];
#pragma unroll
                for (int n = 0; n < NC; ++n) pf[n] = Op<T>::from(s[n][kt], b * KE / 2);
#pragma unroll
                for (int d = 0; d < NT; ++d) {
                    const Frag f = L::columns(vbase, 32 * kt + b * KE, d, lane);
#pragma unroll
                    for (int n = 0; n < NC; ++n) o[n][d] = Op<T>::mma(f, pf[n], o[n][d]);
                }
            }
    }

#pragma unroll
    for (int n = 0; n < NC; ++n) {
        const int r = row0 + 32 * n + (lane & 31);
        const float sum = half_sum(l[n]);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const float lse = sum == 0.0f ? -kInf : m[n] * kLn2 + logf(sum);
        if (r >= rows) continue;
        int token, g;
        row_of(r, a.G, &token, &g);
        const int64_t tok = sq.first + token;
        const int head = hk * a.G + g;
        if (a.splits > 1) {
            const int64_t cell = ((int64_t)split * a.total_q + tok) * a.hq + head;
            float* part = a.part + cell * a.dv;
            if (h == 0) a.part_lse[cell] = lse;
#pragma unroll
            for (int d = 0; d < NT; ++d)
#pragma unroll
                for (int e4 = 0; e4 < 4; ++e4) {
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = o[n][d][4 * e4 + e] * inv;
                    store4<float, FAST>(part, 32 * d + 8 * e4 + 4 * h, a.dv, v);
                }
            continue;
        }
        if (a.lse && h == 0) a.lse[tok * a.hq + head] = lse;
        T* out = (T*)a.out + tok * a.o_ts + (int64_t)head * a.o_hs;
#pragma unroll
        for (int d = 0; d < NT; ++d)
#pragma unroll
            for (int e4 = 0; e4 < 4; ++e4) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = o[n][d][4 * e4 + e] * inv;
                store4<T, FAST>(out, 32 * d + 8 * e4 + 4 * h, a.dv, v);
            }
    }
}

// Joins the parts of each row: a wave a row.
//   l = log sum_s exp l_s,  o = sum_s exp(l_s - l) o_s
template <typename T>
__global__ __launch_bounds__(256) void attn_join(AttnArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t cell = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t tok = cell / a.hq;
    const int head = (int)(cell - tok * a.hq);
    // tokens before the first and behind the last sequence stay as they are
    if (tok >= a.total_q) return;
    if (a.cu_q && (tok < a.cu_q[0] || tok >= a.cu_q[a.n_seq])) return;
    const int64_t stride = a.total_q * a.hq;
    float mx = -kInf;
    for (int s = 0; s < a.splits; ++s) mx = fmaxf(mx, a.part_lse[s * stride + cell]);
    const float use = mx == -kInf ? 0.0f : mx;
    float sum = 0.0f, v0 = 0.0f, v1 = 0.0f;
    for (int s = 0; s < a.splits; ++s) {
        const float w = exp2_fast((a.part_lse[s * stride + cell] - use) * kLog2e);
        const float* p = a.part + (s * stride + cell) * a.dv;
        sum += w;
        if (lane < a.dv) v0 += w * p[lane];
        if (lane + 64 < a.dv) v1 += w * p[lane + 64];
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (a.lse && lane == 0) a.lse[cell] = sum == 0.0f ? -kInf : use + logf(sum);
    T* out = (T*)a.out + tok * a.o_ts + (int64_t)head * a.o_hs;
    if (lane < a.dv) store_f(out, lane, v0 * inv);
    if (lane + 64 < a.dv) store_f(out, lane + 64, v1 * inv);
}

template <typename T, int DP, int NW, bool FAST>
int fwd_go(AttnArgs a, hipStream_t st) {
    a.slots = (int)tile_slots(a.cu_q != nullptr, a.total_q, a.n_seq, a.G, 32 * NW);
    const int64_t grid = grid_size((int64_t)a.slots * a.splits, a.hkv);
    {
        KernelTimer timer("attn_fwd", st);
        if (a.bias) attn_fwd<T, DP, NW, 1, true, FAST><<<(unsigned)grid, 64 * NW, 0, st>>>(a);
        else attn_fwd<T, DP, NW, 1, false, FAST><<<(unsigned)grid, 64 * NW, 0, st>>>(a);
    }
    if (a.splits > 1) {
        KernelTimer timer("attn_join", st);
        attn_join<T><<<(unsigned)((a.total_q * a.hq + 3) / 4), 256, 0, st>>>(a);
    }
    return attn_launched("attention_fwd");
}

template <typename T>
int fwd_typed(const AttnArgs& a, hipStream_t st) {
    const AttnPlan p = attn_plan_fwd(a);
    AttnArgs b = a;
    b.splits = p.splits;
    if (!p.fast) return fwd_go<T, 128, 4, false>(b, st);
#define DISCO_ATTN(DP)                                             \
    do {                                                           \
        if (p.waves == 1) return fwd_go<T, DP, 1, true>(b, st);    \
        return fwd_go<T, DP, 4, true>(b, st);                      \
    } while (0)
    const int d = std::max(a.dk, a.dv);
    if (d <= 32) DISCO_ATTN(32);
    if (d <= 64) DISCO_ATTN(64);
    DISCO_ATTN(128);
#undef DISCO_ATTN
}

}  // namespace

int attn_launched(const char* what) {
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess) return DISCO_OK;
    return set_error(DISCO_EHIP, "%s: launch failed: %s", what, hipGetErrorString(e));
}

int launch_attention_fwd(const AttnArgs& a, void* stream) {
    hipStream_t st = static_cast<hipStream_t>(stream);
    return a.dtype == DISCO_F32 ? fwd_typed<float>(a, st) : fwd_typed<bf16_t>(a, st);
}

}  // namespace disco
