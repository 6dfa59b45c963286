// Attention over points or tokens, forward.
#include "attention_device.h"

#include <algorithm>

namespace disco {

using namespace attn;

namespace {

constexpr int kKeys = 64;   // keys of a tile
// A maximum may lag by 2^8: weights then reach 2^8, which bfloat16 holds as well as 1.
constexpr float kLag = 8.0f;

// A workgroup of NW waves has 32 NC rows a wave and walks over the keys of its
// part in tiles of 64: one pass with the running maximum and sum.
template <typename T, int DP, int NW, int NC, bool BIAS, bool FAST>
__global__ __launch_bounds__(64 * NW, (NC == 1 && NW < 8) ? 2 : 1) void attn_fwd(AttnArgs a) {
    typedef Tile<T, DP> L;
    typedef typename Op<T>::Frag Frag;
    constexpr int KE = Op<T>::KE, NT = DP / 32, TR = 32 * NC * NW, KB = 32 / KE, TB = kKeys * L::RB;
    constexpr int STAGES = FAST ? 2 : 1;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[STAGES * 2 * TB];
    __shared__ __attribute__((aligned(16))) float bias_s[2][kKeys];
    const uint32_t base = (uint32_t)(uintptr_t)(lds_u8*)&smem[0];
    const uint32_t bias_base = (uint32_t)(uintptr_t)(lds_f32*)&bias_s[0][0];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), h = lane >> 5;

    int hk, idx, seq, tile, tiles;
    if (!head_of(blockIdx.x, a.slots * a.splits, a.hkv, &hk, &idx)) return;
    const int split = idx % a.splits;
    if (!locate(a.cu_q, a.n_seq, a.total_q, a.G, TR, idx / a.splits, &seq, &tile, &tiles)) return;
    if (a.causal) tile = tiles - 1 - tile;   // the longest rows first
    const Span sq = span_of(a.cu_q, seq, a.n_seq, a.total_q);
    const Span sk = span_of(a.cu_k, seq, a.n_seq, a.total_k);
    const int rows = sq.len * a.G, lk = sk.len, ahead = sk.len - sq.len;

    // keys that the tile's first and last row see
    int t_first, t_last, unused;
    row_of(tile * TR, a.G, &t_first, &unused);
    row_of(min(tile * TR + TR, rows) - 1, a.G, &t_last, &unused);
    const int most = uniform(a.causal ? min(max(t_last + ahead + 1, 0), lk) : lk);
    const int least = uniform(a.causal ? min(max(t_first + ahead + 1, 0), lk) : lk);
    // this part's tiles of keys
    const int all = (most + kKeys - 1) / kKeys;
    const int t0 = (int)((int64_t)all * split / a.splits), t1 = (int)((int64_t)all * (split + 1) / a.splits);

    const T* K = (const T*)a.k + sk.first * a.k_ts + (int64_t)hk * a.k_hs;
    const T* V = (const T*)a.v + sk.first * a.v_ts + (int64_t)hk * a.v_hs;
    const float* B = BIAS ? a.bias + sk.first : nullptr;
    const float scale2 = a.scale * kLog2e, per_scale = 1.0f / a.scale;

    // a key's bias in units of the raw score, which starts the score's sum; -inf
    // where the key is left out.  What lies there stays out of every product.
    auto bias_of = [&](int k0) -> float {
        const int key = k0 + lane;
        const float b = key < lk ? B[key] : -kInf;
        return b < kLowest ? -kInf : b * per_scale;
    };
    Copy<T, DP, kKeys, FAST ? NW : 1> ck, cv;
    float bias = 0.0f;
    auto start = [&](int t) {   // the copies of tile t; `bias` is tile t's
        const uint32_t at = base + (uint32_t)(t & 1) * (2 * TB);
        uint64_t out = 0;
        if constexpr (BIAS) {
            out = __ballot(bias == -kInf);
            if (wave == 0) bias_s[t & 1][lane] = bias;
        }
        const int64_t k0 = (int64_t)t * kKeys;
        ck.start(K + k0 * a.k_ts, at, lk - (int)k0, out, wave);
        cv.start(V + k0 * a.v_ts, at + TB, lk - (int)k0, out, wave);
    };
    if constexpr (FAST) {
        ck.init(a.k_ts, a.dk, wave, lane);
        cv.init(a.v_ts, a.dv, wave, lane);
        if (t0 < t1) {
            if constexpr (BIAS) bias = bias_of(t0 * kKeys);
            start(t0);
            if constexpr (BIAS) bias = bias_of((t0 + 1) * kKeys);
        }
    }

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
        const uint32_t kbase = base + (FAST ? (uint32_t)(t & 1) * (2 * TB) : 0u), vbase = kbase + TB;
        const uint32_t bbase = bias_base + (FAST ? (uint32_t)(t & 1) * (kKeys * 4) : 0u);
        if constexpr (FAST) {
            all_arrived();
            if (t + 1 < t1) {
                start(t + 1);
                if constexpr (BIAS) bias = bias_of(k0 + 2 * kKeys);
            }
        } else {
            __syncthreads();
            if constexpr (BIAS) {
                bias = bias_of(k0);
                if (wave == 0) bias_s[0][lane] = bias;
            }
            const uint64_t out = BIAS ? __ballot(bias == -kInf) : 0;
#pragma unroll
            for (int i = 0; i < kKeys * L::NCH / (64 * NW); ++i) {
                const int id = tid + i * 64 * NW, row = id / L::NCH, c = id % L::NCH;
                const bool ok = k0 + row < lk && !((out >> row) & 1);
                const int64_t key = k0 + row;
                const u32x4 kw = load_chunk<T, FAST>(K + key * a.k_ts, c * L::EPC, a.dk, ok);
                const u32x4 vw = load_chunk<T, FAST>(V + key * a.v_ts, c * L::EPC, a.dv, ok);
                *(lds_u32x4*)(uintptr_t)(kbase + L::at(row, c)) = kw;
                *(lds_u32x4*)(uintptr_t)(vbase + L::at(row, c)) = vw;
            }
            __syncthreads();
        }

        floatx16 s[NC][kKeys / 32];
#pragma unroll
        for (int kt = 0; kt < kKeys / 32; ++kt) {
#pragma unroll
            for (int e4 = 0; e4 < 4; ++e4) {
                floatx4 b = {0, 0, 0, 0};
                if constexpr (BIAS) b = *(const lds_f32x4*)(uintptr_t)(bbase + 4 * (32 * kt + 8 * e4 + 4 * h));
#pragma unroll
                for (int n = 0; n < NC; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[n][kt][4 * e4 + e] = b[e];
            }
#pragma unroll
            for (int c = 0; c < DP / KE; ++c) {
                const Frag f = L::rows(kbase, 32 * kt, c, lane);
#pragma unroll
                for (int n = 0; n < NC; ++n) s[n][kt] = Op<T>::mma(f, qf[n][c], s[n][kt]);
            }
        }
        if (k0 + kKeys > least) {   // some row does not see all of the tile
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int kt = 0; kt < kKeys / 32; ++kt)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (k0 + 32 * kt + 8 * (e / 4) + 4 * h + e % 4 >= lim[n]) s[n][kt][e] = -kInf;
        }
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            float mx = s[n][0][0];
#pragma unroll
            for (int kt = 0; kt < kKeys / 32; ++kt)
#pragma unroll
                for (int e = 0; e < 16; ++e) mx = fmaxf(mx, s[n][kt][e]);
            mx = half_max(mx) * scale2;
            if (__any(mx > m[n] + kLag)) {
                const float mnew = fmaxf(m[n], mx);
                const float shrink = exp2_fast(m[n] - (mnew == -kInf ? 0.0f : mnew));
                m[n] = mnew;
                l[n] *= shrink;
#pragma unroll
                for (int d = 0; d < NT; ++d)
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[n][d][e] *= shrink;
            }
            const float use = m[n] == -kInf ? 0.0f : m[n];
            float sum[4] = {0, 0, 0, 0};
#pragma unroll
            for (int kt = 0; kt < kKeys / 32; ++kt)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float p = exp2_fast(fmaf(s[n][kt][e], scale2, -use));
                    s[n][kt][e] = p;
                    sum[e % 4] += p;
                }
            l[n] += (sum[0] + sum[1]) + (sum[2] + sum[3]);
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

constexpr int kMostSplits = 128;

// Joins the parts of each row: a workgroup a row, its waves share the parts.
//   l = log sum_s exp l_s,  o = sum_s exp(l_s - l) o_s
template <typename T>
__global__ __launch_bounds__(256) void attn_join(AttnArgs a) {
    __shared__ float w_s[kMostSplits], red[4][128];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t cell = blockIdx.x, tok = cell / a.hq;
    const int head = (int)(cell - tok * a.hq);
    // tokens before the first and behind the last sequence stay as they are
    if (a.cu_q && (tok < a.cu_q[0] || tok >= a.cu_q[a.n_seq])) return;
    const int64_t stride = a.total_q * a.hq;
    const float l0 = lane < a.splits ? a.part_lse[lane * stride + cell] : -kInf;
    const float l1 = lane + 64 < a.splits ? a.part_lse[(lane + 64) * stride + cell] : -kInf;
    float mx = fmaxf(l0, l1);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) mx = fmaxf(mx, __shfl_xor(mx, d, 64));
    const float use = mx == -kInf ? 0.0f : mx;
    const float w0 = exp2_fast((l0 - use) * kLog2e), w1 = exp2_fast((l1 - use) * kLog2e);
    float sum = w0 + w1;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d, 64);
    if (wave == 0) {
        w_s[lane] = w0;
        w_s[lane + 64] = w1;
    }
    __syncthreads();
    float v0 = 0.0f, v1 = 0.0f;
    const float* p = a.part + cell * a.dv;
    const bool has0 = lane < a.dv, has1 = lane + 64 < a.dv;
#pragma unroll 8
    for (int s = wave; s < a.splits; s += 4) {
        const float* q = p + s * stride * a.dv;
        const float w = w_s[s];
        if (has0) v0 = fmaf(w, q[lane], v0);
        if (has1) v1 = fmaf(w, q[lane + 64], v1);
    }
    red[wave][lane] = v0;
    red[wave][lane + 64] = v1;
    __syncthreads();
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (a.lse && threadIdx.x == 0) a.lse[cell] = sum == 0.0f ? -kInf : use + logf(sum);
    T* out = (T*)a.out + tok * a.o_ts + (int64_t)head * a.o_hs;
    const int d = threadIdx.x;
    if (d < a.dv) store_f(out, d, ((red[0][d] + red[1][d]) + (red[2][d] + red[3][d])) * inv);
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
        attn_join<T><<<(unsigned)(a.total_q * a.hq), 256, 0, st>>>(a);
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
