// Attention over points or tokens, forward.
#include "attention_device.h"

#include <algorithm>
#include <type_traits>

namespace disco {

using namespace attn;

namespace {

constexpr int kKeys = 64;   // keys of a tile
// The running maximum may lag: weights of 2^60 keep as many digits as weights of
// 1, in bfloat16 too.  So a tile's maximum is taken only where the sum of its
// weights passes this bound, or where the row has seen no key yet.
constexpr float kMostSum = 1.152921504606846976e18f;

// A workgroup of NW waves has 32 rows a wave and walks over the keys of its part
// in tiles of 64: one pass with a reference close to the running maximum, and
// the running sum.
template <typename T, int DP, int NW, bool BIAS, bool FAST>
__global__ __launch_bounds__(64 * NW, sizeof(T) == 2 && NW == 4 && FAST ? 2 : 1) void attn_fwd(AttnArgs a) {
    typedef Tile<T, DP> L;
    typedef typename Op<T>::Frag Frag;
    constexpr int KE = Op<T>::KE, NT = DP / 32, TR = 32 * NW, KB = 32 / KE, TB = kKeys * L::RB;
    constexpr int STAGES = FAST ? 2 : 1;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[STAGES * 2 * TB];
    __shared__ __attribute__((aligned(16))) float bias_s[STAGES][kKeys];
    const uint32_t base = (uint32_t)(uintptr_t)(lds_u8*)&smem[0];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), h = lane >> 5;

    int hk, idx, seq, tile, tiles;
    if (!head_of(blockIdx.x, a.slots * a.splits, a.hkv, &hk, &idx)) return;
    const int slot = a.splits == 1 ? idx : idx / a.splits, split = idx - slot * a.splits;
    if (!locate(a.cu_q, a.n_seq, (int)a.total_q, a.each_q, a.G, TR, slot, &seq, &tile, &tiles)) return;
    if (a.causal) tile = tiles - 1 - tile;   // the longest rows first
    const Span sq = span_of(a.cu_q, seq, a.each_q, (int)a.total_q);
    const Span sk = span_of(a.cu_k, seq, a.each_k, (int)a.total_k);
    const int rows = sq.len * a.G, lk = sk.len, ahead = sk.len - sq.len;

    // keys that the tile's first and last row see
    int most = lk, least = lk;
    if (a.causal) {
        int t_first, t_last, unused;
        row_of(tile * TR, a.G, &t_first, &unused);
        row_of(min(tile * TR + TR, rows) - 1, a.G, &t_last, &unused);
        most = uniform(min(max(t_last + ahead + 1, 0), lk));
        least = uniform(min(max(t_first + ahead + 1, 0), lk));
    }
    // this part's tiles of keys
    const int all = (most + kKeys - 1) / kKeys;
    int t0 = 0, t1 = all;
    if (a.splits > 1) {
        t0 = (int)((int64_t)all * split / a.splits);
        t1 = (int)((int64_t)all * (split + 1) / a.splits);
    }

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
    typedef Copy<T, DP, FAST ? NW : 1> C;
    C copy;
    uint32_t koff[C::N], voff[C::N];
    float bias = 0.0f;
    auto start = [&](int t, int stage) {   // the copies of tile t; `bias` is tile t's
        const uint32_t at = base + (uint32_t)stage * (2 * TB);
        const int64_t k0 = (int64_t)t * kKeys;
        uint64_t out = from_bit(lk - (int)k0);
        if constexpr (BIAS) {
            out |= __ballot(bias == -kInf);
            if (wave == 0) bias_s[stage][lane] = bias;
        }
        copy.start(K + k0 * a.k_ts, koff, at, V + k0 * a.v_ts, voff, at + TB, out, wave);
    };
    if constexpr (FAST) {
        copy.init(wave, lane);
        copy.offsets(koff, a.k_ts, a.dk, lane);
        copy.offsets(voff, a.v_ts, a.dv, lane);
        if (t0 < t1) {
            if constexpr (BIAS) bias = bias_of(t0 * kKeys);
            start(t0, 0);
            if constexpr (BIAS) bias = bias_of((t0 + 1) * kKeys);
        }
    }

    // queries, and how many keys each sees
    Frag qf[DP / KE];
    const int r = tile * TR + wave * 32 + (lane & 31);
    int token, g;
    row_of(r, a.G, &token, &g);
    const int head = hk * a.G + g;
    load_columns<T, DP, FAST>(qf, (const T*)a.q + (sq.first + token) * a.q_ts + (int64_t)head * a.q_hs, a.dk, r < rows, lane);
    const int lim = a.causal ? min(max(token + ahead + 1, 0), lk) : lk;

    Reader<T, DP> rd;
    rd.init(base, lane);
    const uint32_t bbase = (uint32_t)(uintptr_t)(lds_f32*)&bias_s[0][0] + 16 * h;
    floatx16 o[NT];
    float m = -kInf, l = 0.0f;
#pragma unroll
    for (int d = 0; d < NT; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] = 0.0f;

    auto step = [&](auto stage_c, int t) {
        constexpr int stage = decltype(stage_c)::value;
        constexpr uint32_t koffs = stage * 2 * TB, voffs = koffs + TB;
        const int k0 = t * kKeys;
        if constexpr (FAST) {
            all_arrived();
            if (t + 1 < t1) {
                start(t + 1, stage ^ 1);
                if constexpr (BIAS) bias = bias_of(k0 + 2 * kKeys);
            }
        } else {
            __syncthreads();
            uint64_t out = from_bit(lk - k0);
            if constexpr (BIAS) {
                bias = bias_of(k0);
                out |= __ballot(bias == -kInf);
                if (wave == 0) bias_s[0][lane] = bias;
            }
#pragma unroll 1
            for (int id = tid; id < kKeys * L::NCH; id += 64 * NW) {
                const int row = id / L::NCH, c = id % L::NCH;
                const bool ok = !((out >> row) & 1);
                const int64_t key = k0 + row;
                *(lds_u32x4*)(uintptr_t)(base + L::at(row, c)) = load_chunk<T, FAST>(K + key * a.k_ts, c * L::EPC, a.dk, ok);
                *(lds_u32x4*)(uintptr_t)(base + TB + L::at(row, c)) = load_chunk<T, FAST>(V + key * a.v_ts, c * L::EPC, a.dv, ok);
            }
            __syncthreads();
        }

        floatx16 s[kKeys / 32];
#pragma unroll
        for (int kt = 0; kt < kKeys / 32; ++kt) {
#pragma unroll
            for (int e4 = 0; e4 < 4; ++e4) {
                floatx4 b = {0, 0, 0, 0};
                if constexpr (BIAS)
                    b = *(const lds_f32x4*)(uintptr_t)(bbase + 4 * (stage * kKeys + 32 * kt + 8 * e4));
#pragma unroll
                for (int e = 0; e < 4; ++e) s[kt][4 * e4 + e] = b[e];
            }
#pragma unroll
            for (int c = 0; c < DP / KE; ++c) s[kt] = Op<T>::mma(rd.rows(koffs, kt, c), qf[c], s[kt]);
        }
        if (k0 + kKeys > least) {   // some row does not see all of the tile
            const int room = lim - k0 - 4 * h;
#pragma unroll
            for (int kt = 0; kt < kKeys / 32; ++kt)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (32 * kt + 8 * (e / 4) + e % 4 >= room) s[kt][e] = -kInf;
        }
        Frag pf[kKeys / KE];
        float sum;
        bool late = m == -kInf;   // rows whose reference is taken anew; the others keep their bits
        for (;;) {
            if (__any(late)) {
                float mx = s[0][0];
#pragma unroll
                for (int kt = 0; kt < kKeys / 32; ++kt)
#pragma unroll
                    for (int e = 0; e < 16; ++e) mx = fmaxf(mx, s[kt][e]);
                mx = half_max(mx) * scale2;
                const float mnew = late ? fmaxf(m, mx) : m;
                const float shrink = exp2_fast(m - (mnew == -kInf ? 0.0f : mnew));
                m = mnew;
                l *= shrink;
#pragma unroll
                for (int d = 0; d < NT; ++d)
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[d][e] *= shrink;
            }
            const float use = m == -kInf ? 0.0f : m;
            float part[4] = {0, 0, 0, 0};
#pragma unroll
            for (int kt = 0; kt < kKeys / 32; ++kt) {
                floatx16 p;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    p[e] = exp2_fast(fmaf(s[kt][e], scale2, -use));
                    part[e % 4] += p[e];
                }
#pragma unroll
                for (int b = 0; b < KB; ++b) pf[kt * KB + b] = Op<T>::from(p, b * KE / 2);
            }
            sum = (part[0] + part[1]) + (part[2] + part[3]);
            if (!__any(sum > kMostSum)) break;
            late = half_max(sum) > kMostSum;
        }
        l += sum;
#pragma unroll
        for (int b = 0; b < kKeys / KE; ++b)
#pragma unroll
            for (int d = 0; d < NT; ++d) o[d] = Op<T>::mma(rd.columns(voffs, b, d), pf[b], o[d]);
    };
    if constexpr (FAST) {
        for (int t = t0; t < t1; t += 2) {
            step(std::integral_constant<int, 0>(), t);
            if (t + 1 < t1) step(std::integral_constant<int, 1>(), t + 1);
        }
    } else {
        for (int t = t0; t < t1; ++t) step(std::integral_constant<int, 0>(), t);
    }

    const float total = half_sum(l);
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    const float lse = total == 0.0f ? -kInf : m * kLn2 + logf(total);
    if (r >= rows) return;
    const int64_t tok = sq.first + token;
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
                for (int e = 0; e < 4; ++e) v[e] = o[d][4 * e4 + e] * inv;
                store4<float, FAST>(part, 32 * d + 8 * e4 + 4 * h, a.dv, v);
            }
        return;
    }
    if (a.lse && h == 0) a.lse[tok * a.hq + head] = lse;
    T* out = (T*)a.out + tok * a.o_ts + (int64_t)head * a.o_hs;
#pragma unroll
    for (int d = 0; d < NT; ++d)
#pragma unroll
        for (int e4 = 0; e4 < 4; ++e4) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = o[d][4 * e4 + e] * inv;
            store4<T, FAST>(out, 32 * d + 8 * e4 + 4 * h, a.dv, v);
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
        if (a.bias) attn_fwd<T, DP, NW, true, FAST><<<(unsigned)grid, 64 * NW, 0, st>>>(a);
        else attn_fwd<T, DP, NW, false, FAST><<<(unsigned)grid, 64 * NW, 0, st>>>(a);
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
