// Attention over points or tokens, forward.
//
// 4 D operations a score against 2 / rows of a key's bytes: the matrix cores bound it
// where there are more than a few hundred rows, with an exponential, two products
// and a sum a score on the vector units beside them.  129 x 256 points, 8 heads of 64,
// bf16: 2.9 to 3.0 ms, 0.75 PFLOP/s; the matrix cores take 39 percent of the cycles and
// the vector units 57, mostly in turn, at a clock of 1.8 to 2.0 GHz.  Packed causal series
// of 12001 tokens, 12 heads of 128 over 4: 0.13 ms, 0.82 PFLOP/s.  Few rows over many
// keys are bound by the reading of the keys (8 points over 33024 keys, 34 MB: 20 us).
//
// Tried and not kept: 64 rows a wave (a third fewer reads of LDS, half the waves: 3.6
// ms of the 2.9), registers for four waves a SIMD (spills: 5.4), four stages of tiles
// instead of two (no gain), tiles of 64 keys at heads of 128 (spills).
#include "attention_device.h"

#include <algorithm>
#include <type_traits>

namespace disco {

using namespace attn;

namespace {

// The running maximum may lag: weights of 2^24 keep as many digits as weights of
// 1, in bfloat16 too.  So a tile's maximum is taken only where the sum of its
// weights passes this bound, or where the row has seen no key yet.
constexpr float kMostSum = 16777216.0f;

// A workgroup of NW waves has 32 rows a wave and walks over the keys of its
// part in tiles of KT: one pass with a reference close to the running maximum, and
// the running sum.  bfloat16: three tiles are under way in a wave: while tile i's
// scores become weights on the vector units, the matrix cores take the scores of
// i + 1 and the values of i - 1, which depend on none of it.  float32 products take
// most of the time, so a tile goes through at once and leaves registers for the heads.
template <typename T, int DP, int NW, int KT, bool BIAS, bool FAST>
__global__ __launch_bounds__(64 * NW, sizeof(T) == 2 && NW == 4 && FAST ? 2 : 1) void attn_fwd(AttnArgs a) {
    typedef Tile<T, DP> L;
    typedef typename Op<T>::Frag Frag;
    typedef typename Addend<T>::Word Word;
    constexpr int KE = Op<T>::KE, NT = DP / 32, TR = 32 * NW, KB = 32 / KE, NK = KT / 32, TB = KT * L::RB;
    constexpr bool PIPE = sizeof(T) == 2;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[4 * TB];   // two stages of keys, then of values
    // biases, and zeros for the upper half of the lanes
    __shared__ __attribute__((aligned(16))) Word bias_s[BIAS ? 2 : 1][2][KT];
    __shared__ __attribute__((aligned(16))) float raw_s[BIAS && FAST ? 2 : 1][64];
    const uint32_t base = (uint32_t)(uintptr_t)(lds_u8*)&smem[0];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), h = lane >> 5;

    int hk, idx, seq, tile, tiles;
    if (!head_of(blockIdx.x, a.slots * a.splits, a.hkv, a.causal, &hk, &idx)) return;
    const int slot = a.splits == 1 ? idx : idx / a.splits, split = idx - slot * a.splits;
    if (!locate<GROWS>(a.causal, a.cu_q, a.n_seq, (int)a.total_q, a.each_q, a.G, TR, slot, a.slots, &seq, &tile, &tiles)) return;
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
    const int all = (most + KT - 1) / KT;
    int t0 = 0, t1 = all;
    if (a.splits > 1) {
        t0 = (int)((int64_t)all * split / a.splits);
        t1 = (int)((int64_t)all * (split + 1) / a.splits);
    }

    const T* K = (const T*)a.k + sk.first * a.k_ts + (int64_t)hk * a.k_hs;
    const T* V = (const T*)a.v + sk.first * a.v_ts + (int64_t)hk * a.v_hs;
    const float* B = BIAS ? a.bias + sk.first : nullptr;
    const float scale2 = a.scale * kLog2e, per_scale = 1.0f / a.scale, far = kFarTwo / scale2;

    // a key's bias in units of the raw score, which starts the score's sum; -inf
    // where the key is left out.  What lies there stays out of every product.
    auto scaled = [&](float b, int key) -> float { return key >= lk || b < kLowest ? -kInf : b * per_scale; };
    typedef Copy<T, DP, KT, FAST ? NW : 1> C;
    C copy;
    uint32_t koff[C::N], voff[C::N];
    // Tiles of this part are counted from 0, tile i has stage i % 2.  KT rows from
    // tile i's first into LDS at `at`; rows of `out` become zeros.
    const int n_tiles = t1 - t0;
    auto start = [&](const T*& next, int64_t ts, int d, const uint32_t* off, uint32_t at, uint64_t out) {
        const T* q = next;
        next += KT * ts;
        if constexpr (FAST) {
            copy.start(q, off, at, out, wave);
        } else {
#pragma unroll 1
            for (int id = tid; id < KT * L::NCH; id += 64 * NW) {
                const int row = id / L::NCH, c = id % L::NCH;
                *(lds_u32x4*)(uintptr_t)(at + L::at(row, c)) =
                    load_chunk<T, FAST>(q + row * ts, c * L::EPC, d, !((out >> row) & 1));
            }
        }
    };
    // rows of the next tile to be asked for
    const T *knext = K + (int64_t)t0 * KT * a.k_ts, *vnext = V + (int64_t)t0 * KT * a.v_ts;
    const float* bnext = BIAS ? B + t0 * KT : nullptr;
    uint64_t outs[2];   // rows left out of the tiles under way
    auto start_keys = [&](int i, int stage, float b) {
        outs[stage] = from_bit(lk - (t0 + i) * KT);
        if constexpr (BIAS) {
            b = scaled(b, (t0 + i) * KT + lane);
            outs[stage] |= __ballot(b == -kInf);
            if (wave == 0 && lane < KT) bias_s[stage][0][lane] = Addend<T>::pack(b);
        }
        start(knext, a.k_ts, a.dk, koff, base + (uint32_t)stage * TB, outs[stage]);
    };
    auto start_values = [&](int stage) {
        start(vnext, a.v_ts, a.dv, voff, base + (uint32_t)(2 + stage) * TB, outs[stage]);
    };
    auto bias_of = [&](int i) -> float {
        const int key = (t0 + i) * KT + lane;
        return key < lk ? B[key] : 0.0f;
    };
    auto start_bias = [&](int i, int stage) {   // by the first wave
        const uint32_t off = (t0 + i) * KT + lane < lk ? (uint32_t)lane * 4u : kNowhere;
        copy4(buffer_of(bnext + i * KT), off, (uint32_t)(uintptr_t)(lds_f32*)&raw_s[stage][0]);
    };

    // queries, and how many keys each sees
    const int r = tile * TR + wave * 32 + (lane & 31);
    int token, g;
    row_of(r, a.G, &token, &g);
    const int64_t tok = sq.first + token;
    const int head = hk * a.G + g;
    const int lim = a.causal ? min(max(token + ahead + 1, 0), lk) : lk;
    float m = -kInf, l = 0.0f;      // of raw scores
    Reference ref = {0.0f, 0.0f};   // of m
    Frag qf[DP / KE], pf[PIPE ? 2 : 1][KT / KE];
    floatx16 o[NT], s[PIPE ? 2 : 1][NK];
#pragma unroll
    for (int d = 0; d < NT; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] = 0.0f;
    Reader<T, DP> rd;
    rd.init(base, lane);
    typedef __attribute__((address_space(3))) Word lds_word;
    const uint32_t bbase = (uint32_t)(uintptr_t)(lds_word*)&bias_s[0][h][lane & 31];

    auto score = [&](auto stage_c) {
        constexpr int st = decltype(stage_c)::value;
#pragma unroll
        for (int kt = 0; kt < NK; ++kt) {
            floatx16& x = s[PIPE ? st : 0][kt];
            x = floatx16{};
            if constexpr (BIAS) x = Addend<T>::spread(*(const lds_word*)(uintptr_t)(bbase + (uint32_t)sizeof(Word) * (2 * st * KT + 32 * kt)));
#pragma unroll
            for (int c = 0; c < DP / KE; ++c)
                if (worth<T>(c * KE, a.dk)) x = Op<T>::mma(rd.rows(st * TB, kt, c), qf[c], x);
        }
    };
    auto weigh = [&](auto stage_c) {
        constexpr int st = decltype(stage_c)::value;
#pragma unroll
        for (int b = 0; b < KT / KE; ++b)
#pragma unroll
            for (int d = 0; d < NT; ++d)
                if (worth<T>(32 * d, a.dv)) o[d] = Op<T>::mma(rd.columns((2 + st) * TB, b, d), pf[PIPE ? st : 0][b], o[d]);
    };
    // scores to weights, and this lane's part of their sum.  ANY: of every reference
    auto soften = [&](auto any_c, const floatx16* x, Frag* w) -> float {
        float part[4] = {0, 0, 0, 0};
#pragma unroll
        for (int kt = 0; kt < NK; ++kt) {
            floatx16 p;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                p[e] = exp2_fast(fmaf(decltype(any_c)::value ? x[kt][e] - ref.raw : x[kt][e], scale2, -ref.two));
                part[e % 4] += p[e];
            }
#pragma unroll
            for (int b = 0; b < KB; ++b) w[kt * KB + b] = Op<T>::from(p, b * KE / 2);
        }
        return (part[0] + part[1]) + (part[2] + part[3]);
    };
    float raw = 0.0f;
    auto step = [&](auto stage_c, int i) {
        constexpr int st = decltype(stage_c)::value;
        const int k0 = (t0 + i) * KT;
        constexpr int at = PIPE ? st : 0, next = PIPE ? st : st ^ 1;   // of the scores, of the tile asked for
        constexpr int more = PIPE ? 2 : 1;
        // Here are keys i + 1 and values i - 1, and all waves have left keys i and values
        // i - 2 (float32: tile i is here, and all waves have left tile i - 1).
        all_arrived();
        if constexpr (PIPE) start_values(st);
        if constexpr (BIAS && !FAST) raw = bias_of(i + more);
        start_keys(i + more, next, raw);
        if constexpr (!PIPE) start_values(next);
        if constexpr (BIAS && FAST) {
            if (wave == 0) start_bias(i + more + 2, next);
            raw = raw_s[next ^ 1][lane];   // of tile i + more + 1
        }
        if constexpr (!PIPE) score(std::integral_constant<int, st>());
        if (k0 + KT > least) {   // some row does not see all of the tile
            const int room = lim - k0 - 4 * h;
#pragma unroll
            for (int kt = 0; kt < NK; ++kt)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (32 * kt + 8 * (e / 4) + e % 4 >= room) s[at][kt][e] = -kInf;
        }
        if constexpr (PIPE) {
            score(std::integral_constant<int, st ^ 1>());   // behind the last tile: not used
            weigh(std::integral_constant<int, st ^ 1>());
        }
        float sum = soften(std::false_type(), s[at], pf[at]);
        // NK DP / KE products for the scores and as many for the values (2 percent
        // faster than in the compiler's order)
        if constexpr (PIPE) mix<NK * DP / 8, 6, 2, 320 / DP, 128 / DP>();
        // rows whose reference is taken anew; the others keep their bits.  Rows without one,
        // or with a far one, go this way at every tile
        bool late = !(fabsf(m) < far);
        if (__any(late || sum > kMostSum)) {
            late = late || half_max(sum) > kMostSum;
            float mx = s[at][0][0];
#pragma unroll
            for (int kt = 0; kt < NK; ++kt)
#pragma unroll
                for (int e = 0; e < 16; ++e) mx = fmaxf(mx, s[at][kt][e]);
            mx = half_max(mx);
            const float mnew = late ? fmaxf(m, mx) : m;
            const Reference to = reference_of(mnew, scale2, far);
            const float shrink = m == -kInf ? 0.0f : change_of(ref, to, scale2);
            m = mnew;
            ref = to;
            l *= shrink;
#pragma unroll
            for (int d = 0; d < NT; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[d][e] *= shrink;
            sum = soften(std::true_type(), s[at], pf[at]);
        }
        l += sum;
        if constexpr (!PIPE) weigh(std::integral_constant<int, st>());
    };

    if constexpr (FAST) {
        copy.init(wave, lane);
        copy.offsets(koff, a.k_ts, a.dk, lane);
        copy.offsets(voff, a.v_ts, a.dv, lane);
    }
    if (n_tiles > 0) {
        float b[2] = {0.0f, 0.0f};
        constexpr int first = PIPE ? 2 : 1;   // tiles asked for beforehand
        if constexpr (BIAS) {
            for (int i = 0; i < first; ++i) b[i] = bias_of(i);
            raw = bias_of(first);
        }
        for (int i = 0; i < first; ++i) start_keys(i, i, b[i]);
        if constexpr (!PIPE) start_values(0);
        if constexpr (BIAS) {
            if (FAST && wave == 0) start_bias(first + 1, (first + 1) & 1);
            for (int i = tid; i < 2 * KT; i += 64 * NW) bias_s[i / KT][1][i % KT] = Word{};
        }
        if constexpr (PIPE) {   // no values before the first: zeros, with weights of zero
            for (int i = tid; i < TB / 16; i += 64 * NW)
                *(lds_u32x4*)(uintptr_t)(base + 3 * TB + 16 * i) = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < KT / KE; ++i) pf[1][i] = Frag{};
        }
        load_columns<T, DP, FAST>(qf, (const T*)a.q + tok * a.q_ts + (int64_t)head * a.q_hs, a.dk, r < rows, lane);
        if constexpr (PIPE) {
            all_arrived();
            score(std::integral_constant<int, 0>());
        }
        int i = 0;
        for (;;) {
            step(std::integral_constant<int, 0>(), i);
            if (++i == n_tiles) break;
            step(std::integral_constant<int, 1>(), i);
            if (++i == n_tiles) break;
        }
        all_arrived();   // no copy outlives its workgroup
        if constexpr (PIPE) {
            if (n_tiles & 1) weigh(std::integral_constant<int, 0>());
            else weigh(std::integral_constant<int, 1>());
        }
    }

    const float total = half_sum(l);
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    if (r >= rows) return;
    const int64_t cell = ((int64_t)split * a.total_q + tok) * a.hq + head;
    if (h == 0) {
        if (a.splits > 1) {
            a.part_lse[cell] = m;
            a.part_lse[a.splits * a.total_q * a.hq + cell] = total;
        } else if (a.lse) {
            a.lse[cell] = log_of(ref, a.scale, total);
        }
    }
    float* part = a.part + cell * a.dv;
    T* orow = (T*)a.out + tok * a.o_ts + (int64_t)head * a.o_hs;
#pragma unroll
    for (int d = 0; d < NT; ++d)
#pragma unroll
        for (int e4 = 0; e4 < 4; ++e4) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = o[d][4 * e4 + e] * inv;
            if (a.splits > 1) store4<float, FAST>(part, 32 * d + 8 * e4 + 4 * h, a.dv, v);
            else store4<T, FAST>(orow, 32 * d + 8 * e4 + 4 * h, a.dv, v);
        }
}

constexpr int kMostSplits = 256, kJoinWaves = 16;

// Joins the parts of each row, with weights w_s = sum_s exp(reference_s - reference):
//   l = reference + log sum_s w_s,  o = sum_s w_s o_s / sum_s w_s
// (of a part's l alone a large bias would leave no digit of its sum.)
__device__ __forceinline__ float part_weight(float m, float sum, Reference top, float scale2, float far) {
    return sum == 0.0f ? 0.0f : sum * change_of(reference_of(m, scale2, far), top, scale2);
}

// A wave a row, where the parts are few
template <typename T>
__global__ __launch_bounds__(256) void attn_join_few(AttnArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t cell = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), tok = cell / a.hq;
    const int head = (int)(cell - tok * a.hq);
    // tokens before the first and behind the last sequence stay as they are
    if (tok >= a.total_q || (a.cu_q && (tok < a.cu_q[0] || tok >= a.cu_q[a.n_seq]))) return;
    const int64_t stride = a.total_q * a.hq;
    const float scale2 = a.scale * kLog2e, far = kFarTwo / scale2;
    const float *pm = a.part_lse + cell, *ps = pm + a.splits * stride;
    float mx = -kInf, sum = 0.0f, v0 = 0.0f, v1 = 0.0f;
    for (int s = 0; s < a.splits; ++s) mx = fmaxf(mx, pm[s * stride]);
    const Reference top = reference_of(mx, scale2, far);
    const int d0 = min(lane, a.dv - 1), d1 = min(lane + 64, a.dv - 1);
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
        const float w = part_weight(pm[s * stride], ps[s * stride], top, scale2, far);
        const float* q = a.part + (s * stride + cell) * a.dv;
        sum += w;
        v0 = fmaf(w, q[d0], v0);
        v1 = fmaf(w, q[d1], v1);
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (a.lse && lane == 0) a.lse[cell] = log_of(top, a.scale, sum);
    T* out = (T*)a.out + tok * a.o_ts + (int64_t)head * a.o_hs;
    if (lane < a.dv) store_f(out, lane, v0 * inv);
    if (lane + 64 < a.dv) store_f(out, lane + 64, v1 * inv);
}

// A workgroup a row, its waves share the parts (8 points over 33024 keys, 128 rows
// of 97 parts: 6 us; of 128 parts 10, with a wave a row 120)
template <typename T>
__global__ __launch_bounds__(64 * kJoinWaves) void attn_join(AttnArgs a) {
    constexpr int P = kMostSplits / 64;
    __shared__ float w_s[kMostSplits], red[kJoinWaves][128];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t cell = blockIdx.x, tok = cell / a.hq;
    const int head = (int)(cell - tok * a.hq);
    // tokens before the first and behind the last sequence stay as they are
    if (a.cu_q && (tok < a.cu_q[0] || tok >= a.cu_q[a.n_seq])) return;
    const int64_t stride = a.total_q * a.hq;
    const float scale2 = a.scale * kLog2e, far = kFarTwo / scale2;
    const float *pm = a.part_lse + cell, *ps = pm + a.splits * stride;
    float m[P], l[P], mx = -kInf, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const bool ok = lane + 64 * i < a.splits;
        m[i] = ok ? pm[(lane + 64 * i) * stride] : -kInf;
        l[i] = ok ? ps[(lane + 64 * i) * stride] : 0.0f;
        mx = fmaxf(mx, m[i]);
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) mx = fmaxf(mx, __shfl_xor(mx, d, 64));
    const Reference top = reference_of(mx, scale2, far);
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const float w = part_weight(m[i], l[i], top, scale2, far);
        if (wave == 0) w_s[lane + 64 * i] = w;
        sum += w;
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d, 64);
    __syncthreads();
    float v0 = 0.0f, v1 = 0.0f;
    const float* p = a.part + cell * a.dv;
    const int d0 = min(lane, a.dv - 1), d1 = min(lane + 64, a.dv - 1);
#pragma unroll 8
    for (int s = wave; s < a.splits; s += kJoinWaves) {
        const float* q = p + s * stride * a.dv;
        v0 = fmaf(w_s[s], q[d0], v0);
        v1 = fmaf(w_s[s], q[d1], v1);
    }
    red[wave][lane] = v0;
    red[wave][lane + 64] = v1;
    __syncthreads();
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (a.lse && threadIdx.x == 0) a.lse[cell] = log_of(top, a.scale, sum);
    const int d = threadIdx.x;
    if (d >= a.dv) return;
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kJoinWaves; ++i) v += red[i][d];
    store_f((T*)a.out + tok * a.o_ts + (int64_t)head * a.o_hs, d, v * inv);
}

template <typename T, int DP, int NW, int KT, bool FAST>
int fwd_go(AttnArgs a, hipStream_t st) {
    a.slots = (int)tile_slots(a.cu_q != nullptr, a.total_q, a.n_seq, a.G, 32 * NW);
    const int64_t grid = grid_size((int64_t)a.slots * a.splits, a.hkv);
    {
        KernelTimer timer("attn_fwd", st);
        if (a.bias) attn_fwd<T, DP, NW, KT, true, FAST><<<(unsigned)grid, 64 * NW, 0, st>>>(a);
        else attn_fwd<T, DP, NW, KT, false, FAST><<<(unsigned)grid, 64 * NW, 0, st>>>(a);
    }
    if (a.splits > 1) {
        KernelTimer timer("attn_join", st);
        if (a.splits <= 8) attn_join_few<T><<<(unsigned)((a.total_q * a.hq + 3) / 4), 256, 0, st>>>(a);
        else attn_join<T><<<(unsigned)(a.total_q * a.hq), 64 * kJoinWaves, 0, st>>>(a);
    }
    return attn_launched("attention_fwd");
}

template <typename T, int DP, int KT>
int fwd_waves(const AttnArgs& a, int waves, hipStream_t st) {
    if (waves == 1) return fwd_go<T, DP, 1, KT, true>(a, st);
    if (waves == 2) return fwd_go<T, DP, 2, KT, true>(a, st);
    return fwd_go<T, DP, 4, KT, true>(a, st);
}

template <typename T>
int fwd_typed(AttnArgs a, hipStream_t st) {
    const AttnPlan p = a.plan;
    a.splits = p.splits;
    // keys of a tile: 64 where two waves of a SIMD still hold their scores
    constexpr int KT = sizeof(T) == 2 ? 64 : 32;
    if (!p.fast) return fwd_go<T, 128, 4, KT, false>(a, st);
    const int d = std::max(a.dk, a.dv);
    if (d <= 32) return fwd_waves<T, 32, KT>(a, p.waves, st);
    if (d <= 64) return fwd_waves<T, 64, KT>(a, p.waves, st);
    return fwd_waves<T, 128, 32>(a, p.waves, st);
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
