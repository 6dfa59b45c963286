// Gradients of the attention over points or tokens.
//
//   delta_i = go_i . o_i,  dp_ij = go_i . v_j,  ds_ij = p_ij (dp_ij - delta_i)
//   gq_i = scale sum_j ds_ij k_j,  gk_j = scale sum_i ds_ij q_i,  gv_j = sum_i p_ij go_i
// with p_ij = exp(x_ij - l_i) from the forward's l.  Two kernels, one that walks
// over the keys for tiles of rows (gq) and one that walks over the rows for tiles
// of keys (gk, gv): seven products where one kernel would do with five, but no
// sum is taken in an order that changes from run to run, and no atomics.
//
// p comes from l, which is rounded: rows of |l| above 45426 (all keys behind a mask of
// -1e9, say) have lost it there.  They weigh nothing in the two kernels, and each has a
// slow one behind it that ends at once where there are no such rows (5 us for both).
// Inside the kernels these steps cost the others their registers (gq and gk, gv of 6007
// packed tokens 70 and 151 us instead of 61 and 127).
//
// The matrix cores bound both, 6 D and 8 D operations a score; what they wait for are
// the reads of LDS (each operand of gq, gk and gv is read by columns, at half the
// width) and the vector units.  65 x 128 points, 8 heads of 64, bf16, in four parts:
// gq 260 us (0.82 PFLOP/s of its three products), gk and gv 347 us (0.82 of four).
// Packed causal series of 6007 tokens, 12 heads of 128 over 4: 62 and 129 us; there
// gk and gv of 128 leave one workgroup a compute unit (two workgroups by spilling: 435
// us), and nothing covers the 10 us in which one begins and ends.  float32, 2 x 33 x 64
// points, 4 heads of 32: 86 and 115 us, 0.08 PFLOP/s of the 0.15 that float32 products
// reach.  (Events around each launch under load; a card that has just begun took 277 and
// 377, 62 and 136, 91 and 121.)
//
// The order of instructions is the compiler's: laid out as in the forward kernel,
// gk and gv took 468 us instead of 457 and 190 instead of 147, gq 342 instead of 324.
#include "attention_device.h"
#include "vector_io.h"

#include <algorithm>
#include <type_traits>

namespace disco {

using namespace attn;

namespace {

constexpr int kStep = 32;   // keys (gq) or rows (gk, gv) of a step

// Parts of a tile of so many steps: a causal or packed call's tiles have few or many
__device__ __forceinline__ int parts_of(const AttnArgs& a, int steps) {
    return a.splits == 1 ? 1 : min(max((steps + a.chunk - 1) / a.chunk, 1), a.splits);
}

// A workgroup of NW waves has 32 rows a wave and walks over the keys of its part.
// bfloat16: three steps are under way in a wave: while the scores of step i become ds
// on the vector units, the matrix cores take the scores and dp of step i + 1 and the
// gradient's part of step i - 1.  float32 products take most of the time, so a step
// goes through at once and leaves registers for the heads.
//
// FINE, for queries of up to 32 elements in bfloat16: ds goes into its product in two
// bfloat16 parts (16 bits).  The few keys that such a row weighs most point the same way,
// and as the ds of a row add up to nothing their parts of gq cancel: with one part the
// error was 1.5 to 1.8 times that of rounding the result alone, where heads of 64 have
// 1.4 (65 x 128 points, 8 heads of 32: one part 168 us, two 224).
template <typename T, int DP, int NW, bool BIAS, bool FAST, bool FINE>
__global__ __launch_bounds__(64 * NW, sizeof(T) == 2 && FAST ? 2 : 1) void attn_bwd_q(AttnArgs a) {
    typedef Tile<T, DP> L;
    typedef typename Op<T>::Frag Frag;
    typedef typename Addend<T>::Word Word;
    constexpr int KE = Op<T>::KE, NT = DP / 32, TR = 32 * NW, KB = 32 / KE, TB = kStep * L::RB;
    constexpr bool PIPE = sizeof(T) == 2;
    constexpr int SK = PIPE ? 4 : 2;      // stages of keys; of values two
    __shared__ __attribute__((aligned(1024))) uint8_t smem[(SK + 2) * TB];
    __shared__ __attribute__((aligned(16))) Word bias_s[BIAS ? 2 : 1][2][kStep];
    __shared__ __attribute__((aligned(16))) float raw_s[BIAS && FAST ? 2 : 1][64];
    const uint32_t base = (uint32_t)(uintptr_t)(lds_u8*)&smem[0];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), h = lane >> 5;

    int hk, idx, seq, tile, tiles;
    if (!head_of(blockIdx.x, a.slots * a.splits, a.hkv, a.causal, &hk, &idx)) return;
    // the parts that only the longest tiles have go first
    const int turn = a.splits == 1 ? 0 : idx / a.slots, slot = idx - turn * a.slots, split = a.splits - 1 - turn;
    if (!locate<GROWS>(a.causal, a.cu_q, a.n_seq, (int)a.total_q, a.each_q, a.G, TR, slot, a.slots, &seq, &tile, &tiles)) return;
    const Span sq = span_of(a.cu_q, seq, a.each_q, (int)a.total_q);
    const Span sk = span_of(a.cu_k, seq, a.each_k, (int)a.total_k);
    const int rows = sq.len * a.G, lk = sk.len, ahead = sk.len - sq.len;

    int most = lk, least = lk;
    if (a.causal) {
        int t_first, t_last, unused;
        row_of(tile * TR, a.G, &t_first, &unused);
        row_of(min(tile * TR + TR, rows) - 1, a.G, &t_last, &unused);
        most = uniform(min(max(t_last + ahead + 1, 0), lk));
        least = uniform(min(max(t_first + ahead + 1, 0), lk));
    }
    const int all = (most + kStep - 1) / kStep;
    const int parts = parts_of(a, all);
    if (split >= parts) return;
    const int t0 = (int)((int64_t)all * split / parts), t1 = (int)((int64_t)all * (split + 1) / parts);
    const int n_steps = t1 - t0;

    const int r = tile * TR + wave * 32 + (lane & 31);
    int token, g;
    row_of(r, a.G, &token, &g);
    const int64_t tok = sq.first + token;
    const int head = hk * a.G + g;
    const bool mine = r < rows;
    const int lim = a.causal ? min(max(token + ahead + 1, 0), lk) : lk;
    Frag qf[DP / KE], gf[DP / KE];
    load_columns<T, DP, FAST>(gf, (const T*)a.go + tok * a.go_ts + (int64_t)head * a.go_hs, a.dv, mine, lane);
    float delta = 0.0f;
    const T* orow = (const T*)a.o + tok * a.o_ts + (int64_t)head * a.o_hs;
#pragma unroll
    for (int c = 0; c < DP / KE; ++c) {
        const u32x4 ow = load_chunk<T, FAST>(orow, (2 * c + h) * L::EPC, a.dv, mine);
        const u32x4 gw = __builtin_bit_cast(u32x4, gf[c]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 2) {
                delta = fmaf(__uint_as_float(ow[i] << 16), __uint_as_float(gw[i] << 16), delta);
                delta = fmaf(__uint_as_float(ow[i] & 0xffff0000u), __uint_as_float(gw[i] & 0xffff0000u), delta);
            } else {
                delta = fmaf(__uint_as_float(ow[i]), __uint_as_float(gw[i]), delta);
            }
        }
    }
    delta = half_sum(delta);
    if (split == 0 && h == 0 && mine) {
        a.delta[tok * a.hq + head] = delta;
        if (a.splits > 1) a.count[tok * a.hq + head] = parts;
    }
    // rows that see nothing have no gradient: their l is -inf.  Far rows weigh nothing here
    const float lse = mine ? a.lse_in[tok * a.hq + head] : -kInf;
    const bool far = lse_is_far(lse);
    const float lse2 = lse == -kInf || far ? kInf : lse * kLog2e;
    const int any_far = __any(far) ? 1 : 0;
    if (split == 0 && lane == 0) a.flags[((int64_t)slot * a.hkv + hk) * NW + wave] = any_far;
    if (!a.gq) return;   // only delta is wanted
    load_columns<T, DP, FAST>(qf, (const T*)a.q + tok * a.q_ts + (int64_t)head * a.q_hs, a.dk, mine, lane);

    const float* B = BIAS ? a.bias + sk.first : nullptr;
    const float scale2 = a.scale * kLog2e, per_scale = 1.0f / a.scale;
    typedef Copy<T, DP, kStep, FAST ? NW : 1> C;
    C copy;
    uint32_t koff[C::N], voff[C::N];
    const T* knext = (const T*)a.k + (sk.first + (int64_t)t0 * kStep) * a.k_ts + (int64_t)hk * a.k_hs;
    const T* vnext = (const T*)a.v + (sk.first + (int64_t)t0 * kStep) * a.v_ts + (int64_t)hk * a.v_hs;
    // keys and values of step i; what lies at a key that is left out stays out
    auto start = [&](int i, int stage, float b) {
        const int k0 = (t0 + i) * kStep;
        uint64_t out = from_bit(lk - k0);
        if constexpr (BIAS) {
            b = k0 + lane >= lk || b < kLowest ? -kInf : b * per_scale;
            out |= __ballot(b == -kInf);
            if (wave == 0 && lane < kStep) bias_s[stage & 1][0][lane] = Addend<T>::pack(b);
        }
        const uint32_t kat = base + (uint32_t)(stage & (SK - 1)) * TB, vat = base + (uint32_t)(SK + (stage & 1)) * TB;
        if constexpr (FAST) {
            copy.start(knext, koff, kat, out, wave);
            copy.start(vnext, voff, vat, out, wave);
        } else {
#pragma unroll 1
            for (int id = tid; id < kStep * L::NCH; id += 64 * NW) {
                const int row = id / L::NCH, c = id % L::NCH;
                const bool ok = !((out >> row) & 1);
                *(lds_u32x4*)(uintptr_t)(kat + L::at(row, c)) = load_chunk<T, FAST>(knext + row * a.k_ts, c * L::EPC, a.dk, ok);
                *(lds_u32x4*)(uintptr_t)(vat + L::at(row, c)) = load_chunk<T, FAST>(vnext + row * a.v_ts, c * L::EPC, a.dv, ok);
            }
        }
        knext += kStep * a.k_ts;
        vnext += kStep * a.v_ts;
    };
    auto bias_of = [&](int i) -> float {
        const int key = (t0 + i) * kStep + lane;
        return key < lk ? B[key] : 0.0f;
    };
    auto start_bias = [&](int i, int stage) {   // by the first wave
        const int k0 = (t0 + i) * kStep;
        copy4(buffer_of(B + k0), k0 + lane < lk ? (uint32_t)lane * 4u : kNowhere, (uint32_t)(uintptr_t)(lds_f32*)&raw_s[stage][0]);
    };

    Reader<T, DP> rd;
    rd.init(base, lane);
    typedef __attribute__((address_space(3))) Word lds_word;
    const uint32_t bbase = (uint32_t)(uintptr_t)(lds_word*)&bias_s[0][h][lane & 31];
    constexpr int NQ = FINE ? 1 : NT;   // tiles of a query's elements
    floatx16 gq[NQ], s[PIPE ? 2 : 1], dp[PIPE ? 2 : 1];
    Frag sf[PIPE ? 2 : 1][KB], sr[FINE ? 2 : 1][FINE ? KB : 1];
#pragma unroll
    for (int d = 0; d < NQ; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) gq[d][e] = 0.0f;

    auto score = [&](auto stage_c) {
        constexpr int st = decltype(stage_c)::value, sl = st & 1, p = PIPE ? sl : 0;
        s[p] = dp[p] = floatx16{};
        if constexpr (BIAS) s[p] = Addend<T>::spread(*(const lds_word*)(uintptr_t)(bbase + (uint32_t)sizeof(Word) * (2 * sl * kStep)));
#pragma unroll
        for (int c = 0; c < DP / KE; ++c)
            if (worth<T>(c * KE, a.dk)) s[p] = Op<T>::mma(rd.rows((st & (SK - 1)) * TB, 0, c), qf[c], s[p]);
#pragma unroll
        for (int c = 0; c < DP / KE; ++c)
            if (worth<T>(c * KE, a.dv)) dp[p] = Op<T>::mma(rd.rows((SK + sl) * TB, 0, c), gf[c], dp[p]);
    };
    auto collect = [&](auto stage_c) {
        constexpr int st = decltype(stage_c)::value;
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int d = 0; d < NQ; ++d)
                if (worth<T>(32 * d, a.dk)) {
                    const Frag k = rd.columns((st & (SK - 1)) * TB, b, d);
                    gq[d] = Op<T>::mma(k, sf[PIPE ? st & 1 : 0][b], gq[d]);
                    if constexpr (FINE) gq[d] = Op<T>::mma(k, sr[st & 1][b], gq[d]);
                }
    };
    float raw = 0.0f;
    auto step = [&](auto stage_c, int i) {
        constexpr int st = decltype(stage_c)::value, sl = st & 1, p = PIPE ? sl : 0;
        constexpr int more = PIPE ? 2 : 1, nsl = PIPE ? sl : sl ^ 1;   // steps ahead, and the parity of that one
        const int k0 = (t0 + i) * kStep;
        // Here is step i + 1, and all waves have left the keys of i - 2 and the values of i
        // (float32: step i is here, and all waves have left step i - 1).
        all_arrived();
        if constexpr (BIAS && !FAST) raw = bias_of(i + more);
        start(i + more, (st + more) & 3, raw);
        if constexpr (BIAS && FAST) {
            if (wave == 0) start_bias(i + more + 2, nsl);
            raw = raw_s[nsl ^ 1][lane];   // of step i + more + 1
        }
        if constexpr (!PIPE) score(std::integral_constant<int, st>());
        if (k0 + kStep > least) {   // some row does not see all of it
            const int room = lim - k0 - 4 * h;
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (8 * (e / 4) + e % 4 >= room) s[p][e] = -kInf;
        }
        if constexpr (PIPE) {
            score(std::integral_constant<int, (st + 1) & 3>());   // behind the last step: not used
            collect(std::integral_constant<int, (st + 3) & 3>());
        }
        floatx16 ds;
#pragma unroll
        for (int e = 0; e < 16; ++e) ds[e] = exp2_fast(fmaf(s[p][e], scale2, -lse2)) * (dp[p][e] - delta);
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            sf[p][b] = Op<T>::from(ds, b * KE / 2);
            if constexpr (FINE) sr[p][b] = Op<T>::rest(ds, b * KE / 2, sf[p][b]);
        }
        if constexpr (!PIPE) collect(std::integral_constant<int, st>());
    };

    if constexpr (FAST) {
        copy.init(wave, lane);
        copy.offsets(koff, a.k_ts, a.dk, lane);
        copy.offsets(voff, a.v_ts, a.dv, lane);
    }
    if (n_steps > 0) {
        float b[2] = {0.0f, 0.0f};
        constexpr int first = PIPE ? 2 : 1;   // steps asked for beforehand
        if constexpr (BIAS) {
            for (int i = 0; i < first; ++i) b[i] = bias_of(i);
            raw = bias_of(first);
        }
        for (int i = 0; i < first; ++i) start(i, i, b[i]);
        if constexpr (BIAS) {
            if (FAST && wave == 0) start_bias(first + 1, (first + 1) & 1);
            if (tid < 2 * kStep) bias_s[tid / kStep][1][tid % kStep] = Word{};
        }
        if constexpr (PIPE) {   // no step before the first: zeros
            for (int i = tid; i < TB / 16; i += 64 * NW)
                *(lds_u32x4*)(uintptr_t)(base + 3 * TB + 16 * i) = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < KB; ++i) {
                sf[1][i] = Frag{};
                if constexpr (FINE) sr[1][i] = Frag{};
            }
            all_arrived();
            score(std::integral_constant<int, 0>());
        }
        int i = 0;
        for (;;) {
            step(std::integral_constant<int, 0>(), i);
            if (++i == n_steps) break;
            step(std::integral_constant<int, 1>(), i);
            if (++i == n_steps) break;
            if constexpr (PIPE) {
                step(std::integral_constant<int, 2>(), i);
                if (++i == n_steps) break;
                step(std::integral_constant<int, 3>(), i);
                if (++i == n_steps) break;
            }
        }
        all_arrived();   // no copy outlives its workgroup
        if constexpr (PIPE) switch (n_steps & 3) {
            case 0: collect(std::integral_constant<int, 3>()); break;
            case 1: collect(std::integral_constant<int, 0>()); break;
            case 2: collect(std::integral_constant<int, 1>()); break;
            default: collect(std::integral_constant<int, 2>()); break;
        }
    }

    if (!mine) return;
    float* part = a.part + (((int64_t)split * a.total_q + tok) * a.hq + head) * a.dk;
    T* out = (T*)a.gq + tok * a.gq_ts + (int64_t)head * a.gq_hs;
#pragma unroll
    for (int d = 0; d < NQ; ++d)
#pragma unroll
        for (int e4 = 0; e4 < 4; ++e4) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = gq[d][4 * e4 + e] * a.scale;
            if (parts > 1) store4<float, FAST>(part, 32 * d + 8 * e4 + 4 * h, a.dk, v);
            else store4<T, FAST>(out, 32 * d + 8 * e4 + 4 * h, a.dk, v);
        }
}

// A workgroup has 32 keys a wave and walks over the rows of all heads that read
// its key head, in steps of 32.  Three steps are under way in a wave, as above: the
// scores and dp of step i + 1, the weights of step i, the gradients' parts of
// step i - 1.  -l and -delta of a row are the first summands of its scores and dp
// (float32: they are added afterwards, where the sums are exact to their own size).
template <typename T, int DP, int NW, bool FAST>
__global__ __launch_bounds__(64 * NW, sizeof(T) == 2 && FAST && DP <= 64 ? 2 : 1) void attn_bwd_kv(AttnArgs a) {
    typedef Tile<T, DP> L;
    typedef typename Op<T>::Frag Frag;
    typedef typename Addend<T>::Word Word;
    constexpr int KE = Op<T>::KE, NT = DP / 32, TK = 32 * NW, KB = 32 / KE, TB = kStep * L::RB;
    constexpr bool PIPE = sizeof(T) == 2;
    constexpr int SR = PIPE ? 4 : 2;   // stages
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * SR * TB];   // of queries, of gradients
    // [stage][-l, -delta][values, zeros for the upper half of the lanes][row]
    __shared__ __attribute__((aligned(16))) Word add_s[2][2][2][kStep];
    __shared__ __attribute__((aligned(16))) float raw_s[2][2][64];
    const uint32_t base = (uint32_t)(uintptr_t)(lds_u8*)&smem[0];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), h = lane >> 5;

    int hk, idx, seq, tile, tiles;
    if (!head_of(blockIdx.x, a.slots * a.splits, a.hkv, a.causal, &hk, &idx)) return;
    // the parts that only the longest tiles have go first
    const int turn = a.splits == 1 ? 0 : idx / a.slots, slot = idx - turn * a.slots, split = a.splits - 1 - turn;
    if (!locate<SHRINKS>(a.causal, a.cu_k, a.n_seq, (int)a.total_k, a.each_k, 1, TK, slot, a.slots, &seq, &tile, &tiles)) return;
    const Span sq = span_of(a.cu_q, seq, a.each_q, (int)a.total_q);
    const Span sk = span_of(a.cu_k, seq, a.each_k, (int)a.total_k);
    const int rows = sq.len * a.G, lk = sk.len, ahead = sk.len - sq.len;

    const int key0 = tile * TK + wave * 32, key = key0 + (lane & 31);
    // the first row that sees the tile's first key, the first that sees this lane's key,
    // and the row from which on all of this wave's are seen
    int r_first = 0, r_mine = 0, r_all = 0;
    if (a.causal) {
        r_first = uniform(min(max(tile * TK - ahead, 0), sq.len) * a.G);
        r_mine = min(max(key - ahead, 0), sq.len) * a.G;
        r_all = uniform(min(max(min(key0 + 31, lk - 1) - ahead, 0), sq.len) * a.G);
    }
    const int b0 = r_first / kStep, all = (rows + kStep - 1) / kStep - b0;
    const int parts = parts_of(a, all);
    if (split >= parts) return;
    const int t0 = b0 + (int)((int64_t)all * split / parts), t1 = b0 + (int)((int64_t)all * (split + 1) / parts);
    const int64_t tok = sk.first + key;
    Frag kf[DP / KE], vf[DP / KE];
    bool seen = key < lk;
    if (a.splits > 1 && split == 0 && h == 0 && seen) a.count[tok * a.hkv + hk] = parts;
    float bias = 0.0f;
    if (a.bias && seen) bias = bias2(a.bias[tok]);
    seen = seen && bias != -kInf;
    if (!seen) bias = -kInf;
    load_columns<T, DP, FAST>(kf, (const T*)a.k + tok * a.k_ts + (int64_t)hk * a.k_hs, a.dk, seen, lane);
    load_columns<T, DP, FAST>(vf, (const T*)a.v + tok * a.v_ts + (int64_t)hk * a.v_hs, a.dv, seen, lane);
    const int n_steps = t1 - t0;
    const float scale2 = a.scale * kLog2e, per_scale = 1.0f / a.scale;

    // Row x from a step's first token on is head x % G of token x / G: x is small,
    // so that a float32 product divides it.
    typedef Copy<T, DP, kStep, FAST ? NW : 1> C;
    C copy;
    copy.init(wave, lane);
    const float per_g = 1.0f / (float)a.G;
    auto split_row = [&](int x, int* t, int* gg) {
        *t = a.G == 1 ? x : (int)(((float)x + 0.5f) * per_g);
        *gg = x - *t * a.G;
    };
    const T* Q = (const T*)a.q + sq.first * a.q_ts + (int64_t)hk * a.G * a.q_hs;
    const T* O = (const T*)a.go + sq.first * a.go_ts + (int64_t)hk * a.G * a.go_hs;
    const int64_t cell0 = sq.first * a.hq + (int64_t)hk * a.G;
    auto first_of = [&](int i, int* token) -> int {   // of step i: its first token, rows past that token's first head
        const int r0 = (t0 + i) * kStep;
        *token = a.G == 1 ? r0 : r0 / a.G;
        return r0 - *token * a.G;
    };
    auto start = [&](int i, int stage) {
        int token;
        const int x0 = first_of(i, &token), r0 = (t0 + i) * kStep;
        const T *q = Q + (int64_t)token * a.q_ts, *o = O + (int64_t)token * a.go_ts;
        const uint32_t qat = base + (uint32_t)stage * TB, oat = base + (uint32_t)(SR + stage) * TB;
        if constexpr (FAST) {
            if (!C::shares(wave)) return;
            const u32x4 qb = buffer_of(q), ob = buffer_of(o);
#pragma unroll
            for (int j = 0; j < C::N; ++j) {
                const int row = copy.row + j * (kStep / C::N), src = ((lane % L::NCH) ^ L::turn(row)) * L::EPC;
                int t, gg;
                split_row(x0 + row, &t, &gg);
                const bool ok = r0 + row < rows;
                const uint32_t qo = ((uint32_t)t * (uint32_t)a.q_ts + (uint32_t)gg * (uint32_t)a.q_hs + src) * (uint32_t)sizeof(T);
                const uint32_t oo = ((uint32_t)t * (uint32_t)a.go_ts + (uint32_t)gg * (uint32_t)a.go_hs + src) * (uint32_t)sizeof(T);
                const uint32_t at = (uint32_t)(j * NW + wave) * 1024u;
                copy16(qb, ok && src < a.dk ? qo : kNowhere, qat + at);
                copy16(ob, ok && src < a.dv ? oo : kNowhere, oat + at);
            }
        } else {
#pragma unroll 1
            for (int id = tid; id < kStep * L::NCH; id += 64 * NW) {
                const int row = id / L::NCH, c = id % L::NCH;
                int t, gg;
                split_row(x0 + row, &t, &gg);
                const bool ok = r0 + row < rows;
                *(lds_u32x4*)(uintptr_t)(qat + L::at(row, c)) =
                    load_chunk<T, FAST>(q + t * a.q_ts + gg * a.q_hs, c * L::EPC, a.dk, ok);
                *(lds_u32x4*)(uintptr_t)(oat + L::at(row, c)) =
                    load_chunk<T, FAST>(o + t * a.go_ts + gg * a.go_hs, c * L::EPC, a.dv, ok);
            }
        }
    };
    // l of a row (lanes 0 .. 31) and delta (lanes 32 .. 63) of step i
    const int row = lane & 31;
    auto raw_of = [&](int i) -> float {
        int token, t, gg;
        const int x0 = first_of(i, &token);
        split_row(x0 + row, &t, &gg);
        if ((t0 + i) * kStep + row >= rows) return 0.0f;
        const int64_t cell = cell0 + (int64_t)(token + t) * a.hq + gg;
        return h == 0 ? a.lse_in[cell] : a.delta[cell];
    };
    auto start_raw = [&](int i, int stage) {   // by the first two waves
        int token, t, gg;
        const int x0 = first_of(i, &token);
        split_row(x0 + row, &t, &gg);
        const bool ok = h == 0 && (t0 + i) * kStep + row < rows;
        const float* p = (wave == 0 ? a.lse_in : a.delta) + cell0 + (int64_t)token * a.hq;
        copy4(buffer_of(p), ok ? (uint32_t)(t * a.hq + gg) * 4u : kNowhere, (uint32_t)(uintptr_t)(lds_f32*)&raw_s[stage][wave][0]);
    };
    auto put = [&](int i, int stage, float v) {   // by the first wave
        const bool ok = (t0 + i) * kStep + row < rows;
        // rows that see nothing weigh nothing, nor do far ones here
        if (h == 0) v = !ok || fabsf(v) >= kFarLse ? -kInf : -v * (PIPE ? per_scale : kLog2e);
        else v = ok ? -v : 0.0f;
        add_s[stage][h][0][row] = Addend<T>::pack(v);
    };

    Reader<T, DP> rd;
    rd.init(base, lane);
    typedef __attribute__((address_space(3))) Word lds_word;
    const uint32_t abase = (uint32_t)(uintptr_t)(lds_word*)&add_s[0][0][h][row];
    constexpr uint32_t kAdd = (uint32_t)sizeof(Word) * 2 * kStep;
    floatx16 gk[NT], gv[NT], s[PIPE ? 2 : 1], dp[PIPE ? 2 : 1];
    Frag pf[PIPE ? 2 : 1][KB], sf[PIPE ? 2 : 1][KB];
#pragma unroll
    for (int d = 0; d < NT; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) gk[d][e] = gv[d][e] = 0.0f;

    auto score = [&](auto stage_c) {
        constexpr int st = decltype(stage_c)::value, p = PIPE ? st & 1 : 0;
        if constexpr (PIPE) {
            s[p] = Addend<T>::spread(*(const lds_word*)(uintptr_t)(abase + kAdd * (2 * p)));
            dp[p] = Addend<T>::spread(*(const lds_word*)(uintptr_t)(abase + kAdd * (2 * p + 1)));
        } else {
            s[p] = dp[p] = floatx16{};
        }
#pragma unroll
        for (int c = 0; c < DP / KE; ++c)
            if (worth<T>(c * KE, a.dk)) s[p] = Op<T>::mma(rd.rows(st * TB, 0, c), kf[c], s[p]);
#pragma unroll
        for (int c = 0; c < DP / KE; ++c)
            if (worth<T>(c * KE, a.dv)) dp[p] = Op<T>::mma(rd.rows((SR + st) * TB, 0, c), vf[c], dp[p]);
    };
    auto collect = [&](auto stage_c) {
        constexpr int st = decltype(stage_c)::value, p = PIPE ? st & 1 : 0;
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int d = 0; d < NT; ++d) {
                if (worth<T>(32 * d, a.dv)) gv[d] = Op<T>::mma(rd.columns((SR + st) * TB, b, d), pf[p][b], gv[d]);
                if (worth<T>(32 * d, a.dk)) gk[d] = Op<T>::mma(rd.columns(st * TB, b, d), sf[p][b], gk[d]);
            }
    };
    float raw = 0.0f;
    auto step = [&](auto stage_c, int i) {
        constexpr int st = decltype(stage_c)::value, sl = st & 1, p = PIPE ? sl : 0;
        constexpr int more = PIPE ? 2 : 1, nsl = PIPE ? sl : sl ^ 1;   // steps ahead, and the parity of that one
        const int r0 = (t0 + i) * kStep;
        // Here is step i + 1, and all waves have left step i - 2 (float32: step i is here,
        // and all waves have left step i - 1).
        all_arrived();
        start(i + more, (st + more) & (SR - 1));
        if constexpr (!FAST) raw = raw_of(i + more);
        if (wave == 0) put(i + more, nsl, raw);
        if constexpr (FAST) {
            if (wave < 2) start_raw(i + more + 2, nsl);
            raw = raw_s[nsl ^ 1][h][row];   // of step i + more + 1
        }
        if constexpr (!PIPE) score(std::integral_constant<int, st>());
        if (r0 < r_all) {   // some row does not see all keys of this wave
            const int hidden = r_mine - r0 - 4 * h;
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (8 * (e / 4) + e % 4 < hidden) s[p][e] = -kInf;
        }
        floatx16 w, ds;
        if constexpr (PIPE) {
            score(std::integral_constant<int, (st + 1) & 3>());   // behind the last step: not used
            collect(std::integral_constant<int, (st + 3) & 3>());
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                w[e] = exp2_fast(fmaf(s[p][e], scale2, bias));
                ds[e] = w[e] * dp[p][e];
            }
        } else {
            const uint32_t at = (uint32_t)(uintptr_t)(lds_f32*)&add_s[sl][0][0][4 * h];
#pragma unroll
            for (int e4 = 0; e4 < 4; ++e4) {
                const floatx4 l4 = *(const lds_f32x4*)(uintptr_t)(at + 32 * e4);
                const floatx4 d4 = *(const lds_f32x4*)(uintptr_t)(at + kAdd + 32 * e4);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[4 * e4 + e] = exp2_fast(fmaf(s[p][4 * e4 + e], scale2, bias + l4[e]));
                    ds[4 * e4 + e] = w[4 * e4 + e] * (dp[p][4 * e4 + e] + d4[e]);
                }
            }
        }
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            pf[p][b] = Op<T>::from(w, b * KE / 2);
            sf[p][b] = Op<T>::from(ds, b * KE / 2);
        }
        if constexpr (!PIPE) collect(std::integral_constant<int, st>());
    };

    if (n_steps > 0) {
        constexpr int first = PIPE ? 2 : 1;   // steps asked for beforehand
        float r[2] = {0.0f, 0.0f};
        for (int i = 0; i < first; ++i) r[i] = raw_of(i);
        raw = raw_of(first);
        for (int i = 0; i < first; ++i) {
            start(i, i);
            if (wave == 0) put(i, i, r[i]);
        }
        if constexpr (FAST)
            if (wave < 2) start_raw(first + 1, (first + 1) & 1);
        if (tid < 4 * kStep) add_s[tid >> 6][(tid >> 5) & 1][1][tid & 31] = Word{};
        if constexpr (PIPE) {   // no step before the first: zeros
            for (int i = tid; i < TB / 16; i += 64 * NW) {
                *(lds_u32x4*)(uintptr_t)(base + 3 * TB + 16 * i) = u32x4{0, 0, 0, 0};
                *(lds_u32x4*)(uintptr_t)(base + 7 * TB + 16 * i) = u32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int i = 0; i < KB; ++i) pf[1][i] = sf[1][i] = Frag{};
            all_arrived();
            score(std::integral_constant<int, 0>());
        }
        int i = 0;
        for (;;) {
            step(std::integral_constant<int, 0>(), i);
            if (++i == n_steps) break;
            step(std::integral_constant<int, 1>(), i);
            if (++i == n_steps) break;
            if constexpr (PIPE) {
                step(std::integral_constant<int, 2>(), i);
                if (++i == n_steps) break;
                step(std::integral_constant<int, 3>(), i);
                if (++i == n_steps) break;
            }
        }
        all_arrived();   // no copy outlives its workgroup
        if constexpr (PIPE) switch (n_steps & 3) {
            case 0: collect(std::integral_constant<int, 3>()); break;
            case 1: collect(std::integral_constant<int, 0>()); break;
            case 2: collect(std::integral_constant<int, 1>()); break;
            default: collect(std::integral_constant<int, 2>()); break;
        }
    }

    if (key >= lk) return;
    const int64_t cell = ((int64_t)split * a.total_k + tok) * a.hkv + hk;
    float *pk = a.part + cell * a.dk, *pv = a.part2 + cell * a.dv;
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
                x[e] = gk[d][4 * e4 + e] * a.scale;
                y[e] = gv[d][4 * e4 + e];
            }
            if (parts > 1) {
                store4<float, FAST>(pk, d0, a.dk, x);
                store4<float, FAST>(pv, d0, a.dv, y);
            } else {
                store4<T, FAST>(ok, d0, a.dk, x);
                store4<T, FAST>(ov, d0, a.dv, y);
            }
        }
}

// A tile of kStep rows ts apart into LDS, past d and in rows of `out` zeros
template <typename T, int DP, int NW, bool FAST>
__device__ __forceinline__ void load_tile(const T* p, int64_t ts, int d, uint32_t at, uint64_t out) {
    typedef Tile<T, DP> L;
#pragma unroll 1
    for (int id = threadIdx.x; id < kStep * L::NCH; id += 64 * NW) {
        const int row = id / L::NCH, c = id % L::NCH;
        *(lds_u32x4*)(uintptr_t)(at + L::at(row, c)) = load_chunk<T, FAST>(p + row * ts, c * L::EPC, d, !((out >> row) & 1));
    }
}

// gq of far rows: the maximum and the sum of their scores over all keys, which the
// kernel of gk and gv needs too, then their part of gq, a step at a time.
template <typename T, int DP, int NW, bool FAST, bool FINE>
__global__ __launch_bounds__(64 * NW) void attn_far_q(AttnArgs a) {
    typedef Tile<T, DP> L;
    typedef typename Op<T>::Frag Frag;
    constexpr int KE = Op<T>::KE, NT = FINE ? 1 : DP / 32, TR = 32 * NW, KB = 32 / KE, TB = kStep * L::RB;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * TB];
    const uint32_t base = (uint32_t)(uintptr_t)(lds_u8*)&smem[0];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), h = lane >> 5;
    int hk, idx, seq, tile, tiles;
    if (!head_of(blockIdx.x, a.slots, a.hkv, a.causal, &hk, &idx)) return;
    int* flags = a.flags + ((int64_t)idx * a.hkv + hk) * NW;
    int any = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) any |= flags[i];
    if (!uniform(any)) return;
    if (!locate<GROWS>(a.causal, a.cu_q, a.n_seq, (int)a.total_q, a.each_q, a.G, TR, idx, a.slots, &seq, &tile, &tiles)) {
        if (threadIdx.x < NW) flags[threadIdx.x] = 0;   // no tile: what the workspace held
        return;
    }
    const Span sq = span_of(a.cu_q, seq, a.each_q, (int)a.total_q), sk = span_of(a.cu_k, seq, a.each_k, (int)a.total_k);
    const int rows = sq.len * a.G, lk = sk.len, ahead = sk.len - sq.len;
    int most = lk;
    if (a.causal) {
        int t_last, unused;
        row_of(min(tile * TR + TR, rows) - 1, a.G, &t_last, &unused);
        most = uniform(min(max(t_last + ahead + 1, 0), lk));
    }
    const int all = (most + kStep - 1) / kStep;
    const int r = tile * TR + wave * 32 + (lane & 31);
    int token, g;
    row_of(r, a.G, &token, &g);
    const int64_t tok = sq.first + token;
    const int head = hk * a.G + g;
    const bool far = r < rows && lse_is_far(a.lse_in[tok * a.hq + head]);
    const float delta = far ? a.delta[tok * a.hq + head] : 0.0f;
    const int lim = a.causal ? min(max(token + ahead + 1, 0), lk) : lk;
    const float scale2 = a.scale * kLog2e, per_scale = 1.0f / a.scale;
    Frag qf[DP / KE], gf[DP / KE];
    load_columns<T, DP, FAST>(qf, (const T*)a.q + tok * a.q_ts + (int64_t)head * a.q_hs, a.dk, far, lane);
    load_columns<T, DP, FAST>(gf, (const T*)a.go + tok * a.go_ts + (int64_t)head * a.go_hs, a.dv, far, lane);
    Reader<T, DP> rd;
    rd.init(base, lane);
    floatx16 gq[NT], s, dp;
#pragma unroll
    for (int d = 0; d < NT; ++d) gq[d] = floatx16{};
    float top = -kInf, sum = 0.0f, inv = 0.0f;
    const bool gradient = a.gq != nullptr;
    // once for the maximum and the sum, then for gq
    for (int pass = 0; pass < (gradient ? 2 : 1); ++pass) {
        for (int i = 0; i < all; ++i) {
            const int k0 = i * kStep, key = k0 + (lane & 31);
            float b = 0.0f;
            if (a.bias) b = key < lk ? a.bias[sk.first + key] : 0.0f;
            b = key >= lk || b < kLowest ? -kInf : b * per_scale;
            const uint64_t out = __ballot(b == -kInf);
            const int64_t first = sk.first + k0;
            all_arrived();   // all have left the step before
            load_tile<T, DP, NW, FAST>((const T*)a.k + first * a.k_ts + (int64_t)hk * a.k_hs, a.k_ts, a.dk, base, out);
            load_tile<T, DP, NW, FAST>((const T*)a.v + first * a.v_ts + (int64_t)hk * a.v_hs, a.v_ts, a.dv, base + TB, out);
            all_arrived();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                s[e] = __shfl(b, 8 * (e / 4) + 4 * h + e % 4, 64);
                dp[e] = 0.0f;
            }
#pragma unroll
            for (int c = 0; c < DP / KE; ++c) s = Op<T>::mma(rd.rows(0, 0, c), qf[c], s);
            const int room = lim - k0 - 4 * h;
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (8 * (e / 4) + e % 4 >= room) s[e] = -kInf;
            if (pass == 0) {
                float mx = s[0];
#pragma unroll
                for (int e = 1; e < 16; ++e) mx = fmaxf(mx, s[e]);
                mx = fmaxf(top, half_max(mx));
                if (mx != -kInf) {
                    sum *= exp2_fast((top - mx) * scale2);
                    top = mx;
#pragma unroll
                    for (int e = 0; e < 16; ++e) sum += exp2_fast((s[e] - top) * scale2);
                }
                continue;
            }
#pragma unroll
            for (int c = 0; c < DP / KE; ++c) dp = Op<T>::mma(rd.rows(TB, 0, c), gf[c], dp);
            floatx16 ds;
#pragma unroll
            for (int e = 0; e < 16; ++e) ds[e] = far ? exp2_fast((s[e] - top) * scale2) * inv * (dp[e] - delta) : 0.0f;
#pragma unroll
            for (int k = 0; k < KB; ++k) {
                const Frag w = Op<T>::from(ds, k * KE / 2);
#pragma unroll
                for (int d = 0; d < NT; ++d) gq[d] = Op<T>::mma(rd.columns(0, k, d), w, gq[d]);
                if constexpr (FINE) gq[0] = Op<T>::mma(rd.columns(0, k, 0), Op<T>::rest(ds, k * KE / 2, w), gq[0]);
            }
        }
        if (pass) break;
        sum = half_sum(sum);
        inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        if (top == -kInf) top = 0.0f;
        if (h == 0 && far) {
            a.top[tok * a.hq + head] = top;
            a.inv[tok * a.hq + head] = inv;
        }
    }
    if (!gradient || !far) return;
    T* res = (T*)a.gq + tok * a.gq_ts + (int64_t)head * a.gq_hs;
#pragma unroll
    for (int d = 0; d < NT; ++d)
#pragma unroll
        for (int e4 = 0; e4 < 4; ++e4) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = gq[d][4 * e4 + e] * a.scale;
            store4<T, FAST>(res, 32 * d + 8 * e4 + 4 * h, a.dk, v);
        }
}

// gk and gv of tiles that far rows see, once more and of all rows, a step at a time:
//   p = exp2((x - top) scale2 - two) inv
// with the maximum and the sum that attn_far_q left, or with l for other rows.
template <typename T, int DP, int NW, bool FAST>
__global__ __launch_bounds__(64 * NW) void attn_far_kv(AttnArgs a) {
    typedef Tile<T, DP> L;
    typedef typename Op<T>::Frag Frag;
    constexpr int KE = Op<T>::KE, NT = DP / 32, TK = 32 * NW, KB = 32 / KE, TB = kStep * L::RB;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * TB];
    const uint32_t base = (uint32_t)(uintptr_t)(lds_u8*)&smem[0];
    __shared__ int far_s[2][NW];   // which waves have met far rows
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), h = lane >> 5, row = lane & 31;
    int hk, idx, seq, tile, tiles;
    if (!head_of(blockIdx.x, a.slots, a.hkv, a.causal, &hk, &idx)) return;
    auto none = [&](int which, bool met) -> bool {   // in the workgroup
        if (lane == 0) far_s[which][wave] = 0;
        if (met) far_s[which][wave] = 1;
        all_arrived();
        int any = 0;
#pragma unroll
        for (int i = 0; i < NW; ++i) any |= far_s[which][i];
        return !uniform(any);
    };
    bool met = false;   // in the whole call, then among the rows that the tile meets
#pragma unroll 8
    for (int i = tid; i < a.n_flags; i += 64 * NW) met |= a.flags[i] != 0;
    if (none(0, met)) return;
    if (!locate<SHRINKS>(a.causal, a.cu_k, a.n_seq, (int)a.total_k, a.each_k, 1, TK, idx, a.slots, &seq, &tile, &tiles)) return;
    const Span sq = span_of(a.cu_q, seq, a.each_q, (int)a.total_q), sk = span_of(a.cu_k, seq, a.each_k, (int)a.total_k);
    const int rows = sq.len * a.G, lk = sk.len, ahead = sk.len - sq.len;
    const int key = tile * TK + wave * 32 + row;
    int r_first = 0, r_mine = 0;
    if (a.causal) {
        r_first = uniform(min(max(tile * TK - ahead, 0), sq.len) * a.G);
        r_mine = min(max(key - ahead, 0), sq.len) * a.G;
    }
    const int t0 = r_first / kStep, t1 = (rows + kStep - 1) / kStep;
    auto cell_of = [&](int r) -> int64_t {
        int t, g;
        row_of(r, a.G, &t, &g);
        return (sq.first + t) * a.hq + hk * a.G + g;
    };
    met = false;
    for (int r = r_first + tid; r < rows; r += 64 * NW) met |= lse_is_far(a.lse_in[cell_of(r)]);
    if (none(1, met)) return;
    const int64_t tok = sk.first + key;
    const float scale2 = a.scale * kLog2e;
    bool seen = key < lk;
    float b = a.bias && seen ? a.bias[tok] : 0.0f;
    seen = seen && !(b < kLowest);
    b *= 1.0f / a.scale;
    Frag kf[DP / KE], vf[DP / KE];
    load_columns<T, DP, FAST>(kf, (const T*)a.k + tok * a.k_ts + (int64_t)hk * a.k_hs, a.dk, seen, lane);
    load_columns<T, DP, FAST>(vf, (const T*)a.v + tok * a.v_ts + (int64_t)hk * a.v_hs, a.dv, seen, lane);
    Reader<T, DP> rd;
    rd.init(base, lane);
    floatx16 gk[NT], gv[NT], s, dp;
#pragma unroll
    for (int d = 0; d < NT; ++d) gk[d] = gv[d] = floatx16{};
    for (int i = t0; i < t1; ++i) {
        const int r0 = i * kStep;
        all_arrived();   // all have left the step before
#pragma unroll 1
        for (int n = tid; n < kStep * L::NCH; n += 64 * NW) {
            const int at = n / L::NCH, c = n % L::NCH;
            int t, g;
            row_of(r0 + at, a.G, &t, &g);
            const bool ok = r0 + at < rows;
            const int64_t q = sq.first + t, head = hk * a.G + g;
            *(lds_u32x4*)(uintptr_t)(base + L::at(at, c)) =
                load_chunk<T, FAST>((const T*)a.q + q * a.q_ts + head * a.q_hs, c * L::EPC, a.dk, ok);
            *(lds_u32x4*)(uintptr_t)(base + TB + L::at(at, c)) =
                load_chunk<T, FAST>((const T*)a.go + q * a.go_ts + head * a.go_hs, c * L::EPC, a.dv, ok);
        }
        float top = 0.0f, two = kInf, inv = 0.0f, delta = 0.0f;   // of row r0 + row
        if (r0 + row < rows) {
            const int64_t cell = cell_of(r0 + row);
            const float lse = a.lse_in[cell];
            delta = a.delta[cell];
            inv = 1.0f;
            if (lse_is_far(lse)) {
                top = a.top[cell];
                inv = a.inv[cell];
                two = 0.0f;
            } else if (lse != -kInf) {
                two = lse * kLog2e;
            }
        }
        all_arrived();
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = b, dp[e] = 0.0f;
#pragma unroll
        for (int c = 0; c < DP / KE; ++c) {
            s = Op<T>::mma(rd.rows(0, 0, c), kf[c], s);
            dp = Op<T>::mma(rd.rows(TB, 0, c), vf[c], dp);
        }
        floatx16 w, ds;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int at = 8 * (e / 4) + 4 * h + e % 4;   // of the step's rows
            const float x = fmaf(s[e] - __shfl(top, at, 64), scale2, -__shfl(two, at, 64));
            const float f = __shfl(inv, at, 64), di = __shfl(delta, at, 64);
            w[e] = seen && r0 + at >= r_mine ? exp2_fast(x) * f : 0.0f;
            ds[e] = w[e] * (dp[e] - di);
        }
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            const Frag pf = Op<T>::from(w, k * KE / 2), sf = Op<T>::from(ds, k * KE / 2);
#pragma unroll
            for (int d = 0; d < NT; ++d) {
                gv[d] = Op<T>::mma(rd.columns(TB, k, d), pf, gv[d]);
                gk[d] = Op<T>::mma(rd.columns(0, k, d), sf, gk[d]);
            }
        }
    }
    if (key >= lk) return;
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
                x[e] = gk[d][4 * e4 + e] * a.scale;
                y[e] = gv[d][4 * e4 + e];
            }
            store4<T, FAST>(ok, d0, a.dk, x);
            store4<T, FAST>(ov, d0, a.dv, y);
        }
}

// Sums of the parts of one or two tensors [tokens, heads, d], V elements a thread.
// What came in one part is there already; tokens of no sequence stay as they are.
struct Parts {
    const float* part;
    void* out;
    int64_t ts, hs;
    int d;
};

template <typename T, int V>
__global__ __launch_bounds__(256) void attn_sum(Parts a, Parts b, const int32_t* count, int64_t total, int heads, int splits,
                                                const int32_t* cu, int n_seq) {
    const Parts p = blockIdx.y == 0 ? a : b;
    const int groups = (p.d + V - 1) / V;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, cell = id / groups, tok = cell / heads;
    const int d0 = (int)(id - cell * groups) * V, head = (int)(cell - tok * heads);
    if (tok >= total || (cu && (tok < cu[0] || tok >= cu[n_seq]))) return;
    splits = min(count[cell], splits);   // boundaries out of order leave it undefined
    if (splits <= 1) return;
    const int64_t stride = total * heads * p.d;
    const float* q = p.part + cell * p.d + d0;
    float v[V] = {};
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
        float f[V];
        load_v<float, V>(q + s * stride, f);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += f[i];
    }
    store_v<T, V>((T*)p.out + tok * p.ts + (int64_t)head * p.hs + d0, v);
}

template <typename T>
void sum_parts(const Parts& x, const Parts& y, const int32_t* count, int64_t total, int heads, int splits, const int32_t* cu, int n_seq,
               hipStream_t st) {
    KernelTimer timer("attn_sum", st);
    const int v = x.d % 4 || y.d % 4 ? 1 : 4;
    const dim3 grid((unsigned)((total * heads * (std::max(x.d, y.d) / v) + 255) / 256), y.out ? 2 : 1);
    if (v == 4) attn_sum<T, 4><<<grid, 256, 0, st>>>(x, y, count, total, heads, splits, cu, n_seq);
    else attn_sum<T, 1><<<grid, 256, 0, st>>>(x, y, count, total, heads, splits, cu, n_seq);
}

template <typename T, int DP, bool FAST>
int bwd_go(AttnArgs a, hipStream_t st) {
    constexpr int NW = 4;
    a.slots = (int)tile_slots(a.cu_q != nullptr, a.total_q, a.n_seq, a.G, 32 * NW);
    a.splits = a.gq ? a.plan.splits : 1;
    a.chunk = a.plan.chunk;
    a.n_flags = a.slots * a.hkv * NW;
    if (a.total_q > 0) {   // delta, which gk and gv need too
        KernelTimer timer("attn_bwd_q", st);
        const unsigned grid = (unsigned)grid_size((int64_t)a.slots * a.splits, a.hkv);
        constexpr bool TWO = sizeof(T) == 2;
        if (DP == 32 || (TWO && a.dk <= 32)) {
            if (a.bias) attn_bwd_q<T, DP, NW, true, FAST, TWO><<<grid, 64 * NW, 0, st>>>(a);
            else attn_bwd_q<T, DP, NW, false, FAST, TWO><<<grid, 64 * NW, 0, st>>>(a);
        } else if constexpr (DP > 32) {
            if (a.bias) attn_bwd_q<T, DP, NW, true, FAST, false><<<grid, 64 * NW, 0, st>>>(a);
            else attn_bwd_q<T, DP, NW, false, FAST, false><<<grid, 64 * NW, 0, st>>>(a);
        }
    }
    if (a.splits > 1)
        sum_parts<T>({a.part, a.gq, a.gq_ts, a.gq_hs, a.dk}, {}, a.count, a.total_q, a.hq, a.splits, a.cu_q, a.n_seq, st);
    if (a.total_q > 0 && a.total_k > 0) {
        KernelTimer timer("attn_far_q", st);
        const unsigned grid = (unsigned)grid_size(a.slots, a.hkv);
        constexpr bool TWO = sizeof(T) == 2;
        if (DP == 32 || (TWO && a.dk <= 32)) attn_far_q<T, DP, NW, FAST, TWO><<<grid, 64 * NW, 0, st>>>(a);
        else if constexpr (DP > 32) attn_far_q<T, DP, NW, FAST, false><<<grid, 64 * NW, 0, st>>>(a);
    }
    if (a.gk && a.total_k > 0) {
        a.slots = (int)tile_slots(a.cu_k != nullptr, a.total_k, a.n_seq, 1, 32 * NW);
        a.splits = a.plan_kv.splits;
        a.chunk = a.plan_kv.chunk;
        a.part2 = a.part + (size_t)a.splits * a.total_k * a.hkv * a.dk;
        const unsigned grid = (unsigned)grid_size((int64_t)a.slots * a.splits, a.hkv);
        {
            KernelTimer timer("attn_bwd_kv", st);
            attn_bwd_kv<T, DP, NW, FAST><<<grid, 64 * NW, 0, st>>>(a);
        }
        if (a.splits > 1)
            sum_parts<T>({a.part, a.gk, a.gk_ts, a.gk_hs, a.dk}, {a.part2, a.gv, a.gv_ts, a.gv_hs, a.dv}, a.count, a.total_k,
                         a.hkv, a.splits, a.cu_k, a.n_seq, st);
        if (a.total_q > 0) {
            KernelTimer timer("attn_far_kv", st);
            attn_far_kv<T, DP, NW, FAST><<<(unsigned)grid_size(a.slots, a.hkv), 64 * NW, 0, st>>>(a);
        }
    }
    return attn_launched("attention_bwd");
}

template <typename T>
int bwd_typed(const AttnArgs& a, hipStream_t st) {
    if (!a.plan.fast) return bwd_go<T, 128, false>(a, st);
    const int d = std::max(a.dk, a.dv);
    if (d <= 32) return bwd_go<T, 32, true>(a, st);
    if (d <= 64) return bwd_go<T, 64, true>(a, st);
    return bwd_go<T, 128, true>(a, st);
}

}  // namespace

int launch_attention_bwd(const AttnArgs& a, void* stream) {
    hipStream_t st = static_cast<hipStream_t>(stream);
    return a.dtype == DISCO_F32 ? bwd_typed<float>(a, st) : bwd_typed<bf16_t>(a, st);
}

}  // namespace disco
