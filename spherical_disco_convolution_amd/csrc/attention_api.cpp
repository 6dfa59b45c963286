// C-ABI layer of the attention, of the norm and rotation of its queries and
// keys, and of dropout: argument checks before any launch, and how a call is cut
// up.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <utility>

#include "api_checks.h"
#include "disco_internal.h"

namespace disco {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// 16-byte accesses, and rows near enough for the 32-bit offsets of a tile's copies
bool wide(const AttnArgs& a) {
    const int epc = a.dtype == DISCO_F32 ? 4 : 8;
    if (a.dk % epc || a.dv % epc) return false;
    for (int64_t s : {a.q_ts, a.q_hs, a.k_ts, a.k_hs, a.v_ts, a.v_hs, a.o_ts, a.o_hs, a.go_ts, a.go_hs, a.gq_ts, a.gq_hs,
                      a.gk_ts, a.gk_hs, a.gv_ts, a.gv_hs})
        if (s % epc) return false;
    for (const void* p : {a.q, a.k, a.v, a.o, a.go, (const void*)a.out, (const void*)a.gq, (const void*)a.gk,
                          (const void*)a.gv})
        if (reinterpret_cast<uintptr_t>(p) % 16) return false;
    const int64_t size = 16 / epc, far = ((int64_t)1 << 31) / size;   // elements
    for (int64_t s : {a.k_ts, a.v_ts})
        if (s >= far / 64) return false;
    if (a.go)   // a step's rows of the gradient of k and v: up to 33 tokens of G heads
        for (const auto& s : {std::make_pair(a.q_ts, a.q_hs), std::make_pair(a.go_ts, a.go_hs)})
            if (s.first >= far / 64 || s.second >= far || 33 * s.first + a.G * s.second + 128 >= far) return false;
    return true;
}

// Parts of the keys in a forward call whose `tiles` workgroups of `steps` steps of `us`
// do not fill the chip; `at_once` of them run together, with 3 us before and after.
// Parts cost the writing and reading of their float32 results, `bytes` a part, and a
// launch.
int parts(int64_t tiles, double steps, double us, int64_t at_once, double bytes) {
    int best = 1;
    double least = 0.0;
    for (int s = 1; s <= 256; s += s < 8 ? 1 : s / 4) {
        if (s > 1 && (steps / s * us < 1.5 || steps / s < 1.5)) break;
        double t = (double)ceil_div(tiles * s, at_once) * (steps / s * us + 3.0);
        if (s > 1) t += 8.0 + s * bytes / 2.5e6;
        if (s == 1 || t < 0.95 * least) {
            best = s;
            least = t;
        }
    }
    return best;
}

// The same for a gradient, whose tiles have up to `full` steps.  Equal ones are cut
// alike (65 x 128 points, 8 heads of 64: 520 workgroups, 512 at once: one part 447 us
// (gk, gv) and 324 us (gq), four 345 and 262, joined in 16 us each).  Where tiles have
// steps of different number, causal ones or of packed sequences, a part has `chunk`
// steps, and only tiles of more are cut: else one with all steps of a sequence of
// several times the mean, which is counted on, ends the call (gk and gv of 7 causal
// series of 6007 tokens, 12 heads of 128 over 4: one part 319 us, four 129).
void cut(const AttnArgs& a, AttnPlan* p, int64_t tiles, int64_t full, double us, int64_t at_once, double bytes) {
    p->splits = 1;
    p->chunk = (int)std::max<int64_t>(full, 1);
    if (!a.ragged && !a.causal) {
        p->splits = parts(tiles, (double)full, us, at_once, bytes);
        p->chunk = (int)std::max<int64_t>(ceil_div(full, p->splits), 1);
        return;
    }
    // the longest sequence and the sum of squares of all, over the mean's
    const double n = a.n_seq, far = a.ragged ? std::min({n, 1.5 + 0.15 * n, 4.0}) : 1.0;
    const double skew = a.ragged ? (far * far + (n - far) * (n - far) / (n - 1.0)) / n : 1.0;
    const double around = at_once > 256 ? 5.0 : 10.0;   // us before and after a workgroup's steps
    const double even = tiles * (full * (a.causal ? 0.5 : 1.0) * us * skew + around) / at_once;
    double least = 0.0;
    for (int s = 1; s <= 256; s += s < 8 ? 1 : s / 4) {
        const double chunk = std::ceil(full * far / s);
        if (s > 1 && (chunk * us < 6.0 || s * bytes > 1e9)) break;
        const double t = std::max(even + 0.35 * chunk * us, chunk * us + around) +
                         (s > 1 ? 5.0 + s * bytes / 11e6 + (1.0 - 1.0 / s) * bytes / 2.5e6 + 2.0 * (s - 1) * tiles / at_once : 0.0);
        if (s == 1 || t < 0.92 * least) {
            p->splits = s;
            p->chunk = (int)chunk;
            least = t;
        }
    }
}

struct Mean {   // of a sequence
    int64_t rows, keys;
};
Mean mean_of(const AttnArgs& a) { return {ceil_div(a.total_q, a.n_seq) * a.G, ceil_div(a.total_k, a.n_seq)}; }

// Microseconds of a step of 32 with `products` matrix products: float32 by the rate
// of its products, bfloat16 as measured for two (forward), three (gq) and four (gk, gv)
double step_us(const AttnArgs& a, int products) {
    if (a.dtype == DISCO_F32) return 0.3 + 0.0073 * products * (a.dk + a.dv);
    const bool wide = std::max(a.dk, a.dv) > 64;
    return products == 2 ? (wide ? 0.6 : 0.4) : products == 3 ? (wide ? 0.9 : 0.6) : wide ? 1.6 : 0.86;
}

double steps_of(const AttnArgs& a, int64_t n) { return (double)ceil_div(n, 32) * (a.causal ? 0.5 : 1.0); }

}  // namespace

AttnPlan attn_plan_fwd(const AttnArgs& a) {
    AttnPlan p{};
    p.fast = wide(a);
    const Mean m = mean_of(a);
    p.waves = !p.fast || m.rows > 64 ? 4 : m.rows > 32 ? 2 : 1;
    const int64_t tiles = a.n_seq * ceil_div(m.rows, 32 * p.waves) * a.hkv;
    // more rows than that fill the chip: 129 x 256 points in two parts were no faster
    p.splits = tiles >= 256 ? 1 : parts(tiles, steps_of(a, m.keys), step_us(a, 2), 512, 4.0 * a.total_q * a.hq * a.dv);
    return p;
}

AttnPlan attn_plan_bwd_q(const AttnArgs& a) {
    AttnPlan p{};
    p.fast = wide(a);
    p.waves = 4;
    const Mean m = mean_of(a);
    cut(a, &p, a.n_seq * ceil_div(m.rows, 128) * a.hkv, ceil_div(m.keys, 32), step_us(a, 3),
        a.dtype == DISCO_F32 && std::max(a.dk, a.dv) > 64 ? 256 : 512, 4.0 * a.total_q * a.hq * a.dk);
    return p;
}

AttnPlan attn_plan_bwd_kv(const AttnArgs& a) {
    AttnPlan p{};
    p.fast = wide(a);
    p.waves = 4;
    const Mean m = mean_of(a);
    const int d = std::max(a.dk, a.dv);
    const bool one = d > 64 || (d > 32 && a.dtype == DISCO_F32);   // workgroup of a compute unit
    cut(a, &p, a.n_seq * ceil_div(m.keys, 128) * a.hkv, ceil_div(m.rows, 32),
        step_us(a, 4), one ? 256 : 512, 4.0 * a.total_k * a.hkv * (a.dk + a.dv));
    return p;
}

namespace {

// A tensor [tokens, heads, d] with strides of its own
struct Rows {
    const char* name;
    const void* p;
    int64_t tokens, heads, d, ts, hs;
    int size;            // of an element
    bool output;

    int64_t bytes() const { return tokens && heads && d ? ((tokens - 1) * ts + (heads - 1) * hs + d) * size : 0; }
    int64_t span() const { return ((heads - 1) * hs + d) * size; }   // of a token
};

int check_rows(const Rows& r) {
    if (r.tokens == 0) return DISCO_OK;
    int64_t a = 0, b = 0, c = 0;
    if (r.ts < 0 || r.hs < 0) return set_error(DISCO_EINVAL, "%s has a negative stride", r.name);
    if (__builtin_mul_overflow(r.tokens - 1, r.ts, &a) || __builtin_mul_overflow(r.heads - 1, r.hs, &b) ||
        __builtin_add_overflow(a, b, &c) || c > (INT64_MAX >> 4))
        return set_error(DISCO_EINVAL, "%s's strides are too large", r.name);
    if (!r.output) return DISCO_OK;
    // rows of a result may not share elements
    const bool by_token = (r.heads == 1 || r.hs >= r.d) && (r.tokens == 1 || r.ts >= (r.heads - 1) * r.hs + r.d);
    const bool by_head = (r.tokens == 1 || r.ts >= r.d) && (r.heads == 1 || r.hs >= (r.tokens - 1) * r.ts + r.d);
    if (!by_token && !by_head) return set_error(DISCO_EINVAL, "%s's rows overlap (strides %lld, %lld)", r.name,
                                                (long long)r.ts, (long long)r.hs);
    return DISCO_OK;
}

// Whether two of them share bytes: columns of one buffer, side by side in each
// token, do not.
bool share(const Rows& x, const Rows& y) {
    if (!x.p || !y.p || x.bytes() == 0 || y.bytes() == 0) return false;
    if (!overlap(x.p, x.bytes(), y.p, y.bytes())) return false;
    const int64_t ts = x.ts * x.size;
    if (x.size != y.size || x.ts != y.ts || x.span() > ts || y.span() > ts) return true;
    int64_t d = (int64_t)(reinterpret_cast<intptr_t>(y.p) - reinterpret_cast<intptr_t>(x.p)) % ts;
    if (d < 0) d += ts;
    return !(d >= x.span() && d + y.span() <= ts);
}

// Device, alignment and overlap of row tensors and of dense ones beside them
int check_tensors(const Rows* rows, int n_rows, const Arg* args, int n_args, const bool* arg_is_output) {
    int dev = -1, rc = current_device(&dev);
    if (rc != DISCO_OK) return rc;
    auto device = [&](const char* name, const void* p, int align) {
        const int r = check_device_ptr(p, name, dev);
        if (r != DISCO_OK) return r;
        if (reinterpret_cast<uintptr_t>(p) % align) return set_error(DISCO_EINVAL, "%s is not aligned to its element size", name);
        return DISCO_OK;
    };
    for (int i = 0; i < n_rows; ++i)
        if (rows[i].bytes() > 0 && (rc = device(rows[i].name, rows[i].p, rows[i].size)) != DISCO_OK) return rc;
    for (int i = 0; i < n_args; ++i) {
        if (args[i].bytes == 0 || (!args[i].p && !args[i].required)) continue;
        if ((rc = device(args[i].name, args[i].p, args[i].align)) != DISCO_OK) return rc;
    }
    for (int i = 0; i < n_rows; ++i) {
        if (!rows[i].output) continue;
        for (int k = 0; k < n_rows; ++k)
            if (k != i && !(rows[k].output && k < i) && share(rows[i], rows[k]))
                return set_error(DISCO_EINVAL, "%s overlaps %s", rows[i].name, rows[k].name);
    }
    for (int i = 0; i < n_args; ++i) {
        if (!args[i].p || args[i].bytes == 0) continue;
        for (int k = 0; k < n_rows; ++k)
            if ((arg_is_output[i] || rows[k].output) && rows[k].p && rows[k].bytes() > 0 &&
                overlap(args[i].p, args[i].bytes, rows[k].p, rows[k].bytes()))
                return set_error(DISCO_EINVAL, "%s overlaps %s", args[i].name, rows[k].name);
        for (int k = 0; k < i; ++k)
            if ((arg_is_output[i] || arg_is_output[k]) && args[k].p && args[k].bytes > 0 &&
                overlap(args[i].p, args[i].bytes, args[k].p, args[k].bytes))
                return set_error(DISCO_EINVAL, "%s overlaps %s", args[i].name, args[k].name);
    }
    return DISCO_OK;
}

int check_desc(const disco_attention_desc* d, AttnArgs* a) {
    if (d == nullptr) return set_error(DISCO_EINVAL, "the description is NULL");
    if (!valid_dtype(d->dtype)) return set_error(DISCO_EINVAL, "unknown dtype code %d", d->dtype);
    if (d->total_q < 0 || d->total_k < 0 || d->n_seq < 1)
        return set_error(DISCO_EINVAL, "sizes must be total_q >= 0, total_k >= 0, n_seq >= 1 (got %lld, %lld, %d)",
                         (long long)d->total_q, (long long)d->total_k, d->n_seq);
    if (d->hq < 1 || d->hkv < 1 || d->hq % d->hkv)
        return set_error(DISCO_EINVAL, "the heads of k and v (%d) must divide the heads of q (%d)", d->hkv, d->hq);
    if (d->dk < 1 || d->dv < 1) return set_error(DISCO_EINVAL, "head sizes must be >= 1 (got %d, %d)", d->dk, d->dv);
    if (d->dk > 128 || d->dv > 128)
        return set_error(DISCO_EUNSUPPORTED, "head sizes of at most 128 (got %d, %d)", d->dk, d->dv);
    // a bias is taken in units of the raw score
    if (!(d->scale >= 1e-6f && d->scale <= 1e6f))
        return set_error(DISCO_EINVAL, "scale must lie in [1e-6, 1e6] (got %g)", (double)d->scale);
    if (d->hq > 65535) return set_error(DISCO_EUNSUPPORTED, "at most 65535 heads (got %d)", d->hq);
    // rows of a tile are counted in 32 bits, the threads of a launch too
    constexpr int64_t kMost = ((int64_t)1 << 30) - 4096;
    if (d->total_k > kMost || d->total_q > kMost || d->total_q * d->hq > kMost || d->total_k * d->hkv > kMost)
        return set_error(DISCO_EUNSUPPORTED, "tokens times heads must stay below 2^30 - 4096");
    *a = AttnArgs{};
    a->dtype = d->dtype;
    a->total_q = d->total_q;
    a->total_k = d->total_k;
    a->n_seq = d->n_seq;
    a->hq = d->hq;
    a->hkv = d->hkv;
    a->G = d->hq / d->hkv;
    a->dk = d->dk;
    a->dv = d->dv;
    a->causal = d->causal != 0;
    a->scale = d->scale;
    // every sequence costs a tile for each key head and split
    if ((int64_t)d->n_seq * d->hkv * 256 > kMost)
        return set_error(DISCO_EUNSUPPORTED, "too many sequences in one call (%d of %d key heads)", d->n_seq, d->hkv);
    a->each_q = (int)(d->total_q / d->n_seq);
    a->each_k = (int)(d->total_k / d->n_seq);
    a->q_ts = d->q_stride[0], a->q_hs = d->q_stride[1];
    a->k_ts = d->k_stride[0], a->k_hs = d->k_stride[1];
    a->v_ts = d->v_stride[0], a->v_hs = d->v_stride[1];
    a->o_ts = d->o_stride[0], a->o_hs = d->o_stride[1];
    return DISCO_OK;
}

int check_boundaries(AttnArgs& a) {
    a.ragged = a.n_seq > 1 && (a.cu_q || a.cu_k);
    if (a.cu_q == nullptr && a.total_q % a.n_seq)
        return set_error(DISCO_EINVAL, "without boundaries n_seq (%d) must divide total_q (%lld)", a.n_seq, (long long)a.total_q);
    if (a.cu_k == nullptr && a.total_k % a.n_seq)
        return set_error(DISCO_EINVAL, "without boundaries n_seq (%d) must divide total_k (%lld)", a.n_seq, (long long)a.total_k);
    return DISCO_OK;
}

int64_t fwd_bytes(const AttnArgs& a) {
    const int64_t splits = a.plan.splits;
    // results, references and sums of each part
    return splits > 1 ? ceil_div(splits * a.total_q * a.hq * (a.dv + 2) * 4, 16) * 16 : 0;
}

int64_t bwd_part_bytes(const AttnArgs& a) {
    int64_t n = 0;
    if (a.plan.splits > 1) n = a.plan.splits * a.total_q * a.hq * a.dk * 4;
    if (a.plan_kv.splits > 1) n = std::max(n, a.plan_kv.splits * a.total_k * a.hkv * (a.dk + a.dv) * 4);
    return n;
}

// how many parts each row of gq, or of gk and gv, came in
int64_t bwd_count_bytes(const AttnArgs& a) { return ceil_div(std::max(a.total_q * a.hq, a.total_k * a.hkv) * 4, 256) * 256; }

// of each of delta, top and inv
int64_t bwd_delta_bytes(const AttnArgs& a) { return ceil_div(a.total_q * a.hq * 4, 256) * 256; }

// of the flags of each wave of a tile of 128 rows, as many as a launch may have (tile_slots)
int64_t bwd_flag_bytes(const AttnArgs& a) {
    return ceil_div((a.total_q * a.G / 128 + a.n_seq) * a.hkv * 16, 256) * 256;
}

int need_workspace(const void* ws, int64_t have, int64_t need) {
    if (need > 0 && (ws == nullptr || have < need))
        return set_error(DISCO_EINVAL, "the workspace has %lld bytes, %lld are needed", (long long)(ws ? have : 0), (long long)need);
    return DISCO_OK;
}

}  // namespace

}  // namespace disco

using namespace disco;

extern "C" {

int64_t disco_attention_fwd_workspace(const disco_attention_desc* desc) {
    clear_error();
    AttnArgs a;
    const int rc = check_desc(desc, &a);
    if (rc != DISCO_OK) return rc;
    int64_t most = 0;   // addresses that are not multiples of 16 bytes are cut up like odd strides
    for (int way = 0; way < 2; ++way) {
        if (way) a.q_ts |= 1;
        a.plan = attn_plan_fwd(a);
        most = std::max(most, fwd_bytes(a));
    }
    return most;
}

int disco_attention_fwd(const disco_attention_desc* desc, const void* q, const void* k, const void* v,
                        const float* key_bias, const int32_t* cu_q, const int32_t* cu_k, void* o, float* lse,
                        void* workspace, int64_t workspace_bytes, void* stream) {
    clear_error();
    AttnArgs a;
    int rc = check_desc(desc, &a);
    if (rc != DISCO_OK) return rc;
    a.q = q, a.k = k, a.v = v, a.bias = key_bias, a.cu_q = cu_q, a.cu_k = cu_k, a.out = o, a.lse = lse;
    if ((rc = check_boundaries(a)) != DISCO_OK) return rc;
    const int s = dtype_size(a.dtype);
    const Rows rows[] = {{"q", q, a.total_q, a.hq, a.dk, a.q_ts, a.q_hs, s, false},
                         {"k", k, a.total_k, a.hkv, a.dk, a.k_ts, a.k_hs, s, false},
                         {"v", v, a.total_k, a.hkv, a.dv, a.v_ts, a.v_hs, s, false},
                         {"o", o, a.total_q, a.hq, a.dv, a.o_ts, a.o_hs, s, true}};
    for (const Rows& r : rows)
        if ((rc = check_rows(r)) != DISCO_OK) return rc;
    if (a.total_q == 0) return DISCO_OK;
    a.plan = attn_plan_fwd(a);
    const int64_t need = fwd_bytes(a), cu = (int64_t)(a.n_seq + 1) * 4;
    if ((rc = need_workspace(workspace, workspace_bytes, need)) != DISCO_OK) return rc;
    const Arg args[] = {{"key_bias", key_bias, a.total_k * 4, 4, false},
                        {"cu_q", cu_q, cu, 4, false},
                        {"cu_k", cu_k, cu, 4, false},
                        {"lse", lse, a.total_q * a.hq * 4, 4, false},
                        {"workspace", need ? workspace : nullptr, need, 16, need > 0}};
    const bool outs[] = {false, false, false, true, true};
    if ((rc = check_tensors(rows, 4, args, 5, outs)) != DISCO_OK) return rc;
    a.part = static_cast<float*>(workspace);
    a.part_lse = a.part + (need ? a.plan.splits * a.total_q * a.hq * a.dv : 0);
    return launch_attention_fwd(a, stream);
}

int64_t disco_attention_bwd_workspace(const disco_attention_desc* desc) {
    clear_error();
    AttnArgs a;
    const int rc = check_desc(desc, &a);
    if (rc != DISCO_OK) return rc;
    int64_t most = 0;   // with boundaries or without
    for (int way = 0; way < 2; ++way) {
        a.ragged = way && a.n_seq > 1;
        a.plan = attn_plan_bwd_q(a);
        a.plan_kv = attn_plan_bwd_kv(a);
        most = std::max(most, bwd_part_bytes(a));
    }
    return 3 * bwd_delta_bytes(a) + bwd_count_bytes(a) + bwd_flag_bytes(a) + most;
}

int disco_attention_bwd(const disco_attention_desc* desc, const void* q, const void* k, const void* v,
                        const float* key_bias, const int32_t* cu_q, const int32_t* cu_k, const void* o,
                        const float* lse, const void* go, void* gq, void* gk, void* gv, void* workspace,
                        int64_t workspace_bytes, void* stream) {
    clear_error();
    AttnArgs a;
    int rc = check_desc(desc, &a);
    if (rc != DISCO_OK) return rc;
    if ((gk == nullptr) != (gv == nullptr) && a.total_k > 0)
        return set_error(DISCO_EINVAL, "gk and gv must both be given or both be NULL");
    if (gq == nullptr && gk == nullptr && a.total_q > 0 && a.total_k > 0)
        return set_error(DISCO_EINVAL, "gq, gk and gv are all NULL: nothing to compute");
    a.q = q, a.k = k, a.v = v, a.bias = key_bias, a.cu_q = cu_q, a.cu_k = cu_k, a.o = o, a.go = go, a.lse_in = lse;
    a.gq = gq, a.gk = gk, a.gv = gv;
    a.go_ts = desc->go_stride[0], a.go_hs = desc->go_stride[1];
    if (gq) a.gq_ts = desc->gq_stride[0], a.gq_hs = desc->gq_stride[1];
    if (gk) {
        a.gk_ts = desc->gk_stride[0], a.gk_hs = desc->gk_stride[1];
        a.gv_ts = desc->gv_stride[0], a.gv_hs = desc->gv_stride[1];
    }
    if ((rc = check_boundaries(a)) != DISCO_OK) return rc;
    const int s = dtype_size(a.dtype);
    const int64_t nq = gq ? a.total_q : 0, nk = gk ? a.total_k : 0;
    const Rows rows[] = {{"q", q, a.total_q, a.hq, a.dk, a.q_ts, a.q_hs, s, false},
                         {"k", k, a.total_k, a.hkv, a.dk, a.k_ts, a.k_hs, s, false},
                         {"v", v, a.total_k, a.hkv, a.dv, a.v_ts, a.v_hs, s, false},
                         {"o", o, a.total_q, a.hq, a.dv, a.o_ts, a.o_hs, s, false},
                         {"go", go, a.total_q, a.hq, a.dv, a.go_ts, a.go_hs, s, false},
                         {"gq", gq, nq, a.hq, a.dk, a.gq_ts, a.gq_hs, s, true},
                         {"gk", gk, nk, a.hkv, a.dk, a.gk_ts, a.gk_hs, s, true},
                         {"gv", gv, nk, a.hkv, a.dv, a.gv_ts, a.gv_hs, s, true}};
    for (const Rows& r : rows)
        if ((rc = check_rows(r)) != DISCO_OK) return rc;
    if (nq == 0 && nk == 0) return DISCO_OK;
    a.plan = attn_plan_bwd_q(a);
    a.plan_kv = attn_plan_bwd_kv(a);
    const int64_t delta = bwd_delta_bytes(a), count = bwd_count_bytes(a), flags = bwd_flag_bytes(a);
    const int64_t need = 3 * delta + count + flags + bwd_part_bytes(a);
    const int64_t cu = (int64_t)(a.n_seq + 1) * 4;
    if ((rc = need_workspace(workspace, workspace_bytes, need)) != DISCO_OK) return rc;
    const Arg args[] = {{"key_bias", key_bias, a.total_k * 4, 4, false},
                        {"cu_q", cu_q, cu, 4, false},
                        {"cu_k", cu_k, cu, 4, false},
                        {"lse", lse, a.total_q * a.hq * 4, 4, true},
                        {"workspace", need ? workspace : nullptr, need, 16, need > 0}};
    const bool outs[] = {false, false, false, false, true};
    if ((rc = check_tensors(rows, 8, args, 5, outs)) != DISCO_OK) return rc;
    a.delta = static_cast<float*>(workspace);
    a.top = a.delta + delta / 4;
    a.inv = a.top + delta / 4;
    a.count = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + 3 * delta);
    a.flags = a.count + count / 4;
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + 3 * delta + count + flags);
    return launch_attention_bwd(a, stream);
}

int64_t disco_qk_norm_rope_bwd_workspace(int32_t d) {
    clear_error();
    if (d < 1 || d > 256) return set_error(d < 1 ? DISCO_EINVAL : DISCO_EUNSUPPORTED, "head sizes of 1 to 256 (got %d)", d);
    return (int64_t)qk_norm_rope_bwd_workspace(d);
}

static int qk_call(const disco_qk_desc* d, QkCall* c) {
    if (d == nullptr) return set_error(DISCO_EINVAL, "the description is NULL");
    if (!valid_dtype(d->dtype)) return set_error(DISCO_EINVAL, "unknown dtype code %d", d->dtype);
    if (d->tokens < 0 || d->hq < 1 || d->hkv < 0 || d->d < 1)
        return set_error(DISCO_EINVAL, "sizes must be tokens >= 0, hq >= 1, hkv >= 0, d >= 1 (got %lld, %d, %d, %d)",
                         (long long)d->tokens, d->hq, d->hkv, d->d);
    if (d->d > 256) return set_error(DISCO_EUNSUPPORTED, "head sizes of at most 256 (got %d)", d->d);
    // up to 64 threads a token, and fewer than 2^32 of a launch
    if (d->tokens > ((int64_t)1 << 26) - 64 || (int64_t)d->hq + d->hkv > 65535)
        return set_error(DISCO_EUNSUPPORTED, "at most 2^26 - 64 tokens and 65535 heads");
    if (d->rot < 0 || d->rot % 2 || d->rot > d->d)
        return set_error(DISCO_EINVAL, "rot must be even and lie in 0..%d (got %d)", d->d, d->rot);
    if (d->axes < 1 || d->axes > 4) return set_error(DISCO_EINVAL, "positions have 1 to 4 axes (got %d)", d->axes);
    if (!std::isfinite(d->eps) || d->eps < 0.0f)
        return set_error(DISCO_EINVAL, "eps must be finite and >= 0 (got %g)", (double)d->eps);
    *c = QkCall{};
    c->dtype = d->dtype;
    c->tokens = d->tokens;
    c->hq = d->hq;
    c->hkv = d->hkv;
    c->d = d->d;
    c->rot = d->rot;
    c->axes = d->axes;
    c->pos_is_int = d->positions_int32 != 0;
    c->interleaved = d->interleaved != 0;
    c->eps = d->eps;
    c->q_ts = d->q_stride[0], c->q_hs = d->q_stride[1];
    c->k_ts = d->k_stride[0], c->k_hs = d->k_stride[1];
    c->qo_ts = d->q_out_stride[0], c->qo_hs = d->q_out_stride[1];
    c->ko_ts = d->k_out_stride[0], c->ko_hs = d->k_out_stride[1];
    c->gq_ts = d->gq_stride[0], c->gq_hs = d->gq_stride[1];
    c->gk_ts = d->gk_stride[0], c->gk_hs = d->gk_stride[1];
    return DISCO_OK;
}

int disco_qk_norm_rope_fwd(const disco_qk_desc* desc, const void* q, const void* k, const float* q_weight,
                           const float* k_weight, const void* positions, const float* inv_freq, void* q_out,
                           void* k_out, void* stream) {
    clear_error();
    QkCall c;
    int rc = qk_call(desc, &c);
    if (rc != DISCO_OK) return rc;
    const int s = dtype_size(c.dtype);
    const int64_t nk = c.hkv ? c.tokens : 0;
    const Rows rows[] = {{"q", q, c.tokens, c.hq, c.d, c.q_ts, c.q_hs, s, false},
                         {"k", k, nk, c.hkv, c.d, c.k_ts, c.k_hs, s, false},
                         {"q_out", q_out, c.tokens, c.hq, c.d, c.qo_ts, c.qo_hs, s, true},
                         {"k_out", k_out, nk, c.hkv, c.d, c.ko_ts, c.ko_hs, s, true}};
    for (const Rows& r : rows)
        if ((rc = check_rows(r)) != DISCO_OK) return rc;
    if (c.tokens == 0) return DISCO_OK;
    const Arg args[] = {{"q_weight", q_weight, (int64_t)c.d * 4, 4, false},
                        {"k_weight", k_weight, (int64_t)c.d * 4, 4, false},
                        {"positions", c.rot ? positions : nullptr, c.tokens * c.axes * 4, 4, c.rot > 0},
                        {"inv_freq", c.rot ? inv_freq : nullptr, (int64_t)c.rot * 2, 4, c.rot > 0}};
    const bool outs[] = {false, false, false, false};
    if ((rc = check_tensors(rows, 4, args, 4, outs)) != DISCO_OK) return rc;
    c.q = q, c.k = k, c.q_weight = q_weight, c.k_weight = k_weight, c.positions = positions, c.inv_freq = inv_freq;
    c.q_out = q_out, c.k_out = k_out;
    return launch_qk_norm_rope(c, stream);
}

int disco_qk_norm_rope_bwd(const disco_qk_desc* desc, const void* q, const void* k, const void* gq_out,
                           const void* gk_out, const float* q_weight, const float* k_weight, const void* positions,
                           const float* inv_freq, void* gq, void* gk, float* gq_weight, float* gk_weight,
                           void* workspace, int64_t workspace_bytes, void* stream) {
    clear_error();
    QkCall c;
    int rc = qk_call(desc, &c);
    if (rc != DISCO_OK) return rc;
    const int s = dtype_size(c.dtype);
    const int64_t nk = c.hkv ? c.tokens : 0, nw = (int64_t)c.d * 4;
    const Rows rows[] = {{"q", q, c.tokens, c.hq, c.d, c.q_ts, c.q_hs, s, false},
                         {"k", k, nk, c.hkv, c.d, c.k_ts, c.k_hs, s, false},
                         {"gq_out", gq_out, c.tokens, c.hq, c.d, c.gq_ts, c.gq_hs, s, false},
                         {"gk_out", gk_out, nk, c.hkv, c.d, c.gk_ts, c.gk_hs, s, false},
                         {"gq", gq, c.tokens, c.hq, c.d, c.qo_ts, c.qo_hs, s, true},
                         {"gk", gk, nk, c.hkv, c.d, c.ko_ts, c.ko_hs, s, true}};
    for (const Rows& r : rows)
        if ((rc = check_rows(r)) != DISCO_OK) return rc;
    const bool weights = gq_weight != nullptr || gk_weight != nullptr;
    const int64_t need = weights && c.tokens ? (int64_t)qk_norm_rope_bwd_workspace(c.d) : 0;
    if ((rc = need_workspace(workspace, workspace_bytes, need)) != DISCO_OK) return rc;
    const Arg args[] = {{"q_weight", q_weight, nw, 4, false},
                        {"k_weight", k_weight, nw, 4, false},
                        {"positions", c.rot ? positions : nullptr, c.tokens * c.axes * 4, 4, c.rot > 0},
                        {"inv_freq", c.rot ? inv_freq : nullptr, (int64_t)c.rot * 2, 4, c.rot > 0 && c.tokens > 0},
                        {"gq_weight", gq_weight, nw, 4, false},
                        {"gk_weight", gk_weight, nw, 4, false},
                        {"workspace", need ? workspace : nullptr, need, 16, need > 0}};
    const bool outs[] = {false, false, false, false, true, true, true};
    if (c.tokens == 0) {   // empty sums
        if (!weights) return DISCO_OK;
        if ((rc = check_tensors(nullptr, 0, args + 4, 2, outs + 4)) != DISCO_OK) return rc;
        if (gq_weight && (rc = launch_fill_zero(gq_weight, (size_t)c.d, stream)) != DISCO_OK) return rc;
        if (gk_weight && (rc = launch_fill_zero(gk_weight, (size_t)c.d, stream)) != DISCO_OK) return rc;
        return DISCO_OK;
    }
    if ((rc = check_tensors(rows, 6, args, 7, outs)) != DISCO_OK) return rc;
    c.backward = 1;
    c.q = q, c.k = k, c.gq = gq_out, c.gk = gk_out, c.q_weight = q_weight, c.k_weight = k_weight;
    c.positions = positions, c.inv_freq = inv_freq, c.q_out = gq, c.k_out = gk;
    c.gq_weight = gq_weight, c.gk_weight = gk_weight;
    c.partial = weights ? static_cast<float*>(workspace) : nullptr;
    return launch_qk_norm_rope(c, stream);
}

static int drop_call(const char* in, const void* x, int x_dtype, const void* residual, const char* out, void* y, int y_dtype,
                     int64_t n, double p, uint64_t seed, uint64_t offset, const int64_t* step, void* stream) {
    clear_error();
    if (!valid_dtype(x_dtype) || !valid_dtype(y_dtype))
        return set_error(DISCO_EINVAL, "unknown dtype code (%s %d, %s %d)", in, x_dtype, out, y_dtype);
    const double t = p >= 0.0 && p <= 1.0 ? std::floor(p * 65536.0 + 0.5) : -1.0;
    if (!(t >= 0.0 && t < 65536.0)) return set_error(DISCO_EINVAL, "p must lie in [0, 1 - 2^-17) (got %g)", p);
    if (n < 0) return set_error(DISCO_EINVAL, "n must be >= 0 (got %lld)", (long long)n);
    if (n > (int64_t)1 << 40) return set_error(DISCO_EUNSUPPORTED, "at most 2^40 elements (got %lld)", (long long)n);
    if (n == 0) return DISCO_OK;
    const int sx = dtype_size(x_dtype), sy = dtype_size(y_dtype);
    const Arg ins[] = {{in, x, n * sx, sx, true}, {"residual", residual, n * sx, sx, false}, {"step", step, 8, 8, false}};
    const Arg outs[] = {{out, y, n * sy, sy, true, sx == sy ? 0 : -1}};
    const int rc = check_args(ins, 3, outs, 1);
    if (rc != DISCO_OK) return rc;
    DropoutCall c{};
    c.x = x, c.x_dtype = x_dtype, c.residual = residual, c.y = y, c.y_dtype = y_dtype, c.n = n;
    c.threshold = (uint32_t)t, c.seed = seed, c.offset = offset, c.step = step;
    return launch_dropout(c, stream);
}

int disco_dropout_fwd(const void* x, int x_dtype, const void* residual, void* y, int y_dtype, int64_t n, double p,
                      uint64_t seed, uint64_t offset, const int64_t* step, void* stream) {
    return drop_call("x", x, x_dtype, residual, "y", y, y_dtype, n, p, seed, offset, step, stream);
}

int disco_dropout_bwd(const void* gy, int gy_dtype, void* gx, int gx_dtype, int64_t n, double p, uint64_t seed,
                      uint64_t offset, const int64_t* step, void* stream) {
    return drop_call("gy", gy, gy_dtype, nullptr, "gx", gx, gx_dtype, n, p, seed, offset, step, stream);
}

}  // extern "C"
