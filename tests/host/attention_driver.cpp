// Drives the argument checks of attention_api.cpp on the host, under the
// sanitizers.  The helpers that live in disco_api.cpp and the launchers are
// stubs: addresses above kDevice count as device memory, and a launcher counts
// its calls and checks that what it is handed fits.
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <string>

#include "disco_internal.h"

static std::string g_error;
static int g_launches = 0, g_fills = 0;
static disco::AttnArgs g_attn;
static const uintptr_t kDevice = 0x100000000ull;

namespace disco {
int set_error(int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    g_error = buf;
    return code;
}
void clear_error() { g_error.clear(); }
int dtype_size(int dt) { return dt == DISCO_F32 ? 4 : (dt == DISCO_BF16 ? 2 : 0); }
bool valid_dtype(int dt) { return dt == DISCO_F32 || dt == DISCO_BF16; }
int check_device_ptr(const void* ptr, const char* name, int) {
    if (ptr == nullptr) return set_error(DISCO_EINVAL, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(ptr) < kDevice) return set_error(DISCO_EINVAL, "%s is host memory", name);
    return DISCO_OK;
}
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    return pa < pb + nb && pb < pa + na;
}
int current_device(int* dev) {
    *dev = 0;
    return DISCO_OK;
}
int launch_fill_zero(float*, size_t, void*) {
    ++g_fills;
    return DISCO_OK;
}
int launch_attention_fwd(const AttnArgs& a, void*) {
    ++g_launches;
    g_attn = a;
    return DISCO_OK;
}
int launch_attention_bwd(const AttnArgs& a, void*) {
    ++g_launches;
    g_attn = a;
    return DISCO_OK;
}
size_t qk_norm_rope_bwd_workspace(int d) { return (size_t)d * 64; }
int launch_qk_norm_rope(const QkCall& c, void*) {
    if (c.rot && (!c.positions || !c.inv_freq)) std::abort();
    ++g_launches;
    return DISCO_OK;
}
int launch_dropout(const DropoutCall& c, void*) {
    if (c.threshold > 65535) std::abort();
    ++g_launches;
    return DISCO_OK;
}
}  // namespace disco

static void expect(int64_t got, int64_t want, const char* what) {
    if (got != want) {
        std::printf("%s: got %lld, wanted %lld (%s)\n", what, (long long)got, (long long)want, g_error.c_str());
        std::exit(1);
    }
    if (want < 0 && g_error.empty()) {
        std::printf("%s: no message\n", what);
        std::exit(1);
    }
}

// tensors 1 GB apart
static void* T(int k) { return reinterpret_cast<void*>(kDevice + (uintptr_t)k * (1u << 30)); }
static float* F(int k) { return static_cast<float*>(T(k)); }
static int32_t* I(int k) { return static_cast<int32_t*>(T(k)); }
static void* at(void* p, intptr_t off) { return static_cast<char*>(p) + off; }

static disco_attention_desc desc(int64_t tq, int64_t tk, int hq = 4, int hkv = 2, int d = 16) {
    disco_attention_desc x{};
    x.total_q = tq, x.total_k = tk, x.n_seq = 1, x.hq = hq, x.hkv = hkv, x.dk = x.dv = d;
    x.dtype = DISCO_BF16, x.scale = 0.25f;
    int64_t* q[] = {x.q_stride, x.o_stride, x.go_stride, x.gq_stride};
    int64_t* k[] = {x.k_stride, x.v_stride, x.gk_stride, x.gv_stride};
    for (int64_t* s : q) s[0] = (int64_t)hq * d, s[1] = d;
    for (int64_t* s : k) s[0] = (int64_t)hkv * d, s[1] = d;
    return x;
}

static int fwd(const disco_attention_desc& d, const void* q = T(0), const void* k = T(1), const void* v = T(2),
               void* o = T(3), float* lse = F(4), void* ws = T(5), int64_t n = 1ll << 29, const int32_t* cq = nullptr,
               const int32_t* ck = nullptr, const float* bias = nullptr) {
    return disco_attention_fwd(&d, q, k, v, bias, cq, ck, o, lse, ws, n, nullptr);
}

static int bwd(const disco_attention_desc& d, void* gq = T(8), void* gk = T(9), void* gv = T(10), void* ws = T(5),
               int64_t n = 1ll << 29, const float* lse = F(4), const void* o = T(3), const void* go = T(7)) {
    return disco_attention_bwd(&d, T(0), T(1), T(2), nullptr, nullptr, nullptr, o, lse, go, gq, gk, gv, ws, n, nullptr);
}

int main() {
    const int OK = DISCO_OK, EI = DISCO_EINVAL, EU = DISCO_EUNSUPPORTED;
    disco_attention_desc d = desc(100, 200);
    // ---- the description ----
    expect(fwd(d), OK, "forward");
    expect(g_launches, 1, "forward launched");
    auto with = [&](auto f) {
        disco_attention_desc x = desc(100, 200);
        f(x);
        return fwd(x);
    };
    expect(with([](auto& x) { x.dtype = 2; }), EI, "type");
    expect(with([](auto& x) { x.n_seq = 0; }), EI, "no sequences");
    expect(with([](auto& x) { x.n_seq = 3; }), EI, "unequal shares");
    expect(with([](auto& x) { x.total_q = -1; }), EI, "negative tokens");
    expect(with([](auto& x) { x.hq = 5; }), EI, "heads");
    expect(with([](auto& x) { x.hkv = 0; }), EI, "no heads");
    expect(with([](auto& x) { x.dk = 0; }), EI, "empty heads");
    expect(with([](auto& x) { x.dv = 129; }), EU, "large heads");
    expect(with([](auto& x) { x.scale = 0.0f; }), EI, "scale 0");
    expect(with([](auto& x) { x.scale = -1.0f; }), EI, "scale < 0");
    expect(with([](auto& x) { x.scale = INFINITY; }), EI, "scale infinite");
    expect(with([](auto& x) { x.total_q = INT32_MAX / 4; }), EU, "too many rows");
    expect(with([](auto& x) { x.hq = x.hkv = 65536; }), EU, "too many heads");
    expect(with([](auto& x) { x.total_q = INT64_MAX; }), EU, "far too many rows");
    expect(with([](auto& x) { x.n_seq = 1 << 28; x.total_q = x.total_k = 0; }), EU, "too many sequences");
    expect(with([](auto& x) { x.q_stride[0] = -64; }), EI, "negative stride");
    expect(with([](auto& x) { x.k_stride[0] = INT64_MAX / 4; }), EI, "stride past 64 bits");
    expect(with([](auto& x) { x.k_stride[1] = 0; }), OK, "one key head for all");
    expect(with([](auto& x) { x.o_stride[1] = 8; }), EI, "results on each other");
    expect(with([](auto& x) { x.o_stride[0] = 0; }), EI, "results on each other, tokens");
    expect(with([](auto& x) { x.o_stride[0] = 16; x.o_stride[1] = 1600; }), OK, "heads first");
    expect(disco_attention_fwd(nullptr, T(0), T(1), T(2), nullptr, nullptr, nullptr, T(3), F(4), nullptr, 0, nullptr), EI,
           "no description");
    // ---- pointers ----
    expect(fwd(d, nullptr), EI, "q NULL");
    expect(fwd(d, T(0), nullptr), EI, "k NULL");
    expect(fwd(d, reinterpret_cast<void*>(64)), EI, "host q");
    expect(fwd(d, at(T(0), 1)), EI, "misaligned q");
    expect(fwd(d, at(T(0), 2)), OK, "any element");
    expect(fwd(d, T(0), T(1), T(2), nullptr), EI, "o NULL");
    expect(fwd(d, T(0), T(1), T(2), T(0)), EI, "o on q");
    expect(fwd(d, T(0), T(1), T(2), at(T(1), 2 * 200 * 32 - 2)), EI, "o on k's last element");
    expect(fwd(d, T(0), T(1), T(2), at(T(1), 2 * 200 * 32)), OK, "o behind k");
    expect(fwd(d, T(0), T(1), T(2), T(3), static_cast<float*>(T(3))), EI, "lse on o");
    expect(fwd(d, T(0), T(1), T(2), T(3), nullptr), OK, "no lse");
    expect(fwd(d, T(0), T(1), T(2), T(3), F(4), T(5), 1ll << 29, I(20), I(21), F(22)), OK, "boundaries and bias");
    expect(fwd(d, T(0), T(1), T(2), T(3), F(4), T(5), 1ll << 29, reinterpret_cast<int32_t*>(64)), EI, "host boundaries");
    {
        disco_attention_desc x = desc(100, 200);
        x.n_seq = 7;
        expect(fwd(x, T(0), T(1), T(2), T(3), F(4), T(5), 1ll << 29, I(20), I(21)), OK, "any shares with boundaries");
        expect(fwd(x, T(0), T(1), T(2), T(3), F(4), T(5), 1ll << 29, I(20)), EI, "boundaries of the queries alone");
    }
    // ---- workspaces ----
    {
        const disco_attention_desc x = desc(8, 30000);
        const int64_t n = disco_attention_fwd_workspace(&x);
        expect(n > 0, 1, "a workspace for parts");
        expect(fwd(x, T(0), T(1), T(2), T(3), F(4), T(5), n), OK, "exact workspace");
        expect(g_attn.part_lse >= g_attn.part, 1, "parts in order");
        expect(fwd(x, T(0), T(1), T(2), T(3), F(4), T(5), n - 1), EI, "short workspace");
        expect(fwd(x, T(0), T(1), T(2), T(3), F(4), nullptr, n), EI, "no workspace");
        expect(fwd(x, T(0), T(1), T(2), T(3), F(4), at(T(5), 8), n), EI, "misaligned workspace");
        expect(fwd(x, T(0), T(1), T(2), T(3), F(4), T(1), n), EI, "workspace on k");
        // the workspace holds what any alignment of the tensors asks for
        for (int tq : {1, 5, 8, 33, 100, 300})
            for (int tk : {1, 64, 1000, 30000})
                for (int g : {1, 4})
                    for (int off : {0, 2}) {
                        const disco_attention_desc y = desc(tq, tk, 2 * g, 2, 64);
                        const int64_t need = disco_attention_fwd_workspace(&y);
                        expect(fwd(y, at(T(0), off), T(1), T(2), T(3), F(4), T(5), need), OK, "forward of any size");
                        const int s = disco::attn_plan_fwd(g_attn).splits;
                        if (s > 1) expect((char*)(g_attn.part_lse + (int64_t)s * tq * 2 * g) <= (char*)T(5) + need, 1, "parts fit");
                        const int64_t nb = disco_attention_bwd_workspace(&y);
                        expect(bwd(y, T(8), T(9), T(10), T(5), nb), OK, "backward of any size");
                        const int sq = disco::attn_plan_bwd_q(g_attn).splits, sk = disco::attn_plan_bwd_kv(g_attn).splits;
                        expect((char*)(g_attn.delta + (int64_t)tq * 2 * g) <= (char*)g_attn.part, 1, "delta fits");
                        if (sq > 1) expect((char*)(g_attn.part + (int64_t)sq * tq * 2 * g * 64) <= (char*)T(5) + nb, 1, "gq's parts fit");
                        if (sk > 1) expect((char*)(g_attn.part + (int64_t)sk * tk * 2 * 128) <= (char*)T(5) + nb, 1, "gk's and gv's parts fit");
                    }
        const disco_attention_desc many = desc(30000, 30000);
        expect(disco_attention_fwd_workspace(&many), 0, "none for many rows");
    }
    int before = g_launches;
    expect(fwd(desc(0, 200), nullptr, T(1), T(2), nullptr, nullptr, nullptr, 0), OK, "no queries");
    expect(g_launches, before, "no queries launch nothing");
    expect(fwd(desc(100, 0), T(0), nullptr, nullptr), OK, "no keys");
    expect(g_launches, before + 1, "no keys are launched: zeros");
    // ---- backward ----
    expect(bwd(d), OK, "backward");
    expect(bwd(d, nullptr), OK, "without gq");
    expect(bwd(d, T(8), nullptr, nullptr), OK, "without gk and gv");
    expect(bwd(d, T(8), nullptr), EI, "gv without gk");
    expect(bwd(d, nullptr, nullptr, nullptr), EI, "nothing to compute");
    expect(bwd(d, T(8), T(9), T(10), nullptr, 0), EI, "backward, no workspace");
    expect(bwd(d, T(8), T(9), T(10), T(5), 1ll << 29, nullptr), EI, "lse NULL");
    expect(bwd(d, T(8), T(9), T(10), T(5), 1ll << 29, F(4), nullptr), EI, "o NULL");
    expect(bwd(d, T(8), T(9), T(10), T(5), 1ll << 29, F(4), T(3), nullptr), EI, "go NULL");
    expect(bwd(d, T(0)), EI, "gq on q");
    expect(bwd(d, T(8), T(9), T(9)), EI, "gk on gv");
    expect(bwd(d, T(8), T(9), T(10), T(9)), EI, "workspace on gk");
    {   // gradients side by side in one buffer of (4 + 2 + 2) * 16 columns
        disco_attention_desc x = desc(100, 100);
        x.gq_stride[0] = x.gk_stride[0] = x.gv_stride[0] = 128;
        expect(bwd(x, T(8), at(T(8), 2 * 64), at(T(8), 2 * 96)), OK, "columns of one buffer");
        expect(bwd(x, T(8), at(T(8), 2 * 63), at(T(8), 2 * 96)), EI, "columns that share an element");
        expect(bwd(x, T(8), at(T(8), 2 * 64), at(T(8), 2 * 97)), EI, "columns past the next token");
    }
    before = g_launches;
    expect(disco_attention_bwd(&(d = desc(0, 0)), nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                               nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr), OK, "backward of nothing");
    expect(g_launches, before, "nothing launched");
    // ---- norm and rotation ----
    disco_qk_desc c{};
    auto qk = [&](auto f, const void* pos = T(4), const float* fr = F(5), void* qo = T(2)) {
        c = disco_qk_desc{};
        c.tokens = 50, c.hq = 4, c.hkv = 2, c.d = 32, c.rot = 16, c.axes = 1, c.eps = 1e-6f;
        for (int64_t* s : {c.q_stride, c.q_out_stride, c.gq_stride}) s[0] = 128, s[1] = 32;
        for (int64_t* s : {c.k_stride, c.k_out_stride, c.gk_stride}) s[0] = 64, s[1] = 32;
        f(c);
        return disco_qk_norm_rope_fwd(&c, T(0), T(1), F(6), nullptr, pos, fr, qo, T(3), nullptr);
    };
    auto same = [](disco_qk_desc&) {};
    expect(qk(same), OK, "norm");
    expect(qk(same, nullptr), EI, "no positions");
    expect(qk(same, T(4), nullptr), EI, "no frequencies");
    expect(qk(same, T(4), F(5), T(0)), EI, "in place");
    expect(qk(same, T(4), F(5), T(3)), EI, "q_out on k_out");
    expect(qk([](auto& x) { x.rot = 0; }, nullptr, nullptr), OK, "no rotation");
    expect(qk([](auto& x) { x.rot = 15; }), EI, "odd rot");
    expect(qk([](auto& x) { x.rot = 34; }), EI, "rot past d");
    expect(qk([](auto& x) { x.axes = 5; }), EI, "axes");
    expect(qk([](auto& x) { x.d = 257; }), EU, "large heads");
    expect(qk([](auto& x) { x.eps = NAN; }), EI, "eps");
    expect(qk([](auto& x) { x.tokens = (int64_t)1 << 26; }), EU, "tokens");
    expect(qk([](auto& x) { x.hkv = 0; }), OK, "queries alone");
    expect(qk([](auto& x) { x.tokens = 0; }, nullptr, nullptr, nullptr), OK, "no tokens");
    qk(same);
    auto qb = [&](float* gw, void* ws, int64_t n, void* gk = T(9)) {
        return disco_qk_norm_rope_bwd(&c, T(0), T(1), T(7), T(11), F(6), F(12), T(4), F(5), T(8), gk, gw, nullptr, ws, n,
                                      nullptr);
    };
    expect(qb(F(10), T(13), 2048), OK, "norm backward");
    expect(qb(F(10), T(13), 2047), EI, "norm backward, short workspace");
    expect(qb(nullptr, nullptr, 0), OK, "without weights' gradients");
    expect(qb(F(10), T(13), 2048, T(8)), EI, "gq on gk");
    expect(qb(F(6), T(13), 2048), EI, "a weight's gradient on the weight");
    c.tokens = 0;
    expect(qb(F(10), nullptr, 0), OK, "norm backward of nothing");
    expect(g_fills, 1, "empty sums are filled");
    // ---- dropout ----
    auto drop = [](const void* x, void* y, int yd, int64_t n, double p, const void* res = nullptr, const int64_t* st = nullptr) {
        return disco_dropout_fwd(x, 1, res, y, yd, n, p, 1, 2, st, nullptr);
    };
    expect(drop(T(0), T(1), 1, 1000, 0.5), OK, "dropout");
    expect(drop(T(0), T(0), 1, 1000, 0.5), OK, "in place");
    expect(drop(T(0), T(0), 0, 1000, 0.5), EI, "in place of another type");
    expect(drop(T(0), at(T(0), 2), 1, 1000, 0.5), EI, "shifted onto itself");
    expect(drop(T(0), T(1), 1, 1000, 0.5, T(1)), EI, "y on the residual");
    expect(drop(T(0), T(1), 1, 1000, 0.5, T(2), reinterpret_cast<int64_t*>(at(T(3), 4))), EI, "misaligned step");
    expect(drop(T(0), T(1), 2, 1000, 0.5), EI, "type");
    expect(drop(T(0), T(1), 1, 1000, 0.999999), EI, "all dropped");
    expect(drop(T(0), T(1), 1, 1000, 1.0 - 1.0 / 131072 - 1e-9), OK, "nearly all dropped");
    expect(drop(nullptr, nullptr, 1, 0, 0.5), OK, "nothing");
    std::puts("attention-driver ok");
    return 0;
}
