// Drives the argument checks of training_api.cpp on the host, under the
// sanitizers.  The helpers that live in disco_api.cpp and the launchers are
// stubs: addresses above kDevice count as device memory, and a launcher only
// counts its calls.
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <string>

#include "disco_internal.h"

static std::string g_error;
static int g_launches = 0;
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
    ++g_launches;
    return DISCO_OK;
}
size_t layer_norm_bwd_workspace(int64_t, int C, int64_t) { return (size_t)C * 8; }
int launch_layer_norm_fwd(const void*, int, const void*, const float*, const float*, void*, int, void*, float*,
                          float*, int64_t, int, int64_t, float, void*) {
    ++g_launches;
    return DISCO_OK;
}
int launch_layer_norm_bwd(const void*, int, const void*, int, const float*, const float*, const float*, const void*,
                          void*, int, float*, float*, float*, int64_t, int, int64_t, void*) {
    ++g_launches;
    return DISCO_OK;
}
size_t orthogonalize_workspace(int, int, int) { return 4096; }
int launch_orthogonalize(const OrthoCall& c, void*) {
    if (!std::isfinite(c.keep) || !std::isfinite(c.rate)) std::abort();
    ++g_launches;
    return DISCO_OK;
}
}  // namespace disco

static void expect(int got, int want, const char* what) {
    if (got != want) {
        std::printf("%s: got %d, wanted %d (%s)\n", what, got, want, g_error.c_str());
        std::exit(1);
    }
    if (want < 0 && g_error.empty()) {
        std::printf("%s: no message\n", what);
        std::exit(1);
    }
}

// tensors 16 MB apart
static void* T(int k) { return reinterpret_cast<void*>(kDevice + (uintptr_t)k * (16u << 20)); }
static float* F(int k) { return static_cast<float*>(T(k)); }
static void* at(void* p, intptr_t off) { return static_cast<char*>(p) + off; }

int main() {
    const int OK = DISCO_OK, EI = DISCO_EINVAL, EU = DISCO_EUNSUPPORTED;
    // ---- layer norm forward ----
    auto fwd = [](const void* x, int xd, const void* r, void* y, int yd, void* s, float* m, float* v, int64_t o, int C,
                  int64_t in, float eps) {
        return disco_layer_norm_fwd(x, xd, r, F(20), F(21), y, yd, s, m, v, o, C, in, eps, nullptr);
    };
    expect(fwd(T(0), 0, nullptr, T(1), 1, nullptr, F(2), F(3), 2, 8, 30, 1e-5f), OK, "forward");
    expect(g_launches, 1, "forward launched");
    expect(fwd(T(0), 0, T(4), T(1), 1, T(5), nullptr, nullptr, 2, 8, 30, 0.0f), OK, "with residual");
    expect(fwd(T(0), 2, nullptr, T(1), 1, nullptr, F(2), F(3), 2, 8, 30, 1e-5f), EI, "type");
    expect(fwd(T(0), 0, T(4), T(1), 1, nullptr, F(2), F(3), 2, 8, 30, 1e-5f), EI, "residual without sum");
    expect(fwd(T(0), 0, nullptr, T(1), 1, T(5), F(2), F(3), 2, 8, 30, 1e-5f), EI, "sum without residual");
    expect(fwd(T(0), 0, nullptr, T(1), 1, nullptr, F(2), nullptr, 2, 8, 30, 1e-5f), EI, "half the statistics");
    expect(fwd(T(0), 0, nullptr, T(1), 1, nullptr, F(2), F(3), -1, 8, 30, 1e-5f), EI, "negative size");
    expect(fwd(T(0), 0, nullptr, T(1), 1, nullptr, F(2), F(3), 2, 0, 30, 1e-5f), EI, "no channels");
    expect(fwd(T(0), 0, nullptr, T(1), 1, nullptr, F(2), F(3), INT64_MAX / 2, 8, 30, 1e-5f), EI, "too large");
    expect(fwd(T(0), 0, nullptr, T(1), 1, nullptr, F(2), F(3), 2, 8, 30, -1.0f), EI, "eps < 0");
    expect(fwd(T(0), 0, nullptr, T(1), 1, nullptr, F(2), F(3), 2, 8, 30, NAN), EI, "eps NaN");
    expect(fwd(T(0), 0, nullptr, T(1), 1, nullptr, F(2), F(3), 2, 8, 30, INFINITY), EI, "eps infinite");
    expect(fwd(T(0), 0, nullptr, T(0), 0, nullptr, F(2), F(3), 2, 8, 30, 1e-5f), EI, "in place");
    expect(fwd(T(0), 0, nullptr, at(T(0), 4 * 479), 1, nullptr, F(2), F(3), 2, 8, 30, 1e-5f), EI, "last element shared");
    expect(fwd(T(0), 0, nullptr, at(T(0), 4 * 480), 1, nullptr, F(2), F(3), 2, 8, 30, 1e-5f), OK, "side by side");
    expect(fwd(at(T(0), 2), 0, nullptr, T(1), 1, nullptr, F(2), F(3), 2, 8, 30, 1e-5f), EI, "misaligned float");
    expect(fwd(at(T(0), 2), 1, nullptr, T(1), 1, nullptr, F(2), F(3), 2, 8, 30, 1e-5f), OK, "bfloat16 anywhere");
    expect(fwd(nullptr, 0, nullptr, T(1), 1, nullptr, F(2), F(3), 2, 8, 30, 1e-5f), EI, "x NULL");
    expect(fwd(reinterpret_cast<void*>(64), 0, nullptr, T(1), 1, nullptr, F(2), F(3), 2, 8, 30, 1e-5f), EI, "host x");
    int before = g_launches;
    expect(fwd(nullptr, 0, nullptr, nullptr, 1, nullptr, nullptr, nullptr, 0, 8, 30, 1e-5f), OK, "empty");
    expect(g_launches, before, "empty launches nothing");
    // ---- layer norm backward ----
    auto bwd = [](void* gx, float* gg, float* gb, void* ws, int64_t nws, int64_t o, const void* gsum) {
        return disco_layer_norm_bwd(T(0), 0, T(1), 1, F(2), F(3), F(4), gsum, gx, 0, gg, gb, ws, nws, o, 8, 30,
                                    nullptr);
    };
    expect((int)disco_layer_norm_bwd_workspace(2, 8, 30), 64, "workspace");
    expect((int)disco_layer_norm_bwd_workspace(0, 8, 30), 0, "workspace of nothing");
    expect((int)disco_layer_norm_bwd_workspace(2, 0, 30), EI, "workspace, no channels");
    expect(bwd(T(5), F(6), F(7), T(8), 64, 2, nullptr), OK, "backward");
    expect(bwd(T(5), F(6), F(7), T(8), 63, 2, nullptr), EI, "short workspace");
    expect(bwd(T(5), F(6), F(7), nullptr, 64, 2, nullptr), EI, "no workspace");
    expect(bwd(T(5), F(6), F(7), at(T(8), 8), 64, 2, nullptr), EI, "misaligned workspace");
    expect(bwd(T(5), nullptr, nullptr, nullptr, 0, 2, T(9)), OK, "gx alone needs none");
    expect(bwd(nullptr, nullptr, nullptr, nullptr, 0, 2, nullptr), EI, "nothing to compute");
    expect(bwd(T(9), F(6), F(7), T(8), 64, 2, T(9)), EI, "gx on gsum");
    expect(bwd(T(5), F(6), F(6), T(8), 64, 2, nullptr), EI, "ggamma on gbeta");
    before = g_launches;
    expect(bwd(nullptr, F(6), F(7), nullptr, 0, 0, nullptr), OK, "empty sums");
    expect(g_launches, before + 2, "empty sums are filled");
    // ---- orthogonalisation ----
    auto ortho = [](const void* m, void* o, int b, int r, int c, int steps, const float* co, float eps, void* ws,
                    int64_t nws) { return disco_orthogonalize(m, 1, o, 0, b, r, c, steps, co, eps, ws, nws, nullptr); };
    expect(ortho(T(0), T(1), 2, 30, 40, 5, nullptr, 1e-7f, T(2), 4096), OK, "orthogonalize");
    expect(ortho(T(0), T(1), 2, 30, 40, 5, nullptr, 1e-7f, T(2), 4095), EI, "short workspace");
    expect(ortho(T(0), T(1), -1, 30, 40, 5, nullptr, 1e-7f, T(2), 4096), EI, "negative batch");
    expect(ortho(T(0), T(1), 65536, 1, 1, 5, nullptr, 1e-7f, T(2), 4096), EU, "too many matrices");
    expect(ortho(T(0), T(1), 65535, INT32_MAX, INT32_MAX, 5, nullptr, 1e-7f, T(2), 4096), EI, "too large");
    expect(ortho(T(0), T(1), 2, 30, 40, 0, nullptr, 1e-7f, T(2), 4096), EI, "no steps");
    expect(ortho(T(0), T(1), 2, 30, 40, 65, nullptr, 1e-7f, T(2), 4096), EI, "too many steps");
    expect(ortho(T(0), T(1), 2, 30, 40, 5, nullptr, -1.0f, T(2), 4096), EI, "eps < 0");
    expect(ortho(T(0), T(0), 2, 30, 40, 5, nullptr, 1e-7f, T(2), 4096), EI, "in place");
    expect(ortho(T(0), T(1), 2, 30, 40, 5, nullptr, 1e-7f, T(1), 4096), EI, "workspace on the result");
    const float wild[3] = {50.0f, 0.0f, 0.0f}, nan[3] = {NAN, 0.0f, 0.0f}, mild[3] = {2.0f, -1.5f, 0.5f};
    expect(ortho(T(0), T(1), 2, 30, 40, 5, wild, 1e-7f, T(2), 4096), EU, "growing coefficients");
    expect(ortho(T(0), T(1), 2, 30, 40, 1, wild, 1e-7f, T(2), 4096), EU, "one step of large coefficients");
    expect(ortho(T(0), T(1), 2, 30, 40, 5, nan, 1e-7f, T(2), 4096), EI, "NaN coefficient");
    expect(ortho(T(0), T(1), 2, 30, 40, 64, mild, 1e-7f, T(2), 4096), OK, "other coefficients");
    expect(ortho(nullptr, nullptr, 0, 30, 40, 5, nullptr, 1e-7f, nullptr, 0), OK, "empty");
    expect((int)disco_orthogonalize_workspace(1, 0, 40), 0, "workspace of nothing");
    // ---- the step ----
    auto step = [](const void* g, float* mo, const float* mi, const void* w, int wd, void* wo, void* w16, float lr,
                   float beta) {
        return disco_muon_step(g, 0, mi, mo, w, wd, wo, w16, lr, beta, 1, 0.1f, 1.0f, 2, 30, 40, 5, nullptr, 1e-7f,
                               T(9), 4096, nullptr);
    };
    expect(step(T(0), F(1), F(1), T(2), 0, T(2), T(3), 0.1f, 0.9f), OK, "in place");
    expect(step(T(0), F(4), F(1), T(2), 0, T(5), nullptr, 0.1f, 0.9f), OK, "out of place");
    expect(step(T(2), F(1), F(1), T(2), 0, T(2), nullptr, 0.1f, 0.9f), EI, "gradient is the weight");
    expect(step(T(0), F(1), F(1), T(2), 0, T(1), nullptr, 0.1f, 0.9f), EI, "weights onto the momentum");
    expect(step(T(0), F(1), F(1), T(2), 0, at(T(2), 4), nullptr, 0.1f, 0.9f), EI, "weights shifted onto themselves");
    expect(step(T(0), F(1), F(1), T(2), 0, T(2), T(2), 0.1f, 0.9f), EI, "copy on the weights");
    expect(step(T(0), F(1), F(1), T(2), 1, T(2), T(3), 0.1f, 0.9f), EI, "copy of bfloat16 weights");
    expect(step(T(0), F(1), F(1), T(2), 0, T(2), nullptr, INFINITY, 0.9f), EI, "lr infinite");
    expect(step(T(0), F(1), F(1), T(2), 0, T(2), nullptr, 0.1f, 1.0f), EI, "beta 1");
    expect(step(T(0), F(1), F(1), T(2), 0, T(2), nullptr, 0.1f, NAN), EI, "beta NaN");
    expect(step(T(0), F(1), nullptr, T(2), 0, T(2), nullptr, 0.1f, 0.9f), EI, "no momentum");
    std::puts("training-driver ok");
    return 0;
}
