// C-ABI layer of the layer norm: argument checks before any launch, as in
// disco_api.cpp.
#include <hip/hip_runtime.h>

#include <cmath>

#include "disco_internal.h"

using namespace disco;

namespace {

// One tensor argument: what it is called, where it lies and how long it is.
struct Arg {
    const char* name;
    const void* p;
    int64_t bytes;
    int align;      // of one element
    bool required;
};

// Device, alignment and overlap checks of a call: outputs may overlap nothing.
int check_args(const Arg* ins, int n_in, const Arg* outs, int n_out) {
    int dev = -1;
    int rc = current_device(&dev);
    if (rc != DISCO_OK) return rc;
    for (int k = 0; k < n_in + n_out; ++k) {
        const Arg& a = k < n_in ? ins[k] : outs[k - n_in];
        if (a.p == nullptr && !a.required) continue;
        if ((rc = check_device_ptr(a.p, a.name, dev)) != DISCO_OK) return rc;
        if (reinterpret_cast<uintptr_t>(a.p) % a.align != 0)
            return set_error(DISCO_EINVAL, "%s is not aligned to its element size", a.name);
    }
    for (int i = 0; i < n_out; ++i) {
        if (outs[i].p == nullptr) continue;
        for (int k = 0; k < n_in; ++k)
            if (ins[k].p && overlap(outs[i].p, outs[i].bytes, ins[k].p, ins[k].bytes))
                return set_error(DISCO_EINVAL, "%s overlaps %s", outs[i].name, ins[k].name);
        for (int k = i + 1; k < n_out; ++k)
            if (outs[k].p && overlap(outs[i].p, outs[i].bytes, outs[k].p, outs[k].bytes))
                return set_error(DISCO_EINVAL, "%s overlaps %s", outs[i].name, outs[k].name);
    }
    return DISCO_OK;
}

// outer * C * inner, within what a tensor of float32 can address
int check_norm_sizes(int64_t outer, int32_t C, int64_t inner, int64_t* n) {
    if (outer < 0 || inner < 0 || C < 1)
        return set_error(DISCO_EINVAL, "sizes must be outer >= 0, C >= 1, inner >= 0 (got %lld, %d, "
                         "%lld)", (long long)outer, C, (long long)inner);
    int64_t t = 0;
    if (__builtin_mul_overflow(outer, inner, &t) || __builtin_mul_overflow(t, (int64_t)C, &t) ||
        t > (INT64_MAX >> 4))
        return set_error(DISCO_EINVAL, "outer * C * inner is too large");
    *n = t;
    return DISCO_OK;
}

}  // namespace

extern "C" {

int disco_layer_norm_fwd(const void* x, int x_dtype, const void* residual, const float* gamma,
                         const float* beta, void* y, int y_dtype, void* sum, float* mean,
                         float* rstd, int64_t outer, int32_t C, int64_t inner, float eps,
                         void* stream) {
    clear_error();
    if (!valid_dtype(x_dtype) || !valid_dtype(y_dtype))
        return set_error(DISCO_EINVAL, "unknown dtype code (x %d, y %d)", x_dtype, y_dtype);
    if (!std::isfinite(eps) || eps < 0.0f)
        return set_error(DISCO_EINVAL, "eps must be finite and >= 0 (got %g)", (double)eps);
    if ((residual == nullptr) != (sum == nullptr))
        return set_error(DISCO_EINVAL, "residual and sum must both be given or both be NULL");
    if ((mean == nullptr) != (rstd == nullptr))
        return set_error(DISCO_EINVAL, "mean and rstd must both be given or both be NULL");
    int64_t n = 0;
    int rc = check_norm_sizes(outer, C, inner, &n);
    if (rc != DISCO_OK || n == 0) return rc;
    const int sx = dtype_size(x_dtype), sy = dtype_size(y_dtype);
    const int64_t points = n / C;
    const Arg ins[] = {{"x", x, n * sx, sx, true},
                       {"residual", residual, n * sx, sx, false},
                       {"gamma", gamma, (int64_t)C * 4, 4, false},
                       {"beta", beta, (int64_t)C * 4, 4, false}};
    const Arg outs[] = {{"y", y, n * sy, sy, true},
                        {"sum", sum, n * sx, sx, false},
                        {"mean", mean, points * 4, 4, false},
                        {"rstd", rstd, points * 4, 4, false}};
    if ((rc = check_args(ins, 4, outs, 4)) != DISCO_OK) return rc;
    return launch_layer_norm_fwd(x, x_dtype, residual, gamma, beta, y, y_dtype, sum, mean, rstd,
                                 outer, C, inner, eps, stream);
}

int64_t disco_layer_norm_bwd_workspace(int64_t outer, int32_t C, int64_t inner) {
    clear_error();
    int64_t n = 0;
    const int rc = check_norm_sizes(outer, C, inner, &n);
    if (rc != DISCO_OK) return rc;
    return n == 0 ? 0 : (int64_t)layer_norm_bwd_workspace(outer, C, inner);
}

int disco_layer_norm_bwd(const void* x, int x_dtype, const void* gy, int gy_dtype,
                         const float* mean, const float* rstd, const float* gamma,
                         const void* gsum, void* gx, int gx_dtype, float* ggamma, float* gbeta,
                         void* workspace, int64_t workspace_bytes, int64_t outer, int32_t C,
                         int64_t inner, void* stream) {
    clear_error();
    if (!valid_dtype(x_dtype) || !valid_dtype(gy_dtype) || (gx && !valid_dtype(gx_dtype)))
        return set_error(DISCO_EINVAL, "unknown dtype code (x %d, gy %d, gx %d)", x_dtype, gy_dtype,
                         gx_dtype);
    if (gx == nullptr && ggamma == nullptr && gbeta == nullptr)
        return set_error(DISCO_EINVAL, "gx, ggamma and gbeta are all NULL: nothing to compute");
    int64_t n = 0;
    int rc = check_norm_sizes(outer, C, inner, &n);
    if (rc != DISCO_OK) return rc;
    const int64_t nc = (int64_t)C * 4;
    if (n == 0) {   // empty sums
        const Arg outs[] = {{"ggamma", ggamma, nc, 4, false}, {"gbeta", gbeta, nc, 4, false}};
        if ((rc = check_args(nullptr, 0, outs, 2)) != DISCO_OK) return rc;
        if (ggamma && (rc = launch_fill_zero(ggamma, (size_t)C, stream)) != DISCO_OK) return rc;
        if (gbeta && (rc = launch_fill_zero(gbeta, (size_t)C, stream)) != DISCO_OK) return rc;
        return DISCO_OK;
    }
    const bool params = ggamma != nullptr || gbeta != nullptr;
    const int64_t need = params ? (int64_t)layer_norm_bwd_workspace(outer, C, inner) : 0;
    if (params && (workspace == nullptr || workspace_bytes < need))
        return set_error(DISCO_EINVAL, "the workspace has %lld bytes, %lld are needed",
                         (long long)(workspace ? workspace_bytes : 0), (long long)need);
    const int sx = dtype_size(x_dtype), sg = dtype_size(gy_dtype);
    const int so = gx ? dtype_size(gx_dtype) : 1;
    const int64_t points = n / C;
    const Arg ins[] = {{"x", x, n * sx, sx, true},
                       {"gy", gy, n * sg, sg, true},
                       {"mean", mean, points * 4, 4, true},
                       {"rstd", rstd, points * 4, 4, true},
                       {"gamma", gamma, nc, 4, false},
                       {"gsum", gsum, n * sg, sg, false}};
    const Arg outs[] = {{"gx", gx, n * so, so, false},
                        {"ggamma", ggamma, nc, 4, false},
                        {"gbeta", gbeta, nc, 4, false},
                        {"workspace", params ? workspace : nullptr, need, 16, params}};
    if ((rc = check_args(ins, 6, outs, 4)) != DISCO_OK) return rc;
    return launch_layer_norm_bwd(x, x_dtype, gy, gy_dtype, mean, rstd, gamma, gsum, gx, gx_dtype,
                                 ggamma, gbeta, static_cast<float*>(workspace), outer, C, inner,
                                 stream);
}

}  // extern "C"
