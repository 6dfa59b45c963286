// C-ABI layer of the layer norm and the orthogonalised weight update: argument
// checks before any launch, as in disco_api.cpp.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "api_checks.h"
#include "disco_internal.h"

using namespace disco;

namespace {

// Sizes, steps and coefficients of an orthogonalisation; *n = batch * rows * cols.
int check_ortho(int32_t batch, int32_t rows, int32_t cols, int32_t steps, const float* coeffs,
                float eps, float* out_coeffs, int64_t* n) {
    if (batch < 0 || rows < 0 || cols < 0)
        return set_error(DISCO_EINVAL, "sizes must be >= 0 (batch %d, rows %d, cols %d)", batch, rows,
                         cols);
    if (batch > 65535) return set_error(DISCO_EUNSUPPORTED, "more than 65535 matrices in one call");
    int64_t t = (int64_t)rows * cols;
    if (__builtin_mul_overflow(t, (int64_t)batch, &t) || t > (INT64_MAX >> 8))
        return set_error(DISCO_EINVAL, "batch * rows * cols is too large");
    constexpr int32_t kMostSide = INT32_MAX - 63;   // rounded up to 64 in 32 bits
    if (rows > kMostSide || cols > kMostSide)
        return set_error(DISCO_EUNSUPPORTED, "at most %d rows or columns (got %d x %d)", kMostSide, rows, cols);
    *n = t;
    if (steps < 1 || steps > 64)
        return set_error(DISCO_EINVAL, "steps must lie in 1..64 (got %d)", steps);
    if (!std::isfinite(eps) || eps < 0.0f)
        return set_error(DISCO_EINVAL, "eps must be finite and >= 0 (got %g)", (double)eps);
    static const float kDefault[3] = {3.4445f, -4.7750f, 2.0315f};
    const float* c = coeffs ? coeffs : kDefault;
    for (int k = 0; k < 3; ++k) {
        if (!std::isfinite(c[k])) return set_error(DISCO_EINVAL, "a coefficient is not finite");
        out_coeffs[k] = c[k];
    }
    // The singular values start in [0, 1] and go through s (a + b s^2 + c s^4)
    // step by step; X X^T, the polynomial's part in s and a + that part have to
    // stay in the range of the scaled float16 operands (16, 32 and 32; a quarter
    // is left to sampling).
    double hi = 1.0;
    for (int k = 0; k < steps; ++k) {
        double next = 0.0, poly = 0.0;
        for (int q = 0; q <= 64; ++q) {
            const double s = hi * q / 64.0, s2 = s * s, p = s2 * (c[1] + c[2] * s2);
            poly = std::max(poly, std::max(std::fabs(p), std::fabs(c[0] + p)));
            next = std::max(next, std::fabs(s * (c[0] + p)));
        }
        if (hi * hi > 12.0 || poly > 24.0)
            return set_error(DISCO_EUNSUPPORTED, "with these coefficients the singular values reach "
                             "%.3g and the polynomial %.3g at step %d: out of the operands' range",
                             hi, poly, k + 1);
        hi = next;
    }
    return DISCO_OK;
}

// outer * C * inner, within what a tensor of float32 can address
int check_norm_sizes(int64_t outer, int32_t C, int64_t inner, int64_t* n) {
    if (outer < 0 || inner < 0 || C < 1)
        return set_error(DISCO_EINVAL, "sizes must be outer >= 0, C >= 1, inner >= 0 (got %lld, %d, "
                         "%lld)", (long long)outer, C, (long long)inner);
    constexpr int32_t kMostChannels = 1 << 30;   // kernels add up to 2^16 to a channel in 32 bits
    if (C > kMostChannels)
        return set_error(DISCO_EUNSUPPORTED, "at most %d channels (got %d)", kMostChannels, C);
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

int64_t disco_orthogonalize_workspace(int32_t batch, int32_t rows, int32_t cols) {
    clear_error();
    int64_t n = 0;
    float c[3];
    const int rc = check_ortho(batch, rows, cols, 1, nullptr, 0.0f, c, &n);
    if (rc != DISCO_OK) return rc;
    return n == 0 ? 0 : (int64_t)orthogonalize_workspace(batch, rows, cols);
}

int disco_orthogonalize(const void* m, int m_dtype, void* o, int o_dtype, int32_t batch,
                        int32_t rows, int32_t cols, int32_t steps, const float* coeffs, float eps,
                        void* workspace, int64_t workspace_bytes, void* stream) {
    clear_error();
    if (!valid_dtype(m_dtype) || !valid_dtype(o_dtype))
        return set_error(DISCO_EINVAL, "unknown dtype code (m %d, o %d)", m_dtype, o_dtype);
    OrthoCall call{};
    int64_t n = 0;
    int rc = check_ortho(batch, rows, cols, steps, coeffs, eps, call.coeffs, &n);
    if (rc != DISCO_OK || n == 0) return rc;
    const int64_t need = (int64_t)orthogonalize_workspace(batch, rows, cols);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need))
        return set_error(DISCO_EINVAL, "the workspace has %lld bytes, %lld are needed",
                         (long long)(workspace ? workspace_bytes : 0), (long long)need);
    const int sm = dtype_size(m_dtype), so = dtype_size(o_dtype);
    const Arg ins[] = {{"m", m, n * sm, sm, true}};
    const Arg outs[] = {{"o", o, n * so, so, true}, {"workspace", need ? workspace : nullptr, need, 16, need > 0}};
    if ((rc = check_args(ins, 1, outs, 2)) != DISCO_OK) return rc;
    call.m = m;
    call.m_dtype = m_dtype;
    call.o = o;
    call.out_dtype = o_dtype;
    call.batch = batch;
    call.rows = rows;
    call.cols = cols;
    call.steps = steps;
    call.eps = eps;
    call.workspace = workspace;
    return launch_orthogonalize(call, stream);
}

int disco_muon_step(const void* grad, int grad_dtype, const float* momentum, float* momentum_out,
                    const void* w, int w_dtype, void* w_out, void* w16, float lr, float beta,
                    int nesterov, float weight_decay, float scale, int32_t batch, int32_t rows,
                    int32_t cols, int32_t steps, const float* coeffs, float eps, void* workspace,
                    int64_t workspace_bytes, void* stream) {
    clear_error();
    if (!valid_dtype(grad_dtype) || !valid_dtype(w_dtype))
        return set_error(DISCO_EINVAL, "unknown dtype code (grad %d, w %d)", grad_dtype, w_dtype);
    if (!std::isfinite(lr) || !std::isfinite(weight_decay) || !std::isfinite(scale) ||
        !(beta >= 0.0f && beta < 1.0f))
        return set_error(DISCO_EINVAL, "lr, weight_decay and scale must be finite and beta in [0, 1) "
                         "(got %g, %g, %g, %g)", (double)lr, (double)weight_decay, (double)scale,
                         (double)beta);
    if (w16 != nullptr && w_dtype != DISCO_F32)
        return set_error(DISCO_EINVAL, "w16 is the bfloat16 copy of float32 weights");
    OrthoCall call{};
    int64_t n = 0;
    int rc = check_ortho(batch, rows, cols, steps, coeffs, eps, call.coeffs, &n);
    if (rc != DISCO_OK || n == 0) return rc;
    const int64_t need = (int64_t)orthogonalize_workspace(batch, rows, cols);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need))
        return set_error(DISCO_EINVAL, "the workspace has %lld bytes, %lld are needed",
                         (long long)(workspace ? workspace_bytes : 0), (long long)need);
    const int sg = dtype_size(grad_dtype), sw = dtype_size(w_dtype);
    const Arg ins[] = {{"grad", grad, n * sg, sg, true},
                       {"momentum", momentum, n * 4, 4, true},
                       {"w", w, n * sw, sw, true}};
    const Arg outs[] = {{"momentum_out", momentum_out, n * 4, 4, true, 1},
                        {"w_out", w_out, n * sw, sw, true, 2},
                        {"w16", w16, n * 2, 2, false},
                        {"workspace", need ? workspace : nullptr, need, 16, need > 0}};
    if ((rc = check_args(ins, 3, outs, 4)) != DISCO_OK) return rc;
    call.m = grad;
    call.m_dtype = grad_dtype;
    call.momentum = momentum;
    call.momentum_out = momentum_out;
    call.beta = beta;
    call.nesterov = nesterov;
    call.out_dtype = w_dtype;
    call.w = w;
    call.w_out = w_out;
    call.w16 = w16;
    call.keep = (float)(1.0 - (double)lr * weight_decay);
    call.rate = (float)((double)lr * scale);
    call.batch = batch;
    call.rows = rows;
    call.cols = cols;
    call.steps = steps;
    call.eps = eps;
    call.workspace = workspace;
    return launch_orthogonalize(call, stream);
}

}  // extern "C"
