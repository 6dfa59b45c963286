/*
 * disco.h - C ABI of the MI355X (gfx950) forward DISCO convolution on the 2-sphere.
 *
 * The operation (torch_harmonics.DiscreteContinuousConvS2 page, forward
 * equation and the paragraph defining Psi):
 *
 *   g[b,co,j,q] = sum_{ci,k} w[co,ci,k] * sum_{(i,p)} Psi[k,j,(i,p)] * x[b,ci,i,(q*s+p) mod nlon_in]
 *
 * with s = nlon_in / nlon_out.  Psi holds the piecewise-linear filter-basis
 * values at input points seen from the output point (theta'_j, 0) after it is
 * rotated to the north pole, times the quadrature weights; it does not depend
 * on the output longitude q (p-shift symmetry, same page).
 *
 * Conventions shared by every entry point
 *  - Tensors are caller-owned, dense, row-major (C order), and are never
 *    retained or freed by the library:
 *      x   [B, Ci, nlat_in, nlon_in]            (the layer input; page: forward())
 *      xk  [B, Ci, K, nlat_out, nlon_out]       (K-expanded intermediate; the
 *                                                DistributedDiscreteContinuousConvS2
 *                                                page, polar_mode parameter, names this shape)
 *      w   [Co, Ci/groups, K]
 *      y   [B, Co, nlat_out, nlon_out]          (the layer output)
 *      bias [Co] float32, or NULL for no bias.
 *  - Compute entry points take DEVICE pointers on the current HIP device and a
 *    hipStream_t passed as void* (NULL = default stream).  Work is enqueued on
 *    that stream and the call returns without waiting.  Every argument is
 *    checked before anything is launched; a failed check launches nothing.
 *  - Return value: DISCO_OK or a negative DISCO_E* code; disco_last_error()
 *    then gives a message for the calling thread.  The library never aborts
 *    and never falls back to another code path or to the CPU.
 *  - dtype codes: DISCO_F32 (float32) and DISCO_BF16 (bfloat16).  Products
 *    and sums are accumulated in float32.
 */
#ifndef DISCO_H
#define DISCO_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* status codes */
#define DISCO_OK             0
#define DISCO_EINVAL        -1   /* invalid argument (bad size, null pointer, non-divisible groups, ...) */
#define DISCO_EUNSUPPORTED  -2   /* valid request this library does not implement */
#define DISCO_ENOMEM        -3   /* host or device allocation failed */
#define DISCO_EHIP          -4   /* a HIP runtime call or kernel launch failed */

/* element types */
#define DISCO_F32   0
#define DISCO_BF16  1

/* grids (DiscreteContinuousConvS2 page, grid_in / grid_out parameters) */
/* Every grid is a rule in x = cos(theta) over [-1, 1] (weights sum to 2),
 * times 2*pi/nlon per point; nodes ordered from the north pole.  The pages
 * name the last three (DistributedSpectralConvS2 page, grid_in) without
 * defining them; these are the textbook rules of those names. */
#define DISCO_GRID_EQUIANGULAR 0  /* theta_i = pi*i/(nlat-1) (both poles), Clenshaw-Curtis weights */
#define DISCO_GRID_LEGENDRE_GAUSS 1  /* Gauss-Legendre nodes and weights (no poles) */
#define DISCO_GRID_LOBATTO 2      /* Gauss-Lobatto-Legendre nodes (both poles) and weights */
#define DISCO_GRID_EQUIANGULAR_TRAPEZOIDAL 3  /* equiangular nodes, composite trapezoid in x */

/* basis (same page, basis_type / basis_norm_mode parameters) */
#define DISCO_BASIS_PIECEWISE_LINEAR 0
#define DISCO_NORM_NONE 0         /* Psi = basis value * quadrature weight, no further scaling */

typedef struct disco_psi disco_psi;   /* opaque, library-owned, immutable after build */

/* Problem description (same page: in_shape, out_shape, kernel_shape,
 * basis_type, basis_norm_mode, grid_in, grid_out, theta_cutoff). */
typedef struct disco_psi_desc {
    int32_t nlat_in, nlon_in;       /* input grid */
    int32_t nlat_out, nlon_out;     /* output grid; nlon_in must be a multiple of nlon_out */
    int32_t grid_in, grid_out;      /* DISCO_GRID_* */
    int32_t basis_type;             /* DISCO_BASIS_PIECEWISE_LINEAR */
    int32_t basis_norm;             /* DISCO_NORM_NONE */
    int32_t kernel_shape[2];        /* {nr, nphi}: nphi = 0 -> isotropic (nr,), K = nr;
                                       nphi >= 1 -> K = 1 + (nr-1)*nphi */
    double  theta_cutoff;           /* radians, in (0, pi); <= 0 selects (nr+1)*pi/(nlat_out-1) */
} disco_psi_desc;

/* Build Psi on the host in float64 (DiscreteContinuousConvS2 page, Psi
 * paragraph).  No GPU is touched.  On success *out owns a new handle; free it
 * with disco_psi_free.  EINVAL for inconsistent sizes or cutoff, EUNSUPPORTED
 * for unknown grid codes, other bases/normalisations or K > 64, ENOMEM on
 * allocation failure. */
int disco_psi_build(const disco_psi_desc* desc, disco_psi** out);

/* Sizes of a built Psi: number of basis functions K, support points nnz (the
 * (j,i,p) triples with r < theta_cutoff), entries with a basis value above
 * 1e-12 before weighting, and the cutoff actually used.  Any output pointer
 * may be NULL. */
int disco_psi_query(const disco_psi* psi, int32_t* K, int64_t* nnz,
                    int64_t* nnz_nonzero, double* theta_cutoff);

/* Copy the canonical CSR form to caller-owned host arrays:
 * row_ptr [nlat_out+1], in_lat [nnz], lon_off [nnz] (in [0, nlon_in)),
 * vals [nnz, K] float64 (zeros kept).  Entries of each output row are sorted
 * by (in_lat, lon_off).  Any pointer may be NULL to skip that array. */
int disco_psi_export(const disco_psi* psi, int64_t* row_ptr, int32_t* in_lat,
                     int32_t* lon_off, double* vals);

/* Copy the device form of Psi to the current HIP device (allocates device
 * memory owned by the handle).  Must be called before any compute entry point
 * uses the handle.  Calling it again on the same device does nothing;
 * EINVAL if the handle already lives on another device. */
int disco_psi_to_device(disco_psi* psi);

/* Free host and device memory of the handle, including its workspace (it
 * waits for the last call that used the workspace).  NULL is ignored.  The
 * caller must make sure no enqueued work still uses the handle's tables. */
void disco_psi_free(disco_psi* psi);

/* Sparse contraction (the inner sum of the forward equation):
 *   xk[b,c,k,j,q] = sum_{(i,p)} Psi[k,j,(i,p)] * x[b,c,i,(q*s+p) mod nlon_in]
 * x: [B, C, nlat_in, nlon_in] of x_dtype; xk: [B, C, K, nlat_out, nlon_out]
 * of xk_dtype. */
int disco_contract(const disco_psi* psi, const void* x, int x_dtype,
                   void* xk, int xk_dtype, int32_t B, int32_t C, void* stream);

/* Channel/basis contraction (the outer sums of the forward equation):
 *   y[b,co,j,q] = bias[co] + sum_{ci'<Ci/G} sum_k w[co,ci',k] * xk[b, G(co)*Ci/G + ci', k, j, q]
 * with G(co) = co / (Co/G).  EINVAL unless groups divides Ci and Co
 * (DistributedSpectralConvS2 source on the pages raises ValueError for the
 * same condition).  bf16 xk and w with one group of 64 or 128 output
 * channels, Ci*K a multiple of 32 (at least 160 at Co = 128, 192 at Co = 64)
 * and nlat_out*nlon_out a multiple of 8 and at least 256 take a persistent
 * matrix-core kernel that fills one workgroup per compute unit; the
 * environment variable DISCO_EINSUM_PATH=stream selects the double-buffered
 * kernel instead (same sums, float32 accumulation in another order). */
int disco_einsum(const void* xk, int xk_dtype, const void* w, int w_dtype,
                 const float* bias, void* y, int y_dtype,
                 int32_t B, int32_t Ci, int32_t Co, int32_t groups, int32_t K,
                 int32_t nlat_out, int32_t nlon_out, void* stream);

/* Fused forward (DiscreteContinuousConvS2 page, `fused` parameter): the same
 * result as disco_contract followed by disco_einsum, without storing xk in
 * device memory.  x_dtype and w_dtype must be equal.
 *
 * Some layers run in the longitude-spectral form: the forward equation's
 * longitude shift makes each window a circular correlation, so it is
 * evaluated with real DFTs along longitude (a forward transform, the window
 * and channel/basis sums per frequency, an inverse transform), in a
 * workspace of B*Ci*nlat_in*MP*E + B*Co*nlat_out*MP*E bytes with MP =
 * N_in/2 + 1 rounded up to 32 and E = 4 (bf16 spectra) or 8 (float32
 * spectra).
 *
 * Workspace (this call and disco_fused_bwd): the handle keeps one device
 * buffer, allocated with hipMalloc on first need, grown to the largest
 * request and freed by disco_psi_free.  A call that uses it on a stream
 * other than the previous user's first waits for that user's completion
 * event, so calls through one handle are ordered across streams (use one
 * handle per stream for concurrency).  While the stream is being captured
 * into a HIP graph the call takes stream-ordered memory instead
 * (hipMallocAsync / hipFreeAsync nodes that the graph owns).  They are, with N = nlon_in even, N/2 a product of 2, 3
 * and 5 and N <= 1800, groups == 1 and K <= 8:
 *  - bf16 x and w, Ci a multiple of 32, Co 64 or 128, at most 16 input rows
 *    per output row, and stride 1, or stride 2 with N = 720 or 1440 (the
 *    stride-2 output is the stride-1 correlation at every second longitude,
 *    its spectrum folded onto the output grid's frequencies);
 *  - float32 x and w, stride 1, Co <= 128 (both sums on the vector ALUs).
 * The environment variable DISCO_FUSED_PATH=toeplitz selects the direct
 * kernels for them instead.  Rows with 9 to 16 windows (input rows per
 * output row) are summed in two halves of their windows on the 8-window
 * matrix-core kernel when every row has at least two windows;
 * DISCO_SPEC_HALVES=0 selects the 16-window kernel for them instead (same
 * sums, one workgroup per compute unit).  Other layers run the direct kernels: the
 * matrix-core kernel for bf16 layers it accepts, the vector kernels
 * otherwise. */
int disco_fused_fwd(const disco_psi* psi, const void* x, int x_dtype,
                    const void* w, int w_dtype, const float* bias,
                    void* y, int y_dtype, int32_t B, int32_t Ci, int32_t Co,
                    int32_t groups, void* stream);

/* The same result as disco_fused_fwd for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc): this call allocates nothing.  It always takes the
 * direct algorithms (the matrix-core kernel for the bf16 layers it accepts,
 * the vector kernels otherwise; never the longitude-spectral one, whose
 * workspace grows with the grid), and puts the matrix-core kernel's weight
 * fragments (Ci * Co * 16 bytes) in a fixed 4 MiB device array of the
 * library, held on each device it runs on until the process ends.  EINVAL,
 * before any launch, when a layer needs more than those 4 MiB.  Every call
 * on one device shares that array, so calls that overlap on one device
 * (different streams, or other threads) race and must be ordered by the
 * caller. */
int disco_fused_fwd_noalloc(const disco_psi* psi, const void* x, int x_dtype,
                            const void* w, int w_dtype, const float* bias,
                            void* y, int y_dtype, int32_t B, int32_t Ci, int32_t Co,
                            int32_t groups, void* stream);

/* 1 if disco_fused_fwd with these arguments takes the longitude-spectral
 * path described above, 0 if it takes a direct kernel, negative on error
 * (NULL handle or handle not uploaded).  Reads DISCO_FUSED_PATH like the call
 * itself. */
int disco_fused_is_spectral(const disco_psi* psi, int x_dtype, int32_t Ci, int32_t Co,
                            int32_t groups);

/* ---- Gradients ----------------------------------------------------------
 * The layer trains by backpropagation, and its fused mode recomputes the
 * K-expanded intermediate in the backward pass instead of storing it
 * (DiscreteContinuousConvS2 page, `fused` parameter); with fused=False that
 * intermediate is saved for backward (DistributedDiscreteContinuousConvS2
 * page, `fused` parameter).  The forward equation is linear in x and in w, so
 * the gradients below are the adjoints of its two linear maps.  gy is the
 * gradient of the loss with respect to y, [B, Co, nlat_out, nlon_out].  All
 * sums are accumulated in float32; sums over points run in a fixed order, so
 * results are reproducible.  Work is enqueued on `stream`; disco_fused_bwd
 * takes its scratch from the handle's workspace (described at
 * disco_fused_fwd), disco_einsum_grad_w stream-ordered on that stream. */

/* Adjoint of disco_contract:
 *   gx[b,c,i,n] = sum over (j, q, p) with (q*s + p) mod nlon_in = n of
 *                 sum_k Psi[k,j,(i,p)] * gxk[b,c,k,j,q]
 * gxk: [B, C, K, nlat_out, nlon_out] of gxk_dtype; gx: [B, C, nlat_in,
 * nlon_in] of gx_dtype, overwritten.  Each input row is gathered from the
 * windows that reach it (no atomics).  EUNSUPPORTED when K rows of one
 * output row (K * nlon_out floats) exceed 64 KiB. */
int disco_contract_transpose(const disco_psi* psi, const void* gxk, int gxk_dtype, void* gx,
                             int gx_dtype, int32_t B, int32_t C, void* stream);

/* Adjoint of disco_einsum in xk:
 *   gxk[b, G*Ci/G + ci', k, j, q] = sum_{co in group G} w[co,ci',k] * gy[b,co,j,q]
 * gy [B, Co, nlat_out, nlon_out], w [Co, Ci/groups, K], gxk [B, Ci, K,
 * nlat_out, nlon_out]; any dtype combination. */
int disco_einsum_grad_xk(const void* gy, int gy_dtype, const void* w, int w_dtype, void* gxk,
                         int gxk_dtype, int32_t B, int32_t Ci, int32_t Co, int32_t groups,
                         int32_t K, int32_t nlat_out, int32_t nlon_out, void* stream);

/* Adjoint of disco_einsum in w:
 *   gw[co,ci',k] = sum_{b,j,q} gy[b,co,j,q] * xk[b, G(co)*Ci/G + ci', k, j, q]
 * xk [B, Ci, K, nlat_out, nlon_out] (the saved intermediate), gy [B, Co,
 * nlat_out, nlon_out]; gw [Co, Ci/groups, K] float32, overwritten (zeros for
 * B = 0).  Partial sums over chunks of points, then one reduction.  A bf16
 * gy with groups == 1 and nlon_out a multiple of 8 takes the partial sums
 * on the matrix cores, a float32 xk rounded to bf16 as it is read (the
 * bf16 bar); otherwise they run in float32 on the vector ALUs.  The same
 * holds for disco_fused_bwd's gw. */
int disco_einsum_grad_w(const void* xk, int xk_dtype, const void* gy, int gy_dtype, float* gw,
                        int32_t B, int32_t Ci, int32_t Co, int32_t groups, int32_t K,
                        int32_t nlat_out, int32_t nlon_out, void* stream);

/* Fused-mode backward: from x, w and gy, any of
 *   gx    [B, Ci, nlat_in, nlon_in] of gx_dtype = contract^T(einsum_grad_xk(gy, w)),
 *   gw    [Co, Ci/groups, K] float32            = einsum_grad_w(contract(x), gy),
 *   gbias [Co] float32                          = sum_{b,j,q} gy[b,co,j,q],
 * each overwritten; a NULL pointer skips that gradient (not all three).
 * X_K is recomputed in float32, in slabs of at most ceil(nlat_out / 8)
 * output rows (one slab when the layer's two slab tensors take at most
 * 64 MiB), so neither K-expanded tensor is ever held whole.  The exception
 * is gw of a bf16 layer with a bf16 gy and groups == 1 that the matrix-core
 * contraction takes (Ci a multiple of 32, K <= 8, stride 1 or 2, nlon_in and
 * nlon_out multiples of 8, x and gy 16-byte aligned): its X_K is recomputed
 * whole in bf16 on the matrix cores (at most 4 GiB, in the handle's
 * workspace, which keeps it between calls) and grad_w sums it there (the
 * bf16 bar).  Layers on the longitude-spectral path's tables (stride 1, or stride 2 at
 * 720 or 1440 input longitudes) with bf16 x, w and gy, groups == 1, Ci 64 or
 * 128 and Co a multiple of 32 take gx on the longitude-spectral kernels
 * instead: the adjoint of each window's circular correlation is a circular
 * convolution, so gx = irfft(sum over output rows and k of Psi_hat * sum_co
 * w * rfft(gy)) (at stride 2 gy with a zero inserted after each sample),
 * with bf16 spectra and float32 accumulation (the bf16 bar, not float32
 * exactness); DISCO_FUSED_PATH=toeplitz selects the float32 path for them.
 * Float32 stride-1 layers with a float32 gy (groups == 1, Ci <= 128) take
 * gx on the float32 spectral kernels (float32 spectra, the float32 bar).
 * Layers with one input channel per group take gx with the weights folded
 * into the taps (gy contracted directly, no grad_xk), in float32, and, at
 * stride 1 or 2 with K <= 32, gw with no X_K at all: per window the
 * correlation of gy's output row with x's input row, folded with the
 * window's Psi values, in float32. */
int disco_fused_bwd(const disco_psi* psi, const void* x, int x_dtype, const void* w, int w_dtype,
                    const void* gy, int gy_dtype, void* gx, int gx_dtype, float* gw, float* gbias,
                    int32_t B, int32_t Ci, int32_t Co, int32_t groups, void* stream);

/* ---- Layer norm ----------------------------------------------------------
 * Normalisation over the channels, the step that stands before the
 * convolution in a pre-norm residual block.  Tensors are dense and seen as
 * [outer, C, inner]: a field [B, C, nlat, nlon] is outer = B, inner =
 * nlat*nlon; channel-last rows [n, C] are outer = n, inner = 1.  Pointers
 * need the alignment of their element only.  C is at most 2^30 (EUNSUPPORTED
 * past it).  Statistics are float32, the mean first and then the centred
 * squares.  Outputs may not overlap inputs. */

/* Forward:
 *   s = x, or x + residual rounded to x_dtype and stored in `sum`
 *   mean = 1/C sum_c s,  rstd = 1/sqrt(1/C sum_c (s - mean)^2 + eps)
 *   y = (s - mean) * rstd * gamma[c] + beta[c]
 * x, residual, sum: [outer, C, inner] of x_dtype (residual and sum both given
 * or both NULL); gamma, beta: [C] float32, either NULL for ones / zeros; y:
 * [outer, C, inner] of y_dtype; mean, rstd: [outer, inner] float32, both given
 * (the gradient needs them) or both NULL.  outer == 0 or inner == 0 does
 * nothing.  Points are independent: a NaN or an infinity stays in its own. */
int disco_layer_norm_fwd(const void* x, int x_dtype, const void* residual, const float* gamma,
                         const float* beta, void* y, int y_dtype, void* sum, float* mean,
                         float* rstd, int64_t outer, int32_t C, int64_t inner, float eps,
                         void* stream);

/* Bytes of device workspace that disco_layer_norm_bwd needs for ggamma or
 * gbeta (partial sums per workgroup), or a negative status. */
int64_t disco_layer_norm_bwd_workspace(int64_t outer, int32_t C, int64_t inner);

/* Gradients, with h = (x - mean) * rstd and t = gy * gamma[c]:
 *   gx = rstd * (t - 1/C sum_c t - h * 1/C sum_c t*h) + gsum
 *   ggamma[c] = sum_{outer, inner} gy * h,   gbeta[c] = sum_{outer, inner} gy
 * x: what was normalised (the forward's `sum` where it had a residual);
 * gy, gsum: [outer, C, inner] of gy_dtype; gsum is the gradient that reaches
 * that sum past the norm, NULL for none; gx: [outer, C, inner] of gx_dtype or
 * NULL; ggamma, gbeta: [C] float32, either NULL (not all three).  The
 * parameter sums run in a fixed order in float32, so results are
 * reproducible; they need `workspace` (may be NULL when neither is asked
 * for).  An empty tensor gives zero parameter gradients. */
int disco_layer_norm_bwd(const void* x, int x_dtype, const void* gy, int gy_dtype,
                         const float* mean, const float* rstd, const float* gamma,
                         const void* gsum, void* gx, int gx_dtype, float* ggamma, float* gbeta,
                         void* workspace, int64_t workspace_bytes, int64_t outer, int32_t C,
                         int64_t inner, void* stream);

/* ---- Orthogonalised weight updates --------------------------------------
 * The optimiser step for the layer's weights [Co, Ci/groups, K], seen as
 * `batch` = groups matrices of rows = Co/groups by cols = (Ci/groups)*K, one
 * after another.  A matrix M is replaced by the nearby matrix whose singular
 * values are all near one:
 *   X = M / (|M|_F + eps)
 *   steps times: A = X X^T, X <- a X + (b A + c A^2) X      (coeffs = a, b, c)
 * (X^T in X's place where rows > cols: the same map).  Operands are pairs of
 * float16 (22 bits) and sums float32, whatever the types; the result is rounded
 * once to its own, so that a bfloat16 result is the float32 one rounded.  Before
 * that it is within 1e-5 (relative, of the whole matrix) for five default steps; a
 * further step can amplify its error by up to a, as in any float32 arithmetic.
 * Entries of X are held to 2^-36 at least, so a matrix whose norm is far below eps
 * loses digits.
 * steps lies in 1..64.  coeffs: three floats in HOST memory, or NULL
 * for 3.4445, -4.7750, 2.0315; EUNSUPPORTED where they would carry the
 * singular values (above about 3.5) or the polynomial a + b s^2 + c s^4 (above
 * 24) out of the operands' range.  A NaN or an
 * infinity anywhere in a matrix makes its whole result NaN; a zero matrix
 * stays zero (eps > 0).  A matrix has the same bits by itself as in a
 * batch of any size, and they are reproducible. */

/* Bytes of device workspace that the two calls below need (none for matrices
 * that one workgroup holds: up to 32 x 512 or 64 x 256, either way up), or a
 * negative status (EUNSUPPORTED for more than 65535 matrices or sides past
 * 2^31 - 64). */
int64_t disco_orthogonalize_workspace(int32_t batch, int32_t rows, int32_t cols);

/* o = the orthogonalised m; m [batch, rows, cols] of m_dtype, o of o_dtype. */
int disco_orthogonalize(const void* m, int m_dtype, void* o, int o_dtype, int32_t batch,
                        int32_t rows, int32_t cols, int32_t steps, const float* coeffs, float eps,
                        void* workspace, int64_t workspace_bytes, void* stream);

/* One optimiser step (momentum, orthogonalisation and the weight update of the
 * Muon optimiser):
 *   momentum_out = beta * momentum + grad
 *   u     = grad + beta * momentum_out   (nesterov != 0), or momentum_out
 *   w_out = w * (1 - lr * weight_decay) - lr * scale * orthogonalised(u)
 * grad of grad_dtype, momentum float32, w and w_out of w_dtype (float32, or
 * bfloat16 weights with no float32 master); w16: bfloat16 copy of a float32
 * w_out for a bfloat16 layer, or NULL.  momentum_out may be momentum and
 * w_out may be w; otherwise no output overlaps another tensor. */
int disco_muon_step(const void* grad, int grad_dtype, const float* momentum, float* momentum_out,
                    const void* w, int w_dtype, void* w_out, void* w16, float lr, float beta,
                    int nesterov, float weight_decay, float scale, int32_t batch, int32_t rows,
                    int32_t cols, int32_t steps, const float* coeffs, float eps, void* workspace,
                    int64_t workspace_bytes, void* stream);

/* ---- Attention over points ----------------------------------------------
 * Global mixing beside the convolution's local one: softmax attention over the
 * points of fields or the tokens of series, with quadrature weights as an
 * additive term of each key (the AttentionS2 page: softmax attention whose sums
 * over the sphere are quadratures).  For query i and key j of one sequence, and
 * query head h reading key head h / (hq / hkv):
 *   x_ij = scale * q_i . k_j + key_bias_j,  lse_i = log sum_j exp x_ij
 *   o_i  = sum_j exp(x_ij - lse_i) v_j
 * Tokens of all sequences lie one after another ("packed").  cu_q and cu_k,
 * [n_seq + 1] in DEVICE memory, hold each sequence's first token and the end of
 * the last; NULL stands for n_seq sequences of equal length (a dense batch).
 * Boundaries out of order or out of range are cut to the tensors; tokens before
 * the first and behind the last sequence are not read, and their results are
 * left as they were.
 *  - causal != 0: query i of a sequence of Lq queries and Lk keys sees keys
 *    j <= i + Lk - Lq (the last query sees all keys).
 *  - key_bias [total_k] float32 or NULL, at most 1e30; -inf, or anything below
 *    -1e30, leaves a key out, whatever k and v hold there.  It is a constant: no
 *    gradient.  Any other value is a summand, so a query all of whose keys carry a
 *    mask of -1e9 gets a mean of their values, as large as float32 scores let it be
 *    told apart; beside ordinary keys such a mask weighs nothing.
 *  - a query that sees no key gets o = 0, lse = -inf and gradients of zero.
 *  - values of v are at most 1e25: sums may be that much larger for a while.
 *  - what a causal query does not see has to be finite all the same: a NaN or an
 *    infinity in k or v may reach o and gq of queries that see up to 190 keys less,
 *    one in q, go or o of a query gk and gv of keys up to 158 behind its last one.  In
 *    a query that sees no key it may reach gk and gv of its sequence.
 * float32 tensors are computed in float32; for bfloat16 ones products are of
 * bfloat16 operands summed in float32, with the weights exp(x - max) and the
 * gradients of x rounded to bfloat16 (the bf16 bar).  Sums run in a fixed order:
 * results are reproducible.  Any alignment and strides are taken; head sizes,
 * strides and addresses that are multiples of 16 bytes are much faster. */
typedef struct disco_attention_desc {
    int64_t total_q, total_k;       /* tokens of all sequences; tokens * heads < 2^30 - 4096 */
    int32_t n_seq;                  /* >= 1 */
    int32_t hq, hkv;                /* heads of q and o (at most 65535), of k and v; hkv divides hq */
    int32_t dk, dv;                 /* sizes of a head of q and k, of v and o: 1..128 */
    int32_t dtype;                  /* of every tensor but lse and key_bias */
    int32_t causal;
    float   scale;                  /* 1e-6 .. 1e6 */
    /* strides in elements, token to token and head to head (a head's elements
     * lie together); those of results may be columns of one buffer */
    int64_t q_stride[2], k_stride[2], v_stride[2], o_stride[2];
    int64_t go_stride[2], gq_stride[2], gk_stride[2], gv_stride[2];   /* the gradient call only */
} disco_attention_desc;

/* Bytes of device workspace of the forward call (few rows over many keys are
 * split along the keys and joined), or a negative status. */
int64_t disco_attention_fwd_workspace(const disco_attention_desc* desc);

/* o [total_q, hq, dv]; lse [total_q, hq] float32, dense, or NULL (the gradient
 * needs it). */
int disco_attention_fwd(const disco_attention_desc* desc, const void* q, const void* k, const void* v,
                        const float* key_bias, const int32_t* cu_q, const int32_t* cu_k, void* o, float* lse,
                        void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of device workspace of the gradient call, or a negative status. */
int64_t disco_attention_bwd_workspace(const disco_attention_desc* desc);

/* Gradients of sum(go * o): gq, and gk with gv, NULL to skip (not all); from the
 * forward's o and lse.  gk and gv are summed over the heads of their group. */
int disco_attention_bwd(const disco_attention_desc* desc, const void* q, const void* k, const void* v,
                        const float* key_bias, const int32_t* cu_q, const int32_t* cu_k, const void* o,
                        const float* lse, const void* go, void* gq, void* gk, void* gv, void* workspace,
                        int64_t workspace_bytes, void* stream);

/* ---- Norm and rotation of queries and keys -------------------------------
 * Each head of q [tokens, hq, d] and k [tokens, hkv, d] is divided by its root
 * mean square and turned by its token's position:
 *   n = x / sqrt(mean(x^2) + eps) * weight      (weight [d] float32, NULL for ones)
 *   pair p < rot/2 turns by positions[token, p * axes / (rot/2)] * inv_freq[p]
 * Pairs are (p, p + rot/2), or (2 p, 2 p + 1) where interleaved != 0; elements
 * from rot on do not turn.  positions [tokens, axes], int32 or float32 (times of a
 * series; colatitude and longitude of a point, where whole frequencies are
 * periodic in longitude); scaled tables for long series are the caller's
 * inv_freq.  Angles are taken in float64, squares are summed in float32 (elements of at
 * most 1e18).  Heads are independent: a NaN stays in its own. */
typedef struct disco_qk_desc {
    int64_t tokens;                 /* at most 2^26 - 64 */
    int32_t hq, hkv, d;             /* hkv may be 0; d in 1..256 */
    int32_t dtype;                  /* of every tensor but weights, positions and inv_freq */
    int32_t rot;                    /* elements that turn: even, 0..d */
    int32_t axes;                   /* 1..4 */
    int32_t positions_int32;        /* != 0: int32, else float32 */
    int32_t interleaved;
    float   eps;
    int64_t q_stride[2], k_stride[2];           /* token to token, head to head, in elements */
    int64_t q_out_stride[2], k_out_stride[2];   /* of the results: q_out, k_out; gq, gk of the gradient */
    int64_t gq_stride[2], gk_stride[2];         /* of gq_out, gk_out; the gradient call only */
} disco_qk_desc;

int disco_qk_norm_rope_fwd(const disco_qk_desc* desc, const void* q, const void* k, const float* q_weight,
                           const float* k_weight, const void* positions, const float* inv_freq, void* q_out,
                           void* k_out, void* stream);

/* Bytes of device workspace of the weights' gradients, or a negative status. */
int64_t disco_qk_norm_rope_bwd_workspace(int32_t d);

/* Gradients of sum(gq_out * q_out) + sum(gk_out * k_out) in q, k (what went into
 * the forward) and, where given, the weights ([d] float32, over all tokens and
 * heads; they need the workspace).  No tokens: weights' gradients of zero. */
int disco_qk_norm_rope_bwd(const disco_qk_desc* desc, const void* q, const void* k, const void* gq_out,
                           const void* gk_out, const float* q_weight, const float* k_weight, const void* positions,
                           const float* inv_freq, void* gq, void* gk, float* gq_weight, float* gk_weight,
                           void* workspace, int64_t workspace_bytes, void* stream);

/* ---- Dropout ---------------------------------------------------------------
 *   y = residual + (kept ? x / (1 - P) : 0),   P = t / 65536, t = round(65536 p)
 * Element e of n is kept where half-word e % 8 (the low half of a word first) of
 * block e / 8 is not below t; a block is the four words of the counter-based
 * generator Philox4x32 (ten rounds) at counter (block, offset) under the key
 * seed.  So the mask is a function of (seed, offset, e): the gradient computes it
 * again from the same three, and nothing is stored.  step (device memory, or
 * NULL) is added to offset, so that a captured call draws anew at each replay.
 * x, residual (or NULL) of x_dtype, y of y_dtype; y may be x where the types are
 * the same.  p lies in [0, 1 - 2^-17); n is at most 2^40.  A dropped element is
 * zero whatever x holds. */
int disco_dropout_fwd(const void* x, int x_dtype, const void* residual, void* y, int y_dtype, int64_t n, double p,
                      uint64_t seed, uint64_t offset, const int64_t* step, void* stream);

/* gx = kept ? gy / (1 - P) : 0; the residual's gradient is gy itself. */
int disco_dropout_bwd(const void* gy, int gy_dtype, void* gx, int gx_dtype, int64_t n, double p, uint64_t seed,
                      uint64_t offset, const int64_t* step, void* stream);

/* Per-kernel timing, for benchmarks and profiling (not part of the pages'
 * method).  With enable != 0, every kernel the library launches from then on
 * is bracketed by a pair of HIP events recorded on its launch stream; with 0,
 * no further events are recorded.  Always returns DISCO_OK. */
int disco_kernel_timing(int enable);

/* Drains the recorded event pairs (waiting for each to complete) into totals
 * per kernel, in order of first launch: kernel i's name is the i-th
 * NUL-terminated string packed into names[0 .. names_len), total_ms[i] its
 * summed event time and launches[i] its launch count.  Returns the number of
 * kernels (0 if nothing was recorded), or DISCO_EINVAL if the buffers are too
 * small (the records are then discarded), or DISCO_EHIP. */
int disco_kernel_timing_read(char* names, int32_t names_len, double* total_ms,
                             int64_t* launches, int32_t max_kernels);

/* Message for the last failed call on this thread ("" if none). */
const char* disco_last_error(void);

/* Library version string. */
const char* disco_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DISCO_H */
