/*
 * dora.h - C ABI of libdora.so, the MI355X (gfx950) DoRA module hot path.
 *
 * Sources (by page title and section):
 *   [SD]   "Scaling DoRA: High-Rank Adaptation via Factored Norms and Fused
 *          Kernels" (Zelenin, Zhuravlyova; arXiv 2603.22276), abstract:
 *          the row-wise norm of W + sBA, its factored form (base, cross and
 *          Gram terms through O(d_out r + r^2) intermediates, no dense BA),
 *          and the single-pass, cancellation-safe composition.
 *   [DoRA] "DoRA: Weight-Decomposed Low-Rank Adaptation" (Liu et al. 2024),
 *          summary pages: "Method" (magnitude m and a direction updated by
 *          LoRA) and "Statistical analysis" (a training-memory modification,
 *          read here as a norm held constant in the backward pass).
 *
 * Notation.  W [d_out, d_in] is the frozen weight, A [r, d_in] and
 * B [d_out, r] the LoRA factors, s the LoRA scale, m [d_out] the magnitude,
 * x [T, d_in] the tokens.  V = W + s*B*A is never formed.
 *   n_i  = ||W_i + s*B_i*A||_2                       (row norm, [SD])
 *   g_i  = m_i / n_i
 *   y    = g (.) (x W^T + s * (x A^T) B^T)           ([SD], [DoRA])
 *
 * Conventions shared by every call:
 *   - Every matrix is dense, row-major and contiguous.  Matrix data (x, W,
 *     A, B, dy, y, P, base, lora, dx, dA, dB) has one element type given by
 *     the dora_dtype argument (the 8-bit rows further down: int8 with fp32
 *     scales).  m, n, dm and the optional norm terms are
 *     always fp32.  s is an fp32 scalar passed by value.
 *   - Every pointer is device memory owned by the caller (e.g. torch
 *     tensors).  The library never allocates device memory and keeps no
 *     state between calls; its only scratch is the caller's workspace
 *     `ws` of at least the size the matching *_workspace() query returns.
 *     No workspace size has a d_out*d_in term: no dense [d_out, d_in]
 *     buffer is ever formed.
 *   - `stream` is a hipStream_t (NULL = the null stream).  Arguments are
 *     validated on the host before anything is enqueued; kernels then run
 *     asynchronously on `stream` and results are valid once it is
 *     synchronised.  Nothing inside synchronises the host.
 *   - Every pointer must be 16-byte aligned.  Sizes need not be multiples
 *     of anything: T >= 0, and d_in, d_out, r >= 1 (all < 2^31).  Tails are
 *     masked in the kernels; a bf16 width that leaves rows unaligned to 16
 *     bytes (not a multiple of 8) runs on register-staged tiles, slower than
 *     the pipelined path but with the same arithmetic.
 *   - Results are bitwise deterministic for identical inputs: there are no
 *     floating-point atomics and every reduction runs in a fixed order.
 *   - Arithmetic: products accumulate in fp32; matrix outputs are rounded
 *     once, to nearest even, to the element type.
 *   - Preconditions not checked per element: n_i > 0 (rows of W + sBA are
 *     not zero) and, for dora_backward, m_i != 0.  Violations propagate
 *     IEEE inf/NaN; they never fault.
 *
 * Errors: every call returns a dora_status.  On failure nothing has been
 * enqueued unless the status is DORA_E_HIP (a launch failed part-way; the
 * outputs are then unspecified).  dora_last_error() returns a thread-local
 * message describing the last failure on the calling thread.
 */
#ifndef DORA_H
#define DORA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    DORA_OK = 0,
    DORA_E_NULL = 1,      /* a required pointer is NULL                      */
    DORA_E_SHAPE = 2,     /* a size is out of range                          */
    DORA_E_DTYPE = 3,     /* unknown dora_dtype                              */
    DORA_E_ALIGN = 4,     /* a pointer is not 16-byte aligned                */
    DORA_E_WORKSPACE = 5, /* ws is NULL or ws_bytes is below the query       */
    DORA_E_ALIAS = 6,     /* two buffers overlap where that is not allowed   */
    DORA_E_HIP = 7,       /* a HIP launch or runtime call failed             */
    DORA_E_VALUE = 8      /* a scalar argument is out of range               */
} dora_status;

typedef enum {
    DORA_F32 = 0,  /* IEEE binary32 */
    DORA_BF16 = 1  /* bfloat16 (upper 16 bits of binary32) */
} dora_dtype;

/* Human-readable name of a status code (static string). */
const char *dora_strerror(int status);

/* Message for the last failure on the calling thread ("" if none). */
const char *dora_last_error(void);

/* Workspace sizes in bytes for the calls below (0 if the arguments are
 * invalid).  They are pure host functions.  The norm workspace is
 * O(d_out*r + r^2) for fixed splits, as [SD] states for the factored
 * intermediates; forward and backward add O(T*d_out + T*r) activations. */
size_t dora_norm_workspace(int64_t d_out, int64_t d_in, int64_t r, int dtype);
size_t dora_forward_workspace(int64_t T, int64_t d_in, int64_t d_out, int64_t r, int dtype);
size_t dora_backward_workspace(int64_t T, int64_t d_in, int64_t d_out, int64_t r, int dtype);

/*
 * dora_factored_norm - row norms of W + s*B*A without forming B*A ([SD]
 * abstract, "factored norm"):
 *     n_i^2 = base_i + 2*s*cross_i + s^2*gram_i
 *     base_i  = sum_j W_ij^2
 *     cross_i = sum_k B_ik * U_ik,        U = W A^T      [d_out, r]
 *     gram_i  = sum_k B_ik * (B G)_ik,    G = A A^T      [r, r]
 * n is written as sqrt(max(n^2, 0)) (the factored sum can round below
 * zero only when ||W_i + s B_i A|| << ||W_i||).
 *   W [d_out, d_in], A [r, d_in], B [d_out, r] in `dtype`.
 *   n [d_out] fp32 (required).  base, cross, gram [d_out] fp32, each
 *   optional (NULL to skip).  U_out [d_out, r] fp32, optional: receives
 *   V A^T = (W + s B A) A^T = U + s B G, the two products the norm forms
 *   anyway (U by the cross term's product, s B G added by the Gram term's);
 *   keeping it lets the backward through the norm skip W A^T, A A^T and
 *   B G (its dB term is a row scale of exactly this matrix).
 *   ws: device scratch of dora_norm_workspace(d_out, d_in, r, dtype) bytes.
 */
int dora_factored_norm(const void *W, const void *A, const void *B, float s,
                       int64_t d_out, int64_t d_in, int64_t r, int dtype,
                       float *n, float *base, float *cross, float *gram, float *U_out,
                       void *ws, size_t ws_bytes, void *stream);

/*
 * dora_compose - the single-pass composition ([SD] abstract, fused
 * compose with a numerically stable form for the near-unity regime):
 *     y[t,i] = base[t,i] + ( (g_i - 1) * base[t,i] + g_i * s * lora[t,i] )
 * with g_i - 1 = (m_i - n_i) / n_i and g_i s = m_i s / n_i each rounded once
 * to fp32, the bracket summed in fp32 before base is added, and one rounding
 * to `dtype` at the end.  Mathematically y = (m/n) (.) (base + s*lora).
 *   base, lora, y [T, d_out] in `dtype`; m, n [d_out] fp32.
 *   y may be the same pointer as base (in place); any other overlap of y
 *   with base or lora is DORA_E_ALIAS.
 */
int dora_compose(const void *base, const void *lora, const float *m, const float *n,
                 float s, int64_t T, int64_t d_out, int dtype, void *y, void *stream);

/*
 * dora_forward - the DoRA module forward ([SD], [DoRA]):
 *     n   = factored row norm (as dora_factored_norm), unless n_in is given
 *     P   = x A^T                            [T, r]
 *     h   = x W^T + (s P) B^T                one K-concatenated product,
 *                                            accumulated in fp32
 *     y   = h + ((m - n) / n) h              = (m/n) h, applied by the
 *                                            product's epilogue, rounded once
 *   The base and adapter products share one accumulator, so the composition
 *   happens in the same pass that produces them ([SD]'s single-pass compose,
 *   taken one step further): no [T, d_out] intermediate exists.  P and s P
 *   are each rounded once to the element type from the same fp32 sums of
 *   x A^T (s P is P itself when s = 1).
 *   x [T, d_in], W [d_out, d_in], A [r, d_in], B [d_out, r] in `dtype`;
 *   m [d_out] fp32.  y [T, d_out] in `dtype` (output).
 *   n_out [d_out] fp32: receives n (required; with n_in it receives a copy).
 *   P_out [T, r] in `dtype`: receives x A^T for the backward (NULL: kept in
 *   the workspace only).
 *   n_in [d_out] fp32 or NULL: a norm computed earlier (cached inference);
 *   when given, the norm is not recomputed.
 *   U_out [d_out, r] fp32 or NULL: receives the norm's V A^T = U + s B G
 *   (as in dora_factored_norm) for dora_backward_through_norm; needs n_in
 *   NULL.
 *   y must not overlap any input, n_out, P_out or U_out.
 */
int dora_forward(const void *x, const void *W, const void *A, const void *B, const float *m,
                 float s, int64_t T, int64_t d_in, int64_t d_out, int64_t r, int dtype,
                 void *y, float *n_out, void *P_out, const float *n_in, float *U_out,
                 void *ws, size_t ws_bytes, void *stream);

/*
 * dora_backward - gradients of L = sum(dy (.) y) with the row norm n held
 * constant (stop-gradient; [DoRA] "Statistical analysis", training-memory
 * modification).  With g = m / n and dh = g (.) dy:
 *     dm_i = sum_t dy[t,i] * y[t,i] / m_i    (= sum_t dy h / n_i, h = x V^T)
 *     Q    = s * dh B                        [T, r], in the workspace
 *     dx   = dh W + Q A
 *     dB   = s * dh^T P
 *     dA   = Q^T x
 * W is frozen and gets no gradient.  dx and dm equal the gradients without
 * the stop-gradient (n does not depend on x or m); dA and dB omit the path
 * through n.
 *   dy, y [T, d_out], x [T, d_in], P [T, r] (from dora_forward), W, A, B in
 *   `dtype`; m, n [d_out] fp32 (n as returned by dora_forward).
 *   Outputs: dx [T, d_in], dA [r, d_in], dB [d_out, r] in `dtype`,
 *   dm [d_out] fp32.  Outputs must not overlap each other or any input.
 *   With T = 0, dA, dB and dm are zero.
 */
int dora_backward(const void *dy, const void *x, const void *W, const void *A, const void *B,
                  const float *m, const float *n, float s, const void *P, const void *y,
                  int64_t T, int64_t d_in, int64_t d_out, int64_t r, int dtype,
                  void *dx, void *dA, void *dB, float *dm,
                  void *ws, size_t ws_bytes, void *stream);

/*
 * dora_backward_through_norm - the same gradients without the stop-gradient:
 * the gradient also flows through the row norm n = ||W + s B A|| into A and
 * B.  The DoRA summary page ("Statistical analysis", analysis design) names
 * the gradient with respect to the direction V and the magnitude as derived
 * in the method's gradient analysis; the plain chain rule through n_i =
 * ||V_i|| (dn_i / dV_i = V_i / n_i) gives, with c_i = m_i dm_i / n_i^2,
 *     dV = dh^T x - diag(c) V
 *     dA = s B^T dV = Q^T x - s (c (.) B)^T W - s^2 ((c (.) B)^T B) A
 *     dB = s dV A^T = s dh^T P - s c (.) (W A^T + s B (A A^T))
 * using only [d_out, r] and [r, r] intermediates (no dense V or B A, as in
 * the factored norm of the "Scaling DoRA" abstract).  dx and dm are those of
 * dora_backward, bit for bit.  Arguments, layouts, aliasing rules and the
 * T = 0 case (dm zero, dA and dB then zero as well) are those of
 * dora_backward; n is the norm dora_forward returned and is taken as the
 * exact norm of W + s B A.  U [d_out, r] fp32 or NULL: the norm's
 * V A^T = W A^T + s B (A A^T) as dora_forward's (or dora_factored_norm's)
 * U_out kept it, for the same W, A, B and s (the factored norm's products
 * are reused, so W A^T, A A^T and B G are not formed again); NULL forms
 * them here.
 *   ws: dora_backward_through_norm_workspace(T, d_in, d_out, r, dtype) bytes.
 */
size_t dora_backward_through_norm_workspace(int64_t T, int64_t d_in, int64_t d_out, int64_t r,
                                            int dtype);
int dora_backward_through_norm(const void *dy, const void *x, const void *W, const void *A,
                               const void *B, const float *m, const float *n, float s,
                               const void *P, const void *y, const float *U, int64_t T,
                               int64_t d_in, int64_t d_out, int64_t r, int dtype, void *dx,
                               void *dA, void *dB, float *dm, void *ws, size_t ws_bytes,
                               void *stream);

/*
 * Grouped calls - many adapted modules in few launches.  The "Scaling DoRA"
 * abstract motivates the factored norm with models that carry hundreds of
 * adapted modules; these calls give each kernel of the norm (and of the
 * forward of sibling modules that share one input, such as the query, key
 * and value projections) one launch per 16 modules instead of one per
 * module, with every module's products sharing the GPU at once.
 *
 * dora_module describes one module: W [d_out, d_in], A [r, d_in],
 * B [d_out, r] in `dtype`, m [d_out] fp32 (not read by the norm), scale s.
 * The array is read on the host during the call only.
 */
typedef struct dora_module {
    const void *W;
    const void *A;
    const void *B;
    const float *m;
    float s;
    int64_t d_out, d_in, r;
} dora_module;

/*
 * dora_factored_norm_grouped - n[i] = the row norms of W_i + s_i B_i A_i for
 * every module, as dora_factored_norm computes them (the same terms and
 * precision; the split-K plan may differ, so bits may too).  n is a host
 * array of `count` device pointers ([d_out_i] fp32 each), pairwise disjoint
 * and disjoint from every module's W, A, B and the workspace.  fp32 modules
 * (and bf16 ones whose operands reach 2 GiB) run module by module.
 *   ws: dora_factored_norm_grouped_workspace(mods, count, dtype) bytes.
 */
size_t dora_factored_norm_grouped_workspace(const dora_module *mods, int count, int dtype);
int dora_factored_norm_grouped(const dora_module *mods, int count, int dtype, float *const *n,
                               void *ws, size_t ws_bytes, void *stream);

/*
 * dora_forward_grouped - dora_forward for `count` modules on the same input
 * x [T, d_in] (every module's d_in must equal d_in): y[i] [T, d_out_i],
 * n_out[i] [d_out_i] fp32, optional P_out[i] [T, r_i] (P_out itself may be
 * NULL), optional cached norms n_in[i] (n_in itself may be NULL; a given
 * n_in[i] skips that module's norm and may equal n_out[i]).  Host arrays of
 * device pointers; every output is disjoint from every input and from every
 * other output.  Per 16 modules: one launch of all x A_i^T, one of the s P
 * scalings, one of the fused products with the magnitude epilogue.
 *   ws: dora_forward_grouped_workspace(mods, count, T, dtype, n_in, P_out)
 *   bytes (it depends on which norms are cached and which P are kept).
 */
size_t dora_forward_grouped_workspace(const dora_module *mods, int count, int64_t T, int dtype,
                                      const float *const *n_in, void *const *P_out);
int dora_forward_grouped(const void *x, int64_t T, int64_t d_in, const dora_module *mods,
                         int count, int dtype, void *const *y, float *const *n_out,
                         void *const *P_out, const float *const *n_in, void *ws, size_t ws_bytes,
                         void *stream);

/*
 * dora_merge - the merged weight W' = g (.) (W + s B A), g = m / n by rows,
 * for inference: the DoRA summary pages ("Method"; Key Points 3 and 5) note
 * that the adapted weight folds into the base weight, so inference is a
 * plain linear layer (dora_linear).  n is the factored row norm of the
 * "Scaling DoRA" abstract (computed here unless n_in is given), so no dense
 * B A product is kept: B A is formed tile by tile inside one product whose
 * epilogue writes W'[i, j] = W[i, j] + ((g_i - 1) W[i, j] + g_i s (BA)[i, j])
 * in fp32, rounded once (the near-unity form of dora_compose).
 *   W, W_out [d_out, d_in], A [r, d_in], B [d_out, r] in `dtype`; m and
 *   n_in (nullable) [d_out] fp32.  W_out may be W itself (in place) but must
 *   not overlap it otherwise, nor A, B, m, n_in or the workspace.
 *   ws: dora_merge_workspace(d_out, d_in, r, dtype) bytes.
 */
size_t dora_merge_workspace(int64_t d_out, int64_t d_in, int64_t r, int dtype);
int dora_merge(const void *W, const void *A, const void *B, const float *m, float s,
               int64_t d_out, int64_t d_in, int64_t r, int dtype, const float *n_in, void *W_out,
               void *ws, size_t ws_bytes, void *stream);

/*
 * dora_linear - y = x W^T on the same kernel and launch plan dora_forward
 * uses for its base term.  With W = W' = g (.) (W + sBA), the weight merged
 * after training, this is the whole DoRA inference path: the DoRA summary
 * pages ("Method"; Key Points 3 and 5) note that the adapted weight merges
 * into the base weight, adding no inference latency.
 *   x [T, d_in], W [d_out, d_in], y [T, d_out] in `dtype`; y must not
 *   overlap x or W.  ws: dora_linear_workspace(T, d_in, d_out, dtype) bytes
 *   (0 when the product needs no split-K partials; ws may then be NULL).
 */
size_t dora_linear_workspace(int64_t T, int64_t d_in, int64_t d_out, int dtype);
int dora_linear(const void *x, const void *W, int64_t T, int64_t d_in, int64_t d_out, int dtype,
                void *y, void *ws, size_t ws_bytes, void *stream);

/*
 * dora_forward_noalloc - dora_forward for callers that cannot allocate
 * device memory: code under HIP graph capture, tight serving loops, and
 * harnesses that forbid allocation.  The arguments and results are those
 * of dora_forward without ws / ws_bytes; the scratch comes from a fixed
 * library-owned device array of DORA_NOALLOC_SCRATCH_BYTES (96 MiB), which
 * every GPU the library runs on holds from the library's load until the
 * process ends (its address on a device is looked up on the first call
 * there).  The call allocates nothing.
 *   Modules whose dora_forward_workspace() exceeds the array are rejected
 *   with DORA_E_WORKSPACE before anything touches the device.  The forward
 *   of every module of up to 16384 tokens at widths of the order of 28672
 *   with r = 384 fits.
 *   The array is shared by every call on one GPU and keeps the last call's
 *   contents (nothing in it needs to start at zero): calls that overlap in
 *   time on one GPU (on different streams or threads) race on it and must
 *   be serialised by the caller.  The stream's device is the GPU used.
 */
#define DORA_NOALLOC_SCRATCH_BYTES ((size_t)96 << 20)
int dora_forward_noalloc(const void *x, const void *W, const void *A, const void *B,
                         const float *m, float s, int64_t T, int64_t d_in, int64_t d_out,
                         int64_t r, int dtype, void *y, float *n_out, void *P_out,
                         const float *n_in, float *U_out, void *stream);

/*
 * 8-bit rows.  A matrix [rows, d] is held as int8 values q [rows, d] with fp32
 * scales: one a row (group = 0, scale [rows, 1]) or one for each `group`
 * consecutive columns (group a power of two from 32 to 512, scale
 * [rows, ceil(d / group)]; the last group of a row may be short).  Within a
 * group with values v_j
 *     scale = max_j |v_j| / 127          (0 for a group of zeros)
 *     q_j   = rint(v_j / scale)          ties to even, decided exactly
 * and q_j stands for q_j scale.  The scale is kept between 2^-126 and the
 * largest one for which 127 scale is finite.  A group that holds an infinity
 * or a NaN gets a NaN scale: it stands for NaN throughout.
 * Rows of int8 need no alignment of their own (any d); the buffers do.
 *
 * dora_rmsnorm - the root-mean-square norm in front of an adapted projection,
 * with the residual's addition:
 *     h    = x + residual   summed in fp32, rounded to `dtype` (x without one)
 *     rstd = 1 / sqrt(mean_j h_j^2 + eps)          of the rounded h, in fp32
 *     y    = w (.) h rstd   in fp32, rounded once to `dtype` (y), and / or
 *            held as 8-bit rows (q, scale) taken from the unrounded y
 *   x, residual (nullable) [T, d], w [d] in `dtype`; eps finite, >= 0.  Rows of
 *   any magnitude: squares that leave fp32's range are summed scaled.
 *   y [T, d], h [T, d] in `dtype`, rstd [T] fp32, q [T, d] int8 with scale
 *   [T, groups] fp32: each NULL to skip, but y or q is required and q needs
 *   scale.  h may be x or residual itself, y may be x itself; no other
 *   overlap.
 *   q with group = 0 is dora_linear_quantized's xq; any group serves
 *   dora_backward_checkpoint.
 *
 * dora_rmsnorm_backward - its gradient, from the h and rstd it returned:
 *     dx   = dres + rstd (w (.) dy) - h rstd^3 / d * sum_j w_j dy_j h_j
 *     dw_j = sum_t dy_tj h_tj rstd_t
 *   dx is the gradient of x and, with a residual, of the residual too.  dres
 *   [T, d] (nullable) is the gradient that reaches h along the residual
 *   stream; dx may be dres itself.  dy, h, dres, dx [T, d], w [d] in `dtype`,
 *   rstd [T], dw [d] fp32 (dw NULL to skip; ws may then be NULL).  T = 0
 *   gives dw = 0.
 */
int dora_rmsnorm(const void *x, const void *residual, const void *w, float eps, int64_t T,
                 int64_t d, int dtype, int64_t group, void *y, void *h, float *rstd, void *q,
                 float *scale, void *stream);
size_t dora_rmsnorm_backward_workspace(int64_t T, int64_t d, int dtype);
int dora_rmsnorm_backward(const void *dy, const void *h, const void *w, const float *rstd,
                          const void *dres, int64_t T, int64_t d, int dtype, void *dx, float *dw,
                          void *ws, size_t ws_bytes, void *stream);

/*
 * dora_quantize_rows / dora_dequantize_rows - a matrix [rows, d] of `dtype` to
 * 8-bit rows and back (see above).  With group = 0 and x = the merged weight
 * of dora_merge, q and scale are dora_linear_quantized's wq and wscale.
 * Restored values are q scale in fp32, rounded once to `dtype`, which need not
 * be the type the rows came from.
 */
int dora_quantize_rows(const void *x, int64_t rows, int64_t d, int dtype, int64_t group, void *q,
                       float *scale, void *stream);
int dora_dequantize_rows(const void *q, const float *scale, int64_t rows, int64_t d, int dtype,
                         int64_t group, void *out, void *stream);

/*
 * dora_linear_quantized - dora_linear in 8-bit integers, for a merged weight
 * held as 8-bit rows: one scale per token and one per output channel,
 *     y[t, i] = xs[t] wscale[i] sum_k xq[t, k] wq[i, k]
 * with exact int32 sums, scaled in fp32 (the scales may be any fp32 numbers: no
 * intermediate leaves the range where y does not) and rounded once to `dtype`
 * (the type of y).  xq [T, d_in], wq [d_out, d_in] int8, xs [T], wscale [d_out]
 * fp32.
 * d_in <= 131071 (beyond, int32 sums could overflow).  y must not overlap any
 * input.  ws: dora_linear_quantized_workspace(T, d_in, d_out, dtype) bytes
 * (0: ws may be NULL).
 */
size_t dora_linear_quantized_workspace(int64_t T, int64_t d_in, int64_t d_out, int dtype);
int dora_linear_quantized(const void *xq, const float *xs, const void *wq, const float *wscale,
                          int64_t T, int64_t d_in, int64_t d_out, int dtype, void *y, void *ws,
                          size_t ws_bytes, void *stream);

/*
 * dora_backward_checkpoint - dora_backward (through_norm = 0) or
 * dora_backward_through_norm (otherwise) with the forward's x and y kept
 * between the passes as 8-bit rows, half the bytes of bf16: xq [T, d_in] with
 * xs and yq [T, d_out] with ys, both of this `group`.  The gradients are those
 * of the restored x = xq xs and y = yq ys; y enters dm in fp32.  x enters dA in
 * bf16 modules with group 0, 128, 256 or 512 unrounded, beside a Q = s dh B kept
 * to 16 bits (dA is then rounded once, behind dh); with group 32 or 64, and in
 * fp32 modules, x is rounded to `dtype` and dA is what the two calls make of it.
 * All other arguments, layouts, aliasing rules and the T = 0 case are those of
 * the two calls.
 * ws: dora_backward_checkpoint_workspace(...) bytes, enough for any group.
 */
size_t dora_backward_checkpoint_workspace(int64_t T, int64_t d_in, int64_t d_out, int64_t r,
                                          int dtype, int through_norm);
int dora_backward_checkpoint(const void *dy, const void *xq, const float *xs, const void *W,
                             const void *A, const void *B, const float *m, const float *n, float s,
                             const void *P, const void *yq, const float *ys, int64_t group,
                             const float *U, int through_norm, int64_t T, int64_t d_in,
                             int64_t d_out, int64_t r, int dtype, void *dx, void *dA, void *dB,
                             float *dm, void *ws, size_t ws_bytes, void *stream);

/*
 * dora_block_norm - the norms on both sides of a residual addition, behind one
 * block and in front of the next (dora_rmsnorm is the one in front alone):
 *     u = w_post (.) x / sqrt(mean_j x_j^2 + eps)        (u = x without w_post)
 *     h = residual_scale residual + branch_scale gate (.) u
 *                                formed in fp32, rounded to `dtype`
 *     y = w_pre (.) h / sqrt(mean_j h_j^2 + eps)         of the rounded h
 *   x (the block's output), residual [T, d], w_post (nullable), w_pre [d],
 *   h, y [T, d] in `dtype`.  gate (nullable, then 1): [ceil(T / gate_rows), d] in
 *   `dtype` (one row with T = 0), token t uses row t / gate_rows: gate_rows = T is
 *   a gate a channel, 1 a gate a token and channel, and the length of sequences of
 *   one length a gate vector for each.  rstd_post, rstd_pre [T] fp32 (each NULL to
 *   skip): the two factors 1 / sqrt(...), for the backward.  eps finite, >= 0; rows
 *   of any magnitude whose factor is an fp32 number (with eps = 0 not those of zeros,
 *   NaN as the formula is, nor of fp32 values below 2^-127 alone).  h may be residual
 *   itself, y may be x itself; no other overlap.
 *
 * dora_block_norm_backward - its gradients, from the x, h and factors of the
 * forward; dy is the gradient of y, dh (nullable) the one that reaches h along the
 * residual stream:
 *     Dh        = dh + rstd_pre (w_pre dy - hath mean_j(w_pre dy hath)),
 *                                                     hath = h rstd_pre
 *     dresidual = residual_scale Dh
 *     du        = branch_scale gate (.) Dh
 *     dx        = rstd_post (w_post du - hatx mean_j(w_post du hatx)),
 *                                    hatx = x rstd_post   (du without w_post)
 *     dgate     = sum branch_scale Dh (.) u   over the tokens of a gate row
 *     dw_post   = sum_t du hatx,  dw_pre = sum_t dy hath
 *   dx, dresidual [T, d], dgate (shaped as gate) in `dtype`; dw_post, dw_pre [d]
 *   fp32; the last three NULL to skip.  Dh and du stay in fp32 throughout.
 *   dresidual may be dh itself.  T = 0 gives zeros.
 *   ws: dora_block_norm_backward_workspace(T, d, gate_rows, dtype) bytes, with
 *   gate_rows = 0 for no gate (0 bytes: ws may be NULL).
 */
int dora_block_norm(const void *x, const void *residual, const void *w_post, const void *gate,
                    int64_t gate_rows, const void *w_pre, float residual_scale, float branch_scale,
                    float eps, int64_t T, int64_t d, int dtype, void *h, void *y, float *rstd_post,
                    float *rstd_pre, void *stream);
size_t dora_block_norm_backward_workspace(int64_t T, int64_t d, int64_t gate_rows, int dtype);
int dora_block_norm_backward(const void *dy, const void *dh, const void *x, const void *h,
                             const void *w_post, const void *gate, int64_t gate_rows,
                             const void *w_pre, const float *rstd_post, const float *rstd_pre,
                             float residual_scale, float branch_scale, int64_t T, int64_t d,
                             int dtype, void *dx, void *dresidual, void *dgate, float *dw_post,
                             float *dw_pre, void *ws, size_t ws_bytes, void *stream);

/*
 * 4-bit rows.  A matrix [rows, d] is held as e2m1 codes (sign, two bits of
 * exponent, one of fraction: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) with
 * one bf16 scale for each `group` consecutive columns (a power of two from 32 to
 * 512): codes [rows, groups group / 2] bytes with groups = ceil(d / group), two
 * codes a byte, the even column in the low half, rows of whole groups (what lies
 * past column d is written as zeros and not read as part of the matrix); scale
 * [rows, groups] bf16.  A code stands for its value times its group's scale.
 *
 * dora_quantize_fourbit - rows of `dtype` to this form:
 *     scale = max_j |v_j| / 6 rounded to six significant bits (ties to even)
 *     code  = v_j / scale rounded to the nearest e2m1 value (ties to the even
 *             code, above 6 to 6), decided exactly
 *   With six bits of scale every restored value is a bf16 number: nothing is lost
 *   behind the codes.  A group of zeros has scale 0; the scale is kept between
 *   2^-125 and 1.3125 2^125; a group that holds an infinity or a NaN gets a NaN
 *   scale: it stands for NaN throughout.
 * dora_dequantize_fourbit - code times scale in fp32, rounded once to `dtype`
 *   (exact for the scales above).
 *
 * dora_linear_fourbit - dora_linear for a weight held this way (codes and scale of
 * dora_quantize_fourbit on the merged weight of dora_merge, with group), y = x W^T
 * with fp32 sums, rounded once.  x [T, d_in], y [T, d_out] in `dtype`.
 *   Up to 256 tokens read the codes as they are: products with the codes' values,
 *   each group's fp32 sum times its scale (fp32 tokens of 2^-100 and less in
 *   magnitude may lose bits there, and the sums of six times a group's tokens must
 *   stay finite).  More tokens (or 2^23 columns) restore the weight into the workspace, some of its
 *   rows at a time, rounded once to `dtype`: exact for scales of six bits.
 *   y must not overlap any input.  ws: dora_linear_fourbit_workspace(T, d_in, d_out,
 *   dtype) bytes: none up to 256 tokens (ws may be NULL); beyond, 128 MiB or 256 rows
 *   of the weight at most, and split-K partials of y where the product needs them.
 */
int dora_quantize_fourbit(const void *x, int64_t rows, int64_t d, int dtype, int64_t group,
                          void *codes, void *scale, void *stream);
int dora_dequantize_fourbit(const void *codes, const void *scale, int64_t rows, int64_t d, int dtype,
                            int64_t group, void *out, void *stream);
size_t dora_linear_fourbit_workspace(int64_t T, int64_t d_in, int64_t d_out, int dtype);
int dora_linear_fourbit(const void *x, const void *codes, const void *scale, int64_t group,
                        int64_t T, int64_t d_in, int64_t d_out, int dtype, void *y, void *ws,
                        size_t ws_bytes, void *stream);

/*
 * Orthogonalised updates - the step of an optimiser that moves a matrix along the
 * nearest orthogonal one to its momentum (Muon), for the factors A and B of an
 * adapter and the gradients that dora_backward gives them.
 *
 * dora_orthogonalize - O = Newton-Schulz steps from U [rows, cols]:
 *     X_0 = U / (|U|_F + eps)
 *     X_{k+1} = a X_k + b (X_k X_k^T) X_k + c (X_k X_k^T)^2 X_k     `steps` times
 *   (for rows > cols of the transpose, which is the same matrix), (a, b, c) =
 *   coefficients, a host array, or 3.4445, -4.7750, 2.0315 where it is NULL: after
 *   five steps from a matrix of singular values above 0.0015 of its norm those of O
 *   lie between 0.68 and 1.21.  U, O in `dtype`; O may be U itself.  X X^T and its
 *   polynomials are formed in 64 bits, the product of the last one with U from 24 bits
 *   of both, rounded once, for either `dtype`: as near the steps in exact arithmetic as
 *   the steps in fp32 are.  Like those it loses |a|^steps 2^-24 of |U|_F or so in the
 *   directions that U (of low rank) does not have: 3e-5 after five of these steps, a
 *   hundredth after ten.
 *   1 <= steps <= 16; eps finite, >= 0; the shorter side up to 8192 (or
 *   DORA_E_SHAPE), the matrix up to 2^33 elements with its sides padded to 128s.
 *   U may have any magnitude; an infinity or a NaN in it makes all of O NaN, and a U
 *   of zeros gives an O of zeros, with eps = 0 too.
 *
 * dora_muon - the step of a list of matrices:
 *     momentum_out = mu momentum + grad
 *     U            = grad + mu momentum_out   (nesterov), else momentum_out
 *     param_out    = param - lr (weight_decay param + scale O(U))
 *   param, grad, param_out [rows, cols] in `dtype`, momentum, momentum_out fp32.
 *   param_out may be param, momentum_out momentum (in place); every output is
 *   otherwise disjoint from every other buffer of the list.  Up to 40 matrices (in 256
 *   MiB of workspace) share each launch, and a matrix's share of it decides the order
 *   of its sums; the array is read during the call only.
 *   ws: dora_orthogonalize_workspace / dora_muon_workspace bytes: copies of the
 *   matrices (4 bytes an element, sides padded), and the short sides' squares in 64
 *   bits.
 */
typedef struct dora_update {
    const void *param;
    const void *grad;
    const float *momentum;
    void *param_out;
    float *momentum_out;
    int64_t rows, cols;
    float lr, weight_decay, scale;
} dora_update;

size_t dora_orthogonalize_workspace(int64_t rows, int64_t cols, int dtype);
int dora_orthogonalize(const void *U, int64_t rows, int64_t cols, int dtype, int steps,
                       const float *coefficients, float eps, void *O, void *ws, size_t ws_bytes,
                       void *stream);
size_t dora_muon_workspace(const dora_update *updates, int count, int dtype);
int dora_muon(const dora_update *updates, int count, int dtype, float mu, int nesterov, int steps,
              const float *coefficients, float eps, void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DORA_H */
