/*
 * wtconv.h -- C ABI of libwtconv, the WTConv layer (wavelet convolution) for
 * AMD Instinct MI355X (gfx950), forward and backward.
 *
 * The layer, per channel c of an NCHW activation x (source: "Fast and
 * Memory-Efficient Wavelet Convolutions via I/O-Aware Reformulation", arXiv
 * 2608.10805; its English abstract describes WTConv as a drop-in replacement
 * for a depthwise convolution, and the technical summary's Methodology section
 * describes the analysis, the per-level convolutions with learned per-channel
 * scales, and the synthesis cascade):
 *
 *   y = s0[c] * (W0[c] (*) x + b0[c])
 *     + sum over levels l = 1..L of the Haar synthesis, from level l back to full
 *       resolution, of Z_l^b = s_l[4c+b] * (W_l[4c+b] (*) A_l^b),  b = 0..3,
 *
 * where A_l^0..3 are the four subbands of the orthonormal 2D Haar analysis
 * (2x2 taps of +-1/2) of the level-(l-1) low-pass band (level 0 is x itself),
 * (*) is a k x k cross-correlation with zero 'same' padding at the level's own
 * resolution, and the synthesis of level l adds the reconstruction of level l+1
 * into the low-pass band before its inverse Haar step.  Band order: 0 low-pass,
 * 1 top-row-minus-bottom-row, 2 left-column-minus-right-column, 3 diagonal.
 *
 * Layout
 *   activations  x, y, dy, dx: NCHW contiguous, fp32 (WTCONV_F32) or fp16
 *                (WTCONV_F16) per the descriptor; device memory, 16-byte aligned.
 *   parameters   always fp32, device memory:
 *                w_base [C][k][k], bias [C] (may be NULL: zero bias), s_base [C],
 *                w_lvl [L][4C][k][k] and s_lvl [L][4C] with band b of channel c
 *                at index 4c+b (both may be NULL when L == 0).
 *   gradients    fp32, same shapes as their parameters; OVERWRITTEN, never
 *                accumulated.  dw/ds are gradients of the raw (unfolded)
 *                weights and scales.
 * Shape rules  n, c, h, w >= 1; k in {1, 3, 5, 7}; 0 <= L <= WTCONV_MAX_LEVELS;
 *              h, w and their round-up to multiples of 2^L <= WTCONV_MAX_SIDE.
 * Odd maps     Where 2^L does not divide h or w, every level map with an odd
 *              side is padded with one zero row (bottom) / column (right)
 *              before its Haar analysis and that level's synthesis is cropped
 *              back, so level l is ceil(h / 2^l) x ceil(w / 2^l) (the pages do
 *              not treat odd sides; this is the reading taken).  The library
 *              computes it as the layer on copies zero-padded to multiples of
 *              2^L, cropped, which is the same operator; all three calls then
 *              need a workspace (two padded activation copies plus the padded
 *              layer's own workspace).  The unfused baseline requires 2^L to
 *              divide h and w.
 * fp16 mode    fp16 storage of activations only: every product and sum is fp32,
 *              each output element is rounded once to fp16 (round to nearest
 *              even).
 * Ownership    The caller allocates every buffer, including the workspace
 *              (size from wtconv_workspace_size, 256-byte aligned; its contents
 *              need no initialisation and are scratch after the call).  The
 *              library allocates no device memory and holds no state between
 *              calls; calls are reentrant.  The one exception is
 *              wtconv_backward_weight_noalloc, whose partial results live in a
 *              static device array of the library (see there).
 * Execution    All work is enqueued on `stream` (0 = the null stream) with no
 *              host synchronisation; outputs are ready when the stream reaches
 *              that point.  Inputs and outputs must not overlap (y != x,
 *              dx != dy).  Results are bitwise reproducible run to run (no
 *              floating-point atomics).  Only kernels are enqueued (no memset,
 *              copy or allocation), so calls may be captured into a HIP graph
 *              on a capturing stream and replayed; the workspace and buffers
 *              captured must then stay allocated.
 * Errors       Arguments are validated before any HIP call; a bad argument
 *              returns its status code and enqueues nothing.  A failed kernel
 *              launch returns WTCONV_ERR_HIP.  Asynchronous faults are reported
 *              by the HIP runtime at the caller's next synchronisation.
 */
#ifndef WTCONV_H
#define WTCONV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define WTCONV_MAX_LEVELS 6
#define WTCONV_MAX_SIDE 4096

typedef enum {
    WTCONV_OK = 0,
    WTCONV_ERR_NULL = 1,        /* a required pointer is NULL */
    WTCONV_ERR_SHAPE = 2,       /* sizes, levels or divisibility rule violated */
    WTCONV_ERR_UNSUPPORTED = 3, /* kernel size or dtype not built */
    WTCONV_ERR_WORKSPACE = 4,   /* workspace missing or smaller than required */
    WTCONV_ERR_HIP = 5,         /* the HIP runtime rejected a launch */
    WTCONV_ERR_ALIAS = 6        /* an output overlaps an input */
} wtconv_status_t;

typedef enum {
    WTCONV_F32 = 0,
    WTCONV_F16 = 1,
    WTCONV_BF16 = 2 /* the calls around the layer only; the layer's own refuse it */
} wtconv_dtype_t;

typedef enum {
    WTCONV_OP_FWD = 0,
    WTCONV_OP_BWD_DATA = 1,
    WTCONV_OP_BWD_WEIGHT = 2,
    WTCONV_OP_BWD = 3  /* wtconv_backward: dx and all parameter gradients */
} wtconv_op_t;

typedef struct {
    int64_t n, c, h, w;   /* activation shape, NCHW */
    int32_t k;            /* odd kernel size of the base and every per-level conv */
    int32_t levels;       /* number of Haar levels L */
    int32_t dtype;        /* wtconv_dtype_t of the activations */
} wtconv_desc_t;

/* hipStream_t without pulling in the HIP headers. */
typedef struct ihipStream_t *wtconv_stream_t;

/* Bytes of device workspace `op` needs for `desc` on the current device.  The
 * forward and the data backward need none when a plane fits one workgroup
 * (or L <= 1) and 2^L divides h and w; for larger planes with L >= 2 they keep
 * the level-1 low-pass map and the deeper levels' term there, and for sides
 * 2^L does not divide the zero-padded copies of the input and output.  Errors
 * as for the op itself. */
wtconv_status_t wtconv_workspace_size(const wtconv_desc_t *desc, wtconv_op_t op, size_t *bytes);

/* y = WTConv(x).  The per-channel scales are folded into the weights (and the
 * base scale into the bias) on chip, the Haar analysis is recomputed on chip
 * from the staged input, and the synthesis of all levels is one closed-form
 * pass indexed by the bits of each output coordinate (technical summary,
 * Methodology, reformulations 1-3).  x is read once and y written once. */
wtconv_status_t wtconv_forward(const wtconv_desc_t *desc, const void *x, const float *w_base, const float *bias,
                               const float *s_base, const float *w_lvl, const float *s_lvl, void *y,
                               void *workspace, size_t workspace_bytes, wtconv_stream_t stream);

/* dx = d<dy, WTConv(x)>/dx.  The layer is linear in x and the orthonormal Haar
 * synthesis is the transpose of the analysis, so this is the same fused pass
 * on dy with every kernel turned by 180 degrees and no bias.  Forward outputs
 * and all gradients are part of the method (technical summary, Key
 * Contributions). */
wtconv_status_t wtconv_backward_data(const wtconv_desc_t *desc, const void *dy, const float *w_base,
                                     const float *s_base, const float *w_lvl, const float *s_lvl, void *dx,
                                     void *workspace, size_t workspace_bytes, wtconv_stream_t stream);

/* Parameter gradients of <dy, WTConv(x)>, with the chain rule through the
 * folded scales (technical summary, Methodology, reformulation 3):
 *   dw_base = s0 * G0,  dbias = s0 * Gb,  ds_base = <W0, G0> + b0 * Gb,
 *   dw_lvl  = s_l * G_l, ds_lvl = <W_l, G_l>   (per channel and band),
 * where G0 / G_l are the correlations, summed over N, H and W, of dy (or its
 * Haar analysis) with x (or its Haar analysis) and Gb = sum dy.  Needs the
 * workspace from wtconv_workspace_size(desc, WTCONV_OP_BWD_WEIGHT).  dw_lvl and
 * ds_lvl may be NULL when L == 0. */
wtconv_status_t wtconv_backward_weight(const wtconv_desc_t *desc, const void *x, const void *dy,
                                       const float *w_base, const float *bias, const float *s_base,
                                       const float *w_lvl, const float *s_lvl, float *dw_base, float *dbias,
                                       float *ds_base, float *dw_lvl, float *ds_lvl, void *workspace,
                                       size_t workspace_bytes, wtconv_stream_t stream);

/* dx and all parameter gradients in one call (technical summary, Key
 * Contributions: forward outputs and all parameter gradients).  By default it
 * runs wtconv_backward_data and then wtconv_backward_weight.  With
 * WTCONV_FUSED_BWD=1 in the environment, planes that fit one workgroup run as
 * one fused pass instead: x and dy are read once, dy's Haar pyramid is built
 * once on chip and serves both the data backward's convolution (kernels turned
 * by 180 degrees) and the correlation with x's pyramid, and dx is written once
 * (5 E e bytes of activation traffic instead of 6 E e).  On MI355X the fused
 * pass measured slower than the two calls (it holds both pyramids and the
 * accumulators, so fewer waves stay in flight), hence the default.  The
 * results are those of the two calls (to rounding).  Arguments as theirs; dx
 * must not overlap x or dy; the workspace is wtconv_workspace_size(desc,
 * WTCONV_OP_BWD) under the same environment. */
wtconv_status_t wtconv_backward(const wtconv_desc_t *desc, const void *x, const void *dy, const float *w_base,
                                const float *bias, const float *s_base, const float *w_lvl, const float *s_lvl,
                                void *dx, float *dw_base, float *dbias, float *ds_base, float *dw_lvl, float *ds_lvl,
                                void *workspace, size_t workspace_bytes, wtconv_stream_t stream);

/* ---- The weight backward without a workspace argument --------------------
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation): the same
 * gradients as wtconv_backward_weight, with the partial results kept in a
 * static device array of WTCONV_NOALLOC_SCRATCH_BYTES bytes that the library
 * holds on every GPU it runs on until the process ends.  Nothing is allocated
 * by the call.  Calls whose workspace (wtconv_workspace_size(desc,
 * WTCONV_OP_BWD_WEIGHT)) exceeds the array return WTCONV_ERR_WORKSPACE before
 * anything is enqueued (planes that fit one workgroup need a few MB; the
 * large-plane paths with L >= 2 keep low-pass maps there and are refused).
 * All calls on one GPU share its array: calls that overlap on one GPU (on
 * different streams, or from several threads) race and give wrong gradients;
 * calls in stream order do not.  Other errors as for wtconv_backward_weight;
 * WTCONV_ERR_HIP if the array's device address cannot be obtained. */
#define WTCONV_NOALLOC_SCRATCH_BYTES (16u << 20)
wtconv_status_t wtconv_backward_weight_noalloc(const wtconv_desc_t *desc, const void *x, const void *dy,
                                               const float *w_base, const float *bias, const float *s_base,
                                               const float *w_lvl, const float *s_lvl, float *dw_base, float *dbias,
                                               float *ds_base, float *dw_lvl, float *ds_lvl, wtconv_stream_t stream);

/* ---- Unfused baseline (test and benchmark use only) ----------------------
 * The same layer composed of separate kernels with every intermediate in HBM:
 * per level a Haar analysis pass, a depthwise convolution pass and a scale
 * pass, then per level (deepest first) an add of the low-pass band and a
 * synthesis pass, and the base convolution, scale and final add (the
 * composition the pages measure the fused kernel against: technical summary,
 * Problem Statement, and its count of element moves).  The backward calls are
 * the step-by-step adjoints of that composition.  Same arguments as the fused
 * calls; the caller allocates one workspace of wtconv_unfused_workspace_size()
 * bytes (256-byte aligned) and passes the same workspace to all three calls:
 * the forward leaves its intermediates there and both backward calls read
 * them, so a backward call must follow a forward on the same inputs and
 * parameters.  Intermediates are stored in the activation type.  Errors:
 * WTCONV_ERR_SHAPE for an invalid descriptor, WTCONV_ERR_NULL for a missing
 * pointer, WTCONV_ERR_WORKSPACE when the workspace is too small,
 * WTCONV_ERR_HIP for a launch error. */
wtconv_status_t wtconv_unfused_workspace_size(const wtconv_desc_t *desc, size_t *bytes);
wtconv_status_t wtconv_unfused_forward(const wtconv_desc_t *desc, const void *x, const float *w_base,
                                       const float *bias, const float *s_base, const float *w_lvl,
                                       const float *s_lvl, void *y, void *workspace, size_t workspace_bytes,
                                       wtconv_stream_t stream);
wtconv_status_t wtconv_unfused_backward_data(const wtconv_desc_t *desc, const void *dy, const float *w_base,
                                             const float *s_base, const float *w_lvl, const float *s_lvl, void *dx,
                                             void *workspace, size_t workspace_bytes, wtconv_stream_t stream);
wtconv_status_t wtconv_unfused_backward_weight(const wtconv_desc_t *desc, const void *x, const void *dy,
                                               const float *w_base, const float *bias, const float *s_base,
                                               const float *w_lvl, const float *s_lvl, float *dw_base,
                                               float *dbias, float *ds_base, float *dw_lvl, float *ds_lvl,
                                               void *workspace, size_t workspace_bytes, wtconv_stream_t stream);

/* ---- Group norm with an activation ---------------------------------------
 * What follows the layer in a block.  Channels c of an image fall into
 * `groups` groups of C / groups neighbours; over the K = (C / groups) H W
 * values of a group
 *   mean = sum x / K,  rstd = 1 / sqrt(sum (x - mean)^2 / K + eps),
 *   y = act(gamma[c] * (x - mean) * rstd + beta[c]),
 * act one of wtconv_act_t.
 * Layouts      x (and dx) lie as x_layout says, y (and dy) as y_layout does:
 *              planes (WTCONV_NCHW) or channels last (WTCONV_NHWC), each
 *              without gaps.  The two may differ: planes in and channels last
 *              out is the step from the layer to a product over the channels.
 * Types        activations fp32, fp16 or bf16; gamma, beta [C] fp32, each may
 *              be NULL (ones, zeros); mean, rstd [N][groups] fp32.  All sums,
 *              statistics and products are fp32 (or wider); an output element
 *              is rounded once.
 * Shape rules  n, c, h, w >= 1, groups >= 1 divides c, c * h * w <= 2^31 - 2^16,
 *              n * c < 2^23, eps > 0 and finite.
 * Alignment    activations are aligned to their element; any such address
 *              works, 16-byte aligned ones are faster.
 * Values       a group with a NaN or an infinity comes out as NaN (relu of it
 *              included); other groups are not touched by it.  A group whose sum
 *              of squared differences passes fp32's range has an infinite
 *              variance: rstd 0, y = act(beta).  gelu's erf is within 1.5e-7.
 * Ownership, execution and errors are those of the layer's calls above:
 * kernels only, no allocation, no state, bitwise reproducible; the workspace
 * (256-byte aligned, wtconv_group_norm_workspace_size) belongs to one call at
 * a time. */
typedef enum { WTCONV_NCHW = 0, WTCONV_NHWC = 1 } wtconv_layout_t;

typedef enum {
    WTCONV_ACT_NONE = 0,
    WTCONV_ACT_RELU = 1, /* max(z, 0); slope 0 at z <= 0 */
    WTCONV_ACT_SILU = 2, /* z / (1 + exp(-z)) */
    WTCONV_ACT_GELU = 3  /* z / 2 (1 + erf(z / sqrt 2)) */
} wtconv_act_t;

typedef struct {
    int64_t n, c, h, w;
    int32_t groups;
    int32_t dtype;    /* wtconv_dtype_t of x, y, dy and dx */
    int32_t act;      /* wtconv_act_t */
    int32_t x_layout; /* wtconv_layout_t of x and dx */
    int32_t y_layout; /* wtconv_layout_t of y and dy */
    float eps;
} wtconv_norm_desc_t;

/* Bytes of workspace for op WTCONV_OP_FWD or WTCONV_OP_BWD (other ops:
 * WTCONV_ERR_UNSUPPORTED); may be 0. */
wtconv_status_t wtconv_group_norm_workspace_size(const wtconv_norm_desc_t *desc, wtconv_op_t op, size_t *bytes);

/* y, mean and rstd from x. */
wtconv_status_t wtconv_group_norm_forward(const wtconv_norm_desc_t *desc, const void *x, const float *gamma,
                                          const float *beta, void *y, float *mean, float *rstd, void *workspace,
                                          size_t workspace_bytes, wtconv_stream_t stream);

/* With dz = dy * act'(z), t = gamma dz, xh = (x - mean) rstd and E_g the mean
 * over a group:
 *   dx = rstd (t - E_g[t] - xh E_g[t xh]),
 *   dgamma = sum_{n,h,w} dz xh,  dbeta = sum_{n,h,w} dz.
 * mean and rstd are the forward call's.  dgamma and dbeta may each be NULL. */
wtconv_status_t wtconv_group_norm_backward(const wtconv_norm_desc_t *desc, const void *x, const void *dy,
                                           const float *gamma, const float *beta, const float *mean,
                                           const float *rstd, void *dx, float *dgamma, float *dbeta, void *workspace,
                                           size_t workspace_bytes, wtconv_stream_t stream);

/* ---- Newton-Schulz orthogonalisation and the Muon step --------------------
 * What is done with a weight gradient.  Each of `batch` matrices G of
 * rows x cols is divided by its norm and taken towards the nearest matrix with
 * orthonormal rows (or columns, where rows > cols) by `steps` steps of
 *   X <- a X + (b A + c A^2) X,  A = X X^T,  X_0 = G / (|G|_F + eps),
 *   (a, b, c) = (3.4445, -4.7750, 2.0315)
 * (on X^T where rows > cols), whose odd polynomial lifts every singular value
 * in (0, 1] towards about 1 (0.7 to 1.2).  The layer's parameters are such
 * matrices: w_base one of C x k^2, w_lvl L of 4C x k^2.
 * Types        g and out fp32, fp16 or bf16 (out in g's type, rounded once);
 *              in the Muon step g may be any of them, weight and momentum are
 *              fp32.  Norms sum in fp64.  Products keep 22 bits of each entry
 *              of their factors down to 2^-28 of the matrix's norm (an absolute
 *              2^-49 of it below) and sum in fp32.
 * Shape rules  1 <= batch <= 65535, 1 <= rows, cols <= 2^22, rows * cols < 2^31,
 *              batch * max(rows, 64) * max(cols, 64) < 2^36,
 *              the smaller of rows and cols <= WTCONV_ORTHO_MAX_SIDE, 1 <=
 *              steps <= WTCONV_ORTHO_MAX_STEPS, eps >= 0 and finite (a zero matrix
 *              gives zeros, for eps = 0 NaN).
 * Layout       row-major, matrices one after the other, no gaps; aligned to the
 *              element.
 * Values       a matrix with a NaN or an infinity comes out as NaN; the others
 *              of the batch are not touched by it.
 * Ownership, execution and errors as above; one workspace of
 * wtconv_orthogonalize_workspace_size bytes (256-byte aligned) serves one of
 * the two calls at a time. */
#define WTCONV_ORTHO_MAX_SIDE 16384
#define WTCONV_ORTHO_MAX_STEPS 16

typedef struct {
    int64_t batch, rows, cols;
    int32_t dtype; /* wtconv_dtype_t of g (and out) */
    int32_t steps;
    float eps;
} wtconv_ortho_desc_t;

wtconv_status_t wtconv_orthogonalize_workspace_size(const wtconv_ortho_desc_t *desc, size_t *bytes);

/* out = the iteration above on g; out must not overlap g. */
wtconv_status_t wtconv_orthogonalize(const wtconv_ortho_desc_t *desc, const void *g, void *out, void *workspace,
                                     size_t workspace_bytes, wtconv_stream_t stream);

typedef struct {
    float lr, momentum, weight_decay;
    float scale;      /* factor of the update next to lr, e.g. sqrt(max(1, rows / cols)) */
    int32_t nesterov; /* 0 or 1 */
} wtconv_muon_t;

/* One optimiser step:
 *   momentum_out = mu momentum + (1 - mu) grad,
 *   u = nesterov ? mu momentum_out + (1 - mu) grad : momentum_out,
 *   weight_out = (1 - lr weight_decay) weight - lr scale orthogonalize(u).
 * weight_out may be weight and momentum_out momentum (in place); other
 * overlaps of an output with an argument are refused.  The hyperparameters
 * are passed by value: a captured call replays with those it was captured
 * with. */
wtconv_status_t wtconv_muon_step(const wtconv_ortho_desc_t *desc, const wtconv_muon_t *hyper, const float *weight,
                                 const void *grad, const float *momentum, float *weight_out, float *momentum_out,
                                 void *workspace, size_t workspace_bytes, wtconv_stream_t stream);

/* ---- Root-mean-square norm with the residual's addition --------------------
 * In front of the products over the channels, channels last: for each of `rows`
 * rows of c values
 *   h = x + residual (as stored, in the activations' type; h = x where residual is NULL),
 *   rstd = 1 / sqrt(sum h^2 / c + eps),  y = gamma h rstd.
 * Layout       x, residual, y, h and their gradients row-major [rows][c], no
 *              gaps; gamma [c] fp32 or NULL (ones); rstd [rows] fp32.
 * Types        fp32, fp16 or bf16, one for all of a call's activations.  Sums and
 *              products are fp32 (or wider); an output element is rounded once.
 * Shape rules  rows, c >= 1, c <= 2^24, rows * c < 2^40, rows < 2^31, eps > 0 and
 *              finite.
 * Alignment    to the element; 16-byte aligned activations are faster.
 * Values       a row with a NaN or an infinity comes out as NaN or zero times it;
 *              no other row is touched by it.  A row whose sum of squares passes
 *              fp32's range has rstd 0 and y = 0.
 * Ownership, execution and errors are those of the layer's calls above. */
typedef struct {
    int64_t rows, c;
    int32_t dtype; /* wtconv_dtype_t of the activations */
    float eps;
} wtconv_rms_desc_t;

/* Bytes of workspace for op WTCONV_OP_FWD (0) or WTCONV_OP_BWD. */
wtconv_status_t wtconv_rms_norm_workspace_size(const wtconv_rms_desc_t *desc, wtconv_op_t op, size_t *bytes);

/* y, rstd and, where residual is given, h (else h is not written and may be
 * NULL).  h may be x or residual themselves (in place); other overlaps of an
 * output with an argument are refused. */
wtconv_status_t wtconv_rms_norm_forward(const wtconv_rms_desc_t *desc, const void *x, const void *residual,
                                        const float *gamma, void *y, void *h, float *rstd, wtconv_stream_t stream);

/* With t = gamma dy and hh = h rstd:
 *   dx = rstd (t - hh sum(t hh) / c) + dh   (also the residual's gradient),
 *   dgamma = sum over the rows of dy hh.
 * h and rstd are the forward call's; dh (the gradient that reaches h by its other
 * way) may be NULL, and so may dgamma.  dx may be dh itself (in place). */
wtconv_status_t wtconv_rms_norm_backward(const wtconv_rms_desc_t *desc, const void *h, const void *dy,
                                         const void *dh, const float *gamma, const float *rstd, void *dx,
                                         float *dgamma, void *workspace, size_t workspace_bytes,
                                         wtconv_stream_t stream);

/* ---- Gated product over the channels ---------------------------------------
 * The first half of a gated feed-forward block, both projections, the activation
 * and the product in one kernel: for each row of x (a pixel, channels last)
 *   g = x w_gate^T + b_gate,  u = x w_up^T + b_up,  h = act(g) * u,
 * act one of wtconv_act_t.
 * Layout       x [rows][c], h [rows][f], w_gate and w_up [f][c], all row-major, no
 *              gaps; b_gate, b_up [f] fp32, each may be NULL (zeros).
 * Types        activations, weights and their gradients fp32, fp16 or bf16, one
 *              for all of a call's; biases and their gradients fp32.  Products of
 *              16-bit types are exact and sum in fp32.  fp32 factors are taken as
 *              three bf16 numbers each (24 bits), whose products of up to 2^-16 of
 *              the whole are kept (those left out are at most 2^-24 of it).  The
 *              backward pass holds dg and du in the activations' type between its
 *              products: dx and the weights' gradients see them rounded by half a step
 *              of it.  fp16: they become infinite beyond 65504, lose digits below 2^-14
 *              (steps of 2^-24) and are zero below 2^-25, as any fp16 gradient, so that
 *              losses are to be scaled as for those.  The biases' gradients sum them
 *              before that rounding.
 * Shape rules  rows, c, f >= 1, c and f <= 65536, rows < 2^30, rows * c and rows * f
 *              < 2^36.
 * Alignment    x and the weights 16 bytes in 16-bit types where 8 divides c, else to the
 *              element; the others to the element (16 bytes is faster).
 * Values       a row with a NaN or an infinity gives NaN or an infinity in that
 *              row of h and dx, and in the weights' gradients; no other row is
 *              touched by it.  gelu's erf is within 1.5e-7; relu's slope at a g that
 *              rounds to zero is 0.
 * Ownership, execution and errors are those of the layer's calls above; one
 * workspace of wtconv_gated_workspace_size bytes serves one call at a time. */
typedef struct {
    int64_t rows, c, f;
    int32_t dtype; /* wtconv_dtype_t of activations and weights */
    int32_t act;   /* wtconv_act_t */
} wtconv_gated_desc_t;

/* Bytes of workspace for op WTCONV_OP_FWD or WTCONV_OP_BWD; may be 0. */
wtconv_status_t wtconv_gated_workspace_size(const wtconv_gated_desc_t *desc, wtconv_op_t op, size_t *bytes);

wtconv_status_t wtconv_gated_forward(const wtconv_gated_desc_t *desc, const void *x, const void *w_gate,
                                     const void *w_up, const float *b_gate, const float *b_up, void *h,
                                     void *workspace, size_t workspace_bytes, wtconv_stream_t stream);

/* With dg = dh u act'(g) and du = dh act(g), g and u computed again from x:
 *   dx = dg w_gate + du w_up,
 *   dw_gate = dg^T x,  dw_up = du^T x,  db_gate = sum dg,  db_up = sum du.
 * dx may be NULL, dw_gate and dw_up both, and db_gate and db_up both: what is
 * not asked for is not computed (at least one output is). */
wtconv_status_t wtconv_gated_backward(const wtconv_gated_desc_t *desc, const void *x, const void *dh,
                                      const void *w_gate, const void *w_up, const float *b_gate, const float *b_up,
                                      void *dx, void *dw_gate, void *dw_up, float *db_gate, float *db_up,
                                      void *workspace, size_t workspace_bytes, wtconv_stream_t stream);

/* The same with the weights' gradients in fp32, whatever the activations' type, for
 * parameters that are kept in fp32 under 16-bit activations: the sums come out as they
 * are, with their digits and beyond 65504. */
wtconv_status_t wtconv_gated_backward_f32_grads(const wtconv_gated_desc_t *desc, const void *x, const void *dh,
                                                const void *w_gate, const void *w_up, const float *b_gate,
                                                const float *b_up, void *dx, float *dw_gate, float *dw_up,
                                                float *db_gate, float *db_up, void *workspace,
                                                size_t workspace_bytes, wtconv_stream_t stream);

/* ---- Global gradient norm and clipping --------------------------------------
 * What stands between a backward pass and the optimiser's step: over all elements
 * g of `count` tensors, of any types among fp32, fp16 and bf16,
 *   norm = sqrt(sum g^2),  out = g * min(1, max_norm / (norm + eps)).
 * The squares and their sum are fp64 (fp32's range of g has no effect on it), the
 * result is rounded to fp32 once (infinity beyond fp32's range), an element of out
 * once to its type.  A NaN among the elements makes the norm and every output NaN,
 * an infinity makes the norm infinite, the finite elements' outputs zero and its own
 * NaN.
 * Shape rules  0 <= count <= 65536 (0: norm 0), elems >= 0 each, less than 2^40
 *              together; max_norm >= 0 and eps >= 0, both finite, and not both 0.
 * Layout       contiguous elements, aligned to the element (16 bytes is faster).  The
 *              table is host memory, read before the call returns; a captured
 *              call replays with the addresses it was captured with.
 * An out may be its own grad (in place; where nothing is clipped nothing is then
 * written); other overlaps of an output with a tensor are refused.
 * Ownership, execution and errors are those of the layer's calls above; a workspace
 * of wtconv_grad_norm_workspace_size bytes serves one of the two calls at a time. */
typedef struct {
    const void *grad;
    void *out;      /* wtconv_clip_grad_norm only */
    int64_t elems;
    int32_t dtype;  /* wtconv_dtype_t of grad and out */
    int32_t unused; /* 0 */
} wtconv_tensor_t;

wtconv_status_t wtconv_grad_norm_workspace_size(int64_t count, size_t *bytes);

wtconv_status_t wtconv_grad_norm(const wtconv_tensor_t *tensors, int64_t count, float *norm, void *workspace,
                                 size_t workspace_bytes, wtconv_stream_t stream);

wtconv_status_t wtconv_clip_grad_norm(const wtconv_tensor_t *tensors, int64_t count, float max_norm, float eps,
                                      float *norm, void *workspace, size_t workspace_bytes, wtconv_stream_t stream);

/* Human-readable name of a status code (static string). */
const char *wtconv_status_string(wtconv_status_t status);

/* Library version, "major.minor.patch". */
const char *wtconv_version(void);

#ifdef __cplusplus
}
#endif

#endif /* WTCONV_H */
