/*
 * disco.h — C ABI of the gfx950 DISCO sparse-contraction library (libdisco.so).
 *
 * The operations are the three named on the torch-harmonics "disco-kernel-dev"
 * page, section "Architecture snapshot":
 *   - the CSR sparse contraction from the input grid to the K-expanded output
 *     (B, C, K, Ho, Wo)                                        -> disco_fwd
 *   - the CSR transpose contraction from (B, C, K, Ho, Wo) back to the input
 *     grid, computed as an atomic-free gather (section "Backward direction —
 *     gather vs scatter": each input pixel accumulates from its neighbourhood)
 *                                                              -> disco_bwd
 *   - contraction followed by the dense channel/basis einsum    -> disco_fused_conv
 *
 * With s = Wi / Wo (an integer >= 1) and psi rows r = k*Ho + ho:
 *   out[b,c,k,ho,wo] = sum_{e in row r} val_e * x[b,c,hi_e,(wi_e + s*wo) mod Wi]
 *   gx = F^T gout      (exact transpose of the map above)
 *   y[b,o,ho,wo]     = sum_{c,k} W[o,c,k] * out[b,c,k,ho,wo]
 *
 * Conventions shared by every call
 *   - Tensors are dense, contiguous, row-major, last index fastest; `data` is a
 *     device pointer on the device the psi handle was created on.  The caller
 *     owns every tensor buffer.
 *   - Supported dtypes: DISCO_F32, DISCO_BF16 and DISCO_F16 (the precisions
 *     the page's test rules name, section "Test coverage requirements").  All
 *     tensors of one call share one dtype.  Accumulation is always fp32; a
 *     16-bit output is rounded once (round-to-nearest-even) from the fp32
 *     accumulator.  psi values are fp32 (kpacked section of the page: values
 *     stored as fp32), except on the bf16 matrix-core paths, which take psi
 *     rounded to bf16 as their multiplicand.
 *   - Outputs are fully overwritten (no accumulate flag); rows with no psi
 *     entries are written as exact zeros.
 *   - `stream` is a hipStream_t (0 = the null stream).  Work is enqueued
 *     asynchronously; the calls never synchronise the host with the device.
 *   - Every argument is validated on the host before anything is enqueued; on
 *     any error nothing is written and a status is returned.  The text of the
 *     last error of the calling thread is available from disco_last_error().
 *   - Only gfx950 devices are accepted (the page's kernels check the device
 *     architecture on the host and refuse others; section "Adding a new kernel
 *     variant", step 1).
 */
#ifndef DISCO_H
#define DISCO_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum disco_status {
    DISCO_OK = 0,
    DISCO_ERR_INVALID_ARGUMENT = 1,   /* null handle / tensor / data pointer, wrong device */
    DISCO_ERR_SHAPE = 2,              /* Wi % Wo != 0, or shapes disagree with psi / each other */
    DISCO_ERR_DTYPE = 3,              /* dtype not F32/BF16/F16, unsupported by the op, or dtypes of one call differ */
    DISCO_ERR_PSI = 4,                /* malformed CSR (row_ptr, column range, nnz >= 2^31) */
    DISCO_ERR_UNSUPPORTED_DEVICE = 5, /* device is not gfx950 */
    DISCO_ERR_OOM = 6,                /* device or host allocation failed */
    DISCO_ERR_HIP = 7                 /* a HIP runtime call or kernel launch failed */
} disco_status;

typedef enum disco_dtype {
    DISCO_F32 = 0,
    DISCO_BF16 = 1,
    DISCO_F16 = 2,
    DISCO_F8_E4M3 = 3,        /* 8-bit forms (OCP): disco_rms_norm_f8 and disco_dequantize only */
    DISCO_F8_E5M2 = 4
} disco_dtype;

/* Host-side CSR filter ("psi").  Rows r = k*Ho + ho, K*Ho rows in all.
 * Column of an entry = input pixel (col_hi[e], col_wi[e]): the input latitude
 * and the longitude offset from output longitude 0.  Entries of one row may be
 * in any order; a (hi, wi) pair may appear at most once per row.
 * All arrays are host memory, read during disco_psi_create only. */
typedef struct disco_csr_desc {
    int32_t K, Ho, Wo, Hi, Wi;
    int64_t nnz;              /* must equal row_ptr[K*Ho] and be < 2^31 */
    const int64_t *row_ptr;   /* [K*Ho + 1], row_ptr[0] == 0, non-decreasing */
    const int32_t *col_hi;    /* [nnz], in [0, Hi) */
    const int32_t *col_wi;    /* [nnz], in [0, Wi) */
    const float *val;         /* [nnz] */
} disco_csr_desc;

/* Device tensor view.  shape[0..ndim-1] are used; the rest are ignored. */
typedef struct disco_tensor {
    void *data;               /* device pointer */
    int32_t dtype;            /* disco_dtype */
    int32_t ndim;
    int64_t shape[5];
} disco_tensor;

typedef struct disco_psi_s *disco_psi;

/* Validate the CSR, derive the device plans (longitude-run segments of the
 * forward rows grouped by shared support, and the row-inverted psi used by the
 * backward gather), and upload them to `device` (a HIP device ordinal).
 * Host arrays are copied; the caller may free them on return.  May block the
 * host until the uploads finish.  On success *out_handle owns all device
 * memory of the plan; release it with disco_psi_destroy.  A handle is
 * read-only after creation and may be used from several streams at once. */
disco_status disco_psi_create(const disco_csr_desc *csr, int device, disco_psi *out_handle);

/* Free a handle (NULL is accepted).  The caller must ensure no enqueued call
 * still uses it. */
disco_status disco_psi_destroy(disco_psi h);

/* Forward contraction.  x: (B, C, Hi, Wi) -> out: (B, C, K, Ho, Wo). */
disco_status disco_fwd(disco_psi h, const disco_tensor *x, disco_tensor *out, void *stream);

/* Transpose contraction.  gout: (B, C, K, Ho, Wo) -> gx: (B, C, Hi, Wi).
 * Atomic-free: every gx element is produced by one thread in a fixed order,
 * so results are bitwise reproducible run to run. */
disco_status disco_bwd(disco_psi h, const disco_tensor *gout, disco_tensor *gx, void *stream);

/* Fused convolution.  x: (B, C, Hi, Wi), W: (Co, C, K) -> y: (B, Co, Ho, Wo).
 * The contraction is computed on chip in channel chunks and never written to
 * device memory.  BF16 and F16: the einsum runs on bf16 or fp16 MFMA tiles with
 * fp32 accumulation (contraction chunks are rounded to the data type before the
 * MFMA).  F32: fp32 throughout (fp32 psi, an fp32 contraction chunk, the einsum
 * on the fp32 matrix cores) — the fp32 variant the 16-bit ones are compared
 * with (same page, "Test coverage requirements").
 * Memory: with BF16/F16 data and K < 16 the call takes a temporary of Co * C * 32 bytes from a
 * memory pool the library keeps per device (stream-ordered: taken and returned on `stream`; the pool
 * keeps freed memory for reuse until the process ends) to hold W in rows of 16 elements; if none can be
 * had the kernel stages W element by element instead, with the same result.  With F32 data, and with
 * 16-bit data on shapes outside the matrix-core kernel's plan (K > 16, Wi > 2 Wo, Wo not a multiple of 8),
 * the call takes a temporary of the same pool holding W in the vector-ALU fused kernel's einsum operand
 * order (Co and C rounded up to its 16-channel tiles and channel chunks: about Co * C * K elements); if
 * none can be had the call returns DISCO_ERR_OOM before anything is written. */
disco_status disco_fused_conv(disco_psi h, const disco_tensor *x, const disco_tensor *W,
                              disco_tensor *y, void *stream);

/* Fused convolution that also keeps its contraction, for a training step whose backward then need not
 * recompute it: y as disco_fused_conv, and out[b,c,k,ho,wo] = the contraction F x (B, C, K, Ho, Wo) in
 * the data type (each fp32 accumulator rounded once, RNE).  On the matrix-core fused kernel (BF16 and
 * F16 data on its plan) out holds the very values the einsum multiplied; otherwise (F32 data, shapes
 * outside that plan) out comes from disco_fwd, whose summation order may differ from the fused
 * kernel's by rounding.  Same page, "Python dispatch layer": the fused autograd function keeps what
 * its backward needs.  out is caller-owned and overwritten; it must not overlap x, W or y
 * (DISCO_ERR_INVALID_ARGUMENT). */
disco_status disco_fused_conv_save(disco_psi h, const disco_tensor *x, const disco_tensor *W, disco_tensor *y,
                                   disco_tensor *out, void *stream);

/* The einsum alone: the second half of the fused convolution, for a contraction that is already
 * in device memory (for instance the forward's output kept for the weight gradient).  Same page,
 * "Architecture snapshot" ("contraction + einsum"):
 *   y[b,o,ho,wo] = sum_{c,k} W[o,c,k] * t[b,c,k,ho,wo]
 * t: (B, C, K, Ho, Wo), W: (Co, C, K) -> y: (B, Co, Ho, Wo), on the current device (no psi).
 * BF16 and F16 only, K <= 16 (DISCO_ERR_SHAPE otherwise).  Runs the fused kernel's matrix-core
 * einsum tile with t streamed from device memory: fp32 accumulation in a fixed order, y rounded
 * once (RNE), bitwise reproducible run to run.  All tensors are caller-owned; y is overwritten.
 * K < 16 takes the same stream-ordered W temporary as disco_fused_conv (same fallback). */
disco_status disco_einsum(const disco_tensor *W, const disco_tensor *t, disco_tensor *y, void *stream);

/* Backward of the fused convolution: the gradients of <gy, y> for y = disco_fused_conv(x, W),
 *   gx[b,c]   = F^T g[b,c],  g[b,c,k,ho,wo] = sum_o W[o,c,k] * gy[b,o,ho,wo]
 *   dW[o,c,k] = sum_{b,ho,wo} gy[b,o,ho,wo] * out[b,c,k,ho,wo],  out = F x
 * (torch-harmonics "disco-kernel-dev" page, "Python dispatch layer": the fused autograd function
 * pairs the fused forward with the CSR transpose backward; "Test coverage requirements": fused
 * and unfused agree in output and gradient).
 * x: (B, C, Hi, Wi), W: (Co, C, K), gy: (B, Co, Ho, Wo) -> gx: (B, C, Hi, Wi), dW: (Co, C, K).
 * BF16 and F16; Co and Ho*Wo must be multiples of 8, K <= 256, and one batch of gy, of a channel
 * chunk of g, and W must each stay below 2 GiB (the matrix-core loads address 32-bit offsets).
 * gx: when Wi = Wo and K <= 16, gx[b,c] = sum_{o,k} W[o,c,k] (F_k^T gy[b,o]) is the fused convolution
 * of gy over the per-basis transpose of psi (built by disco_psi_create) with W' = W permuted to
 * (C, Co, K), its contraction rounded to the data type before the einsum as in disco_fused_conv;
 * otherwise channel chunks of g (the data type, on the matrix cores) and the transpose contraction.
 * dW: the forward contraction (the data type) per channel chunk and a split product whose fp32
 * partials are summed in a fixed order.  Results are bitwise reproducible run to run.  gx and dW must not overlap any
 * input (DISCO_ERR_INVALID_ARGUMENT).  `workspace` is caller-owned device memory (256-byte aligned) of at
 * least the size disco_fused_conv_bwd_workspace reports for (B, C, Co); its contents on entry
 * are ignored and on return are unspecified.  Calls sharing one workspace must not overlap.
 * Where gx takes the fused launch, the recomputed contraction and the dW products run on the
 * library's second stream beside it, with the same ordering guarantees as disco_fused_conv_bwd_saved
 * (the call behaves as if everything ran on `stream`). */
disco_status disco_fused_conv_bwd_workspace(disco_psi h, int64_t B, int64_t C, int64_t Co, size_t *bytes);
disco_status disco_fused_conv_bwd(disco_psi h, const disco_tensor *x, const disco_tensor *W, const disco_tensor *gy,
                                  disco_tensor *gx, disco_tensor *dW, void *workspace, size_t workspace_bytes,
                                  void *stream);

/* The same backward with the weight gradient's operand taken from `out`, the contraction that
 * disco_fused_conv_save wrote for the same x, instead of recomputing it from x (x is not needed).
 * out: (B, C, K, Ho, Wo); the other arguments, the workspace and the results as disco_fused_conv_bwd,
 * whose results it reproduces bitwise when out comes from disco_fused_conv_save.
 * The weight-gradient products run on a second stream that the library keeps per device (default
 * priority, created on first use, never destroyed): it waits for everything enqueued on `stream`
 * before the call, and `stream` waits for it before the call returns (also on an error return), so
 * the call behaves as if everything ran on `stream`.  Concurrent calls on one device share that
 * stream, so their weight-gradient work serialises; under graph capture of `stream` the fork and
 * join are captured as event dependencies. */
disco_status disco_fused_conv_bwd_saved(disco_psi h, const disco_tensor *out, const disco_tensor *W,
                                        const disco_tensor *gy, disco_tensor *gx, disco_tensor *dW, void *workspace,
                                        size_t workspace_bytes, void *stream);

/* The backward of the fused convolution (the same operation, results and restrictions as
 * disco_fused_conv_bwd) for callers that cannot allocate device memory: code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation.  It takes no workspace and calls
 * no allocating routine: its workspace is the library's own scratch array of 64 MiB per device
 * (held from the library's load until the process ends).  The channel chunks shrink until the
 * workspace fits; shapes whose workspace cannot fit 64 MiB are refused with DISCO_ERR_SHAPE before
 * anything is enqueued (the fixed buffers alone must fit: 32 C Co bytes of permuted W where gx takes the
 * fused launch over the transposed psi, else 2 (C K Co + B Ho Wo Co) bytes of W^T and gy^T).  Every call on
 * one device uses the same array: calls that overlap on one device (other streams, other threads)
 * race and must not be issued.  The array's contents on entry are ignored. */
disco_status disco_fused_conv_bwd_noalloc(disco_psi h, const disco_tensor *x, const disco_tensor *W,
                                          const disco_tensor *gy, disco_tensor *gx, disco_tensor *dW, void *stream);

/* ---- the operators around the convolution in a residual model's training step -------------------------
 *
 * They take dense tensors of 1 to 5 dimensions and no psi, and run on the current device.  `axis` is the
 * normalised axis (negative: counted from the end): 1 for fields (B, C, H, W), the last one for rows
 * (points, C).  D is the axis's size (at least 1).  Tensors need only their element's alignment, so views
 * into a flat buffer serve.  Outputs must overlap neither inputs nor each other
 * (DISCO_ERR_INVALID_ARGUMENT).  All statistics are fp32 or wider, each output is rounded once (RNE), and
 * results are bitwise reproducible run to run.  Nothing is allocated on the device, so every call can be
 * captured into a graph.  A tensor with no elements is accepted and nothing is launched for it.
 * Squares are fp32 sums: a row whose sum of squares passes fp32's range (|h| near 2^64 / sqrt(D)) has rstd 0, and
 * squares of |h| below 2^-75 are 0, so with eps = 0 a row of nothing else has an infinite rstd. */

/* Root-mean-square norm over `axis`, of x or, with `residual`, of h = x + residual:
 *   y = h * rstd * w,   rstd = (mean(h^2) + eps)^(-1/2)
 * x, residual, y, h: one shape and dtype (F32, BF16 or F16); w: (D,), F32 or that dtype.  With a residual
 * `h` receives the sum (rounded; the norm itself uses the unrounded fp32 sum); residual and h are given
 * together or both NULL.  NaN and infinities follow the formula: one in a row makes that row NaN or zero,
 * and no other. */
disco_status disco_rms_norm(const disco_tensor *x, const disco_tensor *residual, const disco_tensor *w, int axis,
                            float eps, disco_tensor *y, disco_tensor *h, void *stream);

/* The same norm with its output in 8 bits: q (x's shape, DISCO_F8_E4M3 or DISCO_F8_E5M2) and fp32 scales,
 * one for each run of `group` entries along the axis (0: one for the whole axis; else a multiple of 32; the
 * last run may be shorter):
 *   scale = max(max|y| over the run / qmax, 2^-126),  q = y / scale rounded (RNE),  qmax = 448 or 57344
 * from the unrounded fp32 y.  scale: x's shape with the axis replaced by the number of runs.  A NaN in a run
 * makes its scale and all its q NaN. */
disco_status disco_rms_norm_f8(const disco_tensor *x, const disco_tensor *residual, const disco_tensor *w, int axis,
                               float eps, int64_t group, disco_tensor *q, disco_tensor *scale, disco_tensor *h,
                               void *stream);

/* out = q * scale, the reader of that form: q, scale, axis and group as disco_rms_norm_f8 gives them; out: q's
 * shape, F32, BF16 or F16. */
disco_status disco_dequantize(const disco_tensor *q, const disco_tensor *scale, int axis, int64_t group,
                              disco_tensor *out, void *stream);

/* Backward of disco_rms_norm.  h: the tensor the norm was taken of (the stored sum, or x without a residual),
 * gy: the gradient of y, gh: the gradient that reaches h past the norm (the residual path) or NULL.  With g = gy * w:
 *   gx = rstd * g - h * rstd^3 * mean(g h) + gh     (the gradient of x, and of the residual)
 *   dw = sum over all points of gy * h * rstd
 * h, gy, gh, gx: one shape and dtype; w, dw: (D,), F32 or that dtype, both alike.  `workspace` is caller-owned
 * device memory (4-byte aligned) of at least the size disco_rms_norm_bwd_workspace reports for h (its data is not
 * read); its contents on entry are ignored.  Calls sharing one workspace must not overlap.  With no points
 * (an empty h) dw is written as zeros. */
disco_status disco_rms_norm_bwd_workspace(const disco_tensor *h, int axis, size_t *bytes);
disco_status disco_rms_norm_bwd(const disco_tensor *h, const disco_tensor *w, const disco_tensor *gy,
                                const disco_tensor *gh, int axis, float eps, disco_tensor *gx, disco_tensor *dw,
                                void *workspace, size_t workspace_bytes, void *stream);

/* norm = sqrt(sum of the squares of all elements of the n tensors), squares summed in fp64.  The tensors may
 * differ in shape and dtype (F32, BF16, F16) and may be empty; n may be 0 (norm 0).  norm: one F32 element.
 * `workspace`: caller-owned device memory (8-byte aligned) of at least the size disco_grad_norm_workspace
 * reports for these tensors (their data is not read), as disco_rms_norm_bwd's.  Tensors that follow each other in
 * memory are walked as one; all of them together have at most 2^40 elements. */
disco_status disco_grad_norm_workspace(int64_t n, const disco_tensor *grads, size_t *bytes);
disco_status disco_grad_norm(int64_t n, const disco_tensor *grads, disco_tensor *norm, void *workspace,
                             size_t workspace_bytes, void *stream);

/* Clipping by that norm: outs[i] = grads[i] * min(1, max_norm / (norm + eps)), each rounded once; norm is the
 * norm before clipping.  outs[i] has the shape and dtype of grads[i] and is either the same memory (in place;
 * nothing is rewritten where the factor is 1) or disjoint from everything else.  max_norm may be infinite (no
 * limit).  Where norm + eps and max_norm are both 0 the factor is 1.  A NaN gradient makes every output NaN, an infinite
 * one makes finite elements 0 and infinite ones NaN, whatever max_norm is.  The factor stays on the device. */
disco_status disco_clip_grads(int64_t n, const disco_tensor *grads, float max_norm, float eps, disco_tensor *outs,
                              disco_tensor *norm, void *workspace, size_t workspace_bytes, void *stream);

/* Message of the last non-OK status returned on the calling thread ("" if none). */
const char *disco_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* DISCO_H */
