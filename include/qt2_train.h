/*
 * qt2_train.h -- C ABI of the training operators beside the quantized linears (qt2.h) for NVIDIA
 * B200 (sm_100a), in the library libqt2_train.so: layer norm, the head's softmax cross entropy
 * over a large vocabulary, and the global gradient norm with clipping, each with what a training
 * step needs of it.
 *
 * Conventions are those of qt2.h (device pointers owned by the caller, work enqueued on `stream`,
 * arguments validated on the host before any launch, negative qt2_status on error, no allocation,
 * no abort, one NVTX range per call), with these differences:
 *   - Dimensions are any positive ints below 2^30, not multiples of 128 (a matrix of the head loss
 *     has fewer than 2^44 elements).  Matrices are row-major with a leading dimension that is a
 *     multiple of 8 elements, at least the row's length and below 2^40 (x and w of the head loss:
 *     2^39), and 16-byte aligned bases.  Elements between a row's length and its leading dimension
 *     are neither used nor written.  All other arrays are contiguous.
 *   - Outputs and workspaces must not overlap inputs or each other, except where a call says so.
 *     Two calls that can run at the same time need workspaces of their own (as do two captured
 *     graphs that can).
 *   - Inputs may be inf or NaN: what the formulas give for them is what comes out, unless a call
 *     says otherwise.
 *   - Every result is a deterministic function of the inputs: no atomics order any sum.
 *   - The library has a device status word, a fault hook and a checked build of its own
 *     (libqt2_train_checked.so), which work as those of qt2.h do.
 */
#ifndef QT2_TRAIN_H
#define QT2_TRAIN_H

#include "qt2.h"

#ifdef __cplusplus
extern "C" {
#endif

/* qt2_device_status, qt2_set_fault_hook and qt2_build_checked of this library.  Its kernels
 * report QT2_ERR_TIMEOUT, QT2_ERR_INVALID_ARG (a target outside the vocabulary), and in the
 * checked build QT2_ERR_BOUNDS. */
QT2_API qt2_status qt2_train_device_status(qt2_stream_t stream, int *code);
QT2_API void qt2_train_set_fault_hook(qt2_fault_hook hook, void *user);
QT2_API int qt2_train_build_checked(void);

/* ---------------------------------------------------------------------------------------
 * Layer norm over the rows of x [rows][cols]:
 *   mean_r = sum_c x_rc / cols,  rstd_r = 1/sqrt(sum_c (x_rc - mean_r)^2 / cols + eps),
 *   y_rc = (x_rc - mean_r) * rstd_r * weight_c + bias_c.
 * x and y have type x_dtype (QT2_DTYPE_*), weight and bias [cols] w_dtype, 16-byte aligned; a
 * NULL weight stands for ones, a NULL bias for zeros.  mean and rstd [rows] (fp32) are what the
 * backward pass needs; both may be NULL where there is none.  Statistics and products are fp32
 * (the variance from the differences to the mean, not from squares), rounded once on writing.
 * eps >= 0 and finite.  y may be x (with ldy = ldx).
 * --------------------------------------------------------------------------------------- */
QT2_API qt2_status qt2_layernorm_fwd(const void *x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx,
                                     const void *weight, const void *bias, int w_dtype, float eps, void *y,
                                     int64_t ldy, float *mean, float *rstd, qt2_stream_t stream);

/* ---------------------------------------------------------------------------------------
 * Backward of the layer norm, with h_rc = (x_rc - mean_r) * rstd_r and a_rc = dy_rc * weight_c:
 *   dx_rc = rstd_r * (a_rc - sum_c a_rc / cols - h_rc * sum_c (a_rc h_rc) / cols),
 *   dweight_c = sum_r dy_rc h_rc,  dbias_c = sum_r dy_rc.
 * dy, x and dx have type x_dtype; weight (NULL: ones), dweight and dbias w_dtype, 16-byte aligned.
 * dx, dweight and dbias may each be NULL (not wanted), not all of them.  dx may be dy (with lddx = lddy).
 * Sums are fp32.  Workspace: qt2_layernorm_bwd_workspace_size() bytes, 256-byte aligned.
 * --------------------------------------------------------------------------------------- */
QT2_API qt2_status qt2_layernorm_bwd_workspace_size(int64_t rows, int64_t cols, size_t *bytes);
QT2_API qt2_status qt2_layernorm_bwd(const void *dy, int64_t lddy, const void *x, int x_dtype, int64_t rows,
                                     int64_t cols, int64_t ldx, const void *weight, int w_dtype, const float *mean,
                                     const float *rstd, void *dx, int64_t lddx, void *dweight, void *dbias,
                                     void *workspace, size_t ws_bytes, qt2_stream_t stream);

/* ---------------------------------------------------------------------------------------
 * Head loss: softmax cross entropy of the logits l = x w^T, x [T][K] and w [V][K] bf16, against
 * targets [T] (int64):
 *   lse_t = log sum_v exp(l_tv),  loss_t = lse_t - l_t,target(t).
 * The logits are formed piece by piece of the vocabulary on the tensor cores (fp32 sums) and never
 * stored; the target's logit is formed again in fp32.  loss and lse [T] are fp32.  The tensor cores' sums
 * truncate: a logit other than the target's is off by up to (K/16 + 16) 2^-23 of the sum of its products'
 * magnitudes (measured, products of one sign: 3e-6 of it at K = 1024, 1.7e-5 at 4096, 9e-5 at 16384), and so
 * are loss and lse in rows that such a logit dominates.  Where the target dominates they are off by 1e-6 of the
 * largest logit at most, where products have either sign and many entries count by about 2e-7 (2-norm).  Rows whose target is ignore_index have
 * loss 0 (their lse is still written).  Any other target outside [0, V) is treated as ignore_index and
 * reported as QT2_ERR_INVALID_ARG through qt2_train_device_status.
 * Workspace: qt2_linear_xent_fwd_workspace_size() bytes, 256-byte aligned.
 * --------------------------------------------------------------------------------------- */
QT2_API qt2_status qt2_linear_xent_fwd_workspace_size(int64_t T, int64_t K, int64_t V, size_t *bytes);
QT2_API qt2_status qt2_linear_xent_fwd(const void *x, const void *w, const int64_t *targets, int64_t T, int64_t K,
                                       int64_t V, int64_t ldx, int64_t ldw, int64_t ignore_index, float *loss,
                                       float *lse, void *workspace, size_t ws_bytes, qt2_stream_t stream);

/* ---------------------------------------------------------------------------------------
 * Gradient of sum_t dloss_t loss_t, from the forward pass's lse and the same inputs:
 *   P_tv = dloss_t * (exp(l_tv - lse_t) - [v = target(t)])   (0 in rows without a target),
 *   dx = P w  [T][K] bf16,  dw = P^T x  [V][K] of type dw_dtype.
 * The logits are formed again, a piece of the vocabulary at a time; the piece's P, each row divided
 * by the probability that is not its target's, is held in bf16 (rounded once, 2^-8 at most relative
 * to each entry, the target's entry exact) in the workspace while the tensor cores multiply it, with
 * fp32 sums over the whole of V (dx) and T (dw).  dloss and that factor multiply dx's rows in fp32, and
 * x's for dw: a product with a target's entry has 16 bits of it or more, products with the others 8.  The
 * roundings of the other entries are what an fp32 dw shows: 1e-5 to 7e-5 of it (2-norm) at 16 to 8192 tokens and
 * vocabularies of 1000 to 50000 with probability spread over many entries, up to 2^-8 in rows that one wrong entry
 * dominates.  A bf16 dx or dw has its own rounding (1.65e-3) besides.  Rows without a target add nothing to dw, whatever
 * x holds there (inf and NaN included), and have dx 0 for finite w.  Targets outside [0, V) count as
 * ignore_index and are not reported again.
 * dx or dw may be NULL (not wanted), not both.
 * Workspace: qt2_linear_xent_bwd_workspace_size() bytes, 256-byte aligned.
 * --------------------------------------------------------------------------------------- */
QT2_API qt2_status qt2_linear_xent_bwd_workspace_size(int64_t T, int64_t K, int64_t V, size_t *bytes);
QT2_API qt2_status qt2_linear_xent_bwd(const void *x, const void *w, const int64_t *targets, const float *lse,
                                       const float *dloss, int64_t T, int64_t K, int64_t V, int64_t ldx, int64_t ldw,
                                       int64_t ignore_index, void *dx, int64_t lddx, void *dw, int dw_dtype,
                                       int64_t lddw, void *workspace, size_t ws_bytes, qt2_stream_t stream);

/* ---------------------------------------------------------------------------------------
 * Global norm of many gradients, and clipping by it.  A gradient is a contiguous array of numel
 * (>= 0) elements of type dtype, aligned to its element only; `out`, of the same size, type and
 * alignment rule, receives the clipped gradient and may be `grad` itself (it is not used by
 * qt2_grad_norm and may then be NULL).  The list is read on the host during the call.
 * The outputs of two entries must not overlap, nor an output the gradient of another entry.
 *   qt2_grad_norm: *norm = sqrt(sum over all elements of g^2), without overflow or underflow of
 *     the squares for any finite fp32 values (inf where the norm itself exceeds fp32); squares are
 *     summed in fp32 over at most 8 elements, then in fp64.
 *     Workspace: qt2_grad_norm_workspace_size() bytes, 256-byte aligned.
 *   qt2_grad_clip: out = g * min(1, max_norm / (*norm + 1e-6)), max_norm >= 0, *norm read on the
 *     device (so that ranks can combine their norms between the two calls).  A NaN norm makes
 *     every gradient NaN; an infinite one zeroes the finite elements.  Where the factor is 1,
 *     gradients whose out is grad are not touched.
 * --------------------------------------------------------------------------------------- */
typedef struct {
    const void *grad; /* device */
    void *out;        /* device */
    int64_t numel;
    int32_t dtype; /* QT2_DTYPE_* */
    int32_t reserved;
} qt2_grad;
QT2_API qt2_status qt2_grad_norm_workspace_size(const qt2_grad *grads, int64_t count, size_t *bytes);
QT2_API qt2_status qt2_grad_norm(const qt2_grad *grads, int64_t count, float *norm, void *workspace, size_t ws_bytes,
                                 qt2_stream_t stream);
QT2_API qt2_status qt2_grad_clip(const qt2_grad *grads, int64_t count, const float *norm, float max_norm,
                                 qt2_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QT2_TRAIN_H */
