/*
 * qt2_train.h -- C ABI of the training operators beside the quantized linears (qt2.h) for NVIDIA
 * B200 (sm_100a), in the library libqt2_train.so: layer norm, the head's softmax cross entropy
 * over a large vocabulary, the gated feed-forward product on NVFP4 operands, the norm of queries and
 * keys with the position rotation, the global gradient norm with clipping, and the AdamW step of many
 * tensors, each with what a training step needs of it.
 *
 * Conventions are those of qt2.h (device pointers owned by the caller, work enqueued on `stream`,
 * arguments validated on the host before any launch, negative qt2_status on error, no allocation,
 * no abort, one NVTX range per call), with these differences:
 *   - Dimensions are any positive ints below 2^30, not multiples of 128 unless a call says so (a matrix
 *     of the head loss or of a gated product has fewer than 2^44 elements).  Matrices are row-major with a leading dimension that is a
 *     multiple of 8 elements, at least the row's length and below 2^40 (x and w of the head loss, gate and
 *     up of the gated product's backward pass: 2^39), and 16-byte aligned bases.  Elements between a row's length and its leading dimension
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
 * report QT2_ERR_TIMEOUT, QT2_ERR_INVALID_ARG (a target outside the vocabulary, a position outside the
 * tables, a step below 1), and in the checked build QT2_ERR_BOUNDS. */
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
 * Gated feed-forward product: both projections, the activation and the product in one kernel.
 *   g = alpha ga gg sum_k val(a)*sa * val(b_gate)*sg,  u the same of b_up,  h = act(g) * u.
 * a is an [M][K] view (the quantized x), b_gate and b_up are [F][K] views (the two weights, each with a
 * tensor scale of its own), as qt2_gemm_nvfp4 takes them; M, F and K are multiples of 128, the products' steps of
 * 256 x 128 x 256 fewer than 2^31.  act(x) = x s(x):
 *   QT2_ACT_SILU       s = 1 / (1 + exp(-x)),
 *   QT2_ACT_GELU_TANH  s = 1 / (1 + exp(-2 z)), z = sqrt(2/pi) (x + 0.044715 x^3).
 * Sums, activation and product are fp32, each output rounded once.  h [M][F] is bf16; gate and up [M][F]
 * (bf16, both with leading dimension ldgu) are what the backward pass needs: both, or both NULL.  They may
 * be the two halves of one [M][2F] matrix.
 * --------------------------------------------------------------------------------------- */
enum { QT2_ACT_SILU = 0, QT2_ACT_GELU_TANH = 1 };
QT2_API qt2_status qt2_gemm_nvfp4_gated(const qt2_nvfp4_view *a, const qt2_nvfp4_view *b_gate,
                                        const qt2_nvfp4_view *b_up, int64_t M, int64_t F, int64_t K, float alpha,
                                        int act, void *gate, void *up, int64_t ldgu, void *h, int64_t ldh,
                                        qt2_stream_t stream);

/* ---------------------------------------------------------------------------------------
 * Backward of the gated product, in the epilogue of the down projection's dgrad:
 *   dh = alpha ga gb sum_k val(a)*sa * val(b)*sb              (fp32, never stored),
 *   dgate = dh * up * act'(gate),  dup = dh * act(gate),  h = act(gate) * up.
 * a is an [M][K] view (the output's gradient), b an [F][K] view (the down projection's weight with its
 * output dimension contracted): the row view of dy and the column view of the weight that qt2_quant_msedEN
 * gives, with alpha = 2^-7.  gate and up are what the forward pass kept.  dgate and dup [M][F] bf16 (leading
 * dimension lddgu) are the output gradients of the two projections, for qt2_linear_bwd and
 * qt2_linear_bwd_views; h [M][F] bf16, what the down projection's wgrad contracts, may be NULL.
 * M, F and K are multiples of 128.  dgate may be gate and dup may be up (with lddgu = ldgu).
 * --------------------------------------------------------------------------------------- */
QT2_API qt2_status qt2_gemm_nvfp4_gated_bwd(const qt2_nvfp4_view *a, const qt2_nvfp4_view *b, int64_t M, int64_t F,
                                            int64_t K, float alpha, int act, const void *gate, const void *up,
                                            int64_t ldgu, void *dgate, void *dup, int64_t lddgu, void *h, int64_t ldh,
                                            qt2_stream_t stream);

/* ---------------------------------------------------------------------------------------
 * Norm of queries and keys for each head, with the position rotation, in one pass over the QKV linear's
 * output.  x holds Hq + Hk heads of D elements for each of T tokens: head h of token t starts at element
 * t * ldx + h * hsx, the Hq query heads first (with ldx = (Hq + 2 Hk) D and hsx = D they are part of rows
 * that hold the values too, which are not touched; with hsx = T D and ldx = D the heads are outermost).
 * Heads of queries alone or keys alone: Hk = 0 or Hq = 0.  For each head of each token:
 *   r = 1 / sqrt(sum_d x_d^2 / D + eps),  a_d = x_d r w_d  (w = wq or wk, [D]; NULL stands for ones),
 *   y = a with the pairs of its first R elements turned: (p, q) -> (p cos - q sin, q cos + p sin),
 * pair i < R/2 being (i, i + R/2) with QT2_ROPE_HALVES, (2i, 2i + 1) with QT2_ROPE_PAIRS, and cos and sin
 * rows positions[t] of the two fp32 tables [P][R/2].  positions (int64 [T]) NULL: token t is at t (T <= P).
 * A position outside [0, P) leaves its token unturned and is reported as QT2_ERR_INVALID_ARG through
 * qt2_train_device_status.  R = 0: nothing is turned; positions and tables may be NULL.
 * x and y have type x_dtype, wq and wk w_dtype; all of it 16-byte aligned (positions 8), strides multiples of
 * 8 elements below 2^32, such that no two heads overlap.  D and R are multiples of 8, D <= 1024, R <= D.  Statistics and
 * products are fp32, rounded once on writing (a head's sum of squares has to stay within fp32).  y may be x
 * with its strides.  eps >= 0 and finite.  T, Hq and Hk are below 2^30, 2^20 and 2^20, T (Hq + Hk) below 2^32.
 * --------------------------------------------------------------------------------------- */
enum { QT2_ROPE_HALVES = 0, QT2_ROPE_PAIRS = 1 };
QT2_API qt2_status qt2_qk_norm_rope_fwd(const void *x, int x_dtype, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
                                        int64_t ldx, int64_t hsx, const void *wq, const void *wk, int w_dtype,
                                        float eps, const int64_t *positions, const float *cos, const float *sin,
                                        int64_t P, int64_t R, int pairing, void *y, int64_t ldy, int64_t hsy,
                                        qt2_stream_t stream);

/* ---------------------------------------------------------------------------------------
 * Backward of qt2_qk_norm_rope_fwd from its input x, with n = x r and b = dy turned the other way:
 *   dx_d = r (b_d w_d - n_d sum_e (b_e w_e n_e) / D),  dwq_d = sum over tokens and query heads of b_d n_d,
 * dwk the same over the key heads (zeros where there are none).  dy and dx have type x_dtype and strides of
 * their own, dwq and dwk w_dtype.  dx, dwq and dwk may each be NULL (not wanted), not all of them.  dx may be
 * dy or x, with its strides.  Positions outside the tables are not reported again.  Sums are fp32.
 * Workspace: qt2_qk_norm_rope_bwd_workspace_size() bytes, 256-byte aligned.
 * --------------------------------------------------------------------------------------- */
QT2_API qt2_status qt2_qk_norm_rope_bwd_workspace_size(int64_t T, int64_t Hq, int64_t Hk, int64_t D, size_t *bytes);
QT2_API qt2_status qt2_qk_norm_rope_bwd(const void *dy, int64_t lddy, int64_t hsdy, const void *x, int x_dtype,
                                        int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t ldx, int64_t hsx,
                                        const void *wq, const void *wk, int w_dtype, float eps,
                                        const int64_t *positions, const float *cos, const float *sin, int64_t P,
                                        int64_t R, int pairing, void *dx, int64_t lddx, int64_t hsdx, void *dwq,
                                        void *dwk, void *workspace, size_t ws_bytes, qt2_stream_t stream);

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

/* ---------------------------------------------------------------------------------------
 * One AdamW step (decoupled weight decay) of many tensors, in place, the clipping by the global norm taken
 * along.  With f = min(1, max_norm / (*norm + 1e-6)), or 1 where norm is NULL, and t = *step:
 *   g' = g f,  m = beta1 m + (1 - beta1) g',  v = beta2 v + (1 - beta2) g'^2,
 *   p = p - lr weight_decay p - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps).
 * A tensor is numel (>= 0, below 2^40) contiguous elements.  param is bf16 or fp32.  With a master (fp32, for a bf16 param
 * alone; else NULL) p is read from and kept in the master, and param receives it rounded; without one a bf16
 * param is read, and written rounded to nearest.  grad is bf16 or fp32.  States:
 *   QT2_STATE_F32   m and v are fp32; the scales are not used.
 *   QT2_STATE_E4M3  m and v are E4M3 codes, with an fp32 scale for every 256 elements in m_scale and v_scale
 *     [ceil(numel / 256)]: m = code * scale, and sqrt(v) = code * scale (the codes hold the root).  The new
 *     scale is the largest magnitude / 448 (in the step's own update m and v are not rounded); a code is
 *     one of the two neighbours of its value, picked by 16 random bits r so that the mean stays: the fp32
 *     encoding of |value| * (448 / largest) plus r * 2^4, cut to 3 bits of mantissa (below 2^-6 with 2^-6 added
 *     before and taken off after).  A root that is not zero never becomes code 0: where it would, its code is the
 *     smallest, 2^-9, so that no m that rounded up is divided by next to nothing (elements whose root is less than
 *     2^-17.8 of their block's largest move by less than with fp32 states).
 *     Element i draws from word i % 4 of the Philox4x32-10 block of counter
 *     (lo32(i / 4), hi32(i / 4), the tensor's place in the list, lo32(*step)) under the key seed: its low 16 bits
 *     for m, the others for v.  Blocks whose largest magnitude is below 2^-100 become zeros with scale 0; an inf
 *     or NaN makes its block of 256 NaN.  Zeros with scales of zero are a fresh state; states that a caller makes
 *     of others hold no root of code 0 beside an m that is not zero, which the next step would divide by eps.
 * Codes, scales and v are rounded operation by operation in the order above (fp32, no contraction); squares of
 * gradients have to stay within fp32.
 * lr (fp32), step (int64, 1 for the first step) and norm (fp32, what qt2_grad_norm gives) are one element each
 * in device memory, so that a captured graph can be replayed as they change.  A step below 1 is reported as
 * QT2_ERR_INVALID_ARG through qt2_train_device_status; then, and where the norm is inf or NaN, nothing changes.
 * 0 <= beta1, beta2 < 1, eps >= 0, max_norm >= 0, weight_decay finite.  The list is read on the host during
 * the call.  Arrays are aligned to their elements only; those of a tensor go fastest when they start on 16
 * bytes, or equally far (in elements) behind.  Nothing that the step writes may overlap another tensor's
 * arrays or the gradients.
 * --------------------------------------------------------------------------------------- */
enum { QT2_STATE_F32 = 0, QT2_STATE_E4M3 = 1 };
typedef struct {
    void *param;       /* device */
    float *master;     /* device, or NULL */
    const void *grad;  /* device */
    void *m, *v;       /* device */
    float *m_scale, *v_scale; /* device; QT2_STATE_E4M3 */
    int64_t numel;
    int32_t param_dtype, grad_dtype; /* QT2_DTYPE_* */
    int32_t state;                   /* QT2_STATE_* */
    float weight_decay;
} qt2_adamw_tensor;
QT2_API qt2_status qt2_adamw(const qt2_adamw_tensor *tensors, int64_t count, const float *lr, const int64_t *step,
                             double beta1, double beta2, float eps, const float *norm, float max_norm, uint64_t seed,
                             qt2_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QT2_TRAIN_H */
