/*
 * ampops.h - C ABI of the forward/backward operators in libampfp8.so that sit
 * around the optimizer step of ampfp8.h: microscaled 4-bit quantisation,
 * products and linear layers, layer norm, activations whose inputs are kept in
 * 8 bits for the backward pass, dropout, and the log probabilities of tokens.
 *
 *   fp4_quant_mx, fp4_dequant_mx     4-bit blocks (+ transposed copy), and back
 *   fp4_product_mx                   C = A B^T of two such matrices
 *   fp4_linear_mx                    the same with bias, activation, residual and
 *                                    the 8-bit checkpoint in its epilogue
 *   amp_bias_act_backward_mx8        gradients of that bias and activation
 *   amp_dropout_forward/backward     dropout whose mask is never stored
 *   amp_token_logprobs_forward/backward  log probabilities of given tokens,
 *                                    entropy, most probable tokens
 *   amp_layer_norm_forward/backward  layer norm, with both parameters' gradients
 *   amp_act_forward_mx8/backward_mx8 GELU / SiLU, plain or gated, from 8-bit
 *                                    checkpoints of their inputs
 *   amp_ckpt8_save, amp_ckpt8_restore  8-bit checkpoints on their own
 *
 * The conventions of ampfp8.h hold: contiguous device tensors owned by the
 * caller, asynchronous calls on `stream`, no allocation, no host
 * synchronisation, negative status = nothing enqueued, message in
 * amp_last_error(), programmatic dependent launches, one NVTX range per call.
 * A tensor is aligned to its element type (else AMP_EINVAL); where a buffer has
 * to be aligned further its comment says so.  An output shares no memory with
 * another tensor of its call unless its comment allows it.  Empty shapes are
 * accepted everywhere.
 *
 * Block formats (OCP Microscaling Formats specification 1.0: 32 consecutive
 * elements of a row share one E8M0 scale byte e, which stands for 2^(e-127)).
 * With M the element format's largest magnitude (e2m1: 6, e4m3: 448) and
 * a = max |x| of the block:
 *     e  = the smallest byte with a <= M * 2^(e-127)     (0 for a = 0)
 *     q  = RNE(x * 2^(127-e))                            (the product is exact)
 * so no element saturates, and every value q * 2^(e-127) is the nearest of the
 * block's grid to x.  A block that holds a NaN or an infinity gets e = 255 and
 * decodes to NaN throughout (its codes mean nothing), so a non-finite value
 * stays visible to the gradient check.  The last block of a row may be short.
 *
 * Layouts.
 *   4-bit elements  row r of a [rows, cols] matrix takes ceil(cols/32)*16 bytes;
 *                   element j is in byte j/2, the even one in bits 0-3; the
 *                   padding of the last block is zero.  16-byte aligned.
 *   4-bit scales    tiles of 128 rows x 4 blocks, 512 bytes each, tile (R, B) at
 *                   (R * ceil(cols/128) + B) * 512, byte
 *                   (r % 32) * 16 + (r % 128) / 32 * 4 + b % 4 of its tile for
 *                   row r, block b; padding rows and blocks are written as 0.
 *                   The order in which the tensor cores take them.  16-byte
 *                   aligned.
 *   8-bit elements  AMP_DT_E4M3FN bytes, [rows, cols] row-major
 *   8-bit scales    one byte per block, [rows, ceil(cols/32)] row-major
 */
#ifndef AMPOPS_H
#define AMPOPS_H

#include "ampfp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of a [rows, cols] matrix's packed 4-bit elements and of its scales;
 * -1 for a negative or too large size. */
int64_t fp4_mx_bytes(int64_t rows, int64_t cols);
int64_t fp4_mx_scale_bytes(int64_t rows, int64_t cols);

/* x [rows, cols] row-major (AMP_DT_BF16, AMP_DT_F16, AMP_DT_F32) -> out, scales
 * with blocks along the rows, and, if out_t is non-NULL, out_t, scales_t: the
 * transposed matrix [cols, rows], blocks along the columns of x, for products
 * that reduce along the rows of x.  One launch.  A set *skip_if_dev writes
 * nothing.
 * Errors: AMP_EINVAL (NULL x / out / scales, out_t without scales_t, negative
 * or too large size, a misaligned output), AMP_EDTYPE. */
amp_status fp4_quant_mx(const void *x, amp_dtype x_dtype, int64_t rows, int64_t cols, void *out,
                        void *scales, void *out_t, void *scales_t, const int32_t *skip_if_dev,
                        amp_stream_t stream);

/* out [rows, cols] (AMP_DT_BF16, AMP_DT_F16, AMP_DT_F32) = the values that q,
 * scales stand for: exact in f32 and bf16, rounded to nearest even in f16
 * (inf beyond its range).
 * Errors: AMP_EINVAL (NULL pointer, negative or too large size, misaligned q
 * or scales), AMP_EDTYPE. */
amp_status fp4_dequant_mx(const void *q, const void *scales, int64_t rows, int64_t cols, void *out,
                          amp_dtype out_dtype, amp_stream_t stream);

/* out [m, n] row-major = A B^T for 4-bit A [m, k] and B [n, k]:
 *     out[i,j] = RNE(sum_k A[i,k] * B[j,k])
 * summed in fp32 by the tensor cores, rounded once to out_dtype (AMP_DT_BF16,
 * AMP_DT_F16 with inf beyond its range, AMP_DT_F32).  k = 0 writes zeros.  The
 * three products of a linear layer y = x W^T are (x, W), (dy, W^T) and
 * (dy^T, x^T), the transposed operands being the out_t of fp4_quant_mx.
 * The order of the sum depends on the shape and the device alone, so equal
 * calls give equal bits.
 * The kernel's waits on its own copies and products give up after one second
 * of GPU time.  fp4_mx_check reports a call that did; the elements of out that
 * it could not finish are NaN, so the gradient check sees them too.
 * Errors: AMP_EINVAL (NULL or misaligned operands, negative or too large
 * size, k above 2^27), AMP_EDTYPE, AMP_ECUDA. */
amp_status fp4_product_mx(const void *a, const void *a_scales, const void *b, const void *b_scales,
                          int64_t m, int64_t n, int64_t k, void *out, amp_dtype out_dtype,
                          amp_stream_t stream);

/* Waits for `stream`, reads and clears the current device's sticky error word
 * of fp4_product_mx and fp4_linear_mx: AMP_ETIMEOUT if a bounded wait gave up
 * since the last check, AMP_OK otherwise. */
amp_status fp4_mx_check(amp_stream_t stream);

/* fp4_product_mx with waits of at most 2^limit_log2_ns ns (0 to 30) and one of the
 * kernel's roles ended after `stages` stages of 256 along the reduction, counted
 * over all of a CTA's tiles, as if its wait had run out: 0 the loads (where two
 * CTAs share a tile, the first's), 1 the loads of the second, 2 the products.  For
 * tests of what a wait that gave up leaves behind; nothing faults or hangs. */
amp_status fp4_product_mx_selftest(const void *a, const void *a_scales, const void *b,
                                   const void *b_scales, int64_t m, int64_t n, int64_t k,
                                   void *out, amp_dtype out_dtype, int32_t role, int32_t stages,
                                   int32_t limit_log2_ns, amp_stream_t stream);

/* Layer norm over the rows of x [rows, cols] (AMP_DT_BF16, AMP_DT_F16,
 * AMP_DT_F32), in fp32, with the mean taken first and the variance about it:
 *     mean = sum(x) / cols, rstd = 1 / sqrt(sum((x - mean)^2) / cols + eps)
 *     y    = (x - mean) * rstd * weight + bias       rounded to x's type
 *   weight, bias  [cols] of w_dtype (f32, or x's type); either may be NULL
 *                 (1 and 0)
 *   mean, rstd    fp32 [rows], for the backward pass; may be NULL (the inverse
 *                 root is good to 2 units in its last place, and depends on the
 *                 sum under it alone, not on the row's length or address)
 *   ckpt, ckpt_scales  both or neither: the 8-bit checkpoint of x
 * Errors: AMP_EINVAL (NULL x / y, half a checkpoint, negative or too large
 * size, eps < 0 or NaN), AMP_EDTYPE. */
amp_status amp_layer_norm_forward(const void *x, amp_dtype x_dtype, int64_t rows, int64_t cols,
                                  const void *weight, const void *bias, amp_dtype w_dtype,
                                  double eps, void *y, float *mean, float *rstd, void *ckpt,
                                  void *ckpt_scales, amp_stream_t stream);

/* Scratch of amp_layer_norm_backward for this shape, in bytes (a function of
 * the shape and the current device); -1 for a negative or too large size. */
int64_t amp_layer_norm_workspace_bytes(int64_t rows, int64_t cols);

/* Gradients of the layer norm: with xh = (x - mean) * rstd, g = dy * weight,
 *     dx      = rstd * (g - sum(g) / cols - xh * sum(g * xh) / cols)
 *     dweight = sum over rows of dy * xh,   dbias = sum over rows of dy
 * in fp32; the row sums are added in a fixed order, so equal calls give equal
 * bits.  x comes either as x (of dtype) or as the 8-bit checkpoint (x NULL).
 *   weight    [cols] of w_dtype, or NULL (1)
 *   dx        [rows, cols] of dtype, or NULL
 *   dweight, dbias  [cols] of w_dtype; either may be NULL
 *   workspace amp_layer_norm_workspace_bytes(rows, cols) bytes, 16-byte
 *             aligned, free again when the call's work is done; may be NULL
 *             when dweight and dbias are
 * dx may be dy itself (in place), no other outputs may overlap inputs.
 * Errors: AMP_EINVAL, AMP_EDTYPE. */
amp_status amp_layer_norm_backward(const void *dy, const void *x, amp_dtype dtype,
                                   const void *ckpt, const void *ckpt_scales, int64_t rows,
                                   int64_t cols, const void *weight, amp_dtype w_dtype,
                                   const float *mean, const float *rstd, void *dx, void *dweight,
                                   void *dbias, void *workspace, int64_t workspace_bytes,
                                   amp_stream_t stream);

typedef enum {
    AMP_ACT_GELU = 0,      /* x * Phi(x) */
    AMP_ACT_GELU_TANH = 1, /* x/2 * (1 + tanh(sqrt(2/pi) * (x + 0.044715 x^3))) */
    AMP_ACT_SILU = 2       /* x / (1 + exp(-x)) */
} amp_act;

/* y = f(x), or f(x) * up for a non-NULL up, all [rows, cols] of dtype
 * (AMP_DT_BF16, AMP_DT_F16, AMP_DT_F32), computed in fp32; q, scales (and
 * q_up, scales_up with up) take the 8-bit checkpoints of x (and up).  For
 * inference q and scales may both be NULL, which keeps nothing.
 * Before the rounding to the type, f is within 2^-14 |f| + 2^-122 of its exact
 * value for the 16-bit types, tails included.  For f32, with U = 2^-24, it is
 * within (12 + c) U |f| + 2^-122, where c is 1.25 x^2 for AMP_ACT_GELU, 5.5 |t|
 * for AMP_ACT_GELU_TANH with t = 2 sqrt(2/pi) (x + 0.044715 x^3), and 0 for
 * AMP_ACT_SILU: as for f(x) at an x that is off by a unit in its last place.
 * Errors: AMP_EINVAL (NULL, half a checkpoint, up and its checkpoint not
 * together, negative or too large size, unknown act), AMP_EDTYPE. */
amp_status amp_act_forward_mx8(amp_act act, const void *x, const void *up, amp_dtype dtype,
                               int64_t rows, int64_t cols, void *y, void *q, void *scales,
                               void *q_up, void *scales_up, amp_stream_t stream);

/* Gradients of amp_act_forward_mx8 at the checkpointed inputs xh, uh:
 *     dx = dy * f'(xh) [* uh],   dup = dy * f(xh)   (gated: q_up non-NULL)
 * dx (and dup) [rows, cols] of dtype.  dx or dup may be dy itself.
 * Errors: as amp_act_forward_mx8. */
amp_status amp_act_backward_mx8(amp_act act, const void *dy, amp_dtype dtype, int64_t rows,
                                int64_t cols, const void *q, const void *scales, const void *q_up,
                                const void *scales_up, void *dx, void *dup, amp_stream_t stream);

/* The 8-bit checkpoint of x, and the values (rounded to out's type) that one
 * stands for.  Errors: AMP_EINVAL, AMP_EDTYPE. */
amp_status amp_ckpt8_save(const void *x, amp_dtype x_dtype, int64_t rows, int64_t cols, void *q,
                          void *scales, amp_stream_t stream);
amp_status amp_ckpt8_restore(const void *q, const void *scales, int64_t rows, int64_t cols,
                             void *out, amp_dtype out_dtype, amp_stream_t stream);

/* A linear layer in one launch, for 4-bit A [m, k] and B [n, k]:
 *     z   = A B^T + bias                      in fp32, summed as fp4_product_mx
 *     out = f(z) + residual                   rounded once to out_dtype
 *   bias      [n] of bias_dtype (f32, or out's type), or NULL (0)
 *   act       an amp_act, or AMP_ACT_NONE
 *   residual  [m, n] of out_dtype, or NULL (0); may be out itself
 *   q, scales the 8-bit checkpoint of z (before its rounding to any other
 *             type), for amp_bias_act_backward_mx8; both or neither
 * f is as accurate as amp_act_forward_mx8's for out's type.  k = 0: z = bias.
 * Equal calls give equal bits.  Waits are bounded as fp4_product_mx's are:
 * fp4_mx_check reports a call that gave up, what it could not finish is NaN in
 * out and has the NaN scale in the checkpoint.
 * Errors: as fp4_product_mx, AMP_EINVAL (half a checkpoint, unknown act). */
enum { AMP_ACT_NONE = -1 };
amp_status fp4_linear_mx(const void *a, const void *a_scales, const void *b, const void *b_scales,
                         int64_t m, int64_t n, int64_t k, const void *bias, amp_dtype bias_dtype,
                         int32_t act, const void *residual, void *out, amp_dtype out_dtype, void *q,
                         void *scales, amp_stream_t stream);

/* fp4_linear_mx as fp4_product_mx_selftest runs fp4_product_mx. */
amp_status fp4_linear_mx_selftest(const void *a, const void *a_scales, const void *b,
                                  const void *b_scales, int64_t m, int64_t n, int64_t k,
                                  const void *bias, amp_dtype bias_dtype, int32_t act,
                                  const void *residual, void *out, amp_dtype out_dtype, void *q,
                                  void *scales, int32_t role, int32_t stages,
                                  int32_t limit_log2_ns, amp_stream_t stream);

/* Gradients behind a bias and an activation, from the checkpoint of z that
 * fp4_linear_mx made (values zh):
 *     dz = dy * f'(zh),   dbias = sum over rows of dz
 * in fp32; dbias sums dz before its rounding, in an order that depends on the
 * shape, the tensors' alignment and the device alone.  With AMP_ACT_NONE
 * dz = dy: q, scales and dz are NULL and only dbias is written.
 *   dy, dz  [rows, cols] of dtype; dz may be dy
 *   dbias   [cols] of bias_dtype (f32, or dtype); zeros for no rows
 * Errors: AMP_EINVAL (NULL, an activation without q, scales and dz or one of
 * those without it, negative or too large size, unknown act), AMP_EDTYPE. */
amp_status amp_bias_act_backward_mx8(int32_t act, const void *dy, amp_dtype dtype, int64_t rows,
                                     int64_t cols, const void *q, const void *scales, void *dz,
                                     void *dbias, amp_dtype bias_dtype, amp_stream_t stream);

/* Dropout, added to a residual, over [rows, cols] (AMP_DT_BF16, AMP_DT_F16,
 * AMP_DT_F32), in fp32 and rounded once:
 *     y = residual + (u(k) >= T ? x * 65536 / (65536 - T) : 0)
 * with T the whole number nearest to 65536 p (ties to even) and u(k) 16 random
 * bits of element k = row * cols + column, which are a function of seed, step,
 * site and k alone: half (k % 8) % 2, low first, of word (k % 8) / 2 of
 * Philox4x32-10 for the counter {k / 8 low, k / 8 high, step, 2^30 + site}
 * under the key seed.  Nothing is stored: the backward pass makes the same
 * mask.  p = 1 drops everything.  What is dropped is not multiplied: a NaN or an
 * infinity there leaves nothing behind.  The streams of the step's stochastic
 * rounding under the same seed are others (their tensor words are below 2^30,
 * or 2^31 and more).
 *   step_dev  the step, one int32 on the device (so a captured graph draws
 *             another mask each time it is changed); NULL: 0, the same mask in
 *             every call.  A step count that stays where a step was skipped
 *             draws that step's masks again
 *   site      which of a step's dropouts this is, in [0, 2^30).  Calls of one
 *             seed, step and site draw one mask, so each dropout of a model has
 *             its site, each micro-batch of an accumulated step sites of its own
 *             (dropout * micro_batches + micro_batch), and each data-parallel
 *             rank a seed of its own (seed + rank)
 *   residual  of the same type, or NULL (0); y may be x or residual
 * Errors: AMP_EINVAL (NULL x / y, p outside [0, 1] or NaN, site out of range,
 * negative or too large size), AMP_EDTYPE. */
amp_status amp_dropout_forward(const void *x, amp_dtype dtype, int64_t rows, int64_t cols, double p,
                               uint64_t seed, const int32_t *step_dev, int32_t site,
                               const void *residual, void *y, amp_stream_t stream);

/* Its gradients, with the mask of the same seed, step, site and shape:
 *     dx = u(k) >= T ? dy * 65536 / (65536 - T) : 0,   dbias = sum over rows of dx
 * (the residual's is dy).  dx may be dy.  dbias is the gradient of a bias that
 * was added to x before: [cols] of bias_dtype (f32, or dtype), summed as
 * amp_bias_act_backward_mx8's; or NULL.
 * Errors: as amp_dropout_forward. */
amp_status amp_dropout_backward(const void *dy, amp_dtype dtype, int64_t rows, int64_t cols,
                                double p, uint64_t seed, const int32_t *step_dev, int32_t site,
                                void *dx, void *dbias, amp_dtype bias_dtype, amp_stream_t stream);

/* Log probabilities under softmax over the rows of z [rows, cols]
 * (AMP_DT_BF16, AMP_DT_F16, AMP_DT_F32), whose rows start ld >= cols elements
 * apart (what lies between is not read), in fp32:
 *     m = max z_j,  s = sum exp(z_j - m),  log p_j = (z_j - m) - log s
 *   targets  int64 [rows]: the row's token t.  A negative one marks a row that
 *            is not used: it is not read, logp, entropy and stats are 0, and it
 *            has no alternatives.  One of cols or more gives NaN.  NULL: none
 *            (logp NULL too)
 *   logp     fp32 [rows]: log p_t, or NULL
 *   entropy  fp32 [rows]: -sum p_j log p_j, or NULL
 *   stats    fp32 [rows, 2]: m and log s, for the backward pass, or NULL
 *   top_ids, top_logp  int64 and fp32 [rows, top_n], both or neither: the top_n
 *            most probable tokens (at most 32), larger logits first, equal ones
 *            by index; -1 and -inf where there are no more.  Logits of -inf and
 *            NaN are not listed
 * An exponential is within (3 |z_j - m| + 4) 2^-24 of its value, relatively, and
 * 0 below 2^-126.
 * A logit of -inf (a masked token) has probability 0 and log probability -inf.
 * A row with a NaN, with +inf, or with nothing but -inf gives NaN.
 * Errors: AMP_EINVAL (NULL z, logp without targets, top_n outside [0, 32], half
 * of the alternatives, ld < cols, negative or too large size, cols above 2^30),
 * AMP_EDTYPE. */
amp_status amp_token_logprobs_forward(const void *z, amp_dtype dtype, int64_t rows, int64_t cols,
                                      int64_t ld, const int64_t *targets, float *logp,
                                      float *entropy, float *stats, int64_t *top_ids,
                                      float *top_logp, int32_t top_n, amp_stream_t stream);

/* The gradient at the logits, from what the forward call left in stats and
 * entropy, in fp32:
 *     dz_j = S * (dlogp * ([j = t] - p_j) - dentropy * p_j * (log p_j + H))
 *   dlogp     fp32 [rows]: the gradient at logp, or NULL (0)
 *   dentropy  fp32 [rows]: the gradient at the entropy H, or NULL (0); with it
 *             entropy is needed
 *   scale_dev the loss scale S, one fp32 on the device, or NULL (1)
 *   dz        [rows, cols] of dtype, rows dld >= cols elements apart (what lies
 *             between is left as it is); may be z itself with dld = ld, and
 *             otherwise shares no element with it (column slices of one buffer
 *             do not; with two strides the ranges have to be apart)
 * Rows with a negative target get zeros, whatever their logits.
 * Errors: AMP_EINVAL (NULL z / stats / dz, dlogp without targets, dentropy
 * without entropy, ld or dld < cols, dz = z with another dld, dz that overlaps z
 * otherwise, negative or too large size), AMP_EDTYPE. */
amp_status amp_token_logprobs_backward(const float *dlogp, const void *z, amp_dtype dtype,
                                       int64_t rows, int64_t cols, int64_t ld,
                                       const int64_t *targets, const float *stats,
                                       const float *entropy, const float *dentropy,
                                       const float *scale_dev, void *dz, int64_t dld,
                                       amp_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* AMPOPS_H */
