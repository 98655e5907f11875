/*
 * convrot_block.h -- C ABI of the operators that stand between the linears of
 * a transformer block: a linear on 8-bit floating-point codes with block
 * scales, the gated norm with its gradient, and rotary positions.
 *
 * The conventions are convrot.h's: device pointers, row-major layouts with a
 * leading dimension in elements, buffers owned by the caller, arguments
 * checked on the host before anything is enqueued (a non-OK status means that
 * nothing was launched), no allocation and no synchronization, work enqueued
 * on `stream`, deterministic results. Differences are stated at each entry.
 */
#ifndef CONVROT_BLOCK_H_
#define CONVROT_BLOCK_H_

#include "convrot.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the tensors these operators read and write. */
typedef enum { CONVROT_F32 = 0, CONVROT_BF16 = 1, CONVROT_F16 = 2 } convrot_dtype;

/* ------------------------------------------------------------------------
 * The block-scaled linear. Codes are e4m3 (8-bit floating point: 4 exponent
 * and 3 mantissa bits, largest finite value 448), and each block of
 * CONVROT_FP8_BLOCK = 128 consecutive input features has a scale:
 *
 *   activations: one scale for the block of each row,
 *     s_x[r, j] = max(max_{i in block j} |X[r, i]|, 2^-96) / 448
 *     q_x[r, i] = e4m3(X[r, i] * (448 * (1 / max(...))))  nearest, ties to even,
 *                 the operations before it in fp32, each rounded
 *   weights: one scale for each block of 128 rows x 128 features,
 *     s_w[p, j], and q_w[o, i] = e4m3(W[o, i] * (448 * (1 / max(...))))
 *   Y[r, o] = act(sum_j s_x[r, j] s_w[o / 128, j] sum_{i in block j} q_x[r, i] q_w[o, i] + b[o])
 *
 * The last block of a row (and the last row block of a weight) may be short.
 * The inner sums run on the tensor cores and are added up in fp32. A NaN or
 * infinity in X makes the outputs of its row NaN or infinite.
 */
#define CONVROT_FP8_BLOCK 128

/*
 * Quantizes rows [m, k] of X (any dtype, any alignment, ldx >= k) for the
 * linear.
 *   q      [m, ldq] e4m3 codes, 16-byte aligned, ldq >= k, ldq % 16 == 0;
 *          columns past k are neither written nor read.
 *   scale  [ceil(k / 128), lds] fp32, lds >= m: the scale of row r's block j
 *          is scale[j * lds + r] (the linear reads one block's scales of many
 *          rows at once).
 * 1 <= k <= CONVROT_MAX_K; m == 0 launches nothing.
 */
convrot_status convrot_fp8_pack_activations(const void *X, int32_t x_dtype, int64_t m, int64_t k, int64_t ldx,
                                            void *q, int64_t ldq, float *scale, int64_t lds, cudaStream_t stream);

/*
 * Offline: quantizes a weight [n, k] in blocks of 128 x 128.
 *   q      as above, [n, ldq].
 *   scale  [ceil(n / 128), lds] fp32, lds >= ceil(k / 128): scale[p * lds + j].
 * (The layout in which block-scaled checkpoints store a weight and its
 * scales, so such tensors need no call.)
 */
convrot_status convrot_fp8_quantize_weights(const void *W, int32_t w_dtype, int64_t n, int64_t k, int64_t ldw,
                                            void *q, int64_t ldq, float *scale, int64_t lds, cudaStream_t stream);

/*
 * Arguments of the two linears below.
 *   x, ldx     convrot_fp8_linear: codes [m, ldx] (the q of a pack);
 *              convrot_fp8_pack_linear: rows [m, ldx] of type x_dtype, any
 *              alignment.
 *   x_scale    convrot_fp8_linear: the pack's scale, with ld_x_scale.
 *              convrot_fp8_pack_linear: not read.
 *   w, w_scale codes [n, ldw] and scales [ceil(n / 128), ld_w_scale].
 *   bias       fp32 [n] or NULL.
 *   y          [m, ldy] of type y_dtype, any alignment, ldy >= n.
 *   work       convrot_fp8_pack_linear: 256-byte aligned workspace of
 *              convrot_fp8_pack_linear_work_bytes(m, n, k) bytes (which may
 *              be 0: then it is not read); contents undefined afterwards.
 *   dev_status as for convrot_linear.
 */
typedef struct {
    const void *x;
    const float *x_scale;
    const void *w;
    const float *w_scale;
    const float *bias;
    void *y;
    void *work;
    int32_t *dev_status;
    int64_t m, n, k;
    int64_t ldx, ld_x_scale, ldw, ld_w_scale, ldy;
    int64_t work_bytes;
    int32_t x_dtype; /* convrot_fp8_pack_linear */
    int32_t y_dtype;
    int32_t act; /* a convrot_activation */
    int32_t reserved; /* 0 */
} convrot_fp8_linear_args;

/* The linear on packed activations. m == 0 or n == 0 launches nothing. */
convrot_status convrot_fp8_linear(const convrot_fp8_linear_args *a, cudaStream_t stream);

/* The pack of x, then the linear: the same Y as the two calls. */
int64_t convrot_fp8_pack_linear_work_bytes(int64_t m, int64_t n, int64_t k);
convrot_status convrot_fp8_pack_linear(const convrot_fp8_linear_args *a, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * The gated norm: what stands between two linears of a block. Row r belongs
 * to sample b = r / rows_per_batch (the last sample may be shorter).
 *
 *   u = post(y)                                the norm after the branch
 *   h = res_scale * x + gate[b] * u            the residual stream
 *   n = pre(h) * (1 + scale[b]) + shift[b]     the next branch's input
 *
 * post and pre are each CONVROT_NORM_NONE (the identity, times the weight and
 * plus the bias where those are given), CONVROT_NORM_RMS, v / sqrt(mean(v^2)
 * + eps), or CONVROT_NORM_LAYER, (v - mean) / sqrt(var + eps), followed by
 * their weight and bias. Everything between the loads and the one rounding
 * of each result is fp32; n is computed from h before h is rounded. (Where
 * scale meets a bias of pre, or gate one of post, an infinite factor may give
 * NaN for infinity: the products with either part are added up.)
 */
typedef enum { CONVROT_NORM_NONE = 0, CONVROT_NORM_RMS = 1, CONVROT_NORM_LAYER = 2 } convrot_norm_kind;

/* Widest row: it is held in the registers of one block of threads. */
#define CONVROT_NORM_MAX_D 16384

/*
 *   x, y       [m, d] of type dtype; y NULL: no branch (h = res_scale * x;
 *              gate and the post fields are then not read).
 *   gate, scale, shift   [batches, d] of type param_dtype with their leading
 *              dimensions; each may be NULL (1, 0 and 0).
 *   *_weight, *_bias     [d] of type param_dtype, each may be NULL.
 *   h, n       outputs [m, d] of type dtype; either may be NULL. h may be x.
 *   q, q_scale n as convrot_fp8_pack_activations would pack it (from n before
 *              its rounding to dtype), with ldq and ld_q_scale; or NULL.
 *   param_dtype  CONVROT_F32 or dtype. eps >= 0.
 * Any alignment; 1 <= d <= CONVROT_NORM_MAX_D (CONVROT_ERR_UNSUPPORTED
 * above); rows_per_batch >= 1; m == 0 launches nothing. Inputs other than x
 * must not alias outputs.
 */
typedef struct {
    const void *x, *y, *gate, *scale, *shift;
    const void *post_weight, *post_bias, *pre_weight, *pre_bias;
    void *h, *n, *q;
    float *q_scale;
    int64_t m, d, rows_per_batch;
    int64_t ldx, ldy, ldgate, ldscale, ldshift, ldh, ldn, ldq, ld_q_scale;
    float res_scale, eps;
    int32_t post, pre, dtype, param_dtype;
} convrot_gated_norm_args;

convrot_status convrot_gated_norm(const convrot_gated_norm_args *a, cudaStream_t stream);

/*
 * Its gradient. From the forward pass's h (as stored) and y, and the gradients
 * dh and dn of its outputs (either may be NULL: zero):
 *
 *   dx, dy     [m, d] of type dtype
 *   dgate, dscale, dshift             fp32 [batches, d], dense
 *   dpost_weight, dpost_bias, dpre_weight, dpre_bias   fp32 [d]
 *
 * each may be NULL (not wanted). Infinite values of h, or of y, may make the
 * gradients of their row NaN, and the sums over rows with them, also where no
 * norm stands on them. The remaining fields are the forward call's;
 * shift has no part in any gradient. Sums over rows are fp32 in an order that
 * depends on the sizes alone, so results are deterministic.
 *   work       256-byte aligned, convrot_gated_norm_backward_work_bytes(m, d,
 *              rows_per_batch) bytes: 16 d for each run of rows (about one an
 *              SM), and 32 d for each sample where there are more samples than
 *              that (5.4 GB at 32760 samples of one row of 5120).
 */
typedef struct {
    const void *h, *y, *dh, *dn, *gate, *scale;
    const void *post_weight, *post_bias, *pre_weight, *pre_bias;
    void *dx, *dy;
    float *dgate, *dscale, *dshift, *dpost_weight, *dpost_bias, *dpre_weight, *dpre_bias;
    void *work;
    int64_t work_bytes;
    int64_t m, d, rows_per_batch;
    int64_t ldh, ldy, lddh, lddn, ldgate, ldscale, lddx, lddy;
    float res_scale, eps;
    int32_t post, pre, dtype, param_dtype;
} convrot_gated_norm_backward_args;

int64_t convrot_gated_norm_backward_work_bytes(int64_t m, int64_t d, int64_t rows_per_batch);
convrot_status convrot_gated_norm_backward(const convrot_gated_norm_backward_args *a, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Rotary positions: the first rot_dim values of each head are turned in pairs
 * by the angles of the token's position, the others are copied.
 *
 *   (a, b) -> (a cos - b sin, b cos + a sin)
 *   CONVROT_ROTARY_HALF         a = v[i], b = v[i + rot_dim / 2]
 *   CONVROT_ROTARY_INTERLEAVED  a = v[2 i], b = v[2 i + 1]
 *
 * inverse != 0 turns by the opposite angles: the gradient of the rotation.
 *
 *   q, k       [batch, tokens, heads, head_dim] of type dtype with any batch,
 *              token and head strides (elements; >= 0) and head_dim
 *              contiguous. k may be NULL. out_q / out_k likewise, their heads
 *              apart from one another; each may be its input with the same
 *              strides (in place).
 *   cos, sin   fp32 [table_rows, ldt], ldt >= rot_dim / 2.
 *   positions  the table row of each token: int32 or int64 (position_bits)
 *              [batch, tokens] with pos_stride elements between batches
 *              (0: all sequences share them), or NULL: token t uses row t.
 *              A position outside the table gives NaN in its token's rotated
 *              values and CONVROT_ERR_INVALID_ARG in *dev_status.
 *   dev_status device int32 or NULL.
 * 2 <= rot_dim <= head_dim <= CONVROT_ROTARY_MAX_D, rot_dim even.
 */
typedef enum { CONVROT_ROTARY_HALF = 0, CONVROT_ROTARY_INTERLEAVED = 1 } convrot_rotary_layout;
#define CONVROT_ROTARY_MAX_D 4096

typedef struct {
    const void *q, *k;
    void *out_q, *out_k;
    const float *cos, *sin;
    const void *positions;
    int32_t *dev_status;
    int64_t batch, tokens, q_heads, k_heads;
    int64_t q_strides[3], k_strides[3], out_q_strides[3], out_k_strides[3]; /* batch, token, head */
    int64_t table_rows, ldt, pos_stride;
    int32_t head_dim, rot_dim, layout, inverse, dtype, position_bits;
} convrot_rotary_args;

convrot_status convrot_rotary(const convrot_rotary_args *a, cudaStream_t stream);

/*
 * Fills the tables: for row p and pair i, with the angle
 *   positions[p * axes + axis[i]] * freq[i]
 * cos[p, i] = factor * cos(angle), sin[p, i] = factor * sin(angle), the angle
 * reduced in 64 bits so that late positions lose nothing.
 *   positions  fp64 [rows, axes] (image and video tokens have one per axis),
 *              or NULL with axes == 1: row p's position is p.
 *   freq       fp64 [pairs]; axis: int32 [pairs] or NULL (all 0); values
 *              outside [0, axes) give NaN.
 */
convrot_status convrot_rotary_table(const double *positions, int64_t rows, int32_t axes, const double *freq,
                                    const int32_t *axis, int32_t pairs, double factor, float *cos, float *sin,
                                    int64_t ldt, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CONVROT_BLOCK_H_ */
