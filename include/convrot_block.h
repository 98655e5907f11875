/*
 * convrot_block.h -- C ABI of the operators that stand between the linears of
 * a transformer block: a linear on 8-bit floating-point codes with block
 * scales, the gated norm with its gradient, rotary positions, the gated
 * feed-forward's projections and attention to other states, both with their
 * gradients.
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

/* ------------------------------------------------------------------------
 * The input half of a gated feed-forward on 16-bit weights: both projections,
 * the activation and the product.
 *
 *   g = x w_gate^T + b_gate,  u = x w_up^T + b_up
 *   y = act(g) * u
 *
 * act is a convrot_activation or CONVROT_ACT_SILU, v / (1 + e^-v). The products
 * run on the tensor cores with fp32 sums; y is rounded once, from the fp32 g and u.
 *
 *   x          [m, ldx], w_gate, w_up [n, ldw*], all of type dtype (CONVROT_BF16
 *              or CONVROT_F16; CONVROT_F32 is CONVROT_ERR_UNSUPPORTED).
 *   b_gate, b_up   fp32 [n], each may be NULL.
 *   y          [m, ldy] of type dtype.
 *   gate, up   NULL, or both: g and u rounded to dtype, for the gradient.
 *   work       256-byte aligned, convrot_gated_linear_work_bytes(a) bytes: 0
 *              where the rows of x and of the weights start on 16 bytes, else
 *              room for copies of those that do not. The function reads the
 *              tensors' addresses and leading dimensions, and no memory.
 *   dev_status as for convrot_linear.
 * m == 0 or n == 0 launches nothing; 1 <= k. Outputs must not overlap inputs.
 *
 * From here on to the end of this header, 16-bit inputs are read in aligned
 * blocks of 16 bytes: those that hold an element of a tensor may be read whole,
 * so up to 14 bytes before its first element and behind its last one (in the
 * same 16 bytes, so in memory that is there). Nothing depends on what they are,
 * and nothing beside a tensor's elements is written.
 */
enum { CONVROT_ACT_SILU = 3 };

typedef struct {
    const void *x, *w_gate, *w_up;
    const float *b_gate, *b_up;
    void *y, *gate, *up;
    void *work;
    int32_t *dev_status;
    int64_t m, n, k;
    int64_t ldx, ldw_gate, ldw_up, ldy, ldgate, ldup;
    int64_t work_bytes;
    int32_t dtype, act;
} convrot_gated_linear_args;

int64_t convrot_gated_linear_work_bytes(const convrot_gated_linear_args *a);
convrot_status convrot_gated_linear(const convrot_gated_linear_args *a, cudaStream_t stream);

/*
 * Its gradient, from x, the weights, the kept gate and up and the gradient dy of y:
 *
 *   dg = dy u act'(g),  du = dy act(g)
 *   dx = dg w_gate + du w_up          [m, lddx] of type dtype
 *   dw_gate = dg^T x, dw_up = du^T x  [n, lddw*] of type dtype
 *   db_gate, db_up                    column sums of dg and du, fp32 [n]
 *
 * dx, the pair dw_* and the pair db_* may be NULL (not wanted; x is then not read where the
 * weights' gradients are not wanted). dg and du are rounded to dtype for the products, as their
 * operands have to be; the column sums are those of the unrounded fp32 values, added up in an
 * order that depends on the sizes alone.
 *   work       256-byte aligned, convrot_gated_linear_backward_work_bytes(a)
 *              bytes: dg and du, the partial column sums, and copies of operands
 *              whose rows do not start on 16 bytes.
 * m == 0: the gradients of the weights and biases are zero. Outputs must not
 * overlap inputs.
 */
typedef struct {
    const void *x, *w_gate, *w_up, *gate, *up, *dy;
    void *dx, *dw_gate, *dw_up;
    float *db_gate, *db_up;
    void *work;
    int32_t *dev_status;
    int64_t m, n, k;
    int64_t ldx, ldw_gate, ldw_up, ldgate, ldup, lddy, lddx, lddw_gate, lddw_up;
    int64_t work_bytes;
    int32_t dtype, act;
} convrot_gated_linear_backward_args;

int64_t convrot_gated_linear_backward_work_bytes(const convrot_gated_linear_backward_args *a);
convrot_status convrot_gated_linear_backward(const convrot_gated_linear_backward_args *a, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Attention to states of another length (a prompt's, an encoder's):
 *
 *   s_ij = scale q_i . k_j,  lse_i = log(sum_j e^(s_ij))  over the keys that are there
 *   out_i = sum_j e^(s_ij - lse_i) v_j
 *
 * A query without keys (all masked, or kv_tokens == 0) has out 0 and lse -infinity.
 * What stands in a masked key or value (NaN too) does not reach any result.
 * Scores past the floats are infinite: a query with one of +infinity (or NaN)
 * has NaN, one whose scores are all -infinity counts as one without keys.
 *
 *   q, out     [batch, q_tokens, q_heads, head_dim] of type dtype (CONVROT_BF16
 *              or CONVROT_F16; CONVROT_F32 is CONVROT_ERR_UNSUPPORTED),
 *   k, v       [batch, kv_tokens, kv_heads, head_dim]: query head h reads head
 *              h / (q_heads / kv_heads); kv_heads divides q_heads.
 *              Strides (elements, >= 0) of batch, token and head for each,
 *              head_dim contiguous; out's heads apart from one another.
 *   mask       uint8 [batch, kv_tokens] with mask_stride elements between
 *              batches: 0 where a key is not there; or NULL.
 *   lse        fp32 [batch, q_heads, q_tokens], dense.
 *   scale      > 0, at most 1.7e38.
 *   work       256-byte aligned, convrot_attention_work_bytes(a) bytes: 0, or
 *              room for the keys that are there (with a mask of more than 128
 *              keys), for copies of tensors whose heads do not start on 16
 *              bytes, and for partial results of few queries against long
 *              states. The function reads no memory.
 *   dev_status as for convrot_linear.
 * 1 <= head_dim <= CONVROT_ATTENTION_MAX_D (CONVROT_ERR_UNSUPPORTED above).
 * Probabilities are rounded to dtype for their product with v, whose operands
 * have one type; the sums of a softmax are fp32, of the unrounded values.
 * Outputs must not overlap inputs.
 */
#define CONVROT_ATTENTION_MAX_D 128

typedef struct {
    const void *q, *k, *v;
    const uint8_t *mask;
    void *out;
    float *lse;
    void *work;
    int32_t *dev_status;
    int64_t batch, q_tokens, kv_tokens, q_heads, kv_heads;
    int64_t q_strides[3], k_strides[3], v_strides[3], out_strides[3]; /* batch, token, head */
    int64_t mask_stride, work_bytes;
    float scale;
    int32_t head_dim, dtype, reserved; /* 0 */
} convrot_attention_args;

int64_t convrot_attention_work_bytes(const convrot_attention_args *a);
convrot_status convrot_attention(const convrot_attention_args *a, cudaStream_t stream);

/*
 * Its gradient, from the forward call's tensors and the gradient dout of out
 * (with its strides):
 *
 *   P_ij = e^(s_ij - lse_i),  dS_ij = P_ij (dout_i . v_j - dout_i . out_i)
 *   dq_i = scale sum_j dS_ij k_j,  dk_j = scale sum_i dS_ij q_i,  dv_j = sum_i P_ij dout_i
 *
 * dq, dk, dv   dense [batch, tokens, heads, head_dim] of type dtype; dk and dv are
 *              summed over the query heads that share a head and are 0 at
 *              masked keys.
 * P and dS are rounded to dtype for their products; for CONVROT_F16 they are
 * scaled by powers of two first, so that small gradients keep their bits. That
 * of dS is one for all queries of a key head: beside its rounding, dS is off by up
 * to 2^-22 of their largest |dout|, and it is infinite past 2^18 of that (which
 * takes values v past 4096). Sums are fp32, in an order that depends on the sizes
 * (and, with a mask, on the number of keys) alone. Outputs must not overlap inputs.
 *   work       256-byte aligned, convrot_attention_backward_work_bytes(a) bytes:
 *              8 for each query and head, partial sums (50 MB at most), and what
 *              the forward call's has room for.
 */
typedef struct {
    const void *q, *k, *v, *out, *dout;
    const uint8_t *mask;
    const float *lse;
    void *dq, *dk, *dv;
    void *work;
    int32_t *dev_status;
    int64_t batch, q_tokens, kv_tokens, q_heads, kv_heads;
    int64_t q_strides[3], k_strides[3], v_strides[3], out_strides[3], dout_strides[3];
    int64_t mask_stride, work_bytes;
    float scale;
    int32_t head_dim, dtype, reserved; /* 0 */
} convrot_attention_backward_args;

int64_t convrot_attention_backward_work_bytes(const convrot_attention_backward_args *a);
convrot_status convrot_attention_backward(const convrot_attention_backward_args *a, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CONVROT_BLOCK_H_ */
