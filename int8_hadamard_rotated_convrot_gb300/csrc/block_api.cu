// C-ABI entry points of the operators around the linears: host-side
// validation, then launches. The contract is include/convrot_block.h.
#include <climits>

#include "block.h"

namespace {

using namespace convrot;

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int size_of(int dtype) { return dtype == CONVROT_F32 ? 4 : 2; }

bool known(int dtype) { return dtype == CONVROT_F32 || dtype == CONVROT_BF16 || dtype == CONVROT_F16; }

constexpr int64_t kMaxRows = INT_MAX;  // rows and row blocks are counted in 32 bits on the device

int64_t groups(int64_t v, int64_t size) { return (v + size - 1) / size; }

cudaError_t run_linear(const convrot_fp8_linear_args &a, cudaStream_t stream)
{
    return fp8_few_takes(a.m, a.n, a.k) ? launch_fp8_few(a, stream) : launch_fp8_gemm(a, stream);
}

convrot_status done(cudaError_t e) { return e == cudaSuccess ? CONVROT_OK : CONVROT_ERR_CUDA; }

// A matrix [rows, cols] of elements of `bytes` bytes.
convrot_status check_matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, int bytes)
{
    if (ld < cols) return CONVROT_ERR_INVALID_ARG;
    if (rows == 0) return CONVROT_OK;
    if (!p) return CONVROT_ERR_INVALID_ARG;
    return aligned(p, bytes) ? CONVROT_OK : CONVROT_ERR_ALIGNMENT;
}

convrot_status check_optional(const void *p, int64_t rows, int64_t cols, int64_t ld, int bytes)
{
    return p ? check_matrix(p, rows, cols, ld, bytes) : CONVROT_OK;
}

convrot_status first_of(std::initializer_list<convrot_status> all)
{
    for (convrot_status s : all)
        if (s != CONVROT_OK) return s;
    return CONVROT_OK;
}

convrot_status check_codes(const void *q, int64_t rows, int64_t k, int64_t ldq)
{
    if (ldq < k) return CONVROT_ERR_INVALID_ARG;
    if (ldq % 16) return CONVROT_ERR_ALIGNMENT;
    if (rows == 0) return CONVROT_OK;
    if (!q) return CONVROT_ERR_INVALID_ARG;
    return aligned(q, 16) ? CONVROT_OK : CONVROT_ERR_ALIGNMENT;
}

convrot_status check_quantize(const void *src, int dtype, int64_t rows, int64_t k, int64_t ld, const void *q, int64_t ldq)
{
    if (rows < 0 || rows > kMaxRows || !known(dtype)) return CONVROT_ERR_INVALID_ARG;
    if (k < 1 || k > CONVROT_MAX_K) return CONVROT_ERR_K_RANGE;
    return first_of({check_matrix(src, rows, k, ld, size_of(dtype)), check_codes(q, rows, k, ldq)});
}

// What both linears ask for, without x.
convrot_status check_linear(const convrot_fp8_linear_args *a)
{
    if (a->m < 0 || a->m > kMaxRows || a->n < 0 || a->n > kMaxRows || a->reserved) return CONVROT_ERR_INVALID_ARG;
    if (a->k < 1 || a->k > CONVROT_MAX_K) return CONVROT_ERR_K_RANGE;
    if (!known(a->y_dtype) || a->act < CONVROT_ACT_NONE || a->act > CONVROT_ACT_GELU_TANH) return CONVROT_ERR_INVALID_ARG;
    if (a->m == 0) return first_of({check_codes(a->w, 0, a->k, a->ldw)});
    return first_of({check_codes(a->w, a->n, a->k, a->ldw),
                     check_matrix(a->w_scale, groups(a->n, 128), groups(a->k, 128), a->ld_w_scale, 4),
                     check_matrix(a->y, a->n ? a->m : 0, a->n, a->ldy, size_of(a->y_dtype)),
                     check_optional(a->bias, 1, a->n, a->n, 4), check_optional(a->dev_status, 1, 1, 1, 4)});
}

int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }
int64_t work_ldq(int64_t k) { return groups(k, 16) * 16; }
int64_t work_lds(int64_t m) { return groups(m, 4) * 4; }

// Rows of a sample, with no more than there are (so that sums of rows stay far from 64 bits).
int64_t sample_of(int64_t m, int64_t rows) { return rows < m ? rows : m > 1 ? m : 1; }

// Whether an output's heads lie apart from one another (as far as two neighbours show it), and where the output is the
// input itself, each head in its own place: threads read and write different heads in any order.
bool rotary_output(const convrot_rotary_args &a, const void *in, const int64_t *in_strides, const void *out, const int64_t *strides, int64_t heads)
{
    const int64_t n[3] = {a.batch, a.tokens, heads};
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) continue;
        if (strides[i] < a.head_dim || (in == out && strides[i] != in_strides[i])) return false;
        for (int j = 0; j < i; ++j)
            if (n[j] > 1 && strides[i] - strides[j] < a.head_dim && strides[j] - strides[i] < a.head_dim) return false;
    }
    return true;
}

convrot_status check_norm(int64_t m, int64_t d, int64_t rows, int dtype, int param_dtype, int post, int pre, float eps)
{
    if (m < 0 || m > kMaxRows || d < 1 || rows < 1 || !known(dtype)) return CONVROT_ERR_INVALID_ARG;
    if (param_dtype != CONVROT_F32 && param_dtype != dtype) return CONVROT_ERR_INVALID_ARG;
    if (post < CONVROT_NORM_NONE || post > CONVROT_NORM_LAYER || pre < CONVROT_NORM_NONE || pre > CONVROT_NORM_LAYER)
        return CONVROT_ERR_INVALID_ARG;
    if (!(eps >= 0.0f)) return CONVROT_ERR_INVALID_ARG;
    return d > CONVROT_NORM_MAX_D ? CONVROT_ERR_UNSUPPORTED : CONVROT_OK;
}

}  // namespace

extern "C" {

convrot_status convrot_fp8_pack_activations(const void *X, int32_t x_dtype, int64_t m, int64_t k, int64_t ldx,
                                            void *q, int64_t ldq, float *scale, int64_t lds, cudaStream_t stream)
{
    convrot_status st = check_quantize(X, x_dtype, m, k, ldx, q, ldq);
    if (st == CONVROT_OK) st = check_matrix(scale, m, m, lds, 4);
    if (st != CONVROT_OK || m == 0) return st;
    return done(launch_fp8_pack(X, x_dtype, m, k, ldx, q, ldq, scale, lds, stream));
}

convrot_status convrot_fp8_quantize_weights(const void *W, int32_t w_dtype, int64_t n, int64_t k, int64_t ldw,
                                            void *q, int64_t ldq, float *scale, int64_t lds, cudaStream_t stream)
{
    convrot_status st = check_quantize(W, w_dtype, n, k, ldw, q, ldq);
    if (st == CONVROT_OK) st = check_matrix(scale, n, groups(k, 128), lds, 4);
    if (st != CONVROT_OK || n == 0) return st;
    return done(launch_fp8_quantize_weights(W, w_dtype, n, k, ldw, q, ldq, scale, lds, stream));
}

convrot_status convrot_fp8_linear(const convrot_fp8_linear_args *a, cudaStream_t stream)
{
    if (!a) return CONVROT_ERR_INVALID_ARG;
    convrot_status st = check_linear(a);
    if (st == CONVROT_OK)
        st = first_of({check_codes(a->x, a->m, a->k, a->ldx), check_matrix(a->x_scale, a->m, a->m, a->ld_x_scale, 4)});
    if (st != CONVROT_OK || a->m == 0 || a->n == 0) return st;
    return done(run_linear(*a, stream));
}

int64_t convrot_fp8_pack_linear_work_bytes(int64_t m, int64_t n, int64_t k)
{
    if (m < 1 || n < 1 || k < 1 || m > kMaxRows || k > CONVROT_MAX_K || fp8_few_quantizes(m, n, k)) return 0;
    return round256(m * work_ldq(k)) + round256(groups(k, 128) * work_lds(m) * 4);
}

convrot_status convrot_fp8_pack_linear(const convrot_fp8_linear_args *a, cudaStream_t stream)
{
    if (!a) return CONVROT_ERR_INVALID_ARG;
    convrot_status st = check_linear(a);
    if (st != CONVROT_OK) return st;
    if (!known(a->x_dtype)) return CONVROT_ERR_INVALID_ARG;
    st = check_matrix(a->x, a->m, a->k, a->ldx, size_of(a->x_dtype));
    if (st != CONVROT_OK || a->m == 0 || a->n == 0) return st;
    const int64_t need = convrot_fp8_pack_linear_work_bytes(a->m, a->n, a->k);
    if (need > 0 && (!a->work || a->work_bytes < need)) return CONVROT_ERR_INVALID_ARG;
    if (need > 0 && !aligned(a->work, 256)) return CONVROT_ERR_ALIGNMENT;
    if (need == 0) return done(launch_fp8_few_quantize(*a, stream));
    convrot_fp8_linear_args g = *a;
    g.ldx = work_ldq(a->k);
    g.ld_x_scale = work_lds(a->m);
    float *scale = reinterpret_cast<float *>(static_cast<char *>(a->work) + round256(a->m * g.ldx));
    g.x = a->work;
    g.x_scale = scale;
    st = done(launch_fp8_pack(a->x, a->x_dtype, a->m, a->k, a->ldx, a->work, g.ldx, scale, g.ld_x_scale, stream));
    return st == CONVROT_OK ? done(run_linear(g, stream)) : st;
}

convrot_status convrot_gated_norm(const convrot_gated_norm_args *a, cudaStream_t stream)
{
    if (!a) return CONVROT_ERR_INVALID_ARG;
    convrot_status st = check_norm(a->m, a->d, a->rows_per_batch, a->dtype, a->param_dtype, a->post, a->pre, a->eps);
    if (st != CONVROT_OK) return st;
    const int s = size_of(a->dtype), p = size_of(a->param_dtype);
    const int64_t m = a->m, d = a->d, rows = sample_of(m, a->rows_per_batch), batches = groups(m, rows);
    st = first_of({check_matrix(a->x, m, d, a->ldx, s), check_optional(a->y, m, d, a->ldy, s),
                   check_optional(a->gate, batches, d, a->ldgate, p), check_optional(a->scale, batches, d, a->ldscale, p),
                   check_optional(a->shift, batches, d, a->ldshift, p), check_optional(a->post_weight, 1, d, d, p),
                   check_optional(a->post_bias, 1, d, d, p), check_optional(a->pre_weight, 1, d, d, p),
                   check_optional(a->pre_bias, 1, d, d, p), check_optional(a->h, m, d, a->ldh, s),
                   check_optional(a->n, m, d, a->ldn, s)});
    if (st == CONVROT_OK && a->q) st = first_of({check_codes(a->q, m, d, a->ldq), check_matrix(a->q_scale, m, m, a->ld_q_scale, 4)});
    if (st != CONVROT_OK || m == 0) return st;
    if (a->h == a->x && a->ldh != a->ldx) return CONVROT_ERR_INVALID_ARG;
    if (!a->h && !a->n && !a->q) return CONVROT_OK;
    convrot_gated_norm_args b = *a;
    b.rows_per_batch = rows;
    return done(launch_gated_norm(b, stream));
}

int64_t convrot_gated_norm_backward_work_bytes(int64_t m, int64_t d, int64_t rows_per_batch)
{
    if (m < 1 || m > kMaxRows || d < 1 || d > CONVROT_NORM_MAX_D || rows_per_batch < 1) return 0;
    return round256(gated_norm_backward_work_bytes(m, d, sample_of(m, rows_per_batch)));
}

convrot_status convrot_gated_norm_backward(const convrot_gated_norm_backward_args *a, cudaStream_t stream)
{
    if (!a) return CONVROT_ERR_INVALID_ARG;
    convrot_status st = check_norm(a->m, a->d, a->rows_per_batch, a->dtype, a->param_dtype, a->post, a->pre, a->eps);
    if (st != CONVROT_OK) return st;
    const int s = size_of(a->dtype), p = size_of(a->param_dtype);
    const int64_t m = a->m, d = a->d, rows = sample_of(m, a->rows_per_batch), batches = groups(m, rows);
    st = first_of({check_matrix(a->h, m, d, a->ldh, s), check_optional(a->y, m, d, a->ldy, s),
                   check_optional(a->dh, m, d, a->lddh, s), check_optional(a->dn, m, d, a->lddn, s),
                   check_optional(a->gate, batches, d, a->ldgate, p), check_optional(a->scale, batches, d, a->ldscale, p),
                   check_optional(a->post_weight, 1, d, d, p), check_optional(a->post_bias, 1, d, d, p),
                   check_optional(a->pre_weight, 1, d, d, p), check_optional(a->pre_bias, 1, d, d, p),
                   check_optional(a->dx, m, d, a->lddx, s), check_optional(a->dy, m, d, a->lddy, s)});
    for (const float *v : {a->dgate, a->dscale, a->dshift, a->dpost_weight, a->dpost_bias, a->dpre_weight, a->dpre_bias})
        if (st == CONVROT_OK) st = check_optional(v, 1, 1, 1, 4);
    if (st != CONVROT_OK) return st;
    if (!a->y && (a->dy || a->dgate || a->dpost_weight || a->dpost_bias)) return CONVROT_ERR_INVALID_ARG;
    if (m == 0) {  // no rows: the gradients of the weights are zero
        for (float *v : {a->dpost_weight, a->dpost_bias, a->dpre_weight, a->dpre_bias})
            if (v && cudaMemsetAsync(v, 0, d * 4, stream) != cudaSuccess) return CONVROT_ERR_CUDA;
        return CONVROT_OK;
    }
    if (!a->work || a->work_bytes < convrot_gated_norm_backward_work_bytes(m, d, rows)) return CONVROT_ERR_INVALID_ARG;
    if (!aligned(a->work, 256)) return CONVROT_ERR_ALIGNMENT;
    convrot_gated_norm_backward_args b = *a;
    b.rows_per_batch = rows;
    return done(launch_gated_norm_backward(b, stream));
}

convrot_status convrot_rotary(const convrot_rotary_args *a, cudaStream_t stream)
{
    if (!a) return CONVROT_ERR_INVALID_ARG;
    if (a->batch < 0 || a->tokens < 0 || a->q_heads < 0 || a->k_heads < 0 || !known(a->dtype)) return CONVROT_ERR_INVALID_ARG;
    if (a->rot_dim < 2 || a->rot_dim % 2 || a->rot_dim > a->head_dim) return CONVROT_ERR_INVALID_ARG;
    if (a->head_dim > CONVROT_ROTARY_MAX_D) return CONVROT_ERR_UNSUPPORTED;
    if (a->layout != CONVROT_ROTARY_HALF && a->layout != CONVROT_ROTARY_INTERLEAVED) return CONVROT_ERR_INVALID_ARG;
    if (a->tokens && a->batch > kMaxRows / a->tokens) return CONVROT_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i)
        if (a->q_strides[i] < 0 || a->k_strides[i] < 0 || a->out_q_strides[i] < 0 || a->out_k_strides[i] < 0)
            return CONVROT_ERR_INVALID_ARG;
    const int64_t heads = (a->q ? a->q_heads : 0) + (a->k ? a->k_heads : 0);
    if (a->batch == 0 || a->tokens == 0 || heads == 0) return CONVROT_OK;
    if (heads > kMaxRows / CONVROT_ROTARY_MAX_D) return CONVROT_ERR_INVALID_ARG;
    const int s = size_of(a->dtype);
    convrot_status st = first_of({check_matrix(a->cos, 1, a->rot_dim / 2, a->ldt, 4), check_matrix(a->sin, 1, a->rot_dim / 2, a->ldt, 4),
                                  check_optional(a->dev_status, 1, 1, 1, 4), check_optional(a->q, 1, 1, 1, s),
                                  check_optional(a->k, 1, 1, 1, s), check_matrix(a->out_q, a->q && a->q_heads, 1, 1, s),
                                  check_matrix(a->out_k, a->k && a->k_heads, 1, 1, s)});
    if (st != CONVROT_OK) return st;
    if (a->q && a->q_heads && !rotary_output(*a, a->q, a->q_strides, a->out_q, a->out_q_strides, a->q_heads)) return CONVROT_ERR_INVALID_ARG;
    if (a->k && a->k_heads && !rotary_output(*a, a->k, a->k_strides, a->out_k, a->out_k_strides, a->k_heads)) return CONVROT_ERR_INVALID_ARG;
    if (a->positions) {
        if (a->position_bits != 32 && a->position_bits != 64) return CONVROT_ERR_INVALID_ARG;
        if (!aligned(a->positions, a->position_bits / 8)) return CONVROT_ERR_ALIGNMENT;
        if (a->pos_stride < 0 || a->table_rows < 1) return CONVROT_ERR_INVALID_ARG;
    } else if (a->table_rows < a->tokens) {
        return CONVROT_ERR_INVALID_ARG;
    }
    convrot_rotary_args b = *a;
    if (!b.q) b.q_heads = 0;
    if (!b.k) b.k_heads = 0;
    return done(launch_rotary(b, stream));
}

convrot_status convrot_rotary_table(const double *positions, int64_t rows, int32_t axes, const double *freq,
                                    const int32_t *axis, int32_t pairs, double factor, float *cos, float *sin,
                                    int64_t ldt, cudaStream_t stream)
{
    if (rows < 0 || rows > kMaxRows || axes < 1 || pairs < 1 || pairs > CONVROT_ROTARY_MAX_D / 2) return CONVROT_ERR_INVALID_ARG;
    if (!positions && axes != 1 && rows > 0) return CONVROT_ERR_INVALID_ARG;
    convrot_status st = first_of({check_matrix(freq, 1, pairs, pairs, 8), check_optional(positions, 1, 1, 1, 8),
                                  check_optional(axis, 1, 1, 1, 4), check_matrix(cos, rows, pairs, ldt, 4),
                                  check_matrix(sin, rows, pairs, ldt, 4)});
    if (st != CONVROT_OK || rows == 0) return st;
    return done(launch_rotary_table(positions, rows, axes, freq, axis, pairs, factor, cos, sin, ldt, stream));
}

}  // extern "C"
