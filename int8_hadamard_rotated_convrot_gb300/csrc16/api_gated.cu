// C-ABI entry points of the gated feed-forward's projections: host-side
// validation, workspaces, then launches. The contract is
// include/convrot_block.h.
#include "api16.h"
#include "gated.h"
#include "mma16.cuh"

namespace {

using namespace convrot;

int64_t pitch(int64_t cols) { return (cols + 7) / 8 * 8; }

// One call's operands and workspace: first the sizes are added up, then, with a base, the pieces are handed out.
struct Work {
    char *base;
    int64_t used = 0;
    void *take(int64_t bytes)
    {
        void *at = base ? base + used : nullptr;
        used += round256(bytes);
        return at;
    }
};

// An operand of a product: itself, or a copy whose rows start on 16 bytes.
struct Operand {
    const void *p;
    int64_t rows, cols, ld;
    void *copy = nullptr;
    bool copied = false;
    Operand(const void *p_, int64_t rows_, int64_t cols_, int64_t ld_) : p(p_), rows(rows_), cols(cols_), ld(ld_) {}
    void plan(Work &w)
    {
        if (mma16::tma_rows(p, ld, rows)) return;
        copied = true;
        copy = w.take(rows * pitch(cols) * 2);
    }
    cudaError_t make(cudaStream_t stream)
    {
        if (!copied) return cudaSuccess;
        const cudaError_t e = launch_align_rows(p, rows, cols, ld, copy, pitch(cols), stream);
        p = copy;
        ld = pitch(cols);
        return e;
    }
};

bool gated_sizes(int64_t m, int64_t n, int64_t k) { return m >= 0 && n >= 0 && k >= 1 && m <= kMaxSize && n <= kMaxSize && k <= kMaxSize; }

convrot_status check_kind(int64_t m, int64_t n, int64_t k, int dtype, int act)
{
    if (!gated_sizes(m, n, k) || act < CONVROT_ACT_NONE || act > CONVROT_ACT_SILU) return CONVROT_ERR_INVALID_ARG;
    return check_16bit(dtype);
}

struct ForwardWork {
    Operand x, wg, wu;
    int64_t bytes;
    explicit ForwardWork(const convrot_gated_linear_args &a, char *base = nullptr)
        : x(a.x, a.m, a.k, a.ldx), wg(a.w_gate, a.n, a.k, a.ldw_gate), wu(a.w_up, a.n, a.k, a.ldw_up)
    {
        Work w{base};
        x.plan(w);
        wg.plan(w);
        wu.plan(w);
        bytes = w.used;
    }
};

struct BackwardWork {
    Operand x, wg, wu;
    void *dg, *du;
    float *partial = nullptr, *shares = nullptr;
    int64_t bytes, ldd;
    explicit BackwardWork(const convrot_gated_linear_backward_args &a, char *base = nullptr)
        : x(a.x, a.m, a.k, a.ldx), wg(a.w_gate, a.n, a.k, a.ldw_gate), wu(a.w_up, a.n, a.k, a.ldw_up), ldd(pitch(a.n))
    {
        Work w{base};
        dg = w.take(a.m * ldd * 2);
        du = w.take(a.m * ldd * 2);
        if (a.db_gate) partial = static_cast<float *>(w.take(gated_grad_chunks(a.m, a.n) * 2 * a.n * 4));
        if (a.dw_gate) x.plan(w);
        if (a.dx) {
            wg.plan(w);
            wu.plan(w);
            shares = static_cast<float *>(w.take(gated_dx_partial_bytes(a.m, a.n, a.k)));
        }
        bytes = w.used;
    }
};

}  // namespace

extern "C" {

int64_t convrot_gated_linear_work_bytes(const convrot_gated_linear_args *a)
{
    if (!a || !gated_sizes(a->m, a->n, a->k) || a->m == 0 || a->n == 0) return 0;
    return ForwardWork(*a).bytes;
}

convrot_status convrot_gated_linear(const convrot_gated_linear_args *a, cudaStream_t stream)
{
    if (!a) return CONVROT_ERR_INVALID_ARG;
    convrot_status st = check_kind(a->m, a->n, a->k, a->dtype, a->act);
    if (st != CONVROT_OK) return st;
    if (!a->gate != !a->up) return CONVROT_ERR_INVALID_ARG;
    const int64_t m = a->n ? a->m : 0, n = a->m ? a->n : 0;  // nothing is read where there is nothing to write
    st = first_of({check_matrix(a->x, m, a->k, a->ldx, 2), check_matrix(a->w_gate, n, a->k, a->ldw_gate, 2),
                   check_matrix(a->w_up, n, a->k, a->ldw_up, 2), check_matrix(a->y, m, a->n, a->ldy, 2),
                   check_optional(a->gate, m, a->n, a->ldgate, 2), check_optional(a->up, m, a->n, a->ldup, 2),
                   check_optional(a->b_gate, 1, a->n, a->n, 4), check_optional(a->b_up, 1, a->n, a->n, 4),
                   check_optional(a->dev_status, 1, 1, 1, 4)});
    if (st != CONVROT_OK || m == 0 || n == 0) return st;
    ForwardWork w(*a, static_cast<char *>(a->work));
    if ((st = check_work(a->work, a->work_bytes, w.bytes)) != CONVROT_OK) return st;
    convrot_gated_linear_args b = *a;
    for (Operand *o : {&w.x, &w.wg, &w.wu})
        if (o->make(stream) != cudaSuccess) return CONVROT_ERR_CUDA;
    b.x = w.x.p;
    b.ldx = w.x.ld;
    b.w_gate = w.wg.p;
    b.ldw_gate = w.wg.ld;
    b.w_up = w.wu.p;
    b.ldw_up = w.wu.ld;
    return done(gated_few_takes(a->m, a->n, a->k) ? launch_gated_few(b, stream) : launch_gated_gemm(b, stream));
}

int64_t convrot_gated_linear_backward_work_bytes(const convrot_gated_linear_backward_args *a)
{
    if (!a || !gated_sizes(a->m, a->n, a->k) || a->m == 0 || a->n == 0) return 0;
    return BackwardWork(*a).bytes;
}

convrot_status convrot_gated_linear_backward(const convrot_gated_linear_backward_args *a, cudaStream_t stream)
{
    if (!a) return CONVROT_ERR_INVALID_ARG;
    convrot_status st = check_kind(a->m, a->n, a->k, a->dtype, a->act);
    if (st != CONVROT_OK) return st;
    if (!a->dw_gate != !a->dw_up || !a->db_gate != !a->db_up) return CONVROT_ERR_INVALID_ARG;
    const int64_t m = a->m, n = a->n, k = a->k, used = n ? m : 0;
    st = first_of({check_matrix(a->gate, used, n, a->ldgate, 2), check_matrix(a->up, used, n, a->ldup, 2), check_matrix(a->dy, used, n, a->lddy, 2),
                   check_optional(a->dx, m, k, a->lddx, 2), check_optional(a->dw_gate, n, k, a->lddw_gate, 2),
                   check_optional(a->dw_up, n, k, a->lddw_up, 2), check_optional(a->db_gate, 1, n, n, 4), check_optional(a->db_up, 1, n, n, 4),
                   check_optional(a->dev_status, 1, 1, 1, 4)});
    if (st == CONVROT_OK && a->dx)
        st = first_of({check_matrix(a->w_gate, m ? n : 0, k, a->ldw_gate, 2), check_matrix(a->w_up, m ? n : 0, k, a->ldw_up, 2)});
    if (st == CONVROT_OK && a->dw_gate) st = check_matrix(a->x, used, k, a->ldx, 2);
    if (st != CONVROT_OK) return st;
    if (m == 0 || n == 0) {  // sums over nothing
        bool ok = true;
        auto zero = [&](void *p, int64_t rows, int64_t cols, int64_t ld, int bytes) {
            if (ok && p && rows && cols) ok = cudaMemset2DAsync(p, ld * bytes, 0, cols * bytes, rows, stream) == cudaSuccess;
        };
        zero(a->dx, m, k, a->lddx, 2);
        zero(a->dw_gate, n, k, a->lddw_gate, 2);
        zero(a->dw_up, n, k, a->lddw_up, 2);
        zero(a->db_gate, 1, n, n, 4);
        zero(a->db_up, 1, n, n, 4);
        return ok ? CONVROT_OK : CONVROT_ERR_CUDA;
    }
    if (!a->dx && !a->dw_gate && !a->db_gate) return CONVROT_OK;
    BackwardWork w(*a, static_cast<char *>(a->work));
    if ((st = check_work(a->work, a->work_bytes, w.bytes)) != CONVROT_OK) return st;
    if (launch_gated_grad(*a, w.dg, w.du, w.ldd, w.partial, stream) != cudaSuccess) return CONVROT_ERR_CUDA;
    for (Operand *o : {&w.x, &w.wg, &w.wu})
        if (o->make(stream) != cudaSuccess) return CONVROT_ERR_CUDA;
    convrot_gated_linear_backward_args b = *a;
    b.x = w.x.p;
    b.ldx = w.x.ld;
    b.w_gate = w.wg.p;
    b.ldw_gate = w.wg.ld;
    b.w_up = w.wu.p;
    b.ldw_up = w.wu.ld;
    if (a->dx && launch_gated_dx(b, w.dg, w.du, w.ldd, w.shares, stream) != cudaSuccess) return CONVROT_ERR_CUDA;
    if (a->dw_gate && launch_gated_dw(b, w.dg, w.du, w.ldd, stream) != cudaSuccess) return CONVROT_ERR_CUDA;
    return CONVROT_OK;
}

}  // extern "C"
