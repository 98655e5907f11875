// C-ABI entry points of attention to other states: host-side validation,
// workspaces, then launches. The contract is include/convrot_block.h.
#include <cfloat>

#include "api16.h"
#include "attention.cuh"

namespace {

using namespace convrot;

// First the sizes are added up, then, with a base, the pieces are handed out.
struct Work {
    char *base;
    int64_t used = 0;
    template <typename T>
    T *take(int64_t count)
    {
        char *at = base ? base + used : nullptr;
        used += round256(count * static_cast<int64_t>(sizeof(T)));
        return reinterpret_cast<T *>(at);
    }
};

int64_t padded(int64_t d) { return (d + 7) / 8 * 8; }

States states(const void *p, int64_t tokens, int64_t heads, const int64_t (&strides)[3])
{
    return {p, tokens, heads, {strides[0], strides[1], strides[2]}};
}

// Up to two tensors of one shape, each as it is or, where a map cannot describe it or a mask picks its tokens, gathered.
struct Operands {
    States s[2];
    int64_t batch, rows;
    int32_t d;
    int32_t n;
    const uint8_t *mask = nullptr;
    int64_t mask_stride = 0;
    int32_t *counts = nullptr, *index = nullptr;
    bool copied[2] = {};
    uint16_t *copy[2] = {};

    Operands(int64_t batch_, int64_t d_, States a) : s{a, {}}, batch(batch_), rows(a.tokens), d(static_cast<int32_t>(d_)), n(1) {}
    Operands(int64_t batch_, int64_t d_, States a, States b) : s{a, b}, batch(batch_), rows(a.tokens), d(static_cast<int32_t>(d_)), n(2) {}

    void plan(Work &w, const uint8_t *mask_, int64_t stride, bool indexed)
    {
        if (s[0].tokens == 0) return;
        mask = mask_;
        mask_stride = stride;
        if (mask) {
            rows = gathered_rows(s[0].tokens);
            counts = w.take<int32_t>(batch);
            if (indexed) index = w.take<int32_t>(batch * rows);
        }
        for (int i = 0; i < n; ++i) {
            copied[i] = mask || !mma16::heads_on_16_bytes(s[i].p, s[i].strides, batch, s[i].tokens, s[i].heads, d);
            if (copied[i]) copy[i] = w.take<uint16_t>(batch * rows * s[i].heads * padded(d));
        }
    }
    cudaError_t make(cudaStream_t stream, void *zero0 = nullptr, void *zero1 = nullptr)
    {
        GatherArgs g{};
        void *const zero[2] = {zero0, zero1};
        for (int i = 0; i < n; ++i) {
            if (!copied[i]) continue;
            g.src[g.count] = s[i].p;
            for (int k = 0; k < 3; ++k) g.strides[g.count][k] = s[i].strides[k];
            g.dst[g.count] = copy[i];
            g.zero[g.count++] = zero[i];
        }
        if (g.count == 0) return cudaSuccess;
        g.mask = mask;
        g.mask_stride = mask_stride;
        g.counts = counts;
        g.index = index;
        g.batch = batch;
        g.tokens = s[0].tokens;
        g.heads = s[0].heads;
        g.rows = rows;
        g.d = d;
        g.dp = static_cast<int32_t>(padded(d));
        const cudaError_t e = launch_gather(g, stream);
        for (int i = 0; i < n; ++i) {
            if (!copied[i]) continue;
            const int64_t head = padded(d), token = s[i].heads * head;
            s[i] = {copy[i], rows, s[i].heads, {rows * token, token, head}};
        }
        return e;
    }
};

template <typename A>
convrot_status check_shape(const A &a)
{
    const int64_t sizes[] = {a.batch, a.q_tokens, a.kv_tokens, a.q_heads, a.kv_heads};
    for (int64_t v : sizes)
        if (v < 0 || v > kMaxSize) return CONVROT_ERR_INVALID_ARG;
    if (a.head_dim < 1 || a.reserved || a.mask_stride < 0 || !(a.scale > 0.0f && a.scale <= FLT_MAX / 2)) return CONVROT_ERR_INVALID_ARG;
    if (a.q_heads > 0 && (a.kv_heads < 1 || a.q_heads % a.kv_heads)) return CONVROT_ERR_INVALID_ARG;
    if (a.head_dim > CONVROT_ATTENTION_MAX_D) return CONVROT_ERR_UNSUPPORTED;
    // tiles are numbered in 32 bits
    const int64_t heads = a.q_heads > a.kv_heads ? a.q_heads : a.kv_heads, tokens = a.q_tokens > a.kv_tokens ? a.q_tokens : a.kv_tokens;
    const int64_t tiles = (tokens + 63) / 64;
    if (a.batch && heads && tiles && (a.batch > kMaxSize / heads || a.batch * heads > kMaxSize / tiles)) return CONVROT_ERR_INVALID_ARG;
    return check_16bit(a.dtype);
}

convrot_status check_heads(const void *p, const int64_t (&strides)[3], bool empty)
{
    for (int64_t s : strides)
        if (s < 0) return CONVROT_ERR_INVALID_ARG;
    return empty ? CONVROT_OK : check_matrix(p, 1, 1, 1, 2);
}

// Whether heads lie apart from one another, as far as two neighbours show it: they are written in any order.
bool apart(int64_t batch, int64_t tokens, int64_t heads, const int64_t (&strides)[3], int64_t d)
{
    const int64_t n[3] = {batch, tokens, heads};
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (strides[i] < d) return false;
        for (int j = 0; j < i; ++j)
            if (n[j] > 1 && strides[i] - strides[j] < d && strides[j] - strides[i] < d) return false;
    }
    return true;
}

struct ForwardWork {
    Operands q, kv;
    bool few;
    float *partial = nullptr;
    int64_t bytes;
    explicit ForwardWork(const convrot_attention_args &a, char *base = nullptr)
        : q(a.batch, a.head_dim, states(a.q, a.q_tokens, a.q_heads, a.q_strides)),
          kv(a.batch, a.head_dim, states(a.k, a.kv_tokens, a.kv_heads, a.k_strides), states(a.v, a.kv_tokens, a.kv_heads, a.v_strides))
    {
        Work w{base};
        few = a.kv_tokens > 0 && attention_few_takes(a.q_tokens, a.q_heads, a.kv_heads);
        if (few) {
            kv.plan(w, nullptr, 0, false);
            partial = w.take<float>(attention_few_partial_bytes(a.batch, a.kv_tokens, a.kv_heads, a.head_dim) / 4);
        } else {
            q.plan(w, nullptr, 0, false);
            kv.plan(w, mask_in_place(a.kv_tokens) ? nullptr : a.mask, a.mask_stride, false);
            partial = w.take<float>(attention_partial_bytes(a.batch, a.q_tokens, a.kv_tokens, a.q_heads, a.head_dim) / 4);
        }
        bytes = w.used;
    }
};

struct BackwardWork {
    Operands q, kv;  // queries and dout
    float *base2, *delta, *amax = nullptr, *partial, *partial_q;
    int64_t bytes;
    explicit BackwardWork(const convrot_attention_backward_args &a, char *base = nullptr)
        : q(a.batch, a.head_dim, states(a.q, a.q_tokens, a.q_heads, a.q_strides), states(a.dout, a.q_tokens, a.q_heads, a.dout_strides)),
          kv(a.batch, a.head_dim, states(a.k, a.kv_tokens, a.kv_heads, a.k_strides), states(a.v, a.kv_tokens, a.kv_heads, a.v_strides))
    {
        Work w{base};
        const int64_t rows = stat_rows(a.q_tokens);
        base2 = w.take<float>(a.batch * a.q_heads * rows);
        delta = w.take<float>(a.batch * a.q_heads * rows);
        if (a.dtype == CONVROT_F16) amax = w.take<float>(a.batch * a.q_heads * stat_blocks(a.q_tokens, a.q_heads / a.kv_heads));
        partial = w.take<float>(grad_kv_partial_bytes(a.batch, a.q_tokens, a.kv_tokens, a.q_heads, a.kv_heads, a.head_dim) / 4);
        partial_q = w.take<float>(grad_q_partial_bytes(a.batch, a.q_tokens, a.kv_tokens, a.q_heads, a.head_dim) / 4);
        q.plan(w, nullptr, 0, false);
        kv.plan(w, mask_in_place(a.kv_tokens) ? nullptr : a.mask, a.mask_stride, true);
        bytes = w.used;
    }
};

template <typename A>
bool nothing(const A &a)
{
    return a.batch == 0 || a.q_tokens == 0 || a.q_heads == 0;
}

}  // namespace

extern "C" {

int64_t convrot_attention_work_bytes(const convrot_attention_args *a)
{
    if (!a || check_shape(*a) != CONVROT_OK || nothing(*a)) return 0;
    return ForwardWork(*a).bytes;
}

convrot_status convrot_attention(const convrot_attention_args *a, cudaStream_t stream)
{
    if (!a) return CONVROT_ERR_INVALID_ARG;
    convrot_status st = check_shape(*a);
    if (st != CONVROT_OK) return st;
    const bool none = nothing(*a), no_keys = none || a->kv_tokens == 0;
    st = first_of({check_heads(a->q, a->q_strides, none), check_heads(a->k, a->k_strides, no_keys), check_heads(a->v, a->v_strides, no_keys),
                   check_heads(a->out, a->out_strides, none), check_matrix(a->lse, none ? 0 : 1, 1, 1, 4),
                   check_optional(a->dev_status, 1, 1, 1, 4)});
    if (st != CONVROT_OK || none) return st;
    if (!apart(a->batch, a->q_tokens, a->q_heads, a->out_strides, a->head_dim)) return CONVROT_ERR_INVALID_ARG;
    ForwardWork w(*a, static_cast<char *>(a->work));
    if ((st = check_work(a->work, a->work_bytes, w.bytes)) != CONVROT_OK) return st;
    if (w.q.make(stream) != cudaSuccess || w.kv.make(stream) != cudaSuccess) return CONVROT_ERR_CUDA;
    AttentionArgs b{};
    b.q = w.q.s[0];
    b.k = w.kv.s[0];
    b.v = w.kv.s[1];
    b.counts = w.kv.counts;
    if (mask_in_place(a->kv_tokens)) {
        b.mask = a->mask;
        b.mask_stride = a->mask_stride;
    }
    b.out = a->out;
    for (int i = 0; i < 3; ++i) b.out_strides[i] = a->out_strides[i];
    b.lse = a->lse;
    b.dev_status = a->dev_status;
    b.batch = a->batch;
    b.kv_tokens = a->kv_tokens;
    b.scale = a->scale;
    b.d = a->head_dim;
    b.dtype = a->dtype;
    b.splits = attention_splits(a->batch, a->q_tokens, a->kv_tokens, a->q_heads);
    b.partial = w.partial;
    return done(w.few ? launch_attention_few(b, a->mask, a->mask_stride, w.partial, stream) : launch_attention(b, stream));
}

int64_t convrot_attention_backward_work_bytes(const convrot_attention_backward_args *a)
{
    if (!a || check_shape(*a) != CONVROT_OK || nothing(*a) || a->kv_tokens == 0) return 0;
    return BackwardWork(*a).bytes;
}

convrot_status convrot_attention_backward(const convrot_attention_backward_args *a, cudaStream_t stream)
{
    if (!a) return CONVROT_ERR_INVALID_ARG;
    convrot_status st = check_shape(*a);
    if (st != CONVROT_OK) return st;
    const bool none = nothing(*a), no_keys = a->batch == 0 || a->kv_tokens == 0 || a->kv_heads == 0, either = none || no_keys;
    st = first_of({check_heads(a->q, a->q_strides, either), check_heads(a->k, a->k_strides, either), check_heads(a->v, a->v_strides, either),
                   check_heads(a->out, a->out_strides, either), check_heads(a->dout, a->dout_strides, either),
                   check_matrix(a->lse, either ? 0 : 1, 1, 1, 4), check_matrix(a->dq, none ? 0 : 1, 1, 1, 2),
                   check_matrix(a->dk, no_keys ? 0 : 1, 1, 1, 2), check_matrix(a->dv, no_keys ? 0 : 1, 1, 1, 2),
                   check_optional(a->dev_status, 1, 1, 1, 4)});
    if (st != CONVROT_OK) return st;
    const int64_t q_bytes = a->batch * a->q_tokens * a->q_heads * a->head_dim * 2, k_bytes = a->batch * a->kv_tokens * a->kv_heads * a->head_dim * 2;
    if (none) {  // sums over nothing
        if (k_bytes && (cudaMemsetAsync(a->dk, 0, k_bytes, stream) != cudaSuccess || cudaMemsetAsync(a->dv, 0, k_bytes, stream) != cudaSuccess))
            return CONVROT_ERR_CUDA;
        return CONVROT_OK;
    }
    if (no_keys) return done(cudaMemsetAsync(a->dq, 0, q_bytes, stream));
    BackwardWork w(*a, static_cast<char *>(a->work));
    if ((st = check_work(a->work, a->work_bytes, w.bytes)) != CONVROT_OK) return st;
    if (w.q.make(stream) != cudaSuccess || w.kv.make(stream, a->dk, a->dv) != cudaSuccess) return CONVROT_ERR_CUDA;
    AttentionGradArgs b{};
    b.q = w.q.s[0];
    b.dout = w.q.s[1];
    b.k = w.kv.s[0];
    b.v = w.kv.s[1];
    b.counts = w.kv.counts;
    if (mask_in_place(a->kv_tokens)) {
        b.mask = a->mask;
        b.mask_stride = a->mask_stride;
    }
    b.index = w.kv.index;
    b.index_rows = w.kv.rows;
    b.out = a->out;
    b.dout_own = a->dout;
    for (int i = 0; i < 3; ++i) {
        b.out_strides[i] = a->out_strides[i];
        b.dout_own_strides[i] = a->dout_strides[i];
    }
    b.lse = a->lse;
    b.base2 = w.base2;
    b.delta = w.delta;
    b.amax = w.amax;
    b.partial = w.partial;
    b.partial_q = w.partial_q;
    b.dq = a->dq;
    b.dk = a->dk;
    b.dv = a->dv;
    b.dev_status = a->dev_status;
    b.batch = a->batch;
    b.kv_tokens = a->kv_tokens;
    b.scale = a->scale;
    b.d = a->head_dim;
    b.dtype = a->dtype;
    if (launch_attention_stats(b, stream) != cudaSuccess || launch_attention_grad_kv(b, stream) != cudaSuccess) return CONVROT_ERR_CUDA;
    return grad_kv_makes_dq(b.kv_tokens, b.d) ? CONVROT_OK : done(launch_attention_grad_q(b, stream));
}

}  // extern "C"
