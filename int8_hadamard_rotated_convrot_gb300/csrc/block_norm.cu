// The gated norm and its gradient (include/convrot_block.h).
#include "block.h"

namespace convrot {
namespace {

constexpr int kThreads = 256;

// Sum over the block of threads, the same value in each of them.
__device__ float block_sum(float v)
{
    __shared__ float part[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
    for (int i = 0; i < kThreads / 32; ++i) v += part[i];
    return v;
}

// Mean and 1 / sqrt(mean square + eps) of the row in shared memory, as the
// kind of norm has them; each thread reads its own elements.
__device__ void row_stats(const float *v, int d, int kind, float eps, float &mean, float &inv)
{
    mean = 0.0f;
    inv = 1.0f;
    if (kind == CONVROT_NORM_NONE) return;
    float s = 0.0f;
    if (kind == CONVROT_NORM_LAYER) {
        for (int i = threadIdx.x; i < d; i += kThreads) s += v[i];
        mean = block_sum(s) / d;
    }
    s = 0.0f;
    for (int i = threadIdx.x; i < d; i += kThreads) s += (v[i] - mean) * (v[i] - mean);
    inv = 1.0f / sqrtf(block_sum(s) / d + eps);
}

template <typename P>
__device__ __forceinline__ float param(const void *p, int64_t i, float otherwise)
{
    return p ? to_f32(static_cast<const P *>(p)[i]) : otherwise;
}

template <typename T, typename P>
__global__ void __launch_bounds__(kThreads) gated_norm_kernel(const convrot_gated_norm_args a)
{
    extern __shared__ float row_h[];
    const int64_t r = blockIdx.x, b = r / a.rows_per_batch;
    const int d = static_cast<int>(a.d);
    const T *x = static_cast<const T *>(a.x) + r * a.ldx;
    float mean, inv;
    if (a.y) {
        const T *y = static_cast<const T *>(a.y) + r * a.ldy;
        for (int i = threadIdx.x; i < d; i += kThreads) row_h[i] = to_f32(y[i]);
        row_stats(row_h, d, a.post, a.eps, mean, inv);
    }
    for (int i = threadIdx.x; i < d; i += kThreads) {
        float h = a.res_scale * to_f32(x[i]);
        if (a.y) {
            const float u = (row_h[i] - mean) * inv * param<P>(a.post_weight, i, 1.0f) + param<P>(a.post_bias, i, 0.0f);
            h += param<P>(a.gate, b * a.ldgate + i, 1.0f) * u;
        }
        row_h[i] = h;
        if (a.h) static_cast<T *>(a.h)[r * a.ldh + i] = from_f32<T>(h);
    }
    if (!a.n && !a.q) return;
    row_stats(row_h, d, a.pre, a.eps, mean, inv);
    for (int i = threadIdx.x; i < d; i += kThreads) {
        const float v = (row_h[i] - mean) * inv * param<P>(a.pre_weight, i, 1.0f) + param<P>(a.pre_bias, i, 0.0f);
        const float n = v * (1.0f + param<P>(a.scale, b * a.ldscale + i, 0.0f)) + param<P>(a.shift, b * a.ldshift + i, 0.0f);
        if (a.n) static_cast<T *>(a.n)[r * a.ldn + i] = from_f32<T>(n);
        row_h[i] = n;
    }
    if (!a.q) return;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int j = warp; j * 128 < d; j += kThreads / 32) {
        float amax = 0.0f;
        for (int i = j * 128 + lane; i < d && i < j * 128 + 128; i += 32) amax = fmaxf(amax, fabsf(row_h[i]));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        amax = fmaxf(amax, kFp8AmaxFloor);
        if (lane == 0) a.q_scale[j * a.ld_q_scale + r] = amax / kFp8Max;
        const float up = fp8_up(amax);
        for (int i = j * 128 + lane; i < d && i < j * 128 + 128; i += 32)
            static_cast<uint8_t *>(a.q)[r * a.ldq + i] = e4m3(row_h[i] * up);
    }
}

// Gradient, by rows: dx, dy and the row's statistics (mean and 1 / deviation
// of h and y, and the two means that pre's gradient subtracts).
struct RowStats {
    float pre_mean, pre_inv, pre_g, pre_gh, post_mean, post_inv;
};

template <typename T, typename P>
struct Grad {
    const convrot_gated_norm_backward_args &a;
    int64_t r, b;
    __device__ float in(const void *p, int64_t ld, int i) const
    {
        return p ? to_f32(static_cast<const T *>(p)[r * ld + i]) : 0.0f;
    }
    __device__ float dn(int i) const { return in(a.dn, a.lddn, i); }
    // gradient at pre's normalized value
    __device__ float g_pre(int i) const
    {
        return dn(i) * (1.0f + param<P>(a.scale, b * a.ldscale + i, 0.0f)) * param<P>(a.pre_weight, i, 1.0f);
    }
    __device__ float h_hat(int i, const RowStats &s) const { return (in(a.h, a.ldh, i) - s.pre_mean) * s.pre_inv; }
    __device__ float y_hat(int i, const RowStats &s) const { return (in(a.y, a.ldy, i) - s.post_mean) * s.post_inv; }
    // gradient at h, without res_scale
    __device__ float dh(int i, const RowStats &s) const
    {
        return s.pre_inv * (g_pre(i) - s.pre_g - h_hat(i, s) * s.pre_gh) + in(a.dh, a.lddh, i);
    }
    __device__ float gate(int i) const { return param<P>(a.gate, b * a.ldgate + i, 1.0f); }
};

template <typename T, typename P>
__global__ void __launch_bounds__(kThreads) norm_grad_rows_kernel(const convrot_gated_norm_backward_args a, RowStats *stats)
{
    extern __shared__ float row[];
    const int64_t r = blockIdx.x;
    const int d = static_cast<int>(a.d);
    const Grad<T, P> at{a, r, r / a.rows_per_batch};
    RowStats s{};
    for (int i = threadIdx.x; i < d; i += kThreads) row[i] = at.in(a.h, a.ldh, i);
    row_stats(row, d, a.pre, a.eps, s.pre_mean, s.pre_inv);
    if (a.pre != CONVROT_NORM_NONE) {
        float g = 0.0f, gh = 0.0f;
        for (int i = threadIdx.x; i < d; i += kThreads) {
            g += at.g_pre(i);
            gh += at.g_pre(i) * at.h_hat(i, s);
        }
        s.pre_gh = block_sum(gh) / d;
        s.pre_g = a.pre == CONVROT_NORM_LAYER ? block_sum(g) / d : 0.0f;
    }
    if (a.dx)
        for (int i = threadIdx.x; i < d; i += kThreads)
            static_cast<T *>(a.dx)[r * a.lddx + i] = from_f32<T>(a.res_scale * at.dh(i, s));
    s.post_inv = 1.0f;
    if (a.y) {
        for (int i = threadIdx.x; i < d; i += kThreads) row[i] = at.in(a.y, a.ldy, i);
        row_stats(row, d, a.post, a.eps, s.post_mean, s.post_inv);
        if (a.dy) {
            float g = 0.0f, gh = 0.0f;
            for (int i = threadIdx.x; i < d; i += kThreads) {
                row[i] = at.dh(i, s) * at.gate(i) * param<P>(a.post_weight, i, 1.0f);
                g += row[i];
                gh += row[i] * at.y_hat(i, s);
            }
            g = block_sum(g) / d;
            gh = block_sum(gh) / d;
            if (a.post != CONVROT_NORM_LAYER) g = 0.0f;
            if (a.post == CONVROT_NORM_NONE) gh = 0.0f;
            for (int i = threadIdx.x; i < d; i += kThreads)
                static_cast<T *>(a.dy)[r * a.lddy + i] = from_f32<T>(s.post_inv * (row[i] - g - at.y_hat(i, s) * gh));
        }
    }
    if (threadIdx.x == 0) stats[r] = s;
}

// Gradient, by columns: one thread sums one column over the rows of each
// sample in turn.
template <typename T, typename P>
__global__ void __launch_bounds__(kThreads) norm_grad_cols_kernel(const convrot_gated_norm_backward_args a, const RowStats *stats)
{
    const int64_t i64 = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
    if (i64 >= a.d) return;
    const int i = static_cast<int>(i64);
    const float w_pre = param<P>(a.pre_weight, i, 1.0f), b_pre = param<P>(a.pre_bias, i, 0.0f);
    const float w_post = param<P>(a.post_weight, i, 1.0f), b_post = param<P>(a.post_bias, i, 0.0f);
    float dwp = 0.0f, dbp = 0.0f, dwq = 0.0f, dbq = 0.0f;
    for (int64_t b = 0; b * a.rows_per_batch < a.m; ++b) {
        float s0 = 0.0f, s1 = 0.0f, t0 = 0.0f, t1 = 0.0f;
        for (int64_t r = b * a.rows_per_batch; r < a.m && r < (b + 1) * a.rows_per_batch; ++r) {
            const Grad<T, P> at{a, r, b};
            const RowStats s = stats[r];
            s0 += at.dn(i);
            s1 += at.dn(i) * at.h_hat(i, s);
            if (a.y) {
                const float dh = at.dh(i, s);
                t0 += dh;
                t1 += dh * at.y_hat(i, s);
            }
        }
        const float up = 1.0f + param<P>(a.scale, b * a.ldscale + i, 0.0f);
        const float gate = param<P>(a.gate, b * a.ldgate + i, 1.0f);
        if (a.dshift) a.dshift[b * a.d + i] = s0;
        if (a.dscale) a.dscale[b * a.d + i] = w_pre * s1 + b_pre * s0;
        if (a.dgate) a.dgate[b * a.d + i] = w_post * t1 + b_post * t0;
        dwp += up * s1;
        dbp += up * s0;
        dwq += gate * t1;
        dbq += gate * t0;
    }
    if (a.dpre_weight) a.dpre_weight[i] = dwp;
    if (a.dpre_bias) a.dpre_bias[i] = dbp;
    if (a.dpost_weight) a.dpost_weight[i] = dwq;
    if (a.dpost_bias) a.dpost_bias[i] = dbq;
}

// Calls f with null pointers of the tensors' and the parameters' types.
template <typename F>
cudaError_t with_types(int dtype, int param_dtype, F f)
{
    return with_dtype(dtype, [&](auto *t) {
        if (param_dtype == CONVROT_F32) return f(t, static_cast<float *>(nullptr));
        return f(t, t);
    });
}

template <typename K>
cudaError_t allow_smem(K kernel, int bytes)
{
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

}  // namespace

cudaError_t launch_gated_norm(const convrot_gated_norm_args &a, cudaStream_t stream)
{
    return with_types(a.dtype, a.param_dtype, [&](auto *t, auto *p) {
        auto kernel = gated_norm_kernel<std::remove_pointer_t<decltype(t)>, std::remove_pointer_t<decltype(p)>>;
        const int bytes = static_cast<int>(a.d) * 4;
        cudaError_t e = allow_smem(kernel, bytes);
        if (e != cudaSuccess) return e;
        kernel<<<static_cast<unsigned>(a.m), kThreads, bytes, stream>>>(a);
        return cudaGetLastError();
    });
}

int64_t gated_norm_backward_work_bytes(int64_t m, int64_t d, int64_t rows_per_batch)
{
    return m * static_cast<int64_t>(sizeof(RowStats));
}

cudaError_t launch_gated_norm_backward(const convrot_gated_norm_backward_args &a, cudaStream_t stream)
{
    return with_types(a.dtype, a.param_dtype, [&](auto *t, auto *p) {
        using T = std::remove_pointer_t<decltype(t)>;
        using P = std::remove_pointer_t<decltype(p)>;
        const int bytes = static_cast<int>(a.d) * 4;
        RowStats *stats = static_cast<RowStats *>(a.work);
        cudaError_t e = allow_smem(norm_grad_rows_kernel<T, P>, bytes);
        if (e != cudaSuccess) return e;
        norm_grad_rows_kernel<T, P><<<static_cast<unsigned>(a.m), kThreads, bytes, stream>>>(a, stats);
        norm_grad_cols_kernel<T, P><<<static_cast<unsigned>((a.d + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a, stats);
        return cudaGetLastError();
    });
}

}  // namespace convrot
