// Rotary positions (include/convrot_block.h): pairs of values of each query
// and key head turned by the angles of the token's position.
#include <cmath>

#include "block.h"

namespace convrot {
namespace {

template <typename T>
__global__ void rotary_kernel(const convrot_rotary_args a, const T *in, T *out, int64_t heads, int64_t sb,
                              int64_t st, int64_t sh, int64_t ob, int64_t ot, int64_t oh)
{
    const int64_t row = blockIdx.x;  // token of all batches
    const int64_t b = row / a.tokens, t = row % a.tokens;
    int64_t pos = t;
    if (a.positions) {
        const int64_t at = b * a.pos_stride + t;
        pos = a.position_bits == 64 ? static_cast<const int64_t *>(a.positions)[at]
                                    : static_cast<const int32_t *>(a.positions)[at];
    }
    const bool valid = pos >= 0 && pos < a.table_rows;
    if (!valid && threadIdx.x == 0 && a.dev_status) atomicExch(a.dev_status, static_cast<int32_t>(CONVROT_ERR_INVALID_ARG));
    const int half = a.rot_dim / 2, per_head = half + a.head_dim - a.rot_dim;
    for (int64_t i = threadIdx.x; i < heads * per_head; i += blockDim.x) {
        const int64_t h = i / per_head;
        const int e = static_cast<int>(i % per_head);
        const T *src = in + b * sb + t * st + h * sh;
        T *dst = out + b * ob + t * ot + h * oh;
        if (e >= half) {
            dst[a.rot_dim + e - half] = src[a.rot_dim + e - half];
            continue;
        }
        const int p0 = a.layout == CONVROT_ROTARY_HALF ? e : 2 * e, p1 = a.layout == CONVROT_ROTARY_HALF ? e + half : 2 * e + 1;
        const float x = to_f32(src[p0]), y = to_f32(src[p1]);
        float c = nanf(""), s = nanf("");
        if (valid) {
            c = a.cos[pos * a.ldt + e];
            s = a.sin[pos * a.ldt + e];
            if (a.inverse) s = -s;
        }
        dst[p0] = from_f32<T>(x * c - y * s);
        dst[p1] = from_f32<T>(y * c + x * s);
    }
}

// Angles in turns of 2 pi would need the frequency divided by 2 pi first; the
// product itself is exact enough in 64 bits: a position of 10^7 times a
// frequency of 1 is known to 10^-9.
__global__ void rotary_table_kernel(const double *positions, int64_t rows, int32_t axes, const double *freq,
                                    const int32_t *axis, int32_t pairs, double factor, float *cos_out, float *sin_out,
                                    int64_t ldt)
{
    const int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
    if (i >= rows * pairs) return;
    const int64_t p = i / pairs;
    const int e = static_cast<int>(i % pairs);
    const int ax = axis ? axis[e] : 0;
    double s = nan(""), c = nan("");
    if (ax >= 0 && ax < axes) {
        const double at = positions ? positions[p * axes + ax] : static_cast<double>(p);
        sincos(at * freq[e], &s, &c);
    }
    cos_out[p * ldt + e] = static_cast<float>(factor * c);
    sin_out[p * ldt + e] = static_cast<float>(factor * s);
}

}  // namespace

cudaError_t launch_rotary(const convrot_rotary_args &a, cudaStream_t stream)
{
    const unsigned rows = static_cast<unsigned>(a.batch * a.tokens);
    return with_dtype(a.dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        if (a.q_heads > 0)
            rotary_kernel<T><<<rows, 256, 0, stream>>>(a, static_cast<const T *>(a.q), static_cast<T *>(a.out_q),
                                                       a.q_heads, a.q_strides[0], a.q_strides[1], a.q_strides[2],
                                                       a.out_q_strides[0], a.out_q_strides[1], a.out_q_strides[2]);
        if (a.k_heads > 0)
            rotary_kernel<T><<<rows, 256, 0, stream>>>(a, static_cast<const T *>(a.k), static_cast<T *>(a.out_k),
                                                       a.k_heads, a.k_strides[0], a.k_strides[1], a.k_strides[2],
                                                       a.out_k_strides[0], a.out_k_strides[1], a.out_k_strides[2]);
        return cudaGetLastError();
    });
}

cudaError_t launch_rotary_table(const double *positions, int64_t rows, int32_t axes, const double *freq,
                                const int32_t *axis, int32_t pairs, double factor, float *cos, float *sin,
                                int64_t ldt, cudaStream_t stream)
{
    const int64_t blocks = (rows * pairs + 255) / 256;
    rotary_table_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(positions, rows, axes, freq, axis, pairs,
                                                                           factor, cos, sin, ldt);
    return cudaGetLastError();
}

}  // namespace convrot
