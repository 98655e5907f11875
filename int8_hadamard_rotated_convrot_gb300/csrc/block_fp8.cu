// The block-scaled e4m3 linear and its quantizers (include/convrot_block.h).
#include <cuda_fp8.h>

#include "block.h"
#include "internal.h"

namespace convrot {
namespace {

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// One warp quantizes one block of one row: four values a lane.
template <typename T>
__global__ void __launch_bounds__(256) fp8_pack_kernel(const T *x, int64_t m, int64_t k, int64_t ldx, uint8_t *q,
                                                       int64_t ldq, float *scale, int64_t lds)
{
    const int64_t kb = (k + 127) / 128;
    const int64_t w = blockIdx.x * 8ll + (threadIdx.x >> 5);
    if (w >= m * kb) return;
    const int lane = threadIdx.x & 31;
    const int64_t r = w / kb, j = w % kb;
    float v[4], amax = 0.0f;
    for (int e = 0; e < 4; ++e) {
        const int64_t i = j * 128 + e * 32 + lane;
        v[e] = i < k ? to_f32(x[r * ldx + i]) : 0.0f;
        amax = fmaxf(amax, fabsf(v[e]));
    }
    amax = fmaxf(warp_max(amax), kFp8AmaxFloor);
    if (lane == 0) scale[j * lds + r] = amax / kFp8Max;
    for (int e = 0; e < 4; ++e) {
        const int64_t i = j * 128 + e * 32 + lane;
        if (i < k) q[r * ldq + i] = e4m3(v[e] * fp8_up(amax));
    }
}

template <typename T>
__global__ void __launch_bounds__(256) fp8_quantize_weights_kernel(const T *w, int64_t n, int64_t k, int64_t ldw, uint8_t *q,
                                                                   int64_t ldq, float *scale, int64_t lds)
{
    __shared__ float part[8];
    const int64_t j = blockIdx.x, p = blockIdx.y;
    float amax = 0.0f;
    for (int i = threadIdx.x; i < 128 * 128; i += 256) {
        const int64_t r = p * 128 + i / 128, c = j * 128 + i % 128;
        if (r < n && c < k) amax = fmaxf(amax, fabsf(to_f32(w[r * ldw + c])));
    }
    amax = warp_max(amax);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
    __syncthreads();
    amax = kFp8AmaxFloor;
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, part[i]);
    if (threadIdx.x == 0) scale[p * lds + j] = amax / kFp8Max;
    for (int i = threadIdx.x; i < 128 * 128; i += 256) {
        const int64_t r = p * 128 + i / 128, c = j * 128 + i % 128;
        if (r < n && c < k) q[r * ldq + c] = e4m3(to_f32(w[r * ldw + c]) * fp8_up(amax));
    }
}

__device__ __forceinline__ float e4m3_value(uint8_t c)
{
    __nv_fp8_e4m3 v;
    v.__x = c;
    return static_cast<float>(v);
}

// 16 x 16 outputs a block of threads, 128 features at a time.
template <typename T>
__global__ void __launch_bounds__(256) fp8_gemm_kernel(const convrot_fp8_linear_args a)
{
    __shared__ float xs[16][129], ws[16][129];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t r0 = blockIdx.y * 16ll, o0 = blockIdx.x * 16ll;
    const uint8_t *x = static_cast<const uint8_t *>(a.x), *w = static_cast<const uint8_t *>(a.w);
    float acc = 0.0f;
    for (int64_t j = 0; j * 128 < a.k; ++j) {
        for (int i = threadIdx.x; i < 16 * 128; i += 256) {
            const int rr = i / 128, c = i % 128;
            const int64_t kk = j * 128 + c;
            xs[rr][c] = r0 + rr < a.m && kk < a.k ? e4m3_value(x[(r0 + rr) * a.ldx + kk]) : 0.0f;
            ws[rr][c] = o0 + rr < a.n && kk < a.k ? e4m3_value(w[(o0 + rr) * a.ldw + kk]) : 0.0f;
        }
        __syncthreads();
        float s = 0.0f;
        for (int c = 0; c < 128; ++c) s += xs[ty][c] * ws[tx][c];
        if (r0 + ty < a.m && o0 + tx < a.n)
            acc += s * (a.x_scale[j * a.ld_x_scale + r0 + ty] * a.w_scale[(o0 + tx) / 128 * a.ld_w_scale + j]);
        __syncthreads();
    }
    const int64_t r = r0 + ty, o = o0 + tx;
    if (r < a.m && o < a.n)
        static_cast<T *>(a.y)[r * a.ldy + o] = from_f32<T>(apply_act(acc + (a.bias ? a.bias[o] : 0.0f), a.act));
}

}  // namespace

cudaError_t launch_fp8_pack(const void *x, int dtype, int64_t m, int64_t k, int64_t ldx, void *q, int64_t ldq,
                            float *scale, int64_t lds, cudaStream_t stream)
{
    const int64_t blocks = (m * ((k + 127) / 128) + 7) / 8;
    return with_dtype(dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        fp8_pack_kernel<T><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(static_cast<const T *>(x), m, k, ldx,
                                                                              static_cast<uint8_t *>(q), ldq, scale, lds);
        return cudaGetLastError();
    });
}

cudaError_t launch_fp8_quantize_weights(const void *w, int dtype, int64_t n, int64_t k, int64_t ldw, void *q,
                                        int64_t ldq, float *scale, int64_t lds, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>((k + 127) / 128), static_cast<unsigned>((n + 127) / 128));
    return with_dtype(dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        fp8_quantize_weights_kernel<T><<<grid, 256, 0, stream>>>(static_cast<const T *>(w), n, k, ldw,
                                                                 static_cast<uint8_t *>(q), ldq, scale, lds);
        return cudaGetLastError();
    });
}

cudaError_t launch_fp8_gemm(const convrot_fp8_linear_args &a, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>((a.n + 15) / 16), static_cast<unsigned>((a.m + 15) / 16));
    return with_dtype(a.y_dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        fp8_gemm_kernel<T><<<grid, 256, 0, stream>>>(a);
        return cudaGetLastError();
    });
}

}  // namespace convrot
