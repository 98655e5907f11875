// Launch interface between block_api.cu and the kernels of the operators
// around the linears (include/convrot_block.h). Arguments are validated.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/convrot_block.h"

namespace convrot {

cudaError_t launch_fp8_pack(const void *x, int dtype, int64_t m, int64_t k, int64_t ldx, void *q, int64_t ldq,
                            float *scale, int64_t lds, cudaStream_t stream);
cudaError_t launch_fp8_quantize_weights(const void *w, int dtype, int64_t n, int64_t k, int64_t ldw, void *q,
                                        int64_t ldq, float *scale, int64_t lds, cudaStream_t stream);
cudaError_t launch_fp8_gemm(const convrot_fp8_linear_args &a, cudaStream_t stream);

cudaError_t launch_gated_norm(const convrot_gated_norm_args &a, cudaStream_t stream);
cudaError_t launch_gated_norm_backward(const convrot_gated_norm_backward_args &a, cudaStream_t stream);
int64_t gated_norm_backward_work_bytes(int64_t m, int64_t d, int64_t rows_per_batch);

cudaError_t launch_rotary(const convrot_rotary_args &a, cudaStream_t stream);
cudaError_t launch_rotary_table(const double *positions, int64_t rows, int32_t axes, const double *freq,
                                const int32_t *axis, int32_t pairs, double factor, float *cos, float *sin,
                                int64_t ldt, cudaStream_t stream);

// Calls f with a null pointer of the element type that the dtype names.
template <typename F>
auto with_dtype(int dtype, F f)
{
    if (dtype == CONVROT_BF16) return f(static_cast<__nv_bfloat16 *>(nullptr));
    if (dtype == CONVROT_F16) return f(static_cast<__half *>(nullptr));
    return f(static_cast<float *>(nullptr));
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

// Rounded to nearest, ties to even.
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// N consecutive elements as one access of up to 16 bytes (N * sizeof(T) a power
// of two); the address is aligned to it. kStream: the line is not needed again
// (evict-first); the loads stay coherent, so an output may be its own input.
template <int kBytes>
struct Bits;
template <>
struct Bits<2> { using type = unsigned short; };
template <>
struct Bits<4> { using type = unsigned int; };
template <>
struct Bits<8> { using type = uint2; };
template <>
struct Bits<16> { using type = uint4; };

template <typename T, int N>
struct Raw {
    static constexpr int kBytes = N * static_cast<int>(sizeof(T));
    static constexpr int kParts = kBytes > 16 ? kBytes / 16 : 1;
    using B = typename Bits<(kBytes > 16 ? 16 : kBytes)>::type;
    B bits[kParts];
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < kParts; ++i) bits[i] = reinterpret_cast<const B *>(p)[i];
    }
    __device__ __forceinline__ void load_stream(const T *p)
    {
#pragma unroll
        for (int i = 0; i < kParts; ++i) bits[i] = __ldcs(reinterpret_cast<const B *>(p) + i);
    }
    __device__ __forceinline__ void store(T *p) const
    {
#pragma unroll
        for (int i = 0; i < kParts; ++i) reinterpret_cast<B *>(p)[i] = bits[i];
    }
    __device__ __forceinline__ void store_stream(T *p) const
    {
#pragma unroll
        for (int i = 0; i < kParts; ++i) __stcs(reinterpret_cast<B *>(p) + i, bits[i]);
    }
    __device__ __forceinline__ float get(int i) const { return to_f32(reinterpret_cast<const T *>(bits)[i]); }
    __device__ __forceinline__ void set(int i, float v) { reinterpret_cast<T *>(bits)[i] = from_f32<T>(v); }
};

inline bool aligned_to(const void *p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

constexpr float kFp8Max = 448.0f;
constexpr float kFp8AmaxFloor = 1.2621774483536189e-29f;  // 2^-96: no block's scale is 0 or its inverse infinite

// What a block's values are multiplied by before they are rounded to codes.
__device__ __forceinline__ float fp8_up(float amax) { return kFp8Max * __frcp_rn(amax); }

// The four e4m3 codes of four values, nearest with ties to even; values past
// +-448 (a rounding of amax * fp8_up(amax) upwards) become +-448, NaN stays.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

__device__ __forceinline__ uint8_t e4m3(float a)
{
    return static_cast<uint8_t>(e4m3x4(a, 0.0f, 0.0f, 0.0f) & 0xffu);
}

}  // namespace convrot
