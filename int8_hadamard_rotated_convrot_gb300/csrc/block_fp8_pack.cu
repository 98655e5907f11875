// The quantizers of the block-scaled linear (include/convrot_block.h).
#include "block.h"

namespace convrot {
namespace {

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Reads 2 or 4 bytes and writes 1 for a handful of operations: bound by HBM.
// A block of 128 values belongs to 128 / kVec threads with 16 bytes each
// (kWide), or to a warp whose lanes take every 32nd value; a thread has the
// same place in kPackRows rows, all of whose loads are in flight together.
constexpr int kPackRows = 4;

template <typename T, bool kWide>
__global__ void __launch_bounds__(256) fp8_pack_kernel(const T *x, int32_t m, int32_t k, int64_t ldx, uint8_t *q, int64_t ldq,
                                                       float *scale, int64_t lds, int32_t blocks, int32_t scale4)
{
    constexpr int kVec = kWide ? 16 / sizeof(T) : 4, kLanes = kWide ? 128 / kVec : 32;
    const int64_t item = blockIdx.x * 256ll + threadIdx.x;
    const uint32_t group = static_cast<uint32_t>(item / kLanes);  // a block of kPackRows rows
    const int lane = threadIdx.x % kLanes;
    const uint32_t rows4 = group / static_cast<uint32_t>(blocks);
    const int j = static_cast<int>(group - rows4 * blocks);
    const int64_t r0 = static_cast<int64_t>(rows4) * kPackRows;
    after_previous();
    let_next_start();
    if (r0 >= m) return;  // whole groups of lanes
    const int i0 = j * 128 + (kWide ? lane * kVec : lane);
    float v[kPackRows][kVec];
#pragma unroll
    for (int n = 0; n < kPackRows; ++n) {
        const T *p = x + (r0 + n) * ldx;
        if constexpr (kWide) {
            Raw<T, kVec> raw{};
            if (r0 + n < m && i0 < k) raw.load_stream(p + i0);
            raw.unpack(v[n]);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[n][e] = r0 + n < m && i0 + 32 * e < k ? to_f32(p[i0 + 32 * e]) : 0.0f;
        }
    }
    const uint32_t lanes = kLanes == 32 ? 0xffffffffu : 0xffffu << (threadIdx.x & 16);
    float s[kPackRows];
#pragma unroll
    for (int n = 0; n < kPackRows; ++n) {
        float amax = 0.0f;
#pragma unroll
        for (int e = 0; e < kVec; ++e) amax = fmaxf(amax, fabsf(v[n][e]));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(lanes, amax, o));
        amax = fmaxf(amax, kFp8AmaxFloor);
        s[n] = amax / kFp8Max;
        const float up = fp8_up(amax);
        if (r0 + n >= m) continue;
        uint8_t *to = q + (r0 + n) * ldq + i0;
        if constexpr (kWide) {
            if (i0 >= k) continue;
            uint32_t w[kVec / 4];
#pragma unroll
            for (int e = 0; e < kVec; e += 4) w[e / 4] = e4m3x4(v[n][e] * up, v[n][e + 1] * up, v[n][e + 2] * up, v[n][e + 3] * up);
            if constexpr (kVec == 8)
                *reinterpret_cast<uint2 *>(to) = make_uint2(w[0], w[1]);
            else
                *reinterpret_cast<uint32_t *>(to) = w[0];
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (i0 + 32 * e < k) to[32 * e] = e4m3(v[n][e] * up);
        }
    }
    if (lane == 0) {
        float *to = scale + j * lds + r0;
        if (scale4 && r0 + kPackRows <= m)
            *reinterpret_cast<float4 *>(to) = make_float4(s[0], s[1], s[2], s[3]);
        else
#pragma unroll
            for (int n = 0; n < kPackRows; ++n)
                if (r0 + n < m) to[n] = s[n];
    }
}

template <typename T>
__global__ void __launch_bounds__(256) fp8_quantize_weights_kernel(const T *w, int64_t n, int64_t k, int64_t ldw, uint8_t *q,
                                                                   int64_t ldq, float *scale, int64_t lds)
{
    __shared__ float part[8];
    const int64_t p = blockIdx.x, j = blockIdx.y;  // (the grid's second dimension has 16 bits: k's blocks fit)
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

}  // namespace

cudaError_t launch_fp8_pack(const void *x, int dtype, int64_t m, int64_t k, int64_t ldx, void *q, int64_t ldq,
                            float *scale, int64_t lds, cudaStream_t stream)
{
    const int64_t blocks = (k + 127) / 128, groups = blocks * ((m + kPackRows - 1) / kPackRows);
    return with_dtype(dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        constexpr int kVec = 16 / sizeof(T);
        const bool wide = k % kVec == 0 && aligned_to(x, 16) && (m <= 1 || ldx % kVec == 0);
        const int64_t items = groups * (wide ? 128 / kVec : 32);
        const int scale4 = aligned_to(scale, 16) && lds % 4 == 0;
        return launch_after(wide ? fp8_pack_kernel<T, true> : fp8_pack_kernel<T, false>, dim3(static_cast<unsigned>((items + 255) / 256)),
                            256, 0, stream, 1, static_cast<const T *>(x), static_cast<int32_t>(m), static_cast<int32_t>(k), ldx,
                            static_cast<uint8_t *>(q), ldq, scale, lds, static_cast<int32_t>(blocks), scale4);
    });
}

cudaError_t launch_fp8_quantize_weights(const void *w, int dtype, int64_t n, int64_t k, int64_t ldw, void *q,
                                        int64_t ldq, float *scale, int64_t lds, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>((n + 127) / 128), static_cast<unsigned>((k + 127) / 128));
    return with_dtype(dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        fp8_quantize_weights_kernel<T><<<grid, 256, 0, stream>>>(static_cast<const T *>(w), n, k, ldw,
                                                                 static_cast<uint8_t *>(q), ldq, scale, lds);
        return cudaGetLastError();
    });
}

}  // namespace convrot
