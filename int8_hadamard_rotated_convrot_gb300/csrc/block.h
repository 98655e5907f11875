// Launch interface between block_api.cu and the kernels of the operators
// around the linears (include/convrot_block.h). Arguments are validated.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "../../include/convrot_block.h"

namespace convrot {

cudaError_t launch_fp8_pack(const void *x, int dtype, int64_t m, int64_t k, int64_t ldx, void *q, int64_t ldq,
                            float *scale, int64_t lds, cudaStream_t stream);
cudaError_t launch_fp8_quantize_weights(const void *w, int dtype, int64_t n, int64_t k, int64_t ldw, void *q,
                                        int64_t ldq, float *scale, int64_t lds, cudaStream_t stream);
cudaError_t launch_fp8_gemm(const convrot_fp8_linear_args &a, cudaStream_t stream);
// Few rows: whether that kernel takes the sizes, and whether it quantizes x itself.
bool fp8_few_takes(int64_t m, int64_t n, int64_t k);
bool fp8_few_quantizes(int64_t m, int64_t n, int64_t k);
// Shared memory and tensor-memory columns of its CTAs (sizes that it takes).
int fp8_few_shared(int64_t m, int64_t n, int64_t k, bool quantize, int *columns);
cudaError_t launch_fp8_few(const convrot_fp8_linear_args &a, cudaStream_t stream);           // packed x
cudaError_t launch_fp8_few_quantize(const convrot_fp8_linear_args &a, cudaStream_t stream);  // x as rows

cudaError_t launch_gated_norm(const convrot_gated_norm_args &a, cudaStream_t stream);
cudaError_t launch_gated_norm_backward(const convrot_gated_norm_backward_args &a, cudaStream_t stream);
int64_t gated_norm_backward_work_bytes(int64_t m, int64_t d, int64_t rows_per_batch);

cudaError_t launch_rotary(const convrot_rotary_args &a, cudaStream_t stream);
cudaError_t launch_rotary_table(const double *positions, int64_t rows, int32_t axes, const double *freq,
                                const int32_t *axis, int32_t pairs, double factor, float *cos, float *sin,
                                int64_t ldt, cudaStream_t stream);

constexpr int kSms = 152;
constexpr int kMaxShared = 227 * 1024;  // shared memory of a block

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

// Two fp32 values that one instruction works on (fma.rn.f32x2 and its kin:
// each half rounded as the single operation would be).
struct F2 {
    unsigned long long v;
    __device__ __forceinline__ F2() {}
    __device__ __forceinline__ F2(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ explicit F2(float a) : F2(a, a) {}
    __device__ __forceinline__ float lo() const
    {
        float a, b;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
        return a;
    }
    __device__ __forceinline__ float hi() const
    {
        float a, b;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
        return b;
    }
    __device__ __forceinline__ float sum() const { return lo() + hi(); }
};
__device__ __forceinline__ F2 operator+(F2 a, F2 b)
{
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(a.v) : "l"(a.v), "l"(b.v));
    return a;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b)
{
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(a.v) : "l"(a.v), "l"(b.v));
    return a;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(c.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return c;
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// 2^x and 1 / x, approximate (2 and 1 units in the last place).
__device__ __forceinline__ float ex2(float x)
{
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x));
    return x;
}
__device__ __forceinline__ float rcp(float x)
{
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x));
    return x;
}

// GELU of two values (convrot_activation), the forms of internal.h's apply_act
// with their multiplications and additions in pairs, so that the two special
// functions a value are what it costs:
//   tanh form  v / (1 + e^(-2u)), -2u log2(e) = v (c0 + c1 v^2)
//   erf form   v (1/2 + sign(v) (1/2 - q/2)), q = 1 - erf(|v| / sqrt(2)) by Abramowitz & Stegun 7.1.26
template <int kAct>
__device__ __forceinline__ F2 act2(F2 v)
{
    if constexpr (kAct == CONVROT_ACT_GELU_TANH) {
        const F2 z = v * fma2(v * v, F2(-0.10294324f), F2(-2.3022082f));
        const F2 e = F2(ex2(z.lo()), ex2(z.hi())) + F2(1.0f);
        return v * F2(rcp(e.lo()), rcp(e.hi()));
    } else if constexpr (kAct == CONVROT_ACT_GELU_ERF) {
        const F2 x = F2(fabsf(v.lo()), fabsf(v.hi())) * F2(0.70710678f);
        const F2 u = fma2(x, F2(0.3275911f), F2(1.0f));
        const F2 t(rcp(u.lo()), rcp(u.hi()));
        // half of the polynomial: q / 2
        F2 h = fma2(t, F2(0.5f * 1.061405429f), F2(0.5f * -1.453152027f));
        h = fma2(t, h, F2(0.5f * 1.421413741f));
        h = fma2(t, h, F2(0.5f * -0.284496736f));
        h = fma2(t, h, F2(0.5f * 0.254829592f)) * t;
        const F2 z = x * x * F2(-1.4426950f);
        h = fma2(h, F2(-ex2(z.lo()), -ex2(z.hi())), F2(0.5f));
        return v * (F2(copysignf(h.lo(), v.lo()), copysignf(h.hi(), v.hi())) + F2(0.5f));
    } else {
        return v;
    }
}

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
    // N == 1: the value
    __device__ __forceinline__ float value() const
    {
        static_assert(N == 1);
        float v[1];
        unpack(v);
        return v[0];
    }
    __device__ __forceinline__ void set(float f)
    {
        static_assert(N == 1);
        const float v[1] = {f};
        pack(v);
    }
    // All N values; 16-bit types two at a time (one operation a value to widen
    // bf16, one for two values to round).
    __device__ __forceinline__ void unpack(float (&v)[N]) const
    {
        if constexpr (N == 1) {
            v[0] = to_f32(*reinterpret_cast<const T *>(bits));
        } else {
            const uint32_t *w = reinterpret_cast<const uint32_t *>(bits);
#pragma unroll
            for (int i = 0; i < kBytes / 4; ++i) {
                if constexpr (sizeof(T) == 4) {
                    v[i] = __uint_as_float(w[i]);
                } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
                    v[2 * i] = __uint_as_float(w[i] << 16);
                    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                } else {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                    v[2 * i] = f.x;
                    v[2 * i + 1] = f.y;
                }
            }
        }
    }
    __device__ __forceinline__ void unpack(F2 *v) const
    {
        float f[N];
        unpack(f);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) v[i] = F2(f[2 * i], f[2 * i + 1]);
    }
    __device__ __forceinline__ void pack(const F2 *v)
    {
        float f[N];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            f[2 * i] = v[i].lo();
            f[2 * i + 1] = v[i].hi();
        }
        pack(f);
    }
    __device__ __forceinline__ void pack(const float (&v)[N])
    {
        if constexpr (N == 1) {
            *reinterpret_cast<T *>(bits) = from_f32<T>(v[0]);
        } else {
            uint32_t *w = reinterpret_cast<uint32_t *>(bits);
#pragma unroll
            for (int i = 0; i < kBytes / 4; ++i) {
                if constexpr (sizeof(T) == 4) {
                    w[i] = __float_as_uint(v[i]);
                } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t *>(&b);
                } else {
                    const __half2 b = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t *>(&b);
                }
            }
        }
    }
};

// kBytes (4 or 16) from global to shared memory without a register between;
// with bytes = 0 nothing is read and they become zero.
template <int kBytes>
__device__ __forceinline__ void copy_piece(uint32_t to, const void *from, uint32_t bytes)
{
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All of this thread's groups but the last kPending have landed.
template <int kPending>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ uint4 shared16(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

// Allows a kernel the shared memory of a whole SM, once for each kernel (Tag)
// and device: the attribute stays, and setting it costs about as much as a launch.
template <typename Tag, typename K>
cudaError_t allow_shared(K *kernel)
{
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, kernel);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared - static_cast<int>(attr.sharedSizeBytes));
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

template <typename T>
struct Same {
    using type = T;
};

// A launch that may start while the kernel before it drains (and a cluster
// size). Its threads all call after_previous() before they touch global memory:
// that waits until the kernel before is complete and its writes are seen. A
// kernel that calls let_next_start() lets the next such launch set up meanwhile.
template <typename... A>
cudaError_t launch_after(void (*kernel)(A...), dim3 grid, unsigned threads, size_t bytes, cudaStream_t stream, unsigned cluster,
                         typename Same<A>::type... args)
{
    cudaLaunchConfig_t config{};
    config.gridDim = grid;
    config.blockDim = dim3(threads);
    config.dynamicSmemBytes = bytes;
    config.stream = stream;
    cudaLaunchAttribute attrs[2]{};
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim = {cluster, 1, 1};
    config.attrs = attrs;
    config.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&config, kernel, args...);
}

__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// An ordinary load. A kernel that starts before the one ahead of it ends reads what that one writes, so its loads may not
// take the read-only path, which is for data that nobody writes while the kernel runs.
__device__ __forceinline__ float load_f32(const float *p)
{
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ void load_shared(uint32_t at, uint4 &v) { v = shared16(at); }
__device__ __forceinline__ void load_shared(uint32_t at, unsigned int &v)
{
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
}

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
