// What the gated norm and its gradient share.
#pragma once

#include "block.h"

namespace convrot {

template <typename P>
__device__ __forceinline__ float param(const void *p, int64_t i, float otherwise)
{
    return p ? to_f32(static_cast<const P *>(p)[i]) : otherwise;
}

// kVec parameters from index i on, or `otherwise`.
template <typename P, int kVec>
__device__ __forceinline__ void params(const void *p, int64_t i, float otherwise, float (&v)[kVec])
{
    if (p) {
        Raw<P, kVec> r;
        r.load(static_cast<const P *>(p) + i);
        r.unpack(v);
    } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[e] = otherwise;
    }
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

// Whether every address of a [rows, d] operand allows accesses of `vec`
// elements of `size` bytes (at most 16 bytes at a time).
inline bool vectors(const void *p, int64_t rows, int64_t ld, int vec, int size)
{
    const int64_t bytes = vec * size < 16 ? vec * size : 16;
    return !p || (aligned_to(p, bytes) && (rows <= 1 || ld * size % bytes == 0));
}

}  // namespace convrot
