// Host-side checks that the entry points of this folder share.
#pragma once

#include <initializer_list>

#include "../csrc/block.h"

namespace convrot {

// Sizes, and coordinates of tiles past their end, are counted in 32 bits on the device.
constexpr int64_t kMaxSize = int64_t{1} << 30;

inline int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }

inline convrot_status done(cudaError_t e) { return e == cudaSuccess ? CONVROT_OK : CONVROT_ERR_CUDA; }

inline convrot_status first_of(std::initializer_list<convrot_status> all)
{
    for (convrot_status s : all)
        if (s != CONVROT_OK) return s;
    return CONVROT_OK;
}

// A matrix [rows, cols] of elements of `bytes` bytes.
inline convrot_status check_matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, int bytes)
{
    if (ld < cols) return CONVROT_ERR_INVALID_ARG;
    if (rows == 0) return CONVROT_OK;
    if (!p) return CONVROT_ERR_INVALID_ARG;
    return aligned_to(p, bytes) ? CONVROT_OK : CONVROT_ERR_ALIGNMENT;
}

inline convrot_status check_optional(const void *p, int64_t rows, int64_t cols, int64_t ld, int bytes)
{
    return p ? check_matrix(p, rows, cols, ld, bytes) : CONVROT_OK;
}

inline convrot_status check_16bit(int dtype)
{
    if (dtype == CONVROT_F32) return CONVROT_ERR_UNSUPPORTED;
    return dtype == CONVROT_BF16 || dtype == CONVROT_F16 ? CONVROT_OK : CONVROT_ERR_INVALID_ARG;
}

inline convrot_status check_work(const void *work, int64_t has, int64_t need)
{
    if (need == 0) return CONVROT_OK;
    if (!work || has < need) return CONVROT_ERR_INVALID_ARG;
    return aligned_to(work, 256) ? CONVROT_OK : CONVROT_ERR_ALIGNMENT;
}

}  // namespace convrot
