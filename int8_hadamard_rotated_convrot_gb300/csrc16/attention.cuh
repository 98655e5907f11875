// What the attention kernels share: tensor maps over heads, and the work items.
#pragma once

#include "attention.h"
#include "mma16.cuh"

namespace convrot {
namespace mma16 {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// A tensor map over one tensor's heads, in boxes of 64 elements x `rows` tokens of one head. A dimension that is
// broadcast (stride 0) has one entry, at coordinate 0.
struct HeadsMap {
    CUtensorMap map;
    int32_t head_step, batch_step;  // 0 or 1: what a head's and a sample's number is multiplied by
};

inline bool heads_on_16_bytes(const void *p, const int64_t (&strides)[3], int64_t batch, int64_t tokens, int64_t heads, int64_t d)
{
    // (a token stride of 0 is no matrix that a map describes)
    const int64_t n[3] = {batch, tokens, heads};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (strides[i] % 8 || strides[i] > (int64_t{1} << 38))) return false;
    return aligned_to(p, 16) && d % 8 == 0 && (tokens <= 1 || strides[1] >= d);
}

template <typename T>
bool heads_map(HeadsMap *m, const States &s, int64_t batch, int64_t d, uint32_t rows)
{
    auto fn = encode_fn();
    if (!fn) return false;
    m->head_step = s.heads > 1 && s.strides[2] > 0;
    m->batch_step = batch > 1 && s.strides[0] > 0;
    const int64_t dp = (d + 7) / 8 * 8;
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(s.tokens), static_cast<cuuint64_t>(m->head_step ? s.heads : 1),
                          static_cast<cuuint64_t>(m->batch_step ? batch : 1)};
    auto bytes = [&](bool real, int64_t stride) { return static_cast<cuuint64_t>((real ? stride : dp) * 2); };
    cuuint64_t strides[3] = {bytes(s.tokens > 1, s.strides[1]), bytes(m->head_step, s.strides[2]), bytes(m->batch_step, s.strides[0])};
    cuuint32_t box[4] = {kBoxElems, rows, 1, 1}, steps[4] = {1, 1, 1, 1};
    return fn(&m->map, map_type<T>(), 4, const_cast<void *>(s.p), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One tile of a head: kHalves boxes of 64 elements x 128 tokens, one behind the other.
constexpr int kTileBox = 128 * 128;  // bytes

template <int kHalves>
__device__ __forceinline__ void load_tile(uint32_t dst, const HeadsMap &m, int token, int head, int batch, uint32_t bar)
{
#pragma unroll
    for (int i = 0; i < kHalves; ++i)
        tma_load_4d(dst + i * kTileBox, &m.map, i * kBoxElems, token, head * m.head_step, batch * m.batch_step, bar);
}

// Which of 32 keys, one a lane, are there.
__device__ __forceinline__ uint32_t keys_there(const uint8_t *mask, int key, int keys)
{
    bool there = false;
    if (key < keys) there = *reinterpret_cast<const volatile uint8_t *>(mask + key) != 0;
    return __ballot_sync(0xffffffffu, there);
}

// Zeros in the rows of a tile whose key is not there, by two warps, half of the rows each: what stands in a masked key must
// not meet a product over the keys (0 times NaN). The tensor cores see it behind a barrier that each warp's lane 0 arrives at.
template <int kHalves>
__device__ __forceinline__ void clean_rows(uint32_t tile, const uint32_t (&there)[2], int which, int lane)
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int first = which * 64 + i * 32;
        uint32_t gone = ~there[i];
        while (gone) {  // four rows at a time, eight lanes a row
            const int mine = __fns(gone, 0, lane / 8 + 1);
            if (mine >= 0 && mine < 32) {
                const uint32_t at = tile + (first + mine) * 128 + lane % 8 * 16;
#pragma unroll
                for (int h = 0; h < kHalves; ++h) asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at + h * kTileBox), "r"(0) : "memory");
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) gone &= gone - 1;
        }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}

// The cleaning warps' keys of sample b's mask: read again only where the sample changes.
struct MaskedRows {
    uint32_t there[2] = {0, 0};
    int sample = -1;
    __device__ __forceinline__ void of(const uint8_t *mask, int64_t stride, int b, int keys, int which, int lane)
    {
        if (b == sample) return;
        sample = b;
#pragma unroll
        for (int i = 0; i < 2; ++i) there[i] = keys_there(mask + b * stride, which * 64 + i * 32 + lane, keys);
    }
};

// D [128 x 128] = rows of one tile by rows of another, over `steps` times 16 of the head's kD elements.
template <int kD>
__device__ __forceinline__ void tile_product(uint32_t d, uint32_t rows, uint32_t cols, uint32_t id, int steps)
{
    const Desc a(desc_k(rows)), b(desc_k(cols));
#pragma unroll
    for (int kk = 0; kk < kD / kMmaK; ++kk) {
        const uint32_t at = (kk / 4) * (kTileBox >> 4) + (kk % 4) * kStepK;
        if (kk >= steps) break;
        if (kk == 0)
            mma_ss_step<false>(d, a, at, b, at, id);
        else
            mma_ss_step<true>(d, a, at, b, at, id);
    }
}

// sums (+)= a 16-bit [128 x 128] matrix in tensor memory, by a tile's rows. Its K is in kParts parts, each in the first
// half of the columns that its fp32 values had.
template <int kParts>
__device__ __forceinline__ void tile_add(uint32_t sums, uint32_t a, uint32_t tile, uint32_t id, bool fresh)
{
    const Desc b(desc_mn(tile, kTileBox));
    if (fresh)
        mma_ts_step<false>(sums, a, b, 0, id);
    else
        mma_ts_step<true>(sums, a, b, 0, id);
#pragma unroll
    for (int kk = 1; kk < 128 / kMmaK; ++kk) {
        constexpr int kPer = 128 / kMmaK / kParts;
        mma_ts_step<true>(sums, a + (kk / kPer) * (128 / kParts) + (kk % kPer) * (kMmaK / 2), b, kStepMN * kk, id);
    }
}

// float16 has 40 binary orders of magnitude, and gradients may be small: the backward pass takes P 2^15 times as large
// (at most 2^15), and dS by a power of two that brings the largest |dout| of a head to 2^-3 .. 2^-2, both exact and taken back
// at the end. (dS overflows then only where |dout . v| reaches 2^16 of that.)
template <typename T>
constexpr float kProbShift = std::is_same_v<T, __half> ? 15.0f : 0.0f;

// log2 of that power, for a warp: the largest of a head's blocks.
__device__ __forceinline__ int grad_exponent(const float *amax, int64_t blocks, int lane)
{
    float top = 0.0f;
    for (int64_t i = lane; i < blocks; i += 32) top = fmaxf(top, load_f32(amax + i));
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));  // not negative: ordered as integers
    if (!(top > 0.0f) || top > 3e38f) return 0;
    return -3 - (static_cast<int>(__float_as_uint(top) >> 23) - 127);
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// An untiled copy; both addresses and the size are multiples of 16 bytes.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

inline bool heads_wide(const void *p, const int64_t (&strides)[3], int64_t batch, int64_t tokens, int64_t heads)
{
    return aligned_to(p, 16) && (batch <= 1 || strides[0] % 8 == 0) && (tokens <= 1 || strides[1] % 8 == 0) && (heads <= 1 || strides[2] % 8 == 0);
}

}  // namespace mma16
}  // namespace convrot
