// Copies of keys and values for the attention kernels (include/convrot_block.h):
// those that the mask leaves, one behind the other, so that the kernels meet
// whole tiles of keys that are there and zeros behind the last one; and heads
// that do not start on 16 bytes, which a tensor map cannot describe.
//
// A masked key costs the products nothing then, and what stands in it, NaN too,
// is never an operand. A block takes eight tokens of a sample and tensor, or 32
// where blocks of eight would be several rounds of the GPU. Their places are
// the number of tokens that are there before them, which each block counts for
// itself: 4096 bytes of a mask are 16 a thread. Latency is all that counts here
// (2 x 77 tokens of 10 heads of 64: 20 us with 32 tokens a block and a piece at
// a time; 8 x 3525 tokens of 11 heads of 32: 45 us with eight a block, 24 with 32).
#include "attention.h"
#include "mma16.cuh"

namespace convrot {
namespace {

constexpr int kMaxTokens = 32, kThreads = 256, kBatch = 4;  // pieces of a thread in flight

__device__ __forceinline__ bool aligned4(const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

__device__ __forceinline__ uint32_t kept4(uint32_t w)  // bytes that are not 0
{
    return __popc(__vcmpne4(w, 0u)) / 8;
}

// tokens: a block's, 8 or kMaxTokens
__global__ void __launch_bounds__(kThreads) gather_kernel(const __grid_constant__ GatherArgs a, int tokens)
{
    __shared__ int before_s, total_s;
    __shared__ int place[kMaxTokens];
    after_previous();
    let_next_start();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens, b = blockIdx.y;
    const int lane = threadIdx.x & 31;
    int64_t total = a.tokens;
    if (a.mask) {
        if (threadIdx.x == 0) before_s = total_s = 0;
        __syncthreads();
        const uint8_t *mask = a.mask + b * a.mask_stride;
        int before = 0, all = 0;
        // whole words where they are aligned (a word never crosses t0, a multiple of 8 past the mask's own start)
        const bool words = aligned4(mask);
        const int64_t whole = words ? a.tokens / 4 : 0;
#pragma unroll 4
        for (int64_t i = threadIdx.x; i < whole; i += kThreads) {
            const int n = kept4(*reinterpret_cast<const volatile uint32_t *>(mask + 4 * i));
            all += n;
            if (4 * i < t0) before += n;
        }
        for (int64_t i = whole * 4 + threadIdx.x; i < a.tokens; i += kThreads) {
            const int n = *reinterpret_cast<const volatile uint8_t *>(mask + i) != 0;
            all += n;
            if (i < t0) before += n;
        }
        before = __reduce_add_sync(0xffffffffu, before);
        all = __reduce_add_sync(0xffffffffu, all);
        if (lane == 0) {
            atomicAdd(&before_s, before);
            atomicAdd(&total_s, all);
        }
        __syncthreads();
        total = total_s;
        if (threadIdx.x < 32) {
            const int64_t t = t0 + lane;
            const bool there = lane < tokens && t < a.tokens && *reinterpret_cast<const volatile uint8_t *>(mask + t) != 0;
            const uint32_t all_there = __ballot_sync(0xffffffffu, there);
            const int at = before_s + __popc(all_there & ((1u << lane) - 1u));
            if (lane < tokens) place[lane] = there ? at : -1;
            if (there && a.index && blockIdx.z == 0) a.index[b * a.rows + at] = static_cast<int32_t>(t);
        }
        if (blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0) a.counts[b] = static_cast<int32_t>(total);
        __syncthreads();
    }
    const int groups = a.dp / 8;
    const int64_t per_token = a.heads * groups, work = per_token * tokens;
    const int64_t end = (total + kTileKeys - 1) / kTileKeys * kTileKeys;
    const int s = blockIdx.z;
    const uint16_t *src = static_cast<const uint16_t *>(a.src[s]) + b * a.strides[s][0];
    uint16_t *dst = static_cast<uint16_t *>(a.dst[s]) + b * a.rows * a.heads * a.dp;
    uint16_t *zero = static_cast<uint16_t *>(a.zero[s]);
    const bool wide = a.d % 8 == 0 && a.strides[s][0] % 8 == 0 && a.strides[s][1] % 8 == 0 && a.strides[s][2] % 8 == 0 &&
                      reinterpret_cast<uintptr_t>(a.src[s]) % 16 == 0;
    // (a division of 64 bits takes several times as long)
    const bool narrow = work <= INT32_MAX;
    auto divided = [&](int64_t x, int64_t by) { return narrow ? static_cast<uint32_t>(x) / static_cast<uint32_t>(by) : x / by; };
    for (int64_t i0 = threadIdx.x; i0 < work; i0 += kThreads * kBatch) {
        uint4 w[kBatch];
        int64_t to[kBatch];  // place of the piece, or -1
#pragma unroll
        for (int n = 0; n < kBatch; ++n) {
            const int64_t i = i0 + n * kThreads;
            to[n] = -1;
            if (i >= work) continue;
            const int local = static_cast<int>(divided(i, per_token));
            const int64_t rest = i - local * per_token, h = divided(rest, groups), t = t0 + local;
            const int e0 = static_cast<int>(rest - h * groups) * 8, left = a.d - e0 < 8 ? a.d - e0 : 8;
            const int64_t row = t >= a.tokens ? -1 : a.mask ? place[local] : t;
            if (row >= 0) {
                to[n] = (row * a.heads + h) * a.dp + e0;
                const uint16_t *from = src + t * a.strides[s][1] + h * a.strides[s][2] + e0;
                w[n] = wide ? __ldcg(reinterpret_cast<const uint4 *>(from)) : mma16::load8_any(from, left);
            } else if (zero && t < a.tokens) {
                mma16::store8_any(zero + ((b * a.tokens + t) * a.heads + h) * a.d + e0, make_uint4(0, 0, 0, 0), left);
            }
            // the rows behind the last one, to the end of its tile
            if (a.mask && t >= total && t < end) *reinterpret_cast<uint4 *>(dst + (t * a.heads + h) * a.dp + e0) = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int n = 0; n < kBatch; ++n)
            if (to[n] >= 0) *reinterpret_cast<uint4 *>(dst + to[n]) = w[n];
    }
}

}  // namespace

cudaError_t launch_gather(const GatherArgs &a, cudaStream_t stream)
{
    for (int64_t b0 = 0; b0 < a.batch; b0 += 65535) {  // a grid's second dimension ends there
        GatherArgs part = a;
        part.batch = a.batch - b0 < 65535 ? a.batch - b0 : 65535;
        for (int s = 0; s < a.count; ++s) {
            part.src[s] = static_cast<const uint16_t *>(a.src[s]) + b0 * a.strides[s][0];
            part.dst[s] = static_cast<uint16_t *>(a.dst[s]) + b0 * a.rows * a.heads * a.dp;
            if (a.zero[s]) part.zero[s] = static_cast<uint16_t *>(a.zero[s]) + b0 * a.tokens * a.heads * a.d;
        }
        if (a.mask) {
            part.mask = a.mask + b0 * a.mask_stride;
            part.counts = a.counts + b0;
            if (a.index) part.index = a.index + b0 * a.rows;
        }
        const int tokens = (a.rows + 7) / 8 * part.batch * a.count > 2 * 8 * kSms ? kMaxTokens : 8;  // (eight blocks an SM)
        const dim3 grid(static_cast<unsigned>((a.rows + tokens - 1) / tokens), static_cast<unsigned>(part.batch), static_cast<unsigned>(a.count));
        const cudaError_t e = launch_after(gather_kernel, grid, kThreads, 0, stream, 1, part, tokens);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace convrot
