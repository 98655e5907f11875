// What the attention's gradient needs of each query (include/convrot_block.h):
// -lse in base 2, so that a probability is one multiply-add and one exponential,
// and -delta = -dout . out, so that dS = P (dP - delta) needs no sum over keys.
//
// A block takes the queries of 64 tokens (or more) of one head; kLanes lanes
// take one query, 16 bytes of it each, and kBatch of them are loaded together
// (8190 x 40 heads of 128: 74 us with a query a warp and one in flight). A
// block a head, also where heads share keys (4 x 1270 x 43 heads on one of
// keys: 126 us with a block for all 43). Rows behind the last query get -infinity
// for the first, and queries whose lse is -infinity (without keys, or with
// none that counts) too: their probabilities are 0. Bound by HBM: out and dout once
// (8190 x 40 heads of 128: 33 us, 5.1 TB/s).
#include "attention.cuh"

namespace convrot {
namespace {

using namespace mma16;

struct StatParams {
    const void *out, *dout;
    int64_t out_strides[3], dout_strides[3];
    const float *lse;
    float *base2, *delta, *amax;
    int64_t q_tokens, rows;  // rows of a head's statistics
    int64_t blocks, tokens;  // of a head; of a block
    int32_t q_heads, d, wide;
    float shift;
};

template <typename T, int kD>
__global__ void __launch_bounds__(256, 5) attention_stats_kernel(const __grid_constant__ StatParams p)
{
    __shared__ float tops[8];
    after_previous();
    let_next_start();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // (the heads of a stretch of tokens lie together, so they are read together)
    const int64_t bt = blockIdx.x / p.q_heads, h = blockIdx.x - bt * p.q_heads, b = bt / p.blocks, block = bt - b * p.blocks, head = b * p.q_heads + h;
    const int64_t t0 = block * p.tokens;
    constexpr int kLanes = kD / 8, kPerWarp = 32 / kLanes, kBatch = 2, kStride = 8 * kPerWarp;  // queries of a block's round
    const int sub = lane / kLanes, e0 = lane % kLanes * 8;
    const int queries = static_cast<int>(p.tokens);
    float top = 0.0f;
    for (int i0 = warp * kPerWarp + sub; i0 - sub < queries; i0 += kStride * kBatch) {
        Raw<T, 8> ro[kBatch], rg[kBatch];
        float part[kBatch];
#pragma unroll
        for (int n = 0; n < kBatch; ++n) {
            const int i = i0 + n * kStride;
            const int64_t t = t0 + i;
            ro[n].bits[0] = rg[n].bits[0] = make_uint4(0, 0, 0, 0);
            if (i >= queries || t >= p.q_tokens || e0 >= p.d) continue;
            const T *o = static_cast<const T *>(p.out) + b * p.out_strides[0] + t * p.out_strides[1] + h * p.out_strides[2] + e0;
            const T *g = static_cast<const T *>(p.dout) + b * p.dout_strides[0] + t * p.dout_strides[1] + h * p.dout_strides[2] + e0;
            if (p.wide) {
                ro[n].load_stream(o);
                rg[n].load(g);
            } else {
                const int left = p.d - e0 < 8 ? p.d - e0 : 8;
                ro[n].bits[0] = load8_any(o, left);
                rg[n].bits[0] = load8_any(g, left);
            }
        }
#pragma unroll
        for (int n = 0; n < kBatch; ++n) {
            float vo[8], vg[8];
            ro[n].unpack(vo);
            rg[n].unpack(vg);
            part[n] = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                part[n] = fmaf(vo[e], vg[e], part[n]);
                top = fmaxf(top, fabsf(vg[e]));
            }
        }
#pragma unroll
        for (int s = kLanes / 2; s > 0; s >>= 1)
#pragma unroll
            for (int n = 0; n < kBatch; ++n) part[n] += __shfl_xor_sync(0xffffffffu, part[n], s);
        if (e0 == 0) {
#pragma unroll
            for (int n = 0; n < kBatch; ++n) {
                const int i = i0 + n * kStride;
                const int64_t t = t0 + i, at = head * p.rows + t;
                if (i >= queries || t >= p.rows) continue;
                const float lse = t < p.q_tokens ? load_f32(p.lse + head * p.q_tokens + t) : neg_inf();
                p.base2[at] = lse == neg_inf() ? lse : fmaf(lse, -kLog2e, p.shift);
                p.delta[at] = -part[n];
            }
        }
    }
    if (!p.amax) return;
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < 8; ++w) top = fmaxf(top, tops[w]);
        p.amax[head * p.blocks + block] = top;  // (a key head's query heads follow each other)
    }
}

}  // namespace

cudaError_t launch_attention_stats(const AttentionGradArgs &a, cudaStream_t stream)
{
    StatParams p{};
    p.out = a.out;
    p.dout = a.dout_own;
    bool wide = a.d % 8 == 0;
    for (int i = 0; i < 3; ++i) {
        p.out_strides[i] = a.out_strides[i];
        p.dout_strides[i] = a.dout_own_strides[i];
        wide = wide && a.out_strides[i] % 8 == 0 && a.dout_own_strides[i] % 8 == 0;
    }
    p.wide = wide && aligned_to(a.out, 16) && aligned_to(a.dout_own, 16);
    p.lse = a.lse;
    p.base2 = a.base2;
    p.delta = a.delta;
    p.amax = a.amax;
    p.q_tokens = a.q.tokens;
    p.rows = stat_rows(a.q.tokens);
    p.blocks = stat_blocks(a.q.tokens, a.q.heads / a.k.heads);
    p.tokens = stat_tokens(a.q.tokens, a.q.heads / a.k.heads);
    p.q_heads = static_cast<int32_t>(a.q.heads);
    p.d = a.d;
    const int64_t blocks = a.batch * p.q_heads * p.blocks;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(blocks));
    if (a.dtype == CONVROT_BF16)
        return launch_after(a.d <= 64 ? attention_stats_kernel<__nv_bfloat16, 64> : attention_stats_kernel<__nv_bfloat16, 128>, grid, 256, 0, stream, 1, p);
    p.shift = kProbShift<__half>;
    return launch_after(a.d <= 64 ? attention_stats_kernel<__half, 64> : attention_stats_kernel<__half, 128>, grid, 256, 0, stream, 1, p);
}

}  // namespace convrot
