// What the attention's gradient needs of each query (include/convrot_block.h):
// -lse in base 2, so that a probability is one multiply-add and one exponential,
// and -delta = -dout . out, so that dS = P (dP - delta) needs no sum over keys.
//
// A warp takes one query of one head; a block the queries of kStatTokens tokens
// and of the heads that share a key head. Rows behind the last query get -infinity
// for the first: their probabilities are 0. Bound by HBM: out and dout once.
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
    int64_t blocks;
    int32_t q_heads, kv_heads, group, d, wide;
    float shift;
};

template <typename T>
__global__ void __launch_bounds__(256) attention_stats_kernel(const __grid_constant__ StatParams p)
{
    __shared__ float tops[8];
    after_previous();
    let_next_start();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t block = blockIdx.x % p.blocks, bh = blockIdx.x / p.blocks, b = bh / p.kv_heads, hk = bh - b * p.kv_heads;
    const int64_t t0 = block * kStatTokens;
    float top = 0.0f;
    for (int i = warp; i < kStatTokens * p.group; i += 8) {
        const int64_t t = t0 + i / p.group, h = hk * p.group + i % p.group;
        if (t >= p.rows) break;
        float sum = 0.0f;
        if (t < p.q_tokens) {
            const T *o = static_cast<const T *>(p.out) + b * p.out_strides[0] + t * p.out_strides[1] + h * p.out_strides[2];
            const T *g = static_cast<const T *>(p.dout) + b * p.dout_strides[0] + t * p.dout_strides[1] + h * p.dout_strides[2];
            if (p.wide) {  // four elements a lane
                if (lane * 4 < p.d) {
                    Raw<T, 4> ro, rg;
                    float vo[4], vg[4];
                    ro.load(o + lane * 4);
                    rg.load(g + lane * 4);
                    ro.unpack(vo);
                    rg.unpack(vg);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sum = fmaf(vo[e], vg[e], sum);
                        top = fmaxf(top, fabsf(vg[e]));
                    }
                }
            } else {
                for (int e = lane; e < p.d; e += 32) {
                    const float vg = to_f32(g[e]);
                    sum = fmaf(to_f32(o[e]), vg, sum);
                    top = fmaxf(top, fabsf(vg));
                }
            }
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        }
        if (lane == 0) {
            const int64_t head = b * p.q_heads + h, at = head * p.rows + t;
            p.base2[at] = t < p.q_tokens ? fmaf(load_f32(p.lse + head * p.q_tokens + t), -kLog2e, p.shift) : neg_inf();
            p.delta[at] = -sum;
        }
    }
    if (!p.amax) return;
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < 8; ++w) top = fmaxf(top, tops[w]);
        p.amax[bh * p.blocks + block] = top;
    }
}

}  // namespace

cudaError_t launch_attention_stats(const AttentionGradArgs &a, cudaStream_t stream)
{
    StatParams p{};
    p.out = a.out;
    p.dout = a.dout_own;
    bool wide = a.d % 4 == 0;
    for (int i = 0; i < 3; ++i) {
        p.out_strides[i] = a.out_strides[i];
        p.dout_strides[i] = a.dout_own_strides[i];
        wide = wide && a.out_strides[i] % 4 == 0 && a.dout_own_strides[i] % 4 == 0;
    }
    p.wide = wide && aligned_to(a.out, 8) && aligned_to(a.dout_own, 8);
    p.lse = a.lse;
    p.base2 = a.base2;
    p.delta = a.delta;
    p.amax = a.amax;
    p.q_tokens = a.q.tokens;
    p.rows = stat_rows(a.q.tokens);
    p.blocks = p.rows / kStatTokens;
    p.q_heads = static_cast<int32_t>(a.q.heads);
    p.kv_heads = static_cast<int32_t>(a.k.heads);
    p.group = p.q_heads / p.kv_heads;
    p.d = a.d;
    const int64_t blocks = a.batch * p.kv_heads * p.blocks;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(blocks));
    if (a.dtype == CONVROT_BF16) return launch_after(attention_stats_kernel<__nv_bfloat16>, grid, 256, 0, stream, 1, p);
    p.shift = kProbShift<__half>;
    return launch_after(attention_stats_kernel<__half>, grid, 256, 0, stream, 1, p);
}

}  // namespace convrot
