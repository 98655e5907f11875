// The elementwise part of the gated feed-forward's gradient
// (include/convrot_block.h): dg = dy u act'(g) and du = dy act(g), rounded to
// the operands of the products that follow, and their column sums in fp32.
//
// A warp takes 256 columns of a row, eight a lane, and a block's eight warps
// every eighth row of its chunk, so that a thread meets the same columns all
// the way and adds them up in registers; the warps' sums meet in shared
// memory, the chunks' in a second small kernel, in order. Bound by HBM: 6
// bytes read and 4 written a value (8190 x 13824: 174 us, 6.5 TB/s).
#include "gated.h"
#include "mma16.cuh"

namespace convrot {
namespace {

constexpr int kWarps = 8, kCols = 256, kPer = 8;  // warps of a block, columns of a warp and of a lane

// act(v) and its derivative.
template <int kAct>
__device__ __forceinline__ void act_and_slope(float v, float &a, float &slope)
{
    if constexpr (kAct == CONVROT_ACT_SILU) {
        const float p = rcp(1.0f + ex2(-1.4426950f * v));
        a = v * p;
        slope = fmaf(a, 1.0f - p, p);
    } else if constexpr (kAct == CONVROT_ACT_GELU_TANH) {
        // p = 1 / (1 + e^(-2u)), 2u = v (c0 + c1 v^2): a = v p, a' = p + v p (1 - p) (2u)'
        const float v2 = v * v, p = rcp(1.0f + ex2(v * fmaf(v2, -0.10294324f, -2.3022082f)));
        const float w2 = fminf(v2, 400.0f);  // p (1 - p) is 0 there, and v^2 may be infinite
        a = v * p;
        slope = fmaf(a * (1.0f - p), fmaf(w2, 3.0f * 0.071354816f, 1.5957691f), p);
    } else if constexpr (kAct == CONVROT_ACT_GELU_ERF) {
        // Phi(v) + v phi(v), Phi by Abramowitz & Stegun 7.1.26 as in block.h
        const float x = fabsf(v) * 0.70710678f, t = rcp(fmaf(x, 0.3275911f, 1.0f));
        float h = fmaf(t, 0.5f * 1.061405429f, 0.5f * -1.453152027f);
        h = fmaf(t, h, 0.5f * 1.421413741f);
        h = fmaf(t, h, 0.5f * -0.284496736f);
        h = fmaf(t, h, 0.5f * 0.254829592f) * t;
        const float e = ex2(x * x * -1.4426950f);
        const float cdf = 0.5f + copysignf(fmaf(h, -e, 0.5f), v);
        a = v * cdf;
        slope = fmaf(v, e * 0.39894228f, cdf);
    } else {
        a = v;
        slope = 1.0f;
    }
}

struct GradParams {
    const void *gate, *up, *dy;
    int64_t ldgate, ldup, lddy;
    void *dg, *du;
    int64_t ldd;
    float *partial;  // [chunks][2][n] or null
    int64_t m, n;
    int64_t chunk;   // rows of a chunk
    int32_t wide;    // rows of gate, up and dy start on 16 bytes
};

template <typename T, int kAct, bool kSums>
__global__ void __launch_bounds__(32 * kWarps, kSums ? 2 : 3) gated_grad_kernel(const GradParams p)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * kCols + lane * kPer;
    const int64_t row0 = static_cast<int64_t>(blockIdx.y) * p.chunk, row1 = row0 + p.chunk < p.m ? row0 + p.chunk : p.m;
    const int cols = p.n - col >= kPer ? kPer : p.n > col ? static_cast<int>(p.n - col) : 0;
    after_previous();
    let_next_start();
    float sg[kPer] = {}, su[kPer] = {};
    if (cols > 0) {
        constexpr int kRows = 2;  // in flight
        for (int64_t r0 = row0 + warp; r0 < row1; r0 += kWarps * kRows) {
            float g[kRows][kPer], u[kRows][kPer], d[kRows][kPer];
            Raw<T, kPer> in[kRows][3];
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int64_t r = r0 + i * kWarps;
                if (r >= row1) continue;
                const T *from[3] = {static_cast<const T *>(p.gate) + r * p.ldgate + col, static_cast<const T *>(p.up) + r * p.ldup + col,
                                    static_cast<const T *>(p.dy) + r * p.lddy + col};
                if (p.wide && cols == kPer) {
#pragma unroll
                    for (int t = 0; t < 3; ++t) in[i][t].load_stream(from[t]);
                } else {
#pragma unroll
                    for (int t = 0; t < 3; ++t) in[i][t].bits[0] = mma16::load8_any(from[t], cols);
                }
            }
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int64_t r = r0 + i * kWarps;
                if (r >= row1) continue;
                in[i][0].unpack(g[i]);
                in[i][1].unpack(u[i]);
                in[i][2].unpack(d[i]);
                float dg[kPer], du[kPer];
#pragma unroll
                for (int e = 0; e < kPer; ++e) {
                    float a, slope;
                    act_and_slope<kAct>(g[i][e], a, slope);
                    dg[e] = d[i][e] * u[i][e] * slope;
                    du[e] = d[i][e] * a;
                    if constexpr (kSums) {
                        sg[e] += dg[e];
                        su[e] += du[e];
                    }
                }
                Raw<T, kPer> out;
                out.pack(dg);
                out.store(static_cast<T *>(p.dg) + r * p.ldd + col);
                out.pack(du);
                out.store(static_cast<T *>(p.du) + r * p.ldd + col);
            }
        }
    }
    if constexpr (!kSums) return;
    __shared__ float sums[2][kWarps][kCols];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        sums[0][warp][lane * kPer + e] = sg[e];
        sums[1][warp][lane * kPer + e] = su[e];
    }
    __syncthreads();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kCols + threadIdx.x;
    if (c >= p.n) return;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += sums[t][w][threadIdx.x];
        p.partial[(static_cast<int64_t>(blockIdx.y) * 2 + t) * p.n + c] = s;
    }
}

__global__ void __launch_bounds__(256) column_sums_kernel(const float *partial, int64_t chunks, int64_t n, float *gate, float *up)
{
    const int64_t c = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    after_previous();
    let_next_start();
    if (c >= 2 * n) return;
    float s = 0.0f;
    for (int64_t i = 0; i < chunks; ++i) s += load_f32(partial + i * 2 * n + c);
    float *to = c < n ? gate + c : up + (c - n);
    *to = s;
}

// Eight elements a thread, from rows that start anywhere.
__global__ void __launch_bounds__(256) align_rows_kernel(const uint16_t *x, int64_t rows, int64_t cols, int64_t ld, uint16_t *out, int64_t ldo)
{
    after_previous();
    let_next_start();
    const int64_t groups = ldo / 8, total = rows * groups;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t r = i / groups, c = (i - r * groups) * 8;
        const uint4 w = mma16::load8_any(x + r * ld + c, cols - c < 8 ? static_cast<int>(cols - c) : 8);
        *reinterpret_cast<uint4 *>(out + r * ldo + c) = w;
    }
}

template <typename T, int kAct>
cudaError_t launch_form(const GradParams &p, dim3 grid, cudaStream_t stream)
{
    return launch_after(p.partial ? gated_grad_kernel<T, kAct, true> : gated_grad_kernel<T, kAct, false>, grid, 32 * kWarps, 0, stream, 1, p);
}

template <typename T>
cudaError_t launch_act(int act, const GradParams &p, dim3 grid, cudaStream_t stream)
{
    if (act == CONVROT_ACT_SILU) return launch_form<T, 3>(p, grid, stream);
    if (act == CONVROT_ACT_GELU_TANH) return launch_form<T, 2>(p, grid, stream);
    if (act == CONVROT_ACT_GELU_ERF) return launch_form<T, 1>(p, grid, stream);
    return launch_form<T, 0>(p, grid, stream);
}

}  // namespace

// About eight blocks an SM, of sixteen rows or more.
int64_t gated_grad_chunks(int64_t m, int64_t n)
{
    const int64_t across = (n + kCols - 1) / kCols, most = (m + 2 * kWarps - 1) / (2 * kWarps);
    int64_t chunks = (8 * kSms + across - 1) / across;
    if (chunks > most) chunks = most;
    return chunks > 1 ? chunks : 1;
}

cudaError_t launch_gated_grad(const convrot_gated_linear_backward_args &a, void *dg, void *du, int64_t ldd, float *partial, cudaStream_t stream)
{
    GradParams p{a.gate, a.up, a.dy, a.ldgate, a.ldup, a.lddy, dg, du, ldd, partial, a.m, a.n, 0, 0};
    const int64_t chunks = gated_grad_chunks(a.m, a.n);
    // whole rounds of a block: 16 rows
    p.chunk = ((a.m + chunks - 1) / chunks + 2 * kWarps - 1) / (2 * kWarps) * (2 * kWarps);
    p.wide = mma16::tma_rows(a.gate, a.ldgate, a.m) && mma16::tma_rows(a.up, a.ldup, a.m) && mma16::tma_rows(a.dy, a.lddy, a.m);
    const dim3 grid(static_cast<unsigned>((a.n + kCols - 1) / kCols), static_cast<unsigned>(chunks));
    cudaError_t e = a.dtype == CONVROT_BF16 ? launch_act<__nv_bfloat16>(a.act, p, grid, stream) : launch_act<__half>(a.act, p, grid, stream);
    if (e != cudaSuccess || !partial) return e;
    return launch_after(column_sums_kernel, dim3(static_cast<unsigned>((2 * a.n + 255) / 256)), 256, 0, stream, 1,
                        static_cast<const float *>(partial), chunks, a.n, a.db_gate, a.db_up);
}

cudaError_t launch_align_rows(const void *x, int64_t rows, int64_t cols, int64_t ld, void *out, int64_t ldo, cudaStream_t stream)
{
    const int64_t blocks = (rows * (ldo / 8) + 255) / 256;
    return launch_after(align_rows_kernel, dim3(static_cast<unsigned>(blocks < 16 * kSms ? blocks : 16 * kSms)), 256, 0, stream, 1,
                        static_cast<const uint16_t *>(x), rows, cols, ld, static_cast<uint16_t *>(out), ldo);
}

}  // namespace convrot
