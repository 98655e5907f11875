// The gated norm and its gradient (include/convrot_block.h).
//
//   u = post(y), h = res_scale x + gate u, n = pre(h) (1 + scale) + shift
//
// Forward: two reads and two writes of a value for about ten operations on it,
// so HBM is the bound. A row stays in the registers of one block of threads
// (of one warp, up to 32 x 4 vectors) from its load to its store: every tensor
// is moved once, in 16-byte accesses where all addresses allow it and in
// coalesced single elements otherwise. The statistics are two-pass (mean, then
// squares about it), which costs one more trip around the block than a
// one-pass sum of squares and keeps layer norms of rows with a large mean.
#include "block.h"

namespace convrot {
namespace {

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
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[e] = r.get(e);
    } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[e] = otherwise;
    }
}

// Sums over the threads that share a row: a warp, or a block through shared
// memory. Two buffers in turn: a thread that is one sum ahead writes the other
// one, and it cannot be two ahead, so one barrier a sum is enough.
template <bool kWarp>
struct RowSum {
    float2 *slots;  // [2][32]
    int turn = 0;
    __device__ __forceinline__ void operator()(float &a, float &b)
    {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        if (kWarp || blockDim.x == 32) return;
        float2 *s = slots + 32 * turn;
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
        const float2 v = lane < warps ? s[lane] : make_float2(0.0f, 0.0f);
        a = v.x;
        b = v.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
    }
    __device__ __forceinline__ float operator()(float a)
    {
        float b = 0.0f;
        (*this)(a, b);
        return a;
    }
};

// v becomes (v - mean) / sqrt(var + eps) as the kind has it; elements past the
// row (in_row false) are zero on entry and stay out of the sums.
template <int kNv, int kVec, typename Sum, typename In>
__device__ __forceinline__ void normalize(float (&v)[kNv][kVec], int d, int kind, float eps, Sum &sum, In in_row)
{
    if (kind == CONVROT_NORM_NONE) return;
    float mean = 0.0f;
    if (kind == CONVROT_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < kNv; ++j)
#pragma unroll
            for (int e = 0; e < kVec; ++e) s += v[j][e];
        mean = sum(s) / d;
    }
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < kNv; ++j) {
        if (!in_row(j)) continue;
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            v[j][e] -= mean;
            s = fmaf(v[j][e], v[j][e], s);
        }
    }
    const float inv = 1.0f / sqrtf(sum(s) / d + eps);
#pragma unroll
    for (int j = 0; j < kNv; ++j)
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[j][e] *= inv;
}

constexpr int kRowThreads = 512;  // 128 registers a thread: up to 32 values of a row in each

template <typename T, typename P, int kVec, int kNv, bool kWarp>
__global__ void __launch_bounds__(kRowThreads) gated_norm_kernel(const __grid_constant__ convrot_gated_norm_args a)
{
    __shared__ float2 slots[kWarp ? 1 : 64];
    __shared__ float amax32[kVec == 1 ? 512 : 1];  // largest magnitude of each 32 values (single elements, packing)
    const int tid = kWarp ? threadIdx.x & 31 : threadIdx.x, nt = kWarp ? 32 : blockDim.x;
    const int64_t r = kWarp ? blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (kWarp && r >= a.m) return;
    const int64_t b = r / a.rows_per_batch;
    const int d = static_cast<int>(a.d);
    RowSum<kWarp> sum{slots};
    auto at = [&](int j) { return (tid + j * nt) * kVec; };
    auto in_row = [&](int j) { return at(j) < d; };

    Raw<T, kVec> xr[kNv], yr[kNv];
    const T *x = static_cast<const T *>(a.x) + r * a.ldx, *y = static_cast<const T *>(a.y) + r * a.ldy;
#pragma unroll
    for (int j = 0; j < kNv; ++j)
        if (in_row(j)) {
            xr[j].load_stream(x + at(j));
            if (a.y) yr[j].load_stream(y + at(j));
        }
    float h[kNv][kVec];
    if (a.y) {
#pragma unroll
        for (int j = 0; j < kNv; ++j)
#pragma unroll
            for (int e = 0; e < kVec; ++e) h[j][e] = in_row(j) ? yr[j].get(e) : 0.0f;
        normalize(h, d, a.post, a.eps, sum, in_row);
    }
#pragma unroll
    for (int j = 0; j < kNv; ++j) {
        if (!in_row(j)) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) h[j][e] = 0.0f;
            continue;
        }
        const int i = at(j);
        if (a.y) {
            float p[kVec];
            if (a.post_weight) {
                params<P>(a.post_weight, i, 1.0f, p);
#pragma unroll
                for (int e = 0; e < kVec; ++e) h[j][e] *= p[e];
            }
            if (a.post_bias) {
                params<P>(a.post_bias, i, 0.0f, p);
#pragma unroll
                for (int e = 0; e < kVec; ++e) h[j][e] += p[e];
            }
            params<P>(a.gate, b * a.ldgate + i, 1.0f, p);
#pragma unroll
            for (int e = 0; e < kVec; ++e) h[j][e] = fmaf(a.res_scale, xr[j].get(e), p[e] * h[j][e]);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) h[j][e] = a.res_scale * xr[j].get(e);
        }
        if (a.h) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) xr[j].set(e, h[j][e]);
            xr[j].store(static_cast<T *>(a.h) + r * a.ldh + i);
        }
    }
    if (!a.n && !a.q) return;
    normalize(h, d, a.pre, a.eps, sum, in_row);
#pragma unroll
    for (int j = 0; j < kNv; ++j) {
        if (!in_row(j)) continue;
        const int i = at(j);
        float p[kVec];
        if (a.pre_weight) {
            params<P>(a.pre_weight, i, 1.0f, p);
#pragma unroll
            for (int e = 0; e < kVec; ++e) h[j][e] *= p[e];
        }
        if (a.pre_bias) {
            params<P>(a.pre_bias, i, 0.0f, p);
#pragma unroll
            for (int e = 0; e < kVec; ++e) h[j][e] += p[e];
        }
        if (a.scale) {
            params<P>(a.scale, b * a.ldscale + i, 0.0f, p);
#pragma unroll
            for (int e = 0; e < kVec; ++e) h[j][e] *= 1.0f + p[e];
        }
        if (a.shift) {
            params<P>(a.shift, b * a.ldshift + i, 0.0f, p);
#pragma unroll
            for (int e = 0; e < kVec; ++e) h[j][e] += p[e];
        }
        if (a.n) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) xr[j].set(e, h[j][e]);
            xr[j].store(static_cast<T *>(a.n) + r * a.ldn + i);
        }
    }
    if (!a.q) return;
    // n's pack: 128 / kVec threads hold a block of 128 values (a thread's vectors are blockDim vectors apart, a
    // multiple of 32 of them, so the groups of threads are the same for each); single elements of a block lie in
    // four warps, which meet in shared memory.
    uint8_t *q = static_cast<uint8_t *>(a.q) + r * a.ldq;
    if constexpr (kVec == 1 && kWarp) {
        // one warp, single elements: a block is vectors 4 jb .. 4 jb + 3 of every lane
#pragma unroll
        for (int jb = 0; jb < kNv; jb += 4) {
            float m = 0.0f;
#pragma unroll
            for (int j = jb; j < jb + 4 && j < kNv; ++j) m = fmaxf(m, fabsf(h[j][0]));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            m = fmaxf(m, kFp8AmaxFloor);
            if (jb * 32 < d && tid == 0) a.q_scale[(jb / 4) * a.ld_q_scale + r] = m / kFp8Max;
            const float up = fp8_up(m);
#pragma unroll
            for (int j = jb; j < jb + 4 && j < kNv; ++j)
                if (in_row(j)) q[at(j)] = e4m3(h[j][0] * up);
        }
    } else if constexpr (kVec == 1) {
#pragma unroll
        for (int j = 0; j < kNv; ++j) {
            float m = fabsf(h[j][0]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const int g = at(j) >> 5;
            if ((tid & 31) == 0 && g < 512) amax32[g] = m;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kNv; ++j) {
            if (!in_row(j)) continue;
            const int block = at(j) >> 7, groups = (d + 31) >> 5;
            float m = kFp8AmaxFloor;
            for (int g = 4 * block; g < 4 * block + 4 && g < groups; ++g) m = fmaxf(m, amax32[g]);
            if ((at(j) & 127) == 0) a.q_scale[block * a.ld_q_scale + r] = m / kFp8Max;
            q[at(j)] = e4m3(h[j][0] * fp8_up(m));
        }
    } else {
#pragma unroll
        for (int j = 0; j < kNv; ++j) {
            float m = 0.0f;
#pragma unroll
            for (int e = 0; e < kVec; ++e) m = fmaxf(m, fabsf(h[j][e]));
#pragma unroll
            for (int o = 64 / kVec; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (!in_row(j)) continue;
            m = fmaxf(m, kFp8AmaxFloor);
            if (at(j) % 128 == 0) a.q_scale[(at(j) >> 7) * a.ld_q_scale + r] = m / kFp8Max;
            const float up = fp8_up(m);
            uint32_t w[kVec / 4];
#pragma unroll
            for (int e = 0; e < kVec; e += 4)
                w[e / 4] = e4m3x4(h[j][e] * up, h[j][e + 1] * up, h[j][e + 2] * up, h[j][e + 3] * up);
            if constexpr (kVec == 8)
                *reinterpret_cast<uint2 *>(q + at(j)) = make_uint2(w[0], w[1]);
            else
                *reinterpret_cast<uint32_t *>(q + at(j)) = w[0];
        }
    }
}

// ---------------------------------------------------------------------------
// Gradient. With h^ = (h - mean) inv and y^ likewise, g = dn (1 + scale) w_pre:
//   dH  = dh + inv (g - [mean g] - h^ mean(g h^))        [layer norm only]
//   dx  = res_scale dH
//   gy  = dH gate w_post, dy = inv_y (gy - [mean gy] - y^ mean(gy y^))
// and every gradient of a parameter is one of four sums over the rows of a
// sample, times a factor of the column:
//   s0 = sum dn, s1 = sum dn h^, t0 = sum dH, t1 = sum dH y^
//   dshift = s0, dscale = w_pre s1 + b_pre s0, dgate = w_post t1 + b_post t0
//   dw_pre = sum_b (1 + scale) s1, db_pre = sum_b (1 + scale) s0
//   dw_post = sum_b gate t1, db_post = sum_b gate t0
//
// One kernel does rows and sums: a unit (a block of threads, or a cluster of
// them for wide rows) takes a run of rows of one sample, each thread the same
// eight columns of every row, so the four sums of its columns stay in its
// registers; they leave once per unit as a partial, and small kernels add the
// partials up in a fixed order. Four reads and two writes of a value, each
// tensor moved once. The next row's values are loaded before this one's three
// or four sums around the block, which would otherwise leave HBM idle (16-bit
// types; 32-bit rows are twice as long and have no registers to spare).

constexpr int kGradCols = 8;           // columns a thread
constexpr int kGradThreads = 640;      // of one block: 96 registers a thread
constexpr int kGradWidth = kGradCols * kGradThreads;
constexpr int kSms = 152;

// How rows are split: the same on the host that sizes the workspace and at the launch.
struct GradSplit {
    int cluster;        // blocks that share a row
    int width;          // columns a block
    int threads;
    int64_t batches, chunks, rows_per_chunk;
    GradSplit(int64_t m, int64_t d, int64_t rows)
    {
        cluster = d <= kGradWidth ? 1 : d <= 2 * kGradWidth ? 2 : 4;
        width = static_cast<int>(((d + cluster - 1) / cluster + 31) / 32 * 32);
        threads = ((width + kGradCols - 1) / kGradCols + 31) / 32 * 32;
        batches = (m + rows - 1) / rows;
        // one wave of resident blocks, and no unit without a row
        const int64_t resident = kSms * (threads >= kGradThreads ? 1 : kGradThreads / threads < 24 ? kGradThreads / threads : 24);
        const int64_t longest = rows < m ? rows : m;
        chunks = resident / cluster / batches;
        if (chunks > longest) chunks = longest;
        if (chunks < 1) chunks = 1;
        rows_per_chunk = (longest + chunks - 1) / chunks;
        chunks = (longest + rows_per_chunk - 1) / rows_per_chunk;
    }
    int64_t units() const { return batches * chunks; }
};

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sums over the blocks of a cluster that share a row: each block's sum goes to
// a slot in every peer's shared memory (two sets in turn, as in RowSum).
template <int kCluster>
struct GradSum {
    RowSum<false> block;
    float2 *peers;  // [2][kCluster]
    int turn = 0;
    __device__ __forceinline__ void operator()(float &a, float &b)
    {
        block(a, b);
        if constexpr (kCluster > 1) {
            float2 *mine = peers + turn * kCluster;
            turn ^= 1;
            if (threadIdx.x < kCluster) {
                uint32_t to, at = static_cast<uint32_t>(__cvta_generic_to_shared(mine + cluster_rank()));
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(threadIdx.x));
                asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(a), "f"(b) : "memory");
            }
            cluster_barrier();
            a = b = 0.0f;
#pragma unroll
            for (int i = 0; i < kCluster; ++i) {
                a += mine[i].x;
                b += mine[i].y;
            }
        }
    }
};

template <typename T, typename P, int kVec, int kCluster>
__global__ void __launch_bounds__(kGradThreads, 1)
    norm_grad_kernel(const __grid_constant__ convrot_gated_norm_backward_args a, const __grid_constant__ GradSplit split, float *part)
{
    constexpr int kNv = kGradCols / kVec;
    constexpr bool kAhead = sizeof(T) == 2;
    __shared__ float2 slots[64];
    __shared__ float2 peers[2 * kCluster];
    GradSum<kCluster> sum{{slots}, peers};
    const int64_t unit = blockIdx.x / kCluster;
    const int64_t b = unit / split.chunks, chunk = unit - b * split.chunks;
    const int64_t first = b * a.rows_per_batch + chunk * split.rows_per_chunk;
    int64_t last = first + split.rows_per_chunk;
    if (last > (b + 1) * a.rows_per_batch) last = (b + 1) * a.rows_per_batch;
    if (last > a.m) last = a.m;
    const int c0 = kCluster > 1 ? static_cast<int>(cluster_rank()) * split.width : 0;
    const int end = c0 + split.width < a.d ? c0 + split.width : static_cast<int>(a.d);
    const int d = static_cast<int>(a.d);
    auto at = [&](int j) { return c0 + (static_cast<int>(threadIdx.x) + j * static_cast<int>(blockDim.x)) * kVec; };
    auto inside = [&](int j) { return at(j) < end; };

    struct Row {
        Raw<T, kVec> h[kNv], y[kNv], dh[kNv], dn[kNv];
    };
    auto load = [&](Row &v, int64_t r) {
#pragma unroll
        for (int j = 0; j < kNv; ++j) {
            if (!inside(j)) continue;
            v.h[j].load_stream(static_cast<const T *>(a.h) + r * a.ldh + at(j));
            if (a.y) v.y[j].load_stream(static_cast<const T *>(a.y) + r * a.ldy + at(j));
            if (a.dh) v.dh[j].load_stream(static_cast<const T *>(a.dh) + r * a.lddh + at(j));
            if (a.dn) v.dn[j].load_stream(static_cast<const T *>(a.dn) + r * a.lddn + at(j));
        }
    };

    float s0[kNv][kVec] = {}, s1[kNv][kVec] = {}, t0[kNv][kVec] = {}, t1[kNv][kVec] = {};
    Row row;
    if (kAhead && first < last) load(row, first);
    for (int64_t r = first; r < last; ++r) {
        float h[kNv][kVec], y[kNv][kVec], dh[kNv][kVec];
        Raw<T, kVec> dnr[kNv];
        if (!kAhead) load(row, r);
#pragma unroll
        for (int j = 0; j < kNv; ++j) {
            const bool in = inside(j);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                h[j][e] = in ? row.h[j].get(e) : 0.0f;
                y[j][e] = in && a.y ? row.y[j].get(e) : 0.0f;
                dh[j][e] = in && a.dh ? row.dh[j].get(e) : 0.0f;
            }
            if (in && a.dn) {
                dnr[j] = row.dn[j];
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e) dnr[j].set(e, 0.0f);
            }
        }
        if (kAhead && r + 1 < last) load(row, r + 1);

        // h^ and y^
        float hm = 0.0f, ym = 0.0f;
        if (a.pre == CONVROT_NORM_LAYER || (a.y && a.post == CONVROT_NORM_LAYER)) {
#pragma unroll
            for (int j = 0; j < kNv; ++j)
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    hm += h[j][e];
                    ym += y[j][e];
                }
            sum(hm, ym);
            hm = a.pre == CONVROT_NORM_LAYER ? hm / d : 0.0f;
            ym = a.post == CONVROT_NORM_LAYER ? ym / d : 0.0f;
        }
        float hv = 0.0f, yv = 0.0f;
        const bool stats = a.pre != CONVROT_NORM_NONE || (a.y && a.post != CONVROT_NORM_NONE);
        if (stats) {
#pragma unroll
            for (int j = 0; j < kNv; ++j) {
                if (!inside(j)) continue;
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    h[j][e] -= hm;
                    y[j][e] -= ym;
                    hv = fmaf(h[j][e], h[j][e], hv);
                    yv = fmaf(y[j][e], y[j][e], yv);
                }
            }
            sum(hv, yv);
        }
        const float inv = a.pre != CONVROT_NORM_NONE ? 1.0f / sqrtf(hv / d + a.eps) : 1.0f;
        const float inv_y = a.post != CONVROT_NORM_NONE ? 1.0f / sqrtf(yv / d + a.eps) : 1.0f;

        // dH and the means that pre's gradient subtracts
        float g[kNv][kVec], mg = 0.0f, mgh = 0.0f;
#pragma unroll
        for (int j = 0; j < kNv; ++j) {
            if (!inside(j)) continue;
            float up[kVec], w[kVec];
            params<P>(a.scale, b * a.ldscale + at(j), 0.0f, up);
            params<P>(a.pre_weight, at(j), 1.0f, w);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float dn = dnr[j].get(e);
                h[j][e] *= inv;
                y[j][e] *= inv_y;
                s0[j][e] += dn;
                s1[j][e] = fmaf(dn, h[j][e], s1[j][e]);
                g[j][e] = dn * (1.0f + up[e]) * w[e];
                mg += g[j][e];
                mgh = fmaf(g[j][e], h[j][e], mgh);
            }
        }
        if (a.pre != CONVROT_NORM_NONE) {
            sum(mg, mgh);
            mg = a.pre == CONVROT_NORM_LAYER ? mg / d : 0.0f;
            mgh /= d;
        } else {
            mg = mgh = 0.0f;
        }
        float mq = 0.0f, mqy = 0.0f;
#pragma unroll
        for (int j = 0; j < kNv; ++j) {
            if (!inside(j)) continue;
            Raw<T, kVec> out;
            float gate[kVec], w[kVec];
            if (a.y) {
                params<P>(a.gate, b * a.ldgate + at(j), 1.0f, gate);
                params<P>(a.post_weight, at(j), 1.0f, w);
            }
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                dh[j][e] = fmaf(inv, g[j][e] - mg - h[j][e] * mgh, dh[j][e]);
                out.set(e, a.res_scale * dh[j][e]);
                if (a.y) {
                    t0[j][e] += dh[j][e];
                    t1[j][e] = fmaf(dh[j][e], y[j][e], t1[j][e]);
                    g[j][e] = dh[j][e] * gate[e] * w[e];
                    mq += g[j][e];
                    mqy = fmaf(g[j][e], y[j][e], mqy);
                }
            }
            if (a.dx) out.store_stream(static_cast<T *>(a.dx) + r * a.lddx + at(j));
        }
        if (!a.dy) continue;
        if (a.post != CONVROT_NORM_NONE) {
            sum(mq, mqy);
            mq = a.post == CONVROT_NORM_LAYER ? mq / d : 0.0f;
            mqy /= d;
        } else {
            mq = mqy = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < kNv; ++j) {
            if (!inside(j)) continue;
            Raw<T, kVec> out;
#pragma unroll
            for (int e = 0; e < kVec; ++e) out.set(e, inv_y * (g[j][e] - mq - y[j][e] * mqy));
            out.store_stream(static_cast<T *>(a.dy) + r * a.lddy + at(j));
        }
    }
    float *to = part + unit * 4 * a.d;
#pragma unroll
    for (int j = 0; j < kNv; ++j) {
        if (!inside(j)) continue;
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            to[at(j) + e] = s0[j][e];
            to[a.d + at(j) + e] = s1[j][e];
            to[2 * a.d + at(j) + e] = t0[j][e];
            to[3 * a.d + at(j) + e] = t1[j][e];
        }
    }
    if constexpr (kCluster > 1) cluster_barrier();  // no block leaves while a peer may still write into it
}

// Adds up one sample's partials (block (x, y): 32 columns of sample y; warps
// take chunks in turn) and writes that sample's gradients. What the sample adds
// to the weights' gradients goes to `weights` [batches][4][d], or straight to
// them if there is one sample.
template <typename P>
__global__ void norm_grad_sample_kernel(const __grid_constant__ convrot_gated_norm_backward_args a, int64_t chunks,
                                        const float *part, float *weights)
{
    __shared__ float4 sums[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t i = blockIdx.x * 32ll + lane, b = blockIdx.y;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i < a.d)
#pragma unroll 4
        for (int64_t c = warp; c < chunks; c += warps) {
            const float *p = part + (b * chunks + c) * 4 * a.d + i;
            v.x += p[0];
            v.y += p[a.d];
            v.z += p[2 * a.d];
            v.w += p[3 * a.d];
        }
    sums[warp][lane] = v;
    __syncthreads();
    if (warp != 0 || i >= a.d) return;
    for (int w = 1; w < warps; ++w) {
        const float4 o = sums[w][lane];
        v.x += o.x;
        v.y += o.y;
        v.z += o.z;
        v.w += o.w;
    }
    if (a.dshift) a.dshift[b * a.d + i] = v.x;
    if (a.dscale) a.dscale[b * a.d + i] = param<P>(a.pre_weight, i, 1.0f) * v.y + param<P>(a.pre_bias, i, 0.0f) * v.x;
    if (a.dgate) a.dgate[b * a.d + i] = param<P>(a.post_weight, i, 1.0f) * v.w + param<P>(a.post_bias, i, 0.0f) * v.z;
    const float up = 1.0f + param<P>(a.scale, b * a.ldscale + i, 0.0f), gate = param<P>(a.gate, b * a.ldgate + i, 1.0f);
    const float out[4] = {up * v.y, up * v.x, gate * v.w, gate * v.z};
    float *const to[4] = {a.dpre_weight, a.dpre_bias, a.dpost_weight, a.dpost_bias};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (!to[k]) continue;
        if (!weights)
            to[k][i] = out[k];
        else
            weights[(b * 4 + k) * a.d + i] = out[k];
    }
}

__global__ void norm_grad_weights_kernel(const __grid_constant__ convrot_gated_norm_backward_args a, int64_t batches,
                                         const float *weights)
{
    __shared__ float sums[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, k = blockIdx.y;
    const int64_t i = blockIdx.x * 32ll + lane;
    float *const all[4] = {a.dpre_weight, a.dpre_bias, a.dpost_weight, a.dpost_bias};
    float *to = all[0];
#pragma unroll
    for (int j = 1; j < 4; ++j)
        if (j == k) to = all[j];
    if (!to) return;
    float v = 0.0f;
    if (i < a.d)
#pragma unroll 4
        for (int64_t b = warp; b < batches; b += warps) v += weights[(b * 4 + k) * a.d + i];
    sums[warp][lane] = v;
    __syncthreads();
    if (warp != 0 || i >= a.d) return;
    for (int w = 1; w < warps; ++w) v += sums[w][lane];
    to[i] = v;
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
bool vectors(const void *p, int64_t rows, int64_t ld, int vec, int size)
{
    const int64_t bytes = vec * size < 16 ? vec * size : 16;
    return !p || (aligned_to(p, bytes) && (rows <= 1 || ld * size % bytes == 0));
}

// kNv accesses a thread: a block of threads for each row.
template <typename T, typename P, int kVec, int kNv>
cudaError_t launch_block_rows(const convrot_gated_norm_args &a, cudaStream_t stream)
{
    const int64_t per = (a.d + kVec * kNv - 1) / (kVec * kNv);
    gated_norm_kernel<T, P, kVec, kNv, false>
        <<<static_cast<unsigned>(a.m), static_cast<unsigned>((per + 31) / 32 * 32), 0, stream>>>(a);
    return cudaGetLastError();
}

// A warp for each row, four rows a block.
template <typename T, typename P, int kVec, int kNv>
cudaError_t launch_warp_rows(const convrot_gated_norm_args &a, cudaStream_t stream)
{
    gated_norm_kernel<T, P, kVec, kNv, true><<<static_cast<unsigned>((a.m + 3) / 4), 128, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gated_norm(const convrot_gated_norm_args &a, cudaStream_t stream)
{
    return with_types(a.dtype, a.param_dtype, [&](auto *tt, auto *pp) -> cudaError_t {
        using T = std::remove_pointer_t<decltype(tt)>;
        using P = std::remove_pointer_t<decltype(pp)>;
        constexpr int kVec = 16 / sizeof(T), kT = sizeof(T), kP = sizeof(P);
        const int64_t batches = (a.m + a.rows_per_batch - 1) / a.rows_per_batch;
        const bool wide = a.d % kVec == 0 && vectors(a.x, a.m, a.ldx, kVec, kT) && vectors(a.y, a.m, a.ldy, kVec, kT) &&
                          vectors(a.h, a.m, a.ldh, kVec, kT) && vectors(a.n, a.m, a.ldn, kVec, kT) &&
                          vectors(a.gate, batches, a.ldgate, kVec, kP) && vectors(a.scale, batches, a.ldscale, kVec, kP) &&
                          vectors(a.shift, batches, a.ldshift, kVec, kP) && vectors(a.post_weight, 1, a.d, kVec, kP) &&
                          vectors(a.post_bias, 1, a.d, kVec, kP) && vectors(a.pre_weight, 1, a.d, kVec, kP) &&
                          vectors(a.pre_bias, 1, a.d, kVec, kP);
        if (wide) {
            const int64_t n = a.d / kVec;
            if (n <= 32) return launch_warp_rows<T, P, kVec, 1>(a, stream);
            if (n <= kRowThreads) return launch_block_rows<T, P, kVec, 1>(a, stream);
            if (n <= 2 * kRowThreads) return launch_block_rows<T, P, kVec, 2>(a, stream);
            return launch_block_rows<T, P, kVec, 32 / kVec>(a, stream);
        }
        if (a.d <= 128) return launch_warp_rows<T, P, 1, 4>(a, stream);
        if (a.d <= 4 * kRowThreads) return launch_block_rows<T, P, 1, 4>(a, stream);
        if (a.d <= 12 * kRowThreads) return launch_block_rows<T, P, 1, 12>(a, stream);
        return launch_block_rows<T, P, 1, 32>(a, stream);
    });
}

int64_t gated_norm_backward_work_bytes(int64_t m, int64_t d, int64_t rows_per_batch)
{
    const GradSplit s(m, d, rows_per_batch);
    return (s.units() + (s.batches > 1 ? s.batches : 0)) * 4 * d * static_cast<int64_t>(sizeof(float));
}

template <typename T, typename P, int kVec, int kCluster>
cudaError_t launch_grad(const convrot_gated_norm_backward_args &a, const GradSplit &s, float *part, cudaStream_t stream)
{
    cudaLaunchConfig_t config{};
    config.gridDim = dim3(static_cast<unsigned>(s.units() * kCluster));
    config.blockDim = dim3(s.threads);
    config.stream = stream;
    cudaLaunchAttribute cluster{};
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim = {kCluster, 1, 1};
    config.attrs = &cluster;
    config.numAttrs = kCluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&config, norm_grad_kernel<T, P, kVec, kCluster>, a, s, part);
}

cudaError_t launch_gated_norm_backward(const convrot_gated_norm_backward_args &a, cudaStream_t stream)
{
    return with_types(a.dtype, a.param_dtype, [&](auto *tt, auto *pp) -> cudaError_t {
        using T = std::remove_pointer_t<decltype(tt)>;
        using P = std::remove_pointer_t<decltype(pp)>;
        constexpr int kVec = 16 / sizeof(T), kT = sizeof(T), kP = sizeof(P);
        const GradSplit s(a.m, a.d, a.rows_per_batch);
        float *part = static_cast<float *>(a.work), *weights = part + s.units() * 4 * a.d;
        const bool wide = a.d % kVec == 0 && vectors(a.h, a.m, a.ldh, kVec, kT) && vectors(a.y, a.m, a.ldy, kVec, kT) &&
                          vectors(a.dh, a.m, a.lddh, kVec, kT) && vectors(a.dn, a.m, a.lddn, kVec, kT) &&
                          vectors(a.dx, a.m, a.lddx, kVec, kT) && vectors(a.dy, a.m, a.lddy, kVec, kT) &&
                          vectors(a.gate, s.batches, a.ldgate, kVec, kP) && vectors(a.scale, s.batches, a.ldscale, kVec, kP) &&
                          vectors(a.post_weight, 1, a.d, kVec, kP) && vectors(a.pre_weight, 1, a.d, kVec, kP);
        cudaError_t e;
        if (s.cluster == 1)
            e = wide ? launch_grad<T, P, kVec, 1>(a, s, part, stream) : launch_grad<T, P, 1, 1>(a, s, part, stream);
        else if (s.cluster == 2)
            e = wide ? launch_grad<T, P, kVec, 2>(a, s, part, stream) : launch_grad<T, P, 1, 2>(a, s, part, stream);
        else
            e = wide ? launch_grad<T, P, kVec, 4>(a, s, part, stream) : launch_grad<T, P, 1, 4>(a, s, part, stream);
        if (e != cudaSuccess) return e;
        const bool per_weight = a.dpre_weight || a.dpre_bias || a.dpost_weight || a.dpost_bias;
        if (!per_weight && !a.dshift && !a.dscale && !a.dgate) return cudaSuccess;
        const unsigned tiles = static_cast<unsigned>((a.d + 31) / 32);
        const unsigned warps = static_cast<unsigned>(s.chunks < 32 ? s.chunks : 32);
        for (int64_t b0 = 0; b0 < s.batches; b0 += 65535) {  // (the grid's second dimension has 16 bits)
            convrot_gated_norm_backward_args g = a;
            const int64_t n = s.batches - b0 < 65535 ? s.batches - b0 : 65535;
            if (b0 > 0 || n < s.batches) {
                auto move = [&](float *p) { return p ? p + b0 * a.d : p; };
                g.dshift = move(a.dshift);
                g.dscale = move(a.dscale);
                g.dgate = move(a.dgate);
                if (g.scale) g.scale = static_cast<const P *>(a.scale) + b0 * a.ldscale;
                if (g.gate) g.gate = static_cast<const P *>(a.gate) + b0 * a.ldgate;
            }
            norm_grad_sample_kernel<P><<<dim3(tiles, static_cast<unsigned>(n)), warps * 32, 0, stream>>>(
                g, s.chunks, part + b0 * s.chunks * 4 * a.d, s.batches > 1 ? weights + b0 * 4 * a.d : nullptr);
        }
        if (per_weight && s.batches > 1)
            norm_grad_weights_kernel<<<dim3(tiles, 4), static_cast<unsigned>(s.batches < 32 ? s.batches : 32) * 32, 0,
                                       stream>>>(a, s.batches, weights);
        return cudaGetLastError();
    });
}

}  // namespace convrot
