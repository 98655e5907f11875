// The gradient of the gated norm (include/convrot_block.h). With h^ = (h - mean) inv and y^ likewise, g = dn (1 + scale) w_pre:
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
// columns of every row, so the four sums of its columns stay in its
// registers; they leave once per unit as a partial, and small kernels add the
// partials up in a fixed order. Four reads and two writes of a value, each
// tensor moved once.
//
// Registers for the four sums of a whole row allow one block an SM, so nothing
// hides a trip around the block: the sums of a row are gathered in as few of
// them as possible. g does not depend on pre's statistics, so mean(g h^) is inv
// sum(g h) / d in the same trip as sum h^2; and dH is linear in them, so with
// W = gate w_post, for an RMS post norm
//   sum gy y = inv sum g W y - inv mean(g) sum W y - inv^2 mean(g h^) sum h W y + sum dh W y
// goes along too. One trip for RMS norms, one more for the means of a layer
// norm, and one more if post is one. Measured at 8190 x 5120 in bf16 with RMS
// norms: 142 us with the sums, 3.5 TB/s (52 % of a copy); issue slots are 39 %
// busy, the rest is the latency of the trips and of spilled registers: ten warps
// put three on two of an SM's four schedulers, which leaves a thread 168, and
// every form of the kernel spills (bytes stored a thread: 244 here, 256 in
// clusters, 324 to 380 in f32, 352 to 748 in unaligned rows). Any statement more
// in the loop costs (3 to 6 % for one select a value). Clusters of two blocks
// with two of them an SM, for two rows under way: 190 us.
#include "block_norm.cuh"

namespace convrot {
namespace {

// Columns a thread: 16 spread a row's trip around the block over twice the
// values of 8 (146 against 166 us; M8190 D5120 in bf16, RMS norms).
constexpr int kGradCols = 16;
constexpr int kGradThreads = 320;      // of one block: 168 registers a thread
constexpr int kGradWidth = kGradCols * kGradThreads;
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
        // one wave of resident blocks, and no unit without a row (counted by threads: of blocks of 128 to 288 threads
        // registers and shared memory would allow one or two an SM more)
        const int64_t resident = kSms * (threads >= kGradThreads ? 1 : kGradThreads / threads);
        const int64_t longest = rows < m ? rows : m;
        chunks = resident / cluster / batches;
        if (chunks > longest) chunks = longest;
        if (chunks < 1) chunks = 1;
        rows_per_chunk = (longest + chunks - 1) / chunks;
        chunks = (longest + rows_per_chunk - 1) / rows_per_chunk;
    }
    int64_t units() const { return batches * chunks; }
};

// Eight sums at once over the threads that share a row: within a warp each of
// three steps halves the values that a lane carries, a block's warps meet in
// shared memory (two buffers in turn: one barrier a sum is enough), and a cluster's blocks
// write theirs into every peer's.
template <int kCluster>
struct GradSum {
    float *slots;  // [2][8][36]: value, warp (36 keeps the 32 lanes' reads apart)
    float *peers;  // [2][kCluster][8]
    int turn = 0;
    __device__ __forceinline__ void operator()(float (&v)[8])
    {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int n = 4, o = 16; n > 0; n >>= 1, o >>= 1) {
            const bool upper = lane & o;
#pragma unroll
            for (int i = 0; i < n; ++i)
                v[i] = (upper ? v[i + n] : v[i]) + __shfl_xor_sync(0xffffffffu, upper ? v[i] : v[i + n], o);
        }
        float s = v[0];
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        const int which = lane >> 2, part = lane & 3;  // the value that this lane ended up with
        if (blockDim.x > 32) {
            float *to = slots + (turn * 8 + which) * 36;
            if (part == 0) to[threadIdx.x >> 5] = s;
            __syncthreads();
            const int warps = blockDim.x >> 5;
            s = 0.0f;
            for (int w = part; w < warps; w += 4) s += to[w];
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            s += __shfl_xor_sync(0xffffffffu, s, 1);
        }
        if constexpr (kCluster > 1) {
            float *mine = peers + turn * kCluster * 8;
            if (threadIdx.x < 32) {  // a value's four lanes write it to up to four blocks
                const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(mine + cluster_rank() * 8 + which));
                uint32_t to;
                if (part < kCluster) {
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(part));
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(s) : "memory");
                }
            }
            cluster_sync();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = 0.0f;
#pragma unroll
                for (int c = 0; c < kCluster; ++c) v[i] += mine[c * 8 + i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __shfl_sync(0xffffffffu, s, 4 * i);
        }
        turn ^= 1;
    }
};

// Rows of the ring: 4 tensors of 32 bytes a thread and row (64 for 32-bit
// types), 160 KB for the widest block.
template <typename T>
constexpr int grad_stages()
{
    return sizeof(T) == 2 ? 4 : 2;
}

template <typename T, typename P, int kVec, int kCluster>
__global__ void __launch_bounds__(kGradThreads, 1)
    norm_grad_kernel(const __grid_constant__ convrot_gated_norm_backward_args a, const __grid_constant__ GradSplit split, float *part)
{
    // kGradCols columns a thread, in kNv pieces of kVec, and in pairs for the packed arithmetic. Pieces of 16 or 4
    // bytes come through a ring of rows in shared memory that each thread fills for itself, 2-byte ones directly.
    constexpr int kNv = kGradCols / kVec, kPairs = kGradCols / 2, kStages = grad_stages<T>();
    constexpr int kPiece = kVec * static_cast<int>(sizeof(T));
    constexpr bool kRing = kPiece >= 4;
    extern __shared__ uint4 ring[];  // [kStages][h, y, dh, dn][kNv][blockDim] pieces
    __shared__ float slots[2 * 8 * 36];
    __shared__ float peers[2 * kCluster * 8];
    GradSum<kCluster> sum{slots, peers};
    // A peer's shared memory may be written once it is known to run (the first sum does): met under the wait below.
    if constexpr (kCluster > 1) cluster_sync();
    after_previous();
    const int64_t unit = blockIdx.x / kCluster;
    const int64_t b = unit / split.chunks, chunk = unit - b * split.chunks;
    const int64_t first = b * a.rows_per_batch + chunk * split.rows_per_chunk;
    int64_t last = first + split.rows_per_chunk;
    if (last > (b + 1) * a.rows_per_batch) last = (b + 1) * a.rows_per_batch;
    if (last > a.m) last = a.m;
    const int count = last > first ? static_cast<int>(last - first) : 0;
    const int c0 = kCluster > 1 ? static_cast<int>(cluster_rank()) * split.width : 0;
    const int end = c0 + split.width < a.d ? c0 + split.width : static_cast<int>(a.d);
    const float inv_d = 1.0f / static_cast<float>(a.d);
    const int nt = blockDim.x;
    auto at = [&](int j) { return c0 + (static_cast<int>(threadIdx.x) + j * nt) * kVec; };
    auto inside = [&](int j) { return at(j) < end; };

    const T *in[4] = {static_cast<const T *>(a.h) + first * a.ldh + at(0),
                      a.y ? static_cast<const T *>(a.y) + first * a.ldy + at(0) : nullptr,
                      a.dh ? static_cast<const T *>(a.dh) + first * a.lddh + at(0) : nullptr,
                      a.dn ? static_cast<const T *>(a.dn) + first * a.lddn + at(0) : nullptr};
    auto advance = [&]() {
        in[0] += a.ldh;
        if (in[1]) in[1] += a.ldy;
        if (in[2]) in[2] += a.lddh;
        if (in[3]) in[3] += a.lddn;
    };
    const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + threadIdx.x * kPiece;
    const uint32_t piece = nt * kPiece;
    auto fetch = [&](int stage) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (in[k])
#pragma unroll
                for (int j = 0; j < kNv; ++j)
                    copy_piece<kRing ? kPiece : 4>(mine + ((stage * 4 + k) * kNv + j) * piece, in[k] + (inside(j) ? j * nt * kVec : -at(0)),
                                                   inside(j) ? kPiece : 0);
        advance();
    };
    int stage = 0, ahead = kStages - 1;
    // this thread's values of tensor k in the current row, zero where there are none
    auto get = [&](int k, F2 (&v)[kPairs]) {
        if constexpr (kRing) {
#pragma unroll
            for (int j = 0; j < kNv; ++j) {
                Raw<T, kVec> raw{};
                if (in[k]) load_shared(mine + ((stage * 4 + k) * kNv + j) * piece, raw.bits[0]);
                if constexpr (kVec > 1) {
                    raw.unpack(v + j * kVec / 2);
                } else {
                    if (j % 2) v[j / 2] = F2(v[j / 2].lo(), raw.value());
                    else v[j / 2] = F2(raw.value(), 0.0f);
                }
            }
        } else {
            // all loads first, from the row's start where there is no such column
            T raw[2 * kPairs];
            if (in[k]) {
#pragma unroll
                for (int j = 0; j < kNv; ++j) raw[j] = in[k][inside(j) ? j * nt : -at(0)];
            } else {
#pragma unroll
                for (int j = 0; j < kNv; ++j) raw[j] = from_f32<T>(0.0f);
            }
#pragma unroll
            for (int e = 0; e < kPairs; ++e)
                v[e] = F2(inside(2 * e) ? to_f32(raw[2 * e]) : 0.0f, inside(2 * e + 1) ? to_f32(raw[2 * e + 1]) : 0.0f);
        }
    };
    auto put = [&](T *p, const F2 (&v)[kPairs]) {
        if constexpr (kRing) {
#pragma unroll
            for (int j = 0; j < kNv; ++j) {
                if (!inside(j)) continue;
                Raw<T, kVec> raw;
                if constexpr (kVec > 1)
                    raw.pack(v + j * kVec / 2);
                else
                    raw.set(j % 2 ? v[j / 2].hi() : v[j / 2].lo());
                raw.store_stream(p + j * nt * kVec);
            }
        } else {
#pragma unroll
            for (int e = 0; e < kPairs; ++e) {
                if (inside(2 * e)) p[2 * e * nt] = from_f32<T>(v[e].lo());
                if (inside(2 * e + 1)) p[(2 * e + 1) * nt] = from_f32<T>(v[e].hi());
            }
        }
    };
    // the columns' factors, the same for the whole run: (1 + scale) w_pre and gate w_post
    auto column = [&](const void *p, int64_t offset, int i, float otherwise) {
        const int j = i / kVec;
        return inside(j) ? param<P>(p, offset + at(j) + i % kVec, otherwise) : 0.0f;
    };
    F2 w_pre[kPairs], w_post[kPairs], s0[kPairs], s1[kPairs], t0[kPairs], t1[kPairs];
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
        float u[2], v[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            u[i] = (1.0f + column(a.scale, b * a.ldscale, 2 * e + i, 0.0f)) * column(a.pre_weight, 0, 2 * e + i, 1.0f);
            v[i] = column(a.gate, b * a.ldgate, 2 * e + i, 1.0f) * column(a.post_weight, 0, 2 * e + i, 1.0f);
        }
        w_pre[e] = F2(u[0], u[1]);
        w_post[e] = F2(v[0], v[1]);
        s0[e] = s1[e] = t0[e] = t1[e] = F2(0.0f);
    }
    T *dx = a.dx ? static_cast<T *>(a.dx) + first * a.lddx + at(0) : nullptr;
    T *dy = a.dy ? static_cast<T *>(a.dy) + first * a.lddy + at(0) : nullptr;
    const bool y_layer = a.y && a.post == CONVROT_NORM_LAYER;
    const bool trip = a.pre != CONVROT_NORM_NONE || (a.y && a.post != CONVROT_NORM_NONE);

    if constexpr (kRing) {
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) {
            if (s < count) fetch(s);
            copy_commit();
        }
    }
    for (int r = 0; r < count; ++r) {
        if constexpr (kRing) {
            if (r + kStages - 1 < count) fetch(ahead);
            copy_commit();
            if (++ahead == kStages) ahead = 0;
            copy_wait<kStages - 1>();
        }
        F2 h[kPairs], y[kPairs], g[kPairs], v[kPairs];
        float m[8];
        get(0, h);
        get(1, y);
        if (a.pre == CONVROT_NORM_LAYER || y_layer) {
            F2 hs(0.0f), ys(0.0f);
#pragma unroll
            for (int e = 0; e < kPairs; ++e) {
                hs = hs + h[e];
                ys = ys + y[e];
            }
            m[0] = hs.sum();
            m[1] = ys.sum();
            m[2] = m[3] = m[4] = m[5] = m[6] = m[7] = 0.0f;
            sum(m);
            const float hm = a.pre == CONVROT_NORM_LAYER ? -m[0] * inv_d : 0.0f, ym = y_layer ? -m[1] * inv_d : 0.0f;
#pragma unroll
            for (int e = 0; e < kPairs; ++e) {
                const bool lo = inside(2 * e / kVec), hi = inside((2 * e + 1) / kVec);
                h[e] = h[e] + F2(lo ? hm : 0.0f, hi ? hm : 0.0f);
                y[e] = y[e] + F2(lo ? ym : 0.0f, hi ? ym : 0.0f);
            }
        }
        get(3, g);
        float inv = 1.0f, inv_y = 1.0f, mg = 0.0f, mgh = 0.0f, mqy = 0.0f;
        if (trip) {
            F2 hh(0.0f), yy(0.0f), gs(0.0f), gh(0.0f), gwy(0.0f), wys(0.0f), hwy(0.0f), dwy(0.0f);
            get(2, v);
#pragma unroll
            for (int e = 0; e < kPairs; ++e) {
                const F2 u = g[e] * w_pre[e];
                hh = fma2(h[e], h[e], hh);
                gs = gs + u;
                gh = fma2(u, h[e], gh);
                const F2 wy = w_post[e] * y[e];
                yy = fma2(y[e], y[e], yy);
                gwy = fma2(u, wy, gwy);
                wys = wys + wy;
                hwy = fma2(h[e], wy, hwy);
                dwy = fma2(v[e], wy, dwy);
            }
            m[0] = hh.sum();
            m[1] = yy.sum();
            m[2] = gs.sum();
            m[3] = gh.sum();
            m[4] = gwy.sum();
            m[5] = wys.sum();
            m[6] = hwy.sum();
            m[7] = dwy.sum();
            sum(m);
            if (a.pre != CONVROT_NORM_NONE) {
                inv = rsqrtf(fmaf(m[0], inv_d, a.eps));
                mgh = -m[3] * inv * inv_d;
                if (a.pre == CONVROT_NORM_LAYER) mg = -m[2] * inv_d;
            }
            if (a.post != CONVROT_NORM_NONE) {
                inv_y = rsqrtf(fmaf(m[1], inv_d, a.eps));
                mqy = -(inv * (m[4] + mg * m[5] + inv * mgh * m[6]) + m[7]) * inv_y * inv_d;
            }
        }
        get(2, v);
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
            h[e] = h[e] * F2(inv);
            y[e] = y[e] * F2(inv_y);
            s0[e] = s0[e] + g[e];
            s1[e] = fma2(g[e], h[e], s1[e]);
            g[e] = fma2(g[e], w_pre[e], F2(mg));
            v[e] = fma2(F2(inv), fma2(h[e], F2(mgh), g[e]), v[e]);  // dH
            g[e] = v[e] * F2(a.res_scale);
        }
        if (dx) {
            put(dx, g);
            dx += a.lddx;
        }
        if (a.y) {
            F2 gs(0.0f), gy(0.0f);
#pragma unroll
            for (int e = 0; e < kPairs; ++e) {
                t0[e] = t0[e] + v[e];
                t1[e] = fma2(v[e], y[e], t1[e]);
                g[e] = v[e] * w_post[e];
            }
            if (dy) {
                float mq = 0.0f;
                if (y_layer) {
#pragma unroll
                    for (int e = 0; e < kPairs; ++e) {
                        gs = gs + g[e];
                        gy = fma2(g[e], y[e], gy);
                    }
                    m[0] = gs.sum();
                    m[1] = gy.sum();
                    m[2] = m[3] = m[4] = m[5] = m[6] = m[7] = 0.0f;
                    sum(m);
                    mq = -m[0] * inv_d;
                    mqy = -m[1] * inv_d;
                }
#pragma unroll
                for (int e = 0; e < kPairs; ++e) g[e] = F2(inv_y) * fma2(y[e], F2(mqy), g[e] + F2(mq));
                put(dy, g);
                dy += a.lddy;
            }
        }
        if constexpr (kRing) {
            if (++stage == kStages) stage = 0;
        } else {
            advance();
        }
    }
    let_next_start();
    float *to = part + unit * 4 * a.d;
    auto put_sums = [&](float *p, const F2 (&v)[kPairs]) {
#pragma unroll
        for (int j = 0; j < kNv; ++j) {
            if (!inside(j)) continue;
            if constexpr (kVec > 1) {
                Raw<float, kVec> raw;
                raw.pack(v + j * kVec / 2);
                raw.store(p + at(j));
            } else {
                p[at(j)] = j % 2 ? v[j / 2].hi() : v[j / 2].lo();
            }
        }
    };
    put_sums(to, s0);
    put_sums(to + a.d, s1);
    if (a.y) {
        put_sums(to + 2 * a.d, t0);
        put_sums(to + 3 * a.d, t1);
    }
    if constexpr (kCluster > 1) cluster_sync();  // no block leaves while a peer may still write into it
}

// Warps of a block that adds partials up: 8 where that gives every SM two blocks, up to 32 where few columns and
// samples leave a warp many partials to go through.
constexpr int kSumWarps = 32;
int sum_warps(int64_t blocks, int64_t partials)
{
    const int64_t most = blocks >= 2 * kSms ? 8 : kSumWarps;
    return static_cast<int>(partials < most ? partials : most);
}

constexpr int64_t kFewPartials = 128;  // that one block adds up for all samples, instead of a launch more

// Adds up a sample's partials (block (x, y): 32 columns of sample y; warps take
// chunks in turn) and writes that sample's gradients. What the sample adds to
// the weights' gradients goes to `weights` [batches][4][d]; without that (few
// partials) block x goes through the samples in turn and writes the sums itself.
template <typename P>
__global__ void norm_grad_sample_kernel(const __grid_constant__ convrot_gated_norm_backward_args a, int64_t chunks, int64_t samples,
                                        const float *part, float *weights)
{
    __shared__ float4 sums[kSumWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t i = blockIdx.x * 32ll + lane;
    const bool in = i < a.d;
    after_previous();  // the partials are another kernel's
    let_next_start();
    float *const to[4] = {a.dpre_weight, a.dpre_bias, a.dpost_weight, a.dpost_bias};
    float total[4] = {};
    const int64_t first = weights ? blockIdx.y : 0, last = weights ? first + 1 : samples;
    for (int64_t b = first; b < last; ++b) {
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (in)
#pragma unroll 4
            for (int64_t c = warp; c < chunks; c += warps) {
                const float *p = part + (b * chunks + c) * 4 * a.d + i;
                v.x += p[0];
                v.y += p[a.d];
                if (a.y) {
                    v.z += p[2 * a.d];
                    v.w += p[3 * a.d];
                }
            }
        if (b > first) __syncthreads();  // the sums before have been read
        sums[warp][lane] = v;
        __syncthreads();
        if (warp != 0 || !in) continue;
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
        const float adds[4] = {up * v.y, up * v.x, gate * v.w, gate * v.z};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            total[k] += adds[k];
            if (weights && to[k]) weights[(b * 4 + k) * a.d + i] = adds[k];
        }
    }
    if (weights || warp != 0 || !in) return;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (to[k]) to[k][i] = total[k];
}

__global__ void norm_grad_weights_kernel(const __grid_constant__ convrot_gated_norm_backward_args a, int64_t batches,
                                         const float *weights)
{
    __shared__ float sums[kSumWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, k = blockIdx.y;
    const int64_t i = blockIdx.x * 32ll + lane;
    float *const all[4] = {a.dpre_weight, a.dpre_bias, a.dpost_weight, a.dpost_bias};
    float *to = all[0];
#pragma unroll
    for (int j = 1; j < 4; ++j)
        if (j == k) to = all[j];
    after_previous();
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

}  // namespace

int64_t gated_norm_backward_work_bytes(int64_t m, int64_t d, int64_t rows_per_batch)
{
    const GradSplit s(m, d, rows_per_batch);
    return (s.units() + (s.batches > 1 ? s.batches : 0)) * 4 * d * static_cast<int64_t>(sizeof(float));
}

template <typename T, typename P, int kVec, int kCluster>
struct grad_tag;

template <typename T, typename P, int kVec, int kCluster>
cudaError_t launch_grad(const convrot_gated_norm_backward_args &a, const GradSplit &s, float *part, cudaStream_t stream)
{
    const int bytes = kVec * sizeof(T) < 4 ? 0 : grad_stages<T>() * 4 * kGradCols * static_cast<int>(sizeof(T)) * s.threads;
    auto kernel = norm_grad_kernel<T, P, kVec, kCluster>;
    const cudaError_t e = allow_shared<grad_tag<T, P, kVec, kCluster>>(kernel);
    if (e != cudaSuccess) return e;
    return launch_after(kernel, dim3(static_cast<unsigned>(s.units() * kCluster)), static_cast<unsigned>(s.threads), bytes, stream,
                        kCluster, a, s, part);
}

cudaError_t launch_gated_norm_backward(const convrot_gated_norm_backward_args &a, cudaStream_t stream)
{
    return with_types(a.dtype, a.param_dtype, [&](auto *tt, auto *pp) -> cudaError_t {
        using T = std::remove_pointer_t<decltype(tt)>;
        using P = std::remove_pointer_t<decltype(pp)>;
        constexpr int kVec = 16 / sizeof(T), kT = sizeof(T);
        const GradSplit s(a.m, a.d, a.rows_per_batch);
        float *part = static_cast<float *>(a.work), *weights = part + s.units() * 4 * a.d;
        // the rows' pieces: 16 bytes, 4, or single 16-bit elements
        auto pieces = [&](int vec) {
            return a.d % vec == 0 && vectors(a.h, a.m, a.ldh, vec, kT) && vectors(a.y, a.m, a.ldy, vec, kT) &&
                   vectors(a.dh, a.m, a.lddh, vec, kT) && vectors(a.dn, a.m, a.lddn, vec, kT) &&
                   vectors(a.dx, a.m, a.lddx, vec, kT) && vectors(a.dy, a.m, a.lddy, vec, kT);
        };
        auto launch = [&](auto vec) {
            constexpr int kV = decltype(vec)::value;
            if (s.cluster == 1) return launch_grad<T, P, kV, 1>(a, s, part, stream);
            if (s.cluster == 2) return launch_grad<T, P, kV, 2>(a, s, part, stream);
            return launch_grad<T, P, kV, 4>(a, s, part, stream);
        };
        constexpr int kSmall = 4 / kT;
        cudaError_t e;
        if (pieces(kVec))
            e = launch(std::integral_constant<int, kVec>{});
        else if (pieces(kSmall))
            e = launch(std::integral_constant<int, kSmall>{});
        else
            e = launch(std::integral_constant<int, 1>{});
        if (e != cudaSuccess) return e;
        const bool per_weight = a.dpre_weight || a.dpre_bias || a.dpost_weight || a.dpost_bias;
        if (!per_weight && !a.dshift && !a.dscale && !a.dgate) return cudaSuccess;
        const unsigned tiles = static_cast<unsigned>((a.d + 31) / 32);
        if (s.batches == 1 || s.units() <= kFewPartials)
            return launch_after(norm_grad_sample_kernel<P>, dim3(tiles), static_cast<unsigned>(sum_warps(tiles, s.chunks)) * 32, 0, stream,
                                1, a, s.chunks, s.batches, static_cast<const float *>(part), static_cast<float *>(nullptr));
        const unsigned warps = static_cast<unsigned>(sum_warps(tiles * s.batches, s.chunks));
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
            e = launch_after(norm_grad_sample_kernel<P>, dim3(tiles, static_cast<unsigned>(n)), warps * 32, 0, stream, 1, g, s.chunks, n,
                             static_cast<const float *>(part + b0 * s.chunks * 4 * a.d), weights + b0 * 4 * a.d);
            if (e != cudaSuccess) return e;
        }
        if (per_weight)
            return launch_after(norm_grad_weights_kernel, dim3(tiles, 4),
                                static_cast<unsigned>(sum_warps(4 * tiles, s.batches)) * 32, 0, stream, 1, a, s.batches,
                                static_cast<const float *>(weights));
        return cudaSuccess;
    });
}

}  // namespace convrot
