// The gated norm (include/convrot_block.h).
//
//   u = post(y), h = res_scale x + gate u, n = pre(h) (1 + scale) + shift
//
// Forward: two reads and two writes of a value for about ten operations on it,
// so HBM is the bound. A row stays in the registers of one block of threads
// (of one warp, where 32 pieces hold it) from its load to its store: every
// tensor is moved once, in 16-byte accesses where all addresses allow it and in
// coalesced single elements otherwise. The statistics are two-pass (mean, then
// squares about it), which costs one more trip around the block than a
// one-pass sum of squares and keeps layer norms of rows with a large mean.
// Measured on one GB300, 32760 x 5120 in bf16 with RMS norms on both sides: 222
// us, 6.0 TB/s, 89 % of a measured copy (216 us with parameters in f32); 4097 x
// 1155 in f16, single elements: 10.7 us, 2.7 TB/s, bound by instructions. One
// block a row, without the runs of rows below, takes 316 and 24 us; its form for
// single elements of rows above 8192 spills 656 to 760 bytes a thread.
#include <cfloat>

#include "block_norm.cuh"

namespace convrot {
namespace {

// Sums over the threads that share a row: a warp, or a block through shared
// memory. Two buffers in turn: a thread that is one sum ahead writes the other
// one, and it cannot be two ahead, so one barrier a sum is enough.
template <bool kWarp>
struct RowSum {
    float2 *slots;  // [2][32]
    int turn = 0;
    // Two sums at once: the first step leaves a's on one half of the warp and
    // b's on the other, the next four serve both.
    static __device__ __forceinline__ void warp_sum(float &a, float &b)
    {
        const bool upper = threadIdx.x & 16;
        float v = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        a = __shfl_sync(0xffffffffu, v, 0);
        b = __shfl_sync(0xffffffffu, v, 16);
    }
    __device__ __forceinline__ void operator()(float &a, float &b)
    {
        warp_sum(a, b);
        if (kWarp || blockDim.x == 32) return;
        float2 *s = slots + 32 * turn;
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
        const float2 v = lane < warps ? s[lane] : make_float2(0.0f, 0.0f);
        a = v.x;
        b = v.y;
        warp_sum(a, b);
    }
    __device__ __forceinline__ float operator()(float a)
    {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        if (kWarp || blockDim.x == 32) return a;
        float2 *s = slots + 32 * turn;
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5].x = a;
        __syncthreads();
        const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
        a = lane < warps ? s[lane].x : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
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
        mean = sum(s) * (1.0f / d);
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
    const float inv = rsqrtf(fmaf(sum(s), 1.0f / d, eps));
#pragma unroll
    for (int j = 0; j < kNv; ++j)
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[j][e] *= inv;
}

// Codes and scales of a row of n in 16-byte pieces: 128 / kVec threads hold a
// block of 128 values (a thread's pieces are nt apart, a multiple of 32, so the
// same threads share each block). Values past the row are zero.
template <int kVec, int kNv>
__device__ __forceinline__ void pack_row(const convrot_gated_norm_args &a, int64_t r, int d, int tid, int nt, const float (&h)[kNv][kVec])
{
    uint8_t *q = static_cast<uint8_t *>(a.q) + r * a.ldq;
    auto at = [&](int j) { return (tid + j * nt) * kVec; };
#pragma unroll
    for (int j = 0; j < kNv; ++j) {
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < kVec; ++e) m = fmaxf(m, fabsf(h[j][e]));
#pragma unroll
        for (int o = 64 / kVec; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (at(j) >= d) continue;
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

// Rows of a sample in 32 bits (row numbers have 31).
__device__ __forceinline__ uint32_t sample_rows(int64_t rows) { return rows < 0x7fffffff ? static_cast<uint32_t>(rows) : 0x7fffffffu; }

constexpr int kRingThreads = 640;  // 96 registers a thread, so that 640 threads share an SM
constexpr int kRingStages = 3;
constexpr int kRowThreads = 512;  // 128 registers a thread: up to 32 values of a row in each

template <typename T, typename P, int kVec, int kNv, bool kWarp>
__global__ void __launch_bounds__(kRowThreads) gated_norm_kernel(const __grid_constant__ convrot_gated_norm_args a)
{
    __shared__ float2 slots[kWarp ? 1 : 64];
    __shared__ float amax32[kVec == 1 ? 512 : 1];  // largest magnitude of each 32 values (single elements, packing)
    after_previous();
    let_next_start();
    const int tid = kWarp ? threadIdx.x & 31 : threadIdx.x, nt = kWarp ? 32 : blockDim.x;
    const int64_t r = kWarp ? blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (kWarp && r >= a.m) return;
    const int64_t b = static_cast<uint32_t>(r) / sample_rows(a.rows_per_batch);
    const int d = static_cast<int>(a.d);
    RowSum<kWarp> sum{slots};
    auto at = [&](int j) { return (tid + j * nt) * kVec; };
    auto in_row = [&](int j) { return at(j) < d; };

    Raw<T, kVec> xr[kNv], yr[kNv];
    const T *x = static_cast<const T *>(a.x) + r * a.ldx, *y = static_cast<const T *>(a.y) + r * a.ldy;
    // (a piece past the row loads the row's start: loads behind branches would wait for one another)
    auto clamped = [&](int j) { return in_row(j) ? at(j) : 0; };
#pragma unroll
    for (int j = 0; j < kNv; ++j) xr[j].load_stream(x + clamped(j));
    if (a.y) {
#pragma unroll
        for (int j = 0; j < kNv; ++j) yr[j].load_stream(y + clamped(j));
    }
    float h[kNv][kVec];
    if (a.y) {
#pragma unroll
        for (int j = 0; j < kNv; ++j) {
            if (in_row(j)) {
                yr[j].unpack(h[j]);
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e) h[j][e] = 0.0f;
            }
        }
        normalize(h, d, a.post, a.eps, sum, in_row);
    }
    // h[j][e] = f(h[j][e], p[column]) for a vector of columns, if there is one
    auto apply = [&](const void *p, int64_t offset, auto f) {
        if (!p) return;
        float v[kNv][kVec];
#pragma unroll
        for (int j = 0; j < kNv; ++j) params<P>(p, offset + clamped(j), 0.0f, v[j]);
#pragma unroll
        for (int j = 0; j < kNv; ++j)
#pragma unroll
            for (int e = 0; e < kVec; ++e) h[j][e] = f(h[j][e], v[j][e]);
    };
    auto times = [](float v, float p) { return v * p; };
    auto plus = [](float v, float p) { return v + p; };
    if (a.y) {
        apply(a.post_weight, 0, times);
        apply(a.post_bias, 0, plus);
        apply(a.gate, b * a.ldgate, times);
    }
#pragma unroll
    for (int j = 0; j < kNv; ++j) {
        float xv[kVec];
        xr[j].unpack(xv);
#pragma unroll
        for (int e = 0; e < kVec; ++e) h[j][e] = !in_row(j) ? 0.0f : a.y ? fmaf(a.res_scale, xv[e], h[j][e]) : a.res_scale * xv[e];
        if (a.h && in_row(j)) {
            xr[j].pack(h[j]);
            xr[j].store(static_cast<T *>(a.h) + r * a.ldh + at(j));
        }
    }
    if (!a.n && !a.q) return;
    normalize(h, d, a.pre, a.eps, sum, in_row);
    apply(a.pre_weight, 0, times);
    apply(a.pre_bias, 0, plus);
    apply(a.scale, b * a.ldscale, [](float v, float p) { return fmaf(v, p, v); });
    apply(a.shift, b * a.ldshift, plus);
#pragma unroll
    for (int j = 0; j < kNv; ++j) {
        if (!in_row(j)) {  // stays out of the packed block's maximum
#pragma unroll
            for (int e = 0; e < kVec; ++e) h[j][e] = 0.0f;
        } else if (a.n) {
            xr[j].pack(h[j]);
            xr[j].store(static_cast<T *>(a.n) + r * a.ldn + at(j));
        }
    }
    if (!a.q) return;
    // n's pack; single elements of a block of 128 lie in four warps, which meet in shared memory
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
        pack_row<kVec, kNv>(a, r, d, tid, nt, h);
    }
}

// The same for many rows: each block takes a run of them. Per row the
// instructions count as much as the bytes (44 a value are what HBM's rate
// leaves), so everything that a sample's rows share is prepared once, in
// registers: gate w_post, (1 + scale) w_pre and (1 + scale) b_pre + shift;
// values past the row are zeros and need no branch.
// kVec > 0: each thread copies its own pieces (16 or 4 bytes) of the next rows
// into its own places in shared memory (cp.async), kStages - 1 rows ahead. What a thread
// copied it reads back itself, so the ring needs no barrier, and HBM stays busy
// through the sums around the block. Otherwise single elements, kThreads apart,
// the next row's loaded into registers before this one's sums.
template <typename T, typename P, int kNv, int kVec, int kThreads, bool kBranch>
__global__ void __launch_bounds__(kRingThreads, 1) gated_norm_ring_kernel(const __grid_constant__ convrot_gated_norm_args a, int32_t rows)
{
    constexpr int kPiece = kVec * static_cast<int>(sizeof(T));
    constexpr bool kWide = kPiece >= 4;  // through shared memory
    constexpr int kStages = kRingStages, kPieces = kNv * (kBranch ? 2 : 1), kValues = kNv * kVec, kPairs = kValues / 2;
    extern __shared__ uint4 ring[];  // kWide: [kStages][x, y][kNv][blockDim] pieces
    __shared__ float2 slots[64];
    after_previous();
    let_next_start();
    const int nt = kThreads ? kThreads : blockDim.x, d = static_cast<int>(a.d);
    const float inv_d = 1.0f / d;
    RowSum<false> sum{slots};
    const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + threadIdx.x * kPiece;
    const uint32_t step = nt * kPiece, stage_bytes = step * kPieces;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * rows;
    const int count = static_cast<int>(a.m - first < rows ? a.m - first : rows);
    const int pitch = nt * kVec, col = static_cast<int>(threadIdx.x) * kVec;  // piece j: columns col + j pitch on
    bool inside[kNv];
#pragma unroll
    for (int j = 0; j < kNv; ++j) inside[j] = col + j * pitch < d;
    const T *x = static_cast<const T *>(a.x) + first * a.ldx, *y = static_cast<const T *>(a.y) + first * a.ldy;
    T *h_out = static_cast<T *>(a.h) + first * a.ldh + col, *n_out = static_cast<T *>(a.n) + first * a.ldn + col;
    T ahead_x[kWide ? 1 : kNv], ahead_y[kWide || !kBranch ? 1 : kNv];
    auto fetch = [&](uint32_t to) {
#pragma unroll
        for (int j = 0; j < kNv; ++j) {
            if constexpr (kWide) {
                // (a piece past the row reads nothing, but its address stays inside)
                const int at = inside[j] ? col + j * pitch : 0;
                const uint32_t bytes = inside[j] ? kPiece : 0;
                copy_piece<kPiece>(to + j * step, x + at, bytes);
                if constexpr (kBranch) copy_piece<kPiece>(to + (kNv + j) * step, y + at, bytes);
            } else {
                ahead_x[j] = inside[j] ? x[col + j * pitch] : from_f32<T>(0.0f);
                if constexpr (kBranch) ahead_y[j] = inside[j] ? y[col + j * pitch] : from_f32<T>(0.0f);
            }
        }
        x += a.ldx;
        if constexpr (kBranch) y += a.ldy;
    };
    if constexpr (kWide) {
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) {
            if (s < count) fetch(mine + s * stage_bytes);
            copy_commit();
        }
    } else if (count > 0) {
        fetch(0);
    }
    uint32_t sample = static_cast<uint32_t>(first) / sample_rows(a.rows_per_batch);
    int64_t left = (sample + 1ll) * a.rows_per_batch - first;  // rows of this sample
    // kValues of a vector of columns, or `otherwise`; 0 past the row
    auto vector = [&](const void *p, int64_t offset, float otherwise, float (&v)[kValues]) {
#pragma unroll
        for (int j = 0; j < kNv; ++j) {
            float piece[kVec] = {};
            if (inside[j]) params<P>(p, offset + col + j * pitch, otherwise, piece);
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[j * kVec + e] = piece[e];
        }
    };
    F2 w_post[kPairs], w_pre[kPairs], b_pre[kPairs];
    auto prepare = [&]() {
        float u[kValues], v[kValues], w[kValues];
        vector(a.gate, sample * a.ldgate, 1.0f, u);
        vector(a.post_weight, 0, 1.0f, v);
#pragma unroll
        for (int e = 0; e < kPairs; ++e) w_post[e] = F2(u[2 * e] * v[2 * e], u[2 * e + 1] * v[2 * e + 1]);
        vector(a.scale, sample * a.ldscale, 0.0f, u);
        vector(a.pre_weight, 0, 1.0f, v);
#pragma unroll
        for (int e = 0; e < kValues; ++e) u[e] += 1.0f;
#pragma unroll
        for (int e = 0; e < kPairs; ++e) w_pre[e] = F2(u[2 * e] * v[2 * e], u[2 * e + 1] * v[2 * e + 1]);
        vector(a.pre_bias, 0, 0.0f, v);
        vector(a.shift, sample * a.ldshift, 0.0f, w);
        // An infinite scale times a bias that is not there may not become NaN. The choice is made where it costs least in
        // registers: by a select with 16-byte pieces (32760 x 2048 in f32: 170 us, 179 with the other), by a factor kept
        // finite otherwise (27163 x 1537 in bf16: 167 us, 200 with a select).
        if constexpr (kPiece == 16) {
#pragma unroll
            for (int e = 0; e < kPairs; ++e)
                b_pre[e] = !a.pre_bias ? F2(w[2 * e], w[2 * e + 1])
                                       : F2(fmaf(u[2 * e], v[2 * e], w[2 * e]), fmaf(u[2 * e + 1], v[2 * e + 1], w[2 * e + 1]));
        } else {
#pragma unroll
            for (int e = 0; e < kValues; ++e) u[e] = fminf(fmaxf(u[e], -FLT_MAX), FLT_MAX);
#pragma unroll
            for (int e = 0; e < kPairs; ++e)
                b_pre[e] = F2(fmaf(u[2 * e], v[2 * e], w[2 * e]), fmaf(u[2 * e + 1], v[2 * e + 1], w[2 * e + 1]));
        }
    };
    F2 h[kPairs];
    // mean out of h (layer norm), then 1 / deviation
    auto deviation = [&](int kind) {
        if (kind == CONVROT_NORM_LAYER) {
            F2 s = h[0];
#pragma unroll
            for (int e = 1; e < kPairs; ++e) s = s + h[e];
            const float mean = -sum(s.sum()) * inv_d;
#pragma unroll
            for (int e = 0; e < kPairs; ++e)
                h[e] = h[e] + F2(inside[2 * e / kVec] ? mean : 0.0f, inside[(2 * e + 1) / kVec] ? mean : 0.0f);
        }
        F2 s = h[0] * h[0];
#pragma unroll
        for (int e = 1; e < kPairs; ++e) s = fma2(h[e], h[e], s);
        return rsqrtf(fmaf(sum(s.sum()), inv_d, a.eps));
    };
    uint32_t stage = mine, ahead = mine + (kStages - 1) * stage_bytes;
    const uint32_t ring_end = mine + kStages * stage_bytes;
    bool fresh = true;
    for (int r = 0; r < count; ++r) {
        if (fresh) prepare();
        T now_x[kWide ? 1 : kNv], now_y[kWide || !kBranch ? 1 : kNv];
        if constexpr (kWide) {
            if (r + kStages - 1 < count) fetch(ahead);
            copy_commit();
            if ((ahead += stage_bytes) == ring_end) ahead = mine;
            copy_wait<kStages - 1>();
        } else {
#pragma unroll
            for (int j = 0; j < kNv; ++j) {
                now_x[j] = ahead_x[j];
                if constexpr (kBranch) now_y[j] = ahead_y[j];
            }
            if (r + 1 < count) fetch(0);
        }
        // this row's values of x (k = 0) or y (k = 1)
        auto row = [&](int k, F2 (&v)[kPairs]) {
            if constexpr (kWide) {
#pragma unroll
                for (int j = 0; j < kNv; ++j) {
                    Raw<T, kVec> raw;
                    load_shared(stage + (k * kNv + j) * step, raw.bits[0]);
                    if constexpr (kVec > 1)
                        raw.unpack(v + j * kVec / 2);
                    else
                        v[j / 2] = j % 2 ? F2(v[j / 2].lo(), raw.value()) : F2(raw.value(), 0.0f);
                }
            } else {
#pragma unroll
                for (int e = 0; e < kPairs; ++e)
                    v[e] = k ? F2(to_f32(now_y[kBranch ? 2 * e : 0]), to_f32(now_y[kBranch ? 2 * e + 1 : 0]))
                             : F2(to_f32(now_x[2 * e]), to_f32(now_x[2 * e + 1]));
            }
        };
        if constexpr (kBranch) {
            row(1, h);
            if (a.post != CONVROT_NORM_NONE) {
                const F2 inv(deviation(a.post));
#pragma unroll
                for (int e = 0; e < kPairs; ++e) h[e] = h[e] * inv;
            }
#pragma unroll
            for (int e = 0; e < kPairs; ++e) h[e] = h[e] * w_post[e];
            if (a.post_bias) {
                float u[kValues], v[kValues];
                vector(a.gate, sample * a.ldgate, 1.0f, u);
                vector(a.post_bias, 0, 0.0f, v);
#pragma unroll
                for (int e = 0; e < kPairs; ++e) h[e] = fma2(F2(u[2 * e], u[2 * e + 1]), F2(v[2 * e], v[2 * e + 1]), h[e]);
            }
        }
        {
            F2 xv[kPairs];
            row(0, xv);
            const F2 res(a.res_scale);
#pragma unroll
            for (int e = 0; e < kPairs; ++e) h[e] = kBranch ? fma2(res, xv[e], h[e]) : res * xv[e];
        }
        auto put = [&](T *p) {
#pragma unroll
            for (int j = 0; j < kNv; ++j) {
                if constexpr (kVec > 1) {
                    Raw<T, kVec> raw;
                    raw.pack(h + j * kVec / 2);
                    if (inside[j]) raw.store_stream(p + j * pitch);
                } else {
                    if (inside[j]) p[j * pitch] = from_f32<T>(j % 2 ? h[j / 2].hi() : h[j / 2].lo());
                }
            }
        };
        if (a.h) {
            put(h_out);
            h_out += a.ldh;
        }
        if (a.pre != CONVROT_NORM_NONE) {
            const F2 inv(deviation(a.pre));
#pragma unroll
            for (int e = 0; e < kPairs; ++e) h[e] = h[e] * inv;
        }
#pragma unroll
        for (int e = 0; e < kPairs; ++e) h[e] = fma2(h[e], w_pre[e], b_pre[e]);
        if (a.n) {
            put(n_out);
            n_out += a.ldn;
        }
        if constexpr (kPiece == 16) {
            if (a.q) {
                float v[kNv][kVec];
#pragma unroll
                for (int e = 0; e < kPairs; ++e) {
                    v[2 * e / kVec][2 * e % kVec] = h[e].lo();
                    v[2 * e / kVec][2 * e % kVec + 1] = h[e].hi();
                }
                pack_row<kVec, kNv>(a, first + r, d, threadIdx.x, nt, v);
            }
        }
        if constexpr (kWide) {
            if ((stage += stage_bytes) == ring_end) stage = mine;
        }
        fresh = --left == 0;
        if (fresh) {
            ++sample;
            left = a.rows_per_batch;
        }
    }
}

// kNv accesses a thread: a block of threads for each row.
template <typename T, typename P, int kVec, int kNv>
cudaError_t launch_block_rows(const convrot_gated_norm_args &a, cudaStream_t stream)
{
    const int64_t per = (a.d + kVec * kNv - 1) / (kVec * kNv);
    return launch_after(gated_norm_kernel<T, P, kVec, kNv, false>, dim3(static_cast<unsigned>(a.m)), static_cast<unsigned>((per + 31) / 32 * 32), 0, stream, 1, a);
}

constexpr int kRingBytes = 192 * 1024;  // shared memory an SM gives its rings; the rest stays L1 for the vectors

template <typename T, typename P, int kNv, int kVec, int kThreads, bool kBranch>
struct ring_tag;

// Runs of rows, if there are enough of them: four a block, so that preparing the sample's vectors (and filling the
// ring, which has to fit) is a small part.
template <typename T, typename P, int kNv, int kVec, int kThreads, bool kBranch>
bool launch_ring(const convrot_gated_norm_args &a, cudaStream_t stream, cudaError_t *e)
{
    constexpr int kPiece = kVec * static_cast<int>(sizeof(T));
    const int threads = kThreads ? kThreads : static_cast<int>((a.d / kVec + kNv - 1) / kNv + 31) / 32 * 32;
    const int bytes = kPiece >= 4 ? kRingStages * (kBranch ? 2 : 1) * kNv * threads * kPiece : 0;
    int per_sm = kRingThreads / threads;
    if (bytes && kRingBytes / bytes < per_sm) per_sm = kRingBytes / bytes;
    if (per_sm < 1) return false;
    const int64_t blocks = static_cast<int64_t>(per_sm) * kSms;
    if (a.m < 4 * blocks) return false;
    auto kernel = gated_norm_ring_kernel<T, P, kNv, kVec, kThreads, kBranch>;
    *e = allow_shared<ring_tag<T, P, kNv, kVec, kThreads, kBranch>>(kernel);
    if (*e != cudaSuccess) return true;
    const int64_t rows = (a.m + blocks - 1) / blocks;
    *e = launch_after(kernel, dim3(static_cast<unsigned>((a.m + rows - 1) / rows)), static_cast<unsigned>(threads), bytes, stream, 1, a,
                      static_cast<int32_t>(rows));
    return true;
}

template <typename T, typename P, int kNv, int kVec, int kThreads = 0>
bool launch_ring(const convrot_gated_norm_args &a, cudaStream_t stream, cudaError_t *e)
{
    return a.y ? launch_ring<T, P, kNv, kVec, kThreads, true>(a, stream, e) : launch_ring<T, P, kNv, kVec, kThreads, false>(a, stream, e);
}

// A warp for each row, four rows a block.
template <typename T, typename P, int kVec, int kNv>
cudaError_t launch_warp_rows(const convrot_gated_norm_args &a, cudaStream_t stream)
{
    return launch_after(gated_norm_kernel<T, P, kVec, kNv, true>, dim3(static_cast<unsigned>((a.m + 3) / 4)), 128, 0, stream, 1, a);
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
            cudaError_t e;
            if (n > 256 ? launch_ring<T, P, 16 / kVec, kVec>(a, stream, &e) : launch_ring<T, P, 1, kVec>(a, stream, &e)) return e;
            if (n <= 32) return launch_warp_rows<T, P, kVec, 1>(a, stream);
            if (n <= kRowThreads) return launch_block_rows<T, P, kVec, 1>(a, stream);
            if (n <= 2 * kRowThreads) return launch_block_rows<T, P, kVec, 2>(a, stream);
            return launch_block_rows<T, P, kVec, 32 / kVec>(a, stream);
        }
        if (a.d <= 128) return launch_warp_rows<T, P, 1, 4>(a, stream);
        cudaError_t e;
        if (!a.q) {
            // pieces of 4 bytes where rows start on 4, single elements otherwise
            constexpr int kSmall = 4 / kT;
            const bool small = a.d % kSmall == 0 && vectors(a.x, a.m, a.ldx, kSmall, kT) && vectors(a.y, a.m, a.ldy, kSmall, kT) &&
                               vectors(a.h, a.m, a.ldh, kSmall, kT) && vectors(a.n, a.m, a.ldn, kSmall, kT) &&
                               vectors(a.gate, batches, a.ldgate, kSmall, kP) && vectors(a.scale, batches, a.ldscale, kSmall, kP) &&
                               vectors(a.shift, batches, a.ldshift, kSmall, kP) && vectors(a.post_weight, 1, a.d, kSmall, kP) &&
                               vectors(a.post_bias, 1, a.d, kSmall, kP) && vectors(a.pre_weight, 1, a.d, kSmall, kP) &&
                               vectors(a.pre_bias, 1, a.d, kSmall, kP);
            auto runs = [&](auto vec) {
                constexpr int kV = decltype(vec)::value;
                if (a.d <= 512) return launch_ring<T, P, 8 / kV, kV, 64>(a, stream, &e);
                if (a.d <= 1024) return launch_ring<T, P, 8 / kV, kV, 128>(a, stream, &e);
                if (a.d <= 1536) return launch_ring<T, P, 12 / kV, kV, 128>(a, stream, &e);
                if (a.d <= 3072) return launch_ring<T, P, 12 / kV, kV, 256>(a, stream, &e);
                if (a.d <= 6144) return launch_ring<T, P, 12 / kV, kV, 512>(a, stream, &e);
                return false;
            };
            const bool done = small ? runs(std::integral_constant<int, kSmall>{}) : runs(std::integral_constant<int, 1>{});
            if (done) return e;
        }
        // single elements: blocks of 128 to 512 threads, enough values in each that the sums' cost is spread
        if (a.d <= 2048) return launch_block_rows<T, P, 1, 8>(a, stream);
        if (a.d <= 8192) return launch_block_rows<T, P, 1, 16>(a, stream);
        return launch_block_rows<T, P, 1, 32>(a, stream);
    });
}

}  // namespace convrot
