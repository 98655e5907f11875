// Attention with few queries (include/convrot_block.h): one new token, or the
// few that share a key head, against long states. Reading the keys and values
// once is all that counts, so a unit is a key head of a sample with all of its
// query heads' rows (16 at most), its keys are shared out over a cluster of
// CTAs (and, where one cluster is not enough to fill the GPU, over several).
// Each warp goes through its keys 16 at a time with the warp-level matrix
// instruction. (Its rate is of no matter here: 16 keys of 128 elements are 8 KB
// of loads and 32 instructions.) Its keys and values come through a ring of its
// own that TMA copies fill, which its first lane starts, so that no warp waits
// for another and nearly all of an SM's shared memory is on its way. (8
// sequences of one token, 4096 keys, 40 + 8 heads of 128: 32 us with copies by
// the lanes, 16 bytes each, from registers or through queues of any length: 5.2
// TB/s however many were in flight.)
//
// Both orders that the fragments ask for are had by renaming, not by moving
// data. In S = Q K^T the elements of a head are summed in any order: a lane
// takes whole 16-byte pieces of its key, and the same pieces of its query. In
// P V the columns of a result may stand anywhere: a lane takes 16-byte pieces
// of the four keys whose probabilities it holds, and pairs them up by element.
//
// Warps keep a maximum, a sum and sums of their own; they meet in shared
// memory, the cluster's CTAs in distributed shared memory, clusters in a second
// kernel, always added in the same order. The copies bring every key, masked or
// not; a mask takes a key's score and value out where they are used, so it saves
// no time (4 x 2 queries, 8192 keys, half of them masked: 29.5 us).
#include "attention.cuh"

namespace convrot {
namespace {

using namespace mma16;

constexpr int kWarps = 12, kThreads = 32 * kWarps, kRows = 16, kStep = 16;  // keys of a warp's step
constexpr int kPerSm = 1;
constexpr float kGrow = 8.0f;

struct FewParams {
    HeadsMap k, v;
    const void *q;
    int64_t q_strides[3], out_strides[3];
    int32_t *dev_status;
    const uint8_t *mask;
    int64_t mask_stride;
    void *out;
    float *lse;
    float *partial;  // [units][parts][16][kD + 2]: sums, maximum (base 2) and sum of a part, or null
    int32_t q_tokens, q_heads, kv_heads, group, rows;
    int32_t split, parts, d;
    int32_t wide;         // rows of q start on 16 bytes
    int64_t kv_tokens, share;  // keys of a CTA
    float scale_log2;
};

template <typename T>
__device__ __forceinline__ void mma_warp(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (std::is_same_v<T, __nv_bfloat16>)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load16(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

__device__ __forceinline__ float remote4(uint32_t local, uint32_t rank)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(map_to_rank(local, rank)) : "memory");
    return v;
}

// What a part's sums count for beside the largest maximum.
__device__ __forceinline__ float weight_of(float top, float most) { return top == neg_inf() ? 0.0f : ex2(top - most); }

// out and lse of one row from its sums.
template <typename T>
__device__ __forceinline__ void finish(const FewParams &p, int b, int hk, int row, int e, float sum, float total, float most, float shift)
{
    const int t = row / p.group, h = hk * p.group + row % p.group;
    const float inv = total > 0.0f ? 1.0f / total : total == 0.0f ? 0.0f : total;  // NaN stays
    T *out = static_cast<T *>(p.out) + b * p.out_strides[0] + t * p.out_strides[1] + h * p.out_strides[2];
    out[e] = from_f32<T>(total == 0.0f ? 0.0f : sum * inv);
    if (e == 0)
        p.lse[(static_cast<int64_t>(b) * p.q_heads + h) * p.q_tokens + t] = total == 0.0f ? neg_inf() : kLn2 * (most + (log2f(total) - shift));
}

// A warp's ring: steps of 16 keys and values, each a box of 64 elements (128 bytes, swizzled) a row, or two.
template <int kD>
struct Ring {
    static constexpr int kHalves = kD / 64, kBox = kStep * 128, kStepBytes = 2 * kHalves * kBox;
    static constexpr int kSteps = kD == 64 ? 4 : 2;
    static constexpr int kSums = kWarps * kRows * (kD + 2) * 4;
    static constexpr int kBytes = 1024 + (kWarps * kSteps * kStepBytes > kSums ? kWarps * kSteps * kStepBytes : kSums);
    static_assert(kPerSm * (kBytes + 2048) <= kSmShared, "resident");
};

template <typename T, int kD>
__global__ void __launch_bounds__(kThreads, kPerSm) attention_few_kernel(const __grid_constant__ FewParams p)
{
    constexpr float kShift = std::is_same_v<T, __half> ? 7.0f : 0.0f;
    constexpr int kChunks = kD / 8;        // 16-byte pieces of a head
    constexpr int kQ = kChunks / 4;        // of a lane, in S
    constexpr int kV = kChunks / 8;        // of a lane and key, in P V
    constexpr int kPitch = kD + 2;         // of a row in shared memory (its maximum and sum behind it)
    using R = Ring<kD>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[kWarps][R::kSteps];
    __shared__ volatile int abort_flag;
    const uint32_t raw = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw)), base = (raw + 1023u) & ~1023u;
    // the warps' sums, when all their steps are done, over the rings
    float (&sums)[kWarps][kRows][kPitch] = *reinterpret_cast<float (*)[kWarps][kRows][kPitch]>(smem_raw + (base - raw));
    const Waits wait{&abort_flag, p.dev_status};
    if (threadIdx.x == 0) {
        for (int i = 0; i < kWarps * R::kSteps; ++i) mbar_init(static_cast<uint32_t>(__cvta_generic_to_shared(&bars[0][0])) + 8 * i, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&p.k.map);
        prefetch_map(&p.v.map);
    }
    __syncthreads();
    after_previous();
    let_next_start();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t split = static_cast<uint32_t>(p.split), rank = split > 1 ? cluster_rank() : 0;
    const int cluster = static_cast<int>(blockIdx.x / split), unit = cluster / p.parts, part = cluster - unit * p.parts;
    const int b = unit / p.kv_heads, hk = unit - b * p.kv_heads;
    const int chunks = (p.d + 7) / 8;

    // Q: rows g and g + 8 of the unit, pieces t + 4 i
    uint32_t q[2 * kQ][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = g + 8 * r;
        const T *from = static_cast<const T *>(p.q) + b * p.q_strides[0] + row / p.group * p.q_strides[1] + (hk * p.group + row % p.group) * p.q_strides[2];
#pragma unroll
        for (int i = 0; i < kQ; ++i) {
            const int c = t + 4 * i;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (row < p.rows && c < chunks) {
                if (p.wide) {
                    w = load16(from + c * 8);
                } else {
                    const uint16_t *u = reinterpret_cast<const uint16_t *>(from) + c * 8;
                    uint32_t e[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) e[k] = c * 8 + k < p.d ? static_cast<uint32_t>(u[k]) : 0u;
                    w = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
                }
            }
            q[2 * i][r] = w.x;
            q[2 * i][2 + r] = w.y;
            q[2 * i + 1][r] = w.z;
            q[2 * i + 1][2 + r] = w.w;
        }
    }

    const int64_t begin = (static_cast<int64_t>(part) * split + rank) * p.share;
    const int64_t end = begin + p.share < p.kv_tokens ? begin + p.share : p.kv_tokens;
    const uint8_t *mask = p.mask ? p.mask + b * p.mask_stride : nullptr;
    const uint32_t ring = base + warp * R::kSteps * R::kStepBytes, bar = static_cast<uint32_t>(__cvta_generic_to_shared(&bars[warp][0]));
    auto load = [&](int64_t key0, int at) {  // by one lane
        mbar_arrive_expect_tx(bar + 8 * at, R::kStepBytes);
#pragma unroll
        for (int h = 0; h < R::kHalves; ++h) {
            const uint32_t to = ring + at * R::kStepBytes + h * R::kBox;
            tma_load_4d(to, &p.k.map, h * kBoxElems, static_cast<int>(key0), hk * p.k.head_step, b * p.k.batch_step, bar + 8 * at);
            tma_load_4d(to + R::kHalves * R::kBox, &p.v.map, h * kBoxElems, static_cast<int>(key0), hk * p.v.head_step, b * p.v.batch_step, bar + 8 * at);
        }
    };
    // piece c (16 bytes) of a row of keys or, behind them, values
    auto piece = [&](int at, int values, int row, int c) {
        return shared16(ring + at * R::kStepBytes + (values * R::kHalves + c / 8) * R::kBox + row * 128 + ((c ^ row) & 7) * 16);
    };

    float o[8 * kV][4];
#pragma unroll
    for (int n = 0; n < 8 * kV; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] = 0.0f;
    float top[2] = {neg_inf(), neg_inf()}, sum[2] = {0.0f, 0.0f};  // rows g and g + 8; the sum over this lane's keys
    const float c = p.scale_log2;
    const int64_t first = begin + warp * kStep, stride = kWarps * kStep;
    if (lane == 0) {
        for (int n = 0; n < R::kSteps; ++n)
            if (first + n * stride < end) load(first + n * stride, n);
    }
    int at = 0;  // the step's place in the ring
    int flying = 0;  // steps whose copies were started and not waited for
    for (int n = 0; n < R::kSteps; ++n) flying += first + n * stride < end;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t key0 = first; key0 < end; key0 += stride) {
        if (!(ok = wait.together(bar + 8 * at, phase))) break;
        const int left = end - key0 < kStep ? static_cast<int>(end - key0) : kStep;
        bool kept[4];  // keys 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            constexpr int kKeys[4] = {0, 1, 8, 9};
            kept[j] = 2 * t + kKeys[j] < left;
            if (mask && kept[j]) kept[j] = *reinterpret_cast<const volatile uint8_t *>(mask + key0 + 2 * t + kKeys[j]) != 0;
        }
        float s[2][4] = {};
#pragma unroll
        for (int i = 0; i < kQ; ++i)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const uint4 k = piece(at, 0, 8 * n + g, t + 4 * i);
                mma_warp<T>(s[n], q[2 * i], k.x, k.y);
                mma_warp<T>(s[n], q[2 * i + 1], k.z, k.w);
            }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (!kept[2 * n + (e & 1)]) s[n][e] = neg_inf();
        float factor[2] = {1.0f, 1.0f};
        bool grown = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float m = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2)) * c;
            if (m - top[r] > kGrow || (top[r] == neg_inf() && m > top[r])) {
                factor[r] = weight_of(top[r], m);
                top[r] = m;
                sum[r] *= factor[r];
                grown = true;
            }
        }
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
            for (int n = 0; n < 8 * kV; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][e] *= factor[e >> 1];
        }
        uint32_t pk[4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float off = top[r] == neg_inf() ? 0.0f : kShift - top[r];
                const float a = ex2(fmaf(s[n][2 * r], c, off)), d = ex2(fmaf(s[n][2 * r + 1], c, off));
                sum[r] += a + d;
                pk[2 * n + r] = pack2<T>(a, d);
            }
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                constexpr int kKeys[4] = {0, 1, 8, 9};
                v[j] = piece(at, 1, 2 * t + kKeys[j], g + 8 * i);
                if (mask && !kept[j]) v[j] = make_uint4(0, 0, 0, 0);  // (0 times NaN)
            }
            const uint32_t *v0 = reinterpret_cast<const uint32_t *>(&v[0]), *v1 = reinterpret_cast<const uint32_t *>(&v[1]);
            const uint32_t *v2 = reinterpret_cast<const uint32_t *>(&v[2]), *v3 = reinterpret_cast<const uint32_t *>(&v[3]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {  // element e of the piece, of two keys a register
                const uint32_t pick = e & 1 ? 0x7632 : 0x5410;
                mma_warp<T>(o[8 * i + e], pk, __byte_perm(v0[e / 2], v1[e / 2], pick), __byte_perm(v2[e / 2], v3[e / 2], pick));
            }
        }
        __syncwarp();  // every lane has read the step
        --flying;
        if (key0 + R::kSteps * stride < end) {
            if (lane == 0) load(key0 + R::kSteps * stride, at);
            ++flying;
        }
        if (++at == R::kSteps) {
            at = 0;
            phase ^= 1u;
        }
    }
    if (!ok) {
        wait.fail();
        // copies in flight land before shared memory goes away
        for (int n = 0; n < R::kSteps; ++n, at = at + 1 == R::kSteps ? 0 : at + 1) {
            if (at == 0 && n > 0) phase ^= 1u;
            if (n < flying) mbar_wait(bar + 8 * at, phase);
        }
    }
    __syncthreads();  // the rings are done with

    // this warp's rows: o[8 i + e] has columns 2t and 2t + 1, which are elements (2t + 8 i) 8 + e and (2t + 1 + 8 i) 8 + e
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
        sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
        float *to = sums[warp][g + 8 * r];
#pragma unroll
        for (int i = 0; i < kV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                to[(2 * t + 8 * i) * 8 + e] = o[8 * i + e][2 * r];
                to[(2 * t + 1 + 8 * i) * 8 + e] = o[8 * i + e][2 * r + 1];
            }
        if (t == 0) {
            to[kD] = top[r];
            to[kD + 1] = sum[r];
        }
    }
    __syncthreads();
    // the CTA's rows, over the first warp's
    for (int i = threadIdx.x; i < p.rows * kD; i += kThreads) {
        const int row = i / kD, e = i - row * kD;
        float most = neg_inf(), all = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) most = fmaxf(most, sums[w][row][kD]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) all += sums[w][row][e] * weight_of(sums[w][row][kD], most);
        sums[0][row][e] = all;  // (of this thread alone; the maxima stay until all have read them)
    }
    __syncthreads();
    for (int row = threadIdx.x; row < p.rows; row += kThreads) {
        float most = neg_inf(), all = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) most = fmaxf(most, sums[w][row][kD]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) all += sums[w][row][kD + 1] * weight_of(sums[w][row][kD], most);
        sums[0][row][kD] = most;
        sums[0][row][kD + 1] = all;
    }
    if (split > 1)
        cluster_sync();
    else
        __syncthreads();
    // the cluster's: its CTAs share out the elements
    const uint32_t at0 = base;
    for (int i = static_cast<int>(rank) * kThreads + threadIdx.x; i < p.rows * p.d; i += static_cast<int>(split) * kThreads) {
        const int row = i / p.d, e = i - row * p.d;
        const uint32_t at = at0 + row * kPitch * 4;
        float most = neg_inf(), all = 0.0f, total = 0.0f;
        for (uint32_t r = 0; r < split; ++r) most = fmaxf(most, remote4(at + kD * 4, r));
        for (uint32_t r = 0; r < split; ++r) {
            const float w = weight_of(remote4(at + kD * 4, r), most);
            all += remote4(at + e * 4, r) * w;
            total += remote4(at + (kD + 1) * 4, r) * w;
        }
        if (p.partial) {
            float *to = p.partial + (static_cast<int64_t>(cluster) * kRows + row) * kPitch;
            to[e] = all;
            if (e == 0) {
                to[kD] = most;
                to[kD + 1] = total;
            }
        } else {
            finish<T>(p, b, hk, row, e, all, total, most, kShift);
        }
    }
    if (split > 1) cluster_sync();  // a CTA's sums stay until its peers have read them
}

// The parts of a unit, added up in order: a block a row.
template <typename T, int kD>
__global__ void __launch_bounds__(kD) attention_few_join_kernel(const __grid_constant__ FewParams p)
{
    constexpr float kShift = std::is_same_v<T, __half> ? 7.0f : 0.0f;
    constexpr int kPitch = kD + 2;
    after_previous();
    let_next_start();
    const int unit = static_cast<int>(blockIdx.x) / p.rows, row = static_cast<int>(blockIdx.x) - unit * p.rows, e = threadIdx.x;
    if (e >= p.d) return;
    const float *from = p.partial + (static_cast<int64_t>(unit) * p.parts * kRows + row) * kPitch;
    const int64_t next = int64_t{kRows} * kPitch;
    float most = neg_inf(), all = 0.0f, total = 0.0f;
    for (int i = 0; i < p.parts; ++i) most = fmaxf(most, load_f32(from + i * next + kD));
    for (int i = 0; i < p.parts; ++i) {
        const float w = weight_of(load_f32(from + i * next + kD), most);
        all += load_f32(from + i * next + e) * w;
        total += load_f32(from + i * next + kD + 1) * w;
    }
    finish<T>(p, unit / p.kv_heads, unit - unit / p.kv_heads * p.kv_heads, row, e, all, total, most, kShift);
}

// How a unit's keys are shared out: CTAs of a cluster, and clusters.
struct Cut {
    int split, parts;
    int64_t share;
};

// As many CTAs as are resident together, each with 192 keys (a step of its twelve warps) or more; clusters of 1, 2, 4 or 8,
// since clusters of 4 and 8 leave some SMs of a GPC over (36 and 15 of them fit), and of other sizes more (64 of 7: two rounds).
Cut cut_of(int64_t units, int64_t kv_tokens)
{
    const int64_t most = (kv_tokens + kWarps * kStep - 1) / (kWarps * kStep);
    const int room[4] = {kSms, kSms / 2, 36, 15};
    Cut c{1, 1, 0};
    for (int i = 1; i < 4; ++i) {
        const int split = 1 << i;
        if (units > room[i] || most < split) break;
        c.split = split;
    }
    // Long states of few heads: pairs, as many as fill the GPU, and the second kernel, where the one cluster would leave
    // half of the SMs idle for eight steps a warp or more (which take longer than that kernel's 3 us).
    const int64_t pairs = kSms / 2 / units;
    if (pairs >= c.split && most / c.split >= 8) {
        c.split = 2;
        c.parts = static_cast<int>(pairs < most / 2 ? pairs : most / 2);
    }
    const int64_t ctas = int64_t{c.split} * c.parts;
    c.share = (kv_tokens + ctas - 1) / ctas;
    c.share = (c.share + kStep - 1) / kStep * kStep;
    return c;
}

template <typename T, int kD>
struct few_tag;

template <typename T, int kD>
cudaError_t launch(const AttentionArgs &a, const FewParams &p, int64_t units, cudaStream_t stream)
{
    auto kernel = attention_few_kernel<T, kD>;
    cudaError_t e = allow_shared<few_tag<T, kD>>(kernel);
    if (e == cudaSuccess)
        e = launch_after(kernel, dim3(static_cast<unsigned>(units * p.split * p.parts)), kThreads, Ring<kD>::kBytes, stream, static_cast<unsigned>(p.split), p);
    if (e != cudaSuccess || p.parts == 1) return e;
    return launch_after(attention_few_join_kernel<T, kD>, dim3(static_cast<unsigned>(units * p.rows)), kD, 0, stream, 1, p);
}

}  // namespace

bool attention_few_takes(int64_t q_tokens, int64_t q_heads, int64_t kv_heads) { return q_tokens * (q_heads / kv_heads) <= kRows; }

int64_t attention_few_partial_bytes(int64_t batch, int64_t kv_tokens, int64_t kv_heads, int d)
{
    const Cut c = cut_of(batch * kv_heads, kv_tokens);
    return c.parts == 1 ? 0 : batch * kv_heads * c.parts * kRows * ((d <= 64 ? 64 : 128) + 2) * 4;
}

cudaError_t launch_attention_few(const AttentionArgs &a, const uint8_t *mask, int64_t mask_stride, float *partial, cudaStream_t stream)
{
    FewParams p{};
    p.q = a.q.p;
    for (int i = 0; i < 3; ++i) {
        p.q_strides[i] = a.q.strides[i];
        p.out_strides[i] = a.out_strides[i];
    }
    const bool bf16 = a.dtype == CONVROT_BF16;
    if (!(bf16 ? heads_map<__nv_bfloat16>(&p.k, a.k, a.batch, a.d, kStep) && heads_map<__nv_bfloat16>(&p.v, a.v, a.batch, a.d, kStep)
               : heads_map<__half>(&p.k, a.k, a.batch, a.d, kStep) && heads_map<__half>(&p.v, a.v, a.batch, a.d, kStep)))
        return cudaErrorInvalidValue;
    p.dev_status = a.dev_status;
    p.mask = mask;
    p.mask_stride = mask_stride;
    p.out = a.out;
    p.lse = a.lse;
    p.q_tokens = static_cast<int32_t>(a.q.tokens);
    p.q_heads = static_cast<int32_t>(a.q.heads);
    p.kv_heads = static_cast<int32_t>(a.k.heads);
    p.group = p.q_heads / p.kv_heads;
    p.rows = p.q_tokens * p.group;
    p.d = a.d;
    p.wide = a.d % 8 == 0 && heads_wide(a.q.p, a.q.strides, a.batch, a.q.tokens, a.q.heads);
    p.kv_tokens = a.kv_tokens;
    p.scale_log2 = a.scale * kLog2e;
    const int64_t units = a.batch * a.k.heads;
    const Cut c = cut_of(units, a.kv_tokens);
    p.split = c.split;
    p.parts = c.parts;
    p.share = c.share;
    p.partial = c.parts > 1 ? partial : nullptr;
    if (units * c.split * c.parts > INT32_MAX || units * kRows > INT32_MAX) return cudaErrorInvalidValue;
    if (a.dtype == CONVROT_BF16) return a.d <= 64 ? launch<__nv_bfloat16, 64>(a, p, units, stream) : launch<__nv_bfloat16, 128>(a, p, units, stream);
    return a.d <= 64 ? launch<__half, 64>(a, p, units, stream) : launch<__half, 128>(a, p, units, stream);
}

}  // namespace convrot
