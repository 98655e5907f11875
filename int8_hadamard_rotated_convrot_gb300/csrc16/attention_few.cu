// Attention with few queries (include/convrot_block.h): one new token, or the
// few that share a key head, against long states. Reading the keys and values
// once is all that counts, so a unit is a key head of a sample with all of its
// query heads' rows (16 at most), its keys are shared out over a cluster of
// CTAs (and, where one cluster is not enough to fill the GPU, over several),
// and nothing is staged: each warp multiplies straight from registers that wide
// loads fill, 16 keys at a time, with the warp-level matrix instruction. (Its
// rate is of no matter here: 16 keys of 128 elements are 8 KB of loads and 32
// instructions.)
//
// Both orders that the fragments ask for are had by renaming, not by moving
// data. In S = Q K^T the elements of a head are summed in any order: a lane
// takes whole 16-byte pieces of its key, and the same pieces of its query. In
// P V the columns of a result may stand anywhere: a lane takes 16-byte pieces
// of the four keys whose probabilities it holds, and pairs them up by element.
//
// Warps keep a maximum, a sum and sums of their own; they meet in shared
// memory, the cluster's CTAs in distributed shared memory, clusters in a second
// kernel, always added in the same order. A masked key is not read.
#include "attention.cuh"

namespace convrot {
namespace {

using namespace mma16;

constexpr int kWarps = 4, kThreads = 32 * kWarps, kRows = 16, kStep = 16;  // keys of a warp's step
constexpr int kMaxSplit = 8;
constexpr int kPerSm = 2;
constexpr float kGrow = 8.0f;

struct FewParams {
    const void *q, *k, *v;
    int64_t q_strides[3], k_strides[3], v_strides[3], out_strides[3];
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

template <typename T, int kD>
__global__ void __launch_bounds__(kThreads, kPerSm) attention_few_kernel(const __grid_constant__ FewParams p)
{
    constexpr float kShift = std::is_same_v<T, __half> ? 7.0f : 0.0f;
    constexpr int kChunks = kD / 8;        // 16-byte pieces of a head
    constexpr int kQ = kChunks / 4;        // of a lane, in S
    constexpr int kV = kChunks / 8;        // of a lane and key, in P V
    constexpr int kPitch = kD + 2;         // of a row in shared memory (its maximum and sum behind it)
    __shared__ float sums[kWarps][kRows][kPitch];
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
    const T *k_base = static_cast<const T *>(p.k) + b * p.k_strides[0] + hk * p.k_strides[2];
    const T *v_base = static_cast<const T *>(p.v) + b * p.v_strides[0] + hk * p.v_strides[2];
    const uint8_t *mask = p.mask ? p.mask + b * p.mask_stride : nullptr;
    auto there = [&](int64_t key) { return key < end && (!mask || *reinterpret_cast<const volatile uint8_t *>(mask + key) != 0); };

    uint4 kr[2][kQ], vr[4][kV];
    bool kept[4];  // keys 2t, 2t + 1, 2t + 8, 2t + 9 of the step
    auto load_k = [&](int64_t key0) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int64_t key = key0 + 8 * n + g;
            const T *from = k_base + key * p.k_strides[1] + t * 8;
#pragma unroll
            for (int i = 0; i < kQ; ++i) kr[n][i] = key < end && t + 4 * i < chunks ? load16(from + 32 * i) : make_uint4(0, 0, 0, 0);
        }
    };
    auto load_v = [&](int64_t key0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t key = key0 + 2 * t + (j & 1) + (j >> 1) * 8;
            kept[j] = there(key);
            const T *from = v_base + key * p.v_strides[1] + g * 8;
#pragma unroll
            for (int i = 0; i < kV; ++i) vr[j][i] = kept[j] && g + 8 * i < chunks ? load16(from + 64 * i) : make_uint4(0, 0, 0, 0);
        }
    };

    float o[8 * kV][4];
#pragma unroll
    for (int n = 0; n < 8 * kV; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] = 0.0f;
    float top[2] = {neg_inf(), neg_inf()}, sum[2] = {0.0f, 0.0f};  // rows g and g + 8; the sum over this lane's keys
    const float c = p.scale_log2;
    const int64_t first = begin + warp * kStep;
    if (first < end) {
        load_k(first);
        load_v(first);
    }
    for (int64_t key0 = first; key0 < end; key0 += kWarps * kStep) {
        float s[2][4] = {};
#pragma unroll
        for (int i = 0; i < kQ; ++i)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                mma_warp<T>(s[n], q[2 * i], kr[n][i].x, kr[n][i].y);
                mma_warp<T>(s[n], q[2 * i + 1], kr[n][i].z, kr[n][i].w);
            }
        const bool more = key0 + kWarps * kStep < end;
        if (more) load_k(key0 + kWarps * kStep);
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
            const uint32_t *v0 = reinterpret_cast<const uint32_t *>(&vr[0][i]), *v1 = reinterpret_cast<const uint32_t *>(&vr[1][i]);
            const uint32_t *v2 = reinterpret_cast<const uint32_t *>(&vr[2][i]), *v3 = reinterpret_cast<const uint32_t *>(&vr[3][i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {  // element e of the piece, of two keys a register
                const uint32_t pick = e & 1 ? 0x7632 : 0x5410;
                mma_warp<T>(o[8 * i + e], pk, __byte_perm(v0[e / 2], v1[e / 2], pick), __byte_perm(v2[e / 2], v3[e / 2], pick));
            }
        }
        if (more) load_v(key0 + kWarps * kStep);
    }

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
    const uint32_t at0 = static_cast<uint32_t>(__cvta_generic_to_shared(&sums[0][0][0]));
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

// As many CTAs as are resident together, each with 64 keys (a step of its four warps) or more.
Cut cut_of(int64_t units, int64_t kv_tokens)
{
    int64_t want = kPerSm * kSms / units, most = (kv_tokens + kWarps * kStep - 1) / (kWarps * kStep);
    if (want > most) want = most;
    if (want < 1) want = 1;
    Cut c;
    c.split = static_cast<int>(want < kMaxSplit ? want : kMaxSplit);
    c.parts = static_cast<int>(want / c.split);
    const int64_t ctas = int64_t{c.split} * c.parts;
    c.share = (kv_tokens + ctas - 1) / ctas;
    c.share = (c.share + kStep - 1) / kStep * kStep;
    return c;
}

template <typename T, int kD>
cudaError_t launch(const AttentionArgs &a, const FewParams &p, int64_t units, cudaStream_t stream)
{
    cudaError_t e = launch_after(attention_few_kernel<T, kD>, dim3(static_cast<unsigned>(units * p.split * p.parts)), kThreads, 0, stream,
                                 static_cast<unsigned>(p.split), p);
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
    p.k = a.k.p;
    p.v = a.v.p;
    for (int i = 0; i < 3; ++i) {
        p.q_strides[i] = a.q.strides[i];
        p.k_strides[i] = a.k.strides[i];
        p.v_strides[i] = a.v.strides[i];
        p.out_strides[i] = a.out_strides[i];
    }
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
