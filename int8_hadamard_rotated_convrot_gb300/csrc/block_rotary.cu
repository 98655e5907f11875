// Rotary positions (include/convrot_block.h): pairs of values of each query
// and key head turned by the angles of the token's position.
//
//   (a, b) -> (a cos - b sin, b cos + a sin)
//
// Three operations for four bytes moved: the kernel is a copy, bound by HBM.
// One launch covers queries and keys. A thread owns one slot of a head (up to
// 16 bytes of a's and as many of b's in the half layout, 16 bytes of pairs in
// the interleaved one, or 16 bytes past rot_dim, which are copied) and does it
// for kHeads heads of one token: the cosines and sines are read once for all of
// them, and all their loads, 64 bytes a thread, are in flight together. 1536
// threads an SM (40 registers; 1280 where eight pairs a head need more) and
// stores that leave L2 first: the queries and keys of 32760 tokens x 40 heads x
// 128 in bf16 (1.36 GB) take 205 us on one GB300, 6.6 TB/s, 98 % of a measured
// copy; with 960 threads and ordinary stores 259 us.
#include <cmath>

#include "block.h"

namespace convrot {
namespace {

constexpr int kRotaryThreads = 256;

struct RotaryShape {
    int32_t slots;         // of one head
    int32_t pair_slots;    // those that turn pairs
    int32_t head_groups;   // threads that share a slot of one token
    int32_t rows_per_block;
    uint32_t rows;         // tokens of all sequences
    int32_t vec_table;     // cos and sin rows are 16-byte aligned
    int32_t skip_copy;     // in place: nothing to do past rot_dim
};

template <typename T, int kVec, bool kInterleaved, int kHeads>
__global__ void __launch_bounds__(kRotaryThreads, sizeof(T) == 2 && kVec == 8 && !kInterleaved ? 5 : 6) rotary_kernel(const __grid_constant__ convrot_rotary_args a, const RotaryShape s)
{
    // Whether a's and b's are apart: in the half layout, and where single elements are all that is aligned.
    constexpr bool kSplit = !kInterleaved || kVec == 1;
    constexpr int kPairs = kSplit ? kVec : kVec / 2;  // pairs a thread turns in one head
    after_previous();
    let_next_start();
    const int per_row = s.slots * s.head_groups;
    for (int i = threadIdx.x; i < per_row * s.rows_per_block; i += blockDim.x) {
        const int local = i / per_row, rest = i - local * per_row;
        const int group = rest / s.slots, slot = rest - group * s.slots;
        const uint32_t row = blockIdx.x * static_cast<uint32_t>(s.rows_per_block) + local;
        if (row >= s.rows) return;
        const uint32_t b = row / static_cast<uint32_t>(a.tokens), t = row - b * static_cast<uint32_t>(a.tokens);
        const bool copy = slot >= s.pair_slots;
        if (copy && s.skip_copy) continue;
        // first element of the slot's a's, and of its b's where they are apart
        const int e0 = copy ? a.rot_dim + (slot - s.pair_slots) * kVec : slot * (kInterleaved && kSplit ? 2 : kVec);
        const int e1 = e0 + (kInterleaved ? 1 : a.rot_dim / 2);

        Raw<T, kVec> v0[kHeads], v1[kHeads];
        const int heads = static_cast<int>(a.q_heads + a.k_heads);
#pragma unroll
        for (int j = 0; j < kHeads; ++j) {
            const int h = group + j * s.head_groups;
            if (h >= heads) break;
            const bool is_k = h >= a.q_heads;
            const T *p = is_k ? static_cast<const T *>(a.k) + b * a.k_strides[0] + t * a.k_strides[1] +
                                    (h - a.q_heads) * a.k_strides[2]
                              : static_cast<const T *>(a.q) + b * a.q_strides[0] + t * a.q_strides[1] + h * a.q_strides[2];
            v0[j].load_stream(p + e0);
            if (kSplit && !copy) v1[j].load_stream(p + e1);
        }
        float c[kPairs], n[kPairs];
        if (!copy) {
            int64_t pos = t;
            if (a.positions) {
                const int64_t at = b * a.pos_stride + t;
                pos = a.position_bits == 64 ? static_cast<const int64_t *>(a.positions)[at]
                                            : static_cast<const int32_t *>(a.positions)[at];
            }
            const int first = slot * kPairs;
            if (pos < 0 || pos >= a.table_rows) {
                if (a.dev_status) atomicExch(a.dev_status, static_cast<int32_t>(CONVROT_ERR_INVALID_ARG));
#pragma unroll
                for (int e = 0; e < kPairs; ++e) c[e] = n[e] = nanf("");
            } else {
                const float *cp = a.cos + pos * a.ldt + first, *sp = a.sin + pos * a.ldt + first;
                if (kPairs % 4 == 0 && s.vec_table) {
                    Raw<float, (kPairs % 4 ? 4 : kPairs)> cr, sr;
                    cr.load(cp);
                    sr.load(sp);
                    if constexpr (kPairs % 4 == 0) {
                        cr.unpack(c);
                        sr.unpack(n);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < kPairs; ++e) {
                        c[e] = cp[e];
                        n[e] = sp[e];
                    }
                }
                if (a.inverse) {
#pragma unroll
                    for (int e = 0; e < kPairs; ++e) n[e] = -n[e];
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kHeads; ++j) {
            const int h = group + j * s.head_groups;
            if (h >= heads) break;
            const bool is_k = h >= a.q_heads;
            T *p = is_k ? static_cast<T *>(a.out_k) + b * a.out_k_strides[0] + t * a.out_k_strides[1] +
                              (h - a.q_heads) * a.out_k_strides[2]
                        : static_cast<T *>(a.out_q) + b * a.out_q_strides[0] + t * a.out_q_strides[1] +
                              h * a.out_q_strides[2];
            if (copy) {
                v0[j].store_stream(p + e0);
                continue;
            }
            float x[kVec], y[kVec];
            v0[j].unpack(x);
            if (kSplit) v1[j].unpack(y);
#pragma unroll
            for (int e = 0; e < kPairs; ++e) {
                float &pa = kSplit ? x[e] : x[2 * e], &pb = kSplit ? y[e] : x[2 * e + 1];
                const float va = pa, vb = pb;
                // (which product is rounded on its own is fixed, so that every form gives the same bits)
                pa = fmaf(va, c[e], -__fmul_rn(vb, n[e]));
                pb = fmaf(vb, c[e], __fmul_rn(va, n[e]));
            }
            v0[j].pack(x);
            if (kSplit) v1[j].pack(y);
            v0[j].store_stream(p + e0);
            if (kSplit) v1[j].store_stream(p + e1);
        }
    }
}

template <typename T, int kVec, bool kInterleaved, int kHeads>
cudaError_t launch_form(const convrot_rotary_args &a, cudaStream_t stream)
{
    RotaryShape s{};
    const int64_t heads = a.q_heads + a.k_heads;
    const bool same_q = a.q_heads == 0 || (a.q == a.out_q && a.q_strides[0] == a.out_q_strides[0] &&
                                           a.q_strides[1] == a.out_q_strides[1] && a.q_strides[2] == a.out_q_strides[2]);
    const bool same_k = a.k_heads == 0 || (a.k == a.out_k && a.k_strides[0] == a.out_k_strides[0] &&
                                           a.k_strides[1] == a.out_k_strides[1] && a.k_strides[2] == a.out_k_strides[2]);
    s.skip_copy = same_q && same_k;
    s.pair_slots = a.rot_dim / (kInterleaved && kVec > 1 ? kVec : 2 * kVec);
    s.slots = s.pair_slots + (a.head_dim - a.rot_dim) / kVec;
    s.head_groups = static_cast<int32_t>((heads + kHeads - 1) / kHeads);
    s.rows = static_cast<uint32_t>(a.batch * a.tokens);
    s.vec_table = aligned_to(a.cos, 16) && aligned_to(a.sin, 16) && a.ldt % 4 == 0;
    // rows together in a block until few lanes of its warps idle; a row of more items in equal rounds of the block
    const int64_t per_row = static_cast<int64_t>(s.slots) * s.head_groups;
    int best = 1;
    double best_use = 0.0;
    for (int r = 1; r <= 16 && r * per_row <= kRotaryThreads; ++r) {
        const double use = static_cast<double>(r * per_row) / static_cast<double>((r * per_row + 31) / 32 * 32);
        if (use > best_use - 1e-9) {
            best = r;
            best_use = use;
        }
    }
    s.rows_per_block = best;
    const int64_t items = best * per_row, rounds = (items + kRotaryThreads - 1) / kRotaryThreads;
    const unsigned threads = static_cast<unsigned>(((items + rounds - 1) / rounds + 31) / 32 * 32);
    const unsigned blocks = (s.rows + best - 1) / best;
    return launch_after(rotary_kernel<T, kVec, kInterleaved, kHeads>, dim3(blocks), threads, 0, stream, 1, a, s);
}

template <typename T, int kVec>
cudaError_t launch_vec(const convrot_rotary_args &a, cudaStream_t stream)
{
    // Several heads a thread (16 registers of values) once that still fills the GPU (152 SMs of 2048 threads, twice
    // over); one below, where the latency of one load after another would count.
    const int64_t slots = a.head_dim / kVec * (a.q_heads + a.k_heads) * a.batch * a.tokens;
    const bool many = slots / 4 >= 2 * 152 * 2048;
    if (a.layout == CONVROT_ROTARY_INTERLEAVED)
        return many ? launch_form<T, kVec, true, kVec == 1 ? 2 : 4>(a, stream) : launch_form<T, kVec, true, 1>(a, stream);
    return many ? launch_form<T, kVec, false, 2>(a, stream) : launch_form<T, kVec, false, 1>(a, stream);
}

// Whether every access of `vec` consecutive elements is aligned to its size.
bool fits(const convrot_rotary_args &a, int vec, int size)
{
    const int64_t bytes = static_cast<int64_t>(vec) * size;
    const int span = a.layout == CONVROT_ROTARY_HALF ? a.rot_dim / 2 : a.rot_dim;
    if (span % vec || (a.head_dim - a.rot_dim) % vec) return false;
    auto tensor = [&](const void *p, const int64_t *strides, int64_t heads) {
        if (heads == 0) return true;
        const int64_t n[3] = {a.batch, a.tokens, heads};
        if (!aligned_to(p, bytes)) return false;
        for (int i = 0; i < 3; ++i)
            if (n[i] > 1 && strides[i] % vec) return false;
        return true;
    };
    return tensor(a.q, a.q_strides, a.q_heads) && tensor(a.out_q, a.out_q_strides, a.q_heads) &&
           tensor(a.k, a.k_strides, a.k_heads) && tensor(a.out_k, a.out_k_strides, a.k_heads);
}

// The angle of a late position: the product is taken in 64 bits (a position of
// 10^7 times a frequency of 1 is known to 10^-9), and so are its sine and
// cosine. Run once for a table, so the slow 64-bit units do not matter.
__global__ void rotary_table_kernel(const double *positions, int64_t rows, int32_t axes, const double *freq,
                                    const int32_t *axis, int32_t pairs, double factor, float *cos_out, float *sin_out,
                                    int64_t ldt)
{
    const int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
    if (i >= rows * pairs) return;
    const int64_t p = i / pairs;
    const int e = static_cast<int>(i % pairs);
    const int ax = axis ? axis[e] : 0;
    double s = nan(""), c = nan("");
    if (ax >= 0 && ax < axes) {
        const double at = positions ? positions[p * axes + ax] : static_cast<double>(p);
        sincos(at * freq[e], &s, &c);
    }
    cos_out[p * ldt + e] = static_cast<float>(factor * c);
    sin_out[p * ldt + e] = static_cast<float>(factor * s);
}

}  // namespace

cudaError_t launch_rotary(const convrot_rotary_args &a, cudaStream_t stream)
{
    // the widest access that the strides and the sizes of the head's parts allow
    return with_dtype(a.dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        constexpr int size = sizeof(T);
        if (fits(a, 16 / size, size)) return launch_vec<T, 16 / size>(a, stream);
        if (fits(a, 8 / size, size)) return launch_vec<T, 8 / size>(a, stream);
        if (size == 2 && fits(a, 2, size)) return launch_vec<T, 2>(a, stream);
        return launch_vec<T, 1>(a, stream);
    });
}

cudaError_t launch_rotary_table(const double *positions, int64_t rows, int32_t axes, const double *freq,
                                const int32_t *axis, int32_t pairs, double factor, float *cos, float *sin,
                                int64_t ldt, cudaStream_t stream)
{
    const int64_t blocks = (rows * pairs + 255) / 256;
    rotary_table_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(positions, rows, axes, freq, axis, pairs,
                                                                           factor, cos, sin, ldt);
    return cudaGetLastError();
}

}  // namespace convrot
