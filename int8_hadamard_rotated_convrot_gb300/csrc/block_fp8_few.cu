// The block-scaled linear for few rows (include/convrot_block.h), where reading
// the weights and the latency of it all count, not the arithmetic.
//
// The weights are the MMA's M side: a CTA takes 128 rows of w and 16, 32 or 64
// rows of x as the N side, so no tensor-core row is wasted and the accumulator
// of one block of 128 features is 16 to 64 columns of tensor memory, four to
// eight of them in turn. k is split over a cluster of up to eight CTAs, so that
// a projection of a few thousand rows fills the GPU; their partial sums meet in
// distributed shared memory, added in a fixed order.
//
//   warp 0      TMA producer: a block of w (16 KB), and of packed x, a stage
//   warp 1      tensor memory; one thread issues the MMAs
//   warps 2-9   quantize x (kQuantize: at most 16 rows; a call is one launch)
//   warps 2-5   drain: lane = row of w, 16 to 64 sums in registers
//
// Bound by the weights' bytes over HBM (or L2, where they stay there between
// calls) and by its own start and end: at M1 K5120 N5120, weights in L2, the
// first block arrives after 2 us, the ten blocks of a CTA take 3.4 us (7.7
// TB/s), the cluster's sums 0.6 us; 9.1 us a call with the launch.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "block.h"
#include "tc_common.cuh"

namespace convrot {
namespace {

using namespace tc;

constexpr int kBK = 128, kBM = 128, kMmaK = 32;
constexpr int kStages = 4, kStageBytes = kBM * kBK;
constexpr int kXWarps = 8;       // that prepare x
constexpr int kThreads = 64 + 32 * kXWarps;
constexpr int kMaxShare = 128;   // blocks of k a CTA takes: their scales are in shared memory
constexpr int kMaxQuantize = 32; // where it quantizes x: the codes of all its blocks are, too
constexpr int kMaxSplit = 8;     // CTAs of a cluster
// Blocks of rows that a CTA quantizes at most, two rounds of its eight warps; above, a launch of its own (2.4 us) is
// cheaper (M8 K5120 N13824, 160 of them: 22.6 us in one launch, 15.2 in two).
constexpr int kQuantizeUnits = 64;

struct FewParams {
    int32_t m, n, k, blocks, split;
    int32_t groups;       // of kTok rows of x
    int32_t share;        // blocks of k a CTA takes at most
    const void *x;        // kQuantize: the rows
    int64_t ldx;
    int32_t wide_x;       // its rows can be read 4 elements at a time
    const float *x_scale; // packed x
    int64_t ld_x_scale;
    const float *w_scale, *bias;
    int64_t ld_w_scale;
    void *y;
    int64_t ldy;
    int32_t vec_y;        // four elements of a row of y are aligned to their size
    int32_t *dev_status;
};

__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ float4 remote16(uint32_t local, uint32_t rank)
{
    uint32_t at;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(local), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}

template <int kTok, bool kQuantize>
struct Shape {
    static constexpr int TILE = kTok * kBK;  // x's codes of one block
    static constexpr int STAGE = kStageBytes + (kQuantize ? 0 : TILE);
    static constexpr int COLS = kTok == 16 ? 128 : 256, BUFS = COLS / kTok;
    // Shared memory of a CTA that takes up to `share` blocks of k.
    static int bytes(int share)
    {
        const int used = 1024 + kStages * STAGE + share * (kQuantize ? TILE : 0) + share * kTok * 4;
        return used > tmem_share(COLS) ? used : tmem_share(COLS);
    }
};

// kTok: columns of an accumulator (rows of x, rounded up); TX: type of the rows
// that are quantized here (void: x is packed); T: type of y.
template <int kTok, typename TX, typename T, int kAct>
__global__ void __launch_bounds__(kThreads, 2)
    fp8_few_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, const __grid_constant__ FewParams p)
{
    constexpr bool kQuantize = !std::is_void_v<TX>;
    using S = Shape<kTok, kQuantize>;
    // kind::f8f6f4: D fp32, A and B e4m3, K-major, M = 128, N = kTok
    constexpr uint32_t kIdesc = (1u << 4) | (uint32_t(kTok >> 3) << 17) | (uint32_t(kBM >> 4) << 24);
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * kStages + 2 * S::BUFS + (kQuantize ? kMaxQuantize : 0) + 1];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    const uint32_t raw = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw));
    const uint32_t base = (raw + 1023u) & ~1023u;  // swizzle atoms are 1024-byte aligned
    const uint32_t xtiles = base + kStages * S::STAGE;  // kQuantize: x's codes of every block
    // [block][row of x]: s_x s_w
    float *scales = reinterpret_cast<float *>(smem_raw + (xtiles - raw) + (kQuantize ? p.share * S::TILE : 0));
    const uint32_t bar0 = static_cast<uint32_t>(__cvta_generic_to_shared(bars));
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (kStages + s); };
    auto sum_bar = [&](int b) { return bar0 + 8u * (2 * kStages + b); };              // an accumulator is finished
    auto drained_bar = [&](int b) { return bar0 + 8u * (2 * kStages + S::BUFS + b); };  // and free again
    const uint32_t done_bar = bar0 + 8u * (2 * kStages + 2 * S::BUFS);
    auto x_bar = [&](int j) { return done_bar + 8u * (1 + j); };                      // kQuantize: x's codes of the block are there

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t split = static_cast<uint32_t>(p.split), rank = split > 1 ? cluster_rank() : 0;
    const uint32_t unit = blockIdx.x / split, groups = static_cast<uint32_t>(p.groups);
    const int tile = static_cast<int>(unit / groups), row0 = static_cast<int>(unit % groups) * kTok;
    const int m = p.m - row0 < kTok ? p.m - row0 : kTok;  // this CTA's rows of x
    const int j0 = static_cast<int>(static_cast<int64_t>(p.blocks) * rank / split);
    const int count = static_cast<int>(static_cast<int64_t>(p.blocks) * (rank + 1) / split) - j0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < S::BUFS; ++b) {
            mbar_init(sum_bar(b), 1);
            mbar_init(drained_bar(b), 4);
        }
        if constexpr (kQuantize)
            for (int j = 0; j < count; ++j) mbar_init(x_bar(j), kXWarps);
        mbar_init(done_bar, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmW)) : "memory");
        if constexpr (!kQuantize) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmX)) : "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         static_cast<uint32_t>(__cvta_generic_to_shared(&tmem_slot))),
                     "r"(static_cast<uint32_t>(S::COLS))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    after_previous();  // what the kernel before wrote is there
    let_next_start();

    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = globaltimer();
        for (;;) {
#pragma unroll 1
            for (int i = 0; i < 16; ++i)
                if (mbar_try_wait(bar, parity)) return true;
            if (abort_flag || globaltimer() - t0 > kTimeoutNs) return false;
        }
    };
    auto fail = [&]() {
        abort_flag = 1;
        if (p.dev_status) atomicExch(p.dev_status, static_cast<int32_t>(CONVROT_ERR_TIMEOUT));
    };

    if (warp == 0) {
        if (lane == 0) {
            bool ok = true;
            int issued = 0;
            for (int j = 0; j < count; ++j) {
                const int s = j % kStages;
                if (!wait(empty_bar(s), (j / kStages + 1) & 1)) {
                    ok = false;
                    break;
                }
                const uint32_t sa = base + s * S::STAGE;
                mbar_arrive_expect_tx(full_bar(s), S::STAGE);
                tma_load_2d(sa, &tmW, (j0 + j) * kBK, tile * kBM, full_bar(s));
                if constexpr (!kQuantize) tma_load_2d(sa + kStageBytes, &tmX, (j0 + j) * kBK, row0, full_bar(s));
                ++issued;
            }
            if (!ok) {
                fail();
                // copies in flight land before shared memory goes away
                for (int j = issued > kStages ? issued - kStages : 0; j < issued; ++j) mbar_wait(full_bar(j % kStages), (j / kStages) & 1);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            bool ok = true;
            for (int j = 0; j < count; ++j) {
                const int s = j % kStages, buf = j % S::BUFS;
                if (kQuantize && !wait(x_bar(j), 0)) ok = false;
                if (!ok || !wait(drained_bar(buf), (j / S::BUFS + 1) & 1) || !wait(full_bar(s), (j / kStages) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sa = base + s * S::STAGE;
                const uint64_t da = smem_desc(sa), db = smem_desc(kQuantize ? xtiles + j * S::TILE : sa + kStageBytes);
#pragma unroll
                for (int kk = 0; kk < kBK / kMmaK; ++kk)  // 32 bytes along K inside the swizzle span
                    mma(tmem + buf * kTok, da + 2u * kk, db + 2u * kk, kIdesc, kk > 0 ? 1u : 0u);
                mma_commit(empty_bar(s));
                mma_commit(sum_bar(buf));
            }
            if (!ok) fail();
            mma_commit(done_bar);
            mbar_wait(done_bar, 0);
        }
        __syncwarp();
    } else {
        const int w = warp - 2;
        const float *sw = p.w_scale + static_cast<int64_t>(tile) * p.ld_w_scale + j0;
        if constexpr (kQuantize) {
            // A row's block is a warp's at a time, four values a lane; kBatch of them are loaded together. Codes go to
            // the layout that the MMA reads (16-byte chunk c of row r at c ^ (r & 7)).
            constexpr int kBatch = 4;
            const int units = count * m;
            int arrived = 0;  // blocks that this warp has nothing left to add to
            for (int u0 = w; u0 - w < units || arrived < count; u0 += kXWarps * kBatch) {
                float v[kBatch][4], sw_j[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int u = u0 + i * kXWarps, j = u / m, r = u - j * m, c = (j0 + j) * kBK + lane * 4;
                    if (u >= units) break;
                    const TX *from = static_cast<const TX *>(p.x) + r * p.ldx + c;
                    sw_j[i] = load_f32(sw + j);
                    if (p.wide_x && c + 4 <= p.k) {
                        Raw<TX, 4> four;
                        four.load(from);
                        four.unpack(v[i]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[i][e] = c + e < p.k ? to_f32(from[e]) : 0.0f;
                    }
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int u = u0 + i * kXWarps, j = u / m, r = u - j * m;
                    if (u >= units) break;
                    float amax = fmaxf(fmaxf(fabsf(v[i][0]), fabsf(v[i][1])), fmaxf(fabsf(v[i][2]), fabsf(v[i][3])));
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                    amax = fmaxf(amax, kFp8AmaxFloor);
                    const float up = fp8_up(amax);
                    const uint32_t to = xtiles + j * S::TILE + r * kBK + (((lane >> 2) ^ (r & 7)) << 4) + ((lane & 3) << 2);
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(e4m3x4(v[i][0] * up, v[i][1] * up, v[i][2] * up, v[i][3] * up))
                                 : "memory");
                    if (lane == 0) scales[j * kTok + r] = (amax / kFp8Max) * sw_j[i];
                }
                // blocks before the next batch's first are done as far as this warp goes
                const int next = u0 + kXWarps * kBatch, until = next < units ? next / m : count;
                if (arrived < until) {
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the tensor cores read these bytes
                    __syncwarp();
                    if (lane == 0)
                        for (int j = arrived; j < until; ++j) mbar_arrive(x_bar(j));
                    arrived = until;
                }
            }
        } else {
            for (int i = threadIdx.x - 64; i < count * kTok; i += 32 * kXWarps) {
                const int j = i / kTok, r = i % kTok;
                scales[i] = r < m ? load_f32(p.x_scale + (j0 + j) * p.ld_x_scale + row0 + r) * load_f32(sw + j) : 0.0f;
            }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kXWarps) : "memory");  // every row's scales, among these warps
        if (w < 4) {
            const int q = warp & 3;  // tensor-memory lanes of this warp
            float acc[kTok];
#pragma unroll
            for (int i = 0; i < kTok; ++i) acc[i] = 0.0f;
            bool ok = true;
            for (int j = 0; j < count; ++j) {
                const int buf = j % S::BUFS;
                if (!all_lanes(wait(sum_bar(buf), (j / S::BUFS) & 1))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < kTok; c += 16) {
                    if (c >= m) break;
                    uint32_t r[16];
                    tmem_ld16(tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * kTok + c, r);
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 s = *reinterpret_cast<const float4 *>(&scales[j * kTok + c + i]);
                        acc[c + i] = fmaf(__uint_as_float(r[i]), s.x, acc[c + i]);
                        acc[c + i + 1] = fmaf(__uint_as_float(r[i + 1]), s.y, acc[c + i + 1]);
                        acc[c + i + 2] = fmaf(__uint_as_float(r[i + 2]), s.z, acc[c + i + 2]);
                        acc[c + i + 3] = fmaf(__uint_as_float(r[i + 3]), s.w, acc[c + i + 3]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(drained_bar(buf));
            }
            if (!ok) fail();
            // this CTA's sums, [row of x][row of w], over the ring's stages: the last MMA has read them (sum_bar)
            const uint32_t sums = base + (q * 32 + lane) * 4;
#pragma unroll
            for (int i = 0; i < kTok; ++i)
                if (i < m && ok) asm volatile("st.shared.f32 [%0], %1;" ::"r"(sums + i * kBM * 4), "f"(acc[i]) : "memory");
        }
    }

    tc_fence_before();
    if (split > 1)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(static_cast<uint32_t>(S::COLS)) : "memory");
    } else if (warp > 1) {
        // the cluster's warps share out the rows of x, four columns of y a lane; a row's partial sums are all in flight
        const int64_t col = static_cast<int64_t>(tile) * kBM + lane * 4;
        float bias[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) bias[e] = p.bias && col + e < p.n ? load_f32(p.bias + col + e) : 0.0f;
        for (int r = static_cast<int>(rank) * kXWarps + warp - 2; r < m; r += static_cast<int>(split) * kXWarps) {
            const uint32_t at = base + (r * kBM + lane * 4) * 4;
            float4 part[kMaxSplit];
#pragma unroll
            for (uint32_t c = 0; c < kMaxSplit; ++c)
                if (c < split) part[c] = remote16(at, split > 1 ? c : 0);
            float v[4] = {};
#pragma unroll
            for (uint32_t c = 0; c < kMaxSplit; ++c) {
                if (c >= split) break;
                v[0] += part[c].x;
                v[1] += part[c].y;
                v[2] += part[c].z;
                v[3] += part[c].w;
            }
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const F2 two = act2<kAct>(F2(v[e] + bias[e], v[e + 1] + bias[e + 1]));
                v[e] = two.lo();
                v[e + 1] = two.hi();
            }
            T *y = static_cast<T *>(p.y) + (row0 + r) * p.ldy + col;
            if (p.vec_y && col + 4 <= p.n) {
                Raw<T, 4> raw;
                raw.pack(v);
                raw.store(y);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (col + e < p.n) y[e] = from_f32<T>(v[e]);
            }
        }
    }
    if (split > 1) cluster_sync();  // a CTA's sums stay until its peers have read them
}

template <int kTok, typename TX, typename T, int kAct>
struct kernel_tag;

// How a call is cut: groups of tok rows of x, and CTAs that share k.
struct Cut {
    int tok = 0, groups = 0, split = 0, share = 0;
};

template <int kTok, typename TX, typename T, int kAct>
cudaError_t launch_form(const convrot_fp8_linear_args &a, const Cut &cut, cudaStream_t stream)
{
    constexpr bool kQuantize = !std::is_void_v<TX>;
    using S = Shape<kTok, kQuantize>;
    CUtensorMap tmX{}, tmW;
    if (!make_map_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, a.n, a.k, a.ldw, kBK, kBM)) return cudaErrorInvalidValue;
    if constexpr (!kQuantize)
        if (!make_map_2d(&tmX, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.x, a.m, a.k, a.ldx, kBK, kTok)) return cudaErrorInvalidValue;
    FewParams p{};
    p.m = static_cast<int32_t>(a.m);
    p.n = static_cast<int32_t>(a.n);
    p.k = static_cast<int32_t>(a.k);
    p.blocks = static_cast<int32_t>((a.k + kBK - 1) / kBK);
    p.split = cut.split;
    p.groups = cut.groups;
    p.share = cut.share;
    p.x = a.x;
    p.ldx = a.ldx;
    if constexpr (kQuantize) p.wide_x = aligned_to(a.x, 4 * sizeof(TX)) && (a.m <= 1 || a.ldx % 4 == 0);
    p.x_scale = a.x_scale;
    p.ld_x_scale = a.ld_x_scale;
    p.w_scale = a.w_scale;
    p.ld_w_scale = a.ld_w_scale;
    p.bias = a.bias;
    p.y = a.y;
    p.ldy = a.ldy;
    p.vec_y = aligned_to(a.y, 4 * sizeof(T)) && (a.m <= 1 || a.ldy % 4 == 0);
    p.dev_status = a.dev_status;
    const int bytes = S::bytes(cut.share);
    auto kernel = fp8_few_kernel<kTok, TX, T, kAct>;
    cudaError_t e = allow_shared<kernel_tag<kTok, TX, T, kAct>>(kernel);
    if (e != cudaSuccess) return e;
    return launch_after(kernel, dim3(static_cast<unsigned>((a.n + kBM - 1) / kBM * cut.groups * cut.split)), kThreads, bytes, stream,
                        static_cast<unsigned>(cut.split), tmX, tmW, p);
}

// CTAs that are resident together, two an SM: clusters of 4 and 8 leave some SMs of a GPC over (36 and 15 of them fit
// at one CTA an SM).
int resident(int split) { return split <= 2 ? 2 * kSms : split == 4 ? 2 * 36 * 4 : 2 * 15 * 8; }

// The widest cluster (1, 2, 4 or 8) with which every CTA is still resident and has two blocks of k. Up to 64 rows
// this kernel takes any call whose shares fit; more rows only where all groups of them are resident together.
Cut cut_of(int64_t m, int64_t n, int64_t k)
{
    const int64_t tiles = (n + kBM - 1) / kBM, blocks = (k + kBK - 1) / kBK;
    Cut best;
    for (int tok : {16, 32, 64}) {
        if (tok == 16 && m > 16) continue;
        Cut c;
        c.tok = tok;
        c.groups = static_cast<int>((m + tok - 1) / tok);
        const int64_t units = c.groups * tiles;
        if (c.groups > 1 && units > resident(1)) continue;
        c.split = 1;
        while (c.split < kMaxSplit &&
               ((units * 2 * c.split <= resident(2 * c.split) && blocks >= 4 * c.split) || (blocks + c.split - 1) / c.split > kMaxShare))
            c.split *= 2;
        c.share = static_cast<int>((blocks + c.split - 1) / c.split);
        if (c.share > kMaxShare) continue;
        // a CTA's time is that of its blocks, the wider ones a little longer
        if (!best.tok || c.share * (64 + c.tok) < best.share * (64 + best.tok)) best = c;
        if (m <= tok) break;
    }
    return best;
}

template <int kTok, typename TX>
cudaError_t launch_types(const convrot_fp8_linear_args &a, const Cut &cut, cudaStream_t stream)
{
    return with_dtype(a.y_dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        if (a.act == CONVROT_ACT_GELU_ERF) return launch_form<kTok, TX, T, 1>(a, cut, stream);
        if (a.act == CONVROT_ACT_GELU_TANH) return launch_form<kTok, TX, T, 2>(a, cut, stream);
        return launch_form<kTok, TX, T, 0>(a, cut, stream);
    });
}

}  // namespace

bool fp8_few_takes(int64_t m, int64_t n, int64_t k) { return cut_of(m, n, k).tok > 0; }

bool fp8_few_quantizes(int64_t m, int64_t n, int64_t k)
{
    const Cut c = cut_of(m, n, k);
    return c.tok == 16 && c.share <= kMaxQuantize && c.share * m <= kQuantizeUnits;
}

int fp8_few_shared(int64_t m, int64_t n, int64_t k, bool quantize, int *columns)
{
    const Cut c = cut_of(m, n, k);
    *columns = c.tok == 16 ? Shape<16, true>::COLS : Shape<32, false>::COLS;
    static_assert(Shape<32, false>::COLS == Shape<64, false>::COLS);
    if (c.tok == 16) return quantize ? Shape<16, true>::bytes(c.share) : Shape<16, false>::bytes(c.share);
    return c.tok == 32 ? Shape<32, false>::bytes(c.share) : Shape<64, false>::bytes(c.share);
}

cudaError_t launch_fp8_few(const convrot_fp8_linear_args &a, cudaStream_t stream)
{
    const Cut c = cut_of(a.m, a.n, a.k);
    if (c.tok == 16) return launch_types<16, void>(a, c, stream);
    if (c.tok == 32) return launch_types<32, void>(a, c, stream);
    return launch_types<64, void>(a, c, stream);
}

cudaError_t launch_fp8_few_quantize(const convrot_fp8_linear_args &a, cudaStream_t stream)
{
    const Cut c = cut_of(a.m, a.n, a.k);
    return with_dtype(a.x_dtype, [&](auto *tag) { return launch_types<16, std::remove_pointer_t<decltype(tag)>>(a, c, stream); });
}

}  // namespace convrot
