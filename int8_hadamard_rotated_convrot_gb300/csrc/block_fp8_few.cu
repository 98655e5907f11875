// The block-scaled linear for few rows (include/convrot_block.h): at most 64,
// where reading the weights once is all the work.
//
// The weights are the MMA's M side: a CTA takes 128 rows of w and all rows of
// x as the N side (16, 32 or 64 columns), so no tensor-core row is wasted and
// an accumulator of one block of 128 features is 16 to 64 columns of tensor
// memory. k is split over a cluster of up to eight CTAs, so that a projection
// of a few thousand rows fills the GPU; their partial sums meet in distributed
// shared memory, added in a fixed order. Every block of k has its accumulator
// (at most 512 columns for a CTA's share), so nothing waits for a drain.
//
//   warp 0      TMA producer: 16 KB of w a block into a ring of kStages
//   warp 1      tensor memory; one thread issues the MMAs
//   warps 2-9   quantize x (kQuantize: at most 16 rows; a call is one launch)
//   warps 2-5   drain: lane = row of w, 16 to 64 sums in registers
//
// Bound: the weights' bytes over HBM (or L2, where they stay there between
// calls), and the latency of one launch.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "block.h"
#include "internal.h"
#include "tc_common.cuh"

namespace convrot {
namespace {

using namespace tc;

constexpr int kBK = 128, kBM = 128, kMmaK = 32;
constexpr int kStages = 4, kStageBytes = kBM * kBK;
constexpr int kXWarps = 8;       // that prepare x
constexpr int kThreads = 64 + 32 * kXWarps;
constexpr int kMaxBlocks = 32;   // a CTA's share of k: 512 columns of tensor memory / 16
constexpr int kMaxSplit = 8;     // CTAs of a cluster

struct FewParams {
    int32_t m, n, k, blocks, split;
    const void *x;        // kQuantize: the rows
    int64_t ldx;
    int32_t wide_x;       // its rows can be read 4 elements at a time
    const float *x_scale; // packed x
    int64_t ld_x_scale;
    const float *w_scale, *bias;
    int64_t ld_w_scale;
    void *y;
    int64_t ldy;
    int32_t *dev_status;
    uint32_t tmem_cols;
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

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ float remote_f32(uint32_t local, uint32_t rank)
{
    uint32_t at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(local), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

// kTok: columns of an accumulator (rows of x, rounded up); TX: type of the rows
// that are quantized here (void: x is packed); T: type of y.
template <int kTok, typename TX, typename T, int kAct>
__global__ void __launch_bounds__(kThreads)
    fp8_few_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, const __grid_constant__ FewParams p)
{
    constexpr bool kQuantize = !std::is_void_v<TX>;
    constexpr int kTile = kTok * kBK;  // x's codes of one block
    // kind::f8f6f4: D fp32, A and B e4m3, K-major, M = 128, N = kTok
    constexpr uint32_t kIdesc = (1u << 4) | (uint32_t(kTok >> 3) << 17) | (uint32_t(kBM >> 4) << 24);
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * kStages + 2 * kMaxBlocks + 1];
    __shared__ __align__(16) float scales[512];  // [block][row of x]: s_x s_w
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    const uint32_t raw = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw));
    const uint32_t base = (raw + 1023u) & ~1023u;  // swizzle atoms are 1024-byte aligned
    const uint32_t xtiles = base + kStages * kStageBytes;
    const uint32_t bar0 = static_cast<uint32_t>(__cvta_generic_to_shared(bars));
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (kStages + s); };
    auto x_bar = [&](int j) { return bar0 + 8u * (2 * kStages + j); };                  // x's codes of the block are there
    auto sum_bar = [&](int j) { return bar0 + 8u * (2 * kStages + kMaxBlocks + j); };   // the block's sums are
    const uint32_t done_bar = bar0 + 8u * (2 * kStages + 2 * kMaxBlocks);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t split = static_cast<uint32_t>(p.split), rank = split > 1 ? cluster_rank() : 0;
    const int tile = static_cast<int>(blockIdx.x / split);
    const int j0 = static_cast<int>(static_cast<int64_t>(p.blocks) * rank / split);
    const int count = static_cast<int>(static_cast<int64_t>(p.blocks) * (rank + 1) / split) - j0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int j = 0; j < count; ++j) {
            mbar_init(x_bar(j), kQuantize ? kXWarps : 1);
            mbar_init(sum_bar(j), 1);
        }
        mbar_init(done_bar, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmW)) : "memory");
        if constexpr (!kQuantize) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmX)) : "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         static_cast<uint32_t>(__cvta_generic_to_shared(&tmem_slot))),
                     "r"(p.tmem_cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what the kernel before wrote is there

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
            if constexpr (!kQuantize) {
                for (int j = 0; j < count; ++j) {  // all of this CTA's x at once
                    mbar_arrive_expect_tx(x_bar(j), kTile);
                    tma_load_2d(xtiles + j * kTile, &tmX, (j0 + j) * kBK, 0, x_bar(j));
                }
            }
            for (int j = 0; j < count; ++j) {
                const int s = j % kStages;
                if (!wait(empty_bar(s), (j / kStages + 1) & 1)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(full_bar(s), kStageBytes);
                tma_load_2d(base + s * kStageBytes, &tmW, (j0 + j) * kBK, tile * kBM, full_bar(s));
                ++issued;
            }
            if (!ok) {
                fail();
                // copies in flight land before shared memory goes away
                for (int j = issued > kStages ? issued - kStages : 0; j < issued; ++j) mbar_wait(full_bar(j % kStages), (j / kStages) & 1);
                if constexpr (!kQuantize)
                    for (int j = 0; j < count; ++j) mbar_wait(x_bar(j), 0);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            bool ok = true;
            for (int j = 0; j < count; ++j) {
                const int s = j % kStages;
                if (!wait(x_bar(j), 0) || !wait(full_bar(s), (j / kStages) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t da = smem_desc(base + s * kStageBytes), db = smem_desc(xtiles + j * kTile);
#pragma unroll
                for (int kk = 0; kk < kBK / kMmaK; ++kk)  // 32 bytes along K inside the swizzle span
                    mma(tmem + j * kTok, da + 2u * kk, db + 2u * kk, kIdesc, kk > 0 ? 1u : 0u);
                mma_commit(empty_bar(s));
                mma_commit(sum_bar(j));
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
            const int units = count * p.m;
            int arrived = 0;  // blocks that this warp has nothing left to add to
            for (int u0 = w; u0 - w < units || arrived < count; u0 += kXWarps * kBatch) {
                float v[kBatch][4], sw_j[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int u = u0 + i * kXWarps, j = u / p.m, r = u - j * p.m, c = (j0 + j) * kBK + lane * 4;
                    if (u >= units) break;
                    const TX *from = static_cast<const TX *>(p.x) + r * p.ldx + c;
                    sw_j[i] = __ldg(sw + j);
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
                    const int u = u0 + i * kXWarps, j = u / p.m, r = u - j * p.m;
                    if (u >= units) break;
                    float amax = fmaxf(fmaxf(fabsf(v[i][0]), fabsf(v[i][1])), fmaxf(fabsf(v[i][2]), fabsf(v[i][3])));
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                    amax = fmaxf(amax, kFp8AmaxFloor);
                    const float up = fp8_up(amax);
                    const uint32_t to = xtiles + j * kTile + r * kBK + (((lane >> 2) ^ (r & 7)) << 4) + ((lane & 3) << 2);
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(e4m3x4(v[i][0] * up, v[i][1] * up, v[i][2] * up, v[i][3] * up))
                                 : "memory");
                    if (lane == 0) scales[j * kTok + r] = (amax / kFp8Max) * sw_j[i];
                }
                // blocks before the next batch's first are done as far as this warp goes
                const int next = u0 + kXWarps * kBatch, until = next < units ? next / p.m : count;
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
                scales[i] = r < p.m ? __ldg(p.x_scale + (j0 + j) * p.ld_x_scale + r) * __ldg(sw + j) : 0.0f;
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
                if (!wait(sum_bar(j), 0)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < kTok; c += 16) {
                    if (c >= p.m) break;
                    uint32_t r[16];
                    tmem_ld16(tmem + (static_cast<uint32_t>(q * 32) << 16) + j * kTok + c, r);
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 s = *reinterpret_cast<const float4 *>(&scales[j * kTok + c + i]);
                        acc[c + i] = fmaf(__uint_as_float(r[i]), s.x, acc[c + i]);
                        acc[c + i + 1] = fmaf(__uint_as_float(r[i + 1]), s.y, acc[c + i + 1]);
                        acc[c + i + 2] = fmaf(__uint_as_float(r[i + 2]), s.z, acc[c + i + 2]);
                        acc[c + i + 3] = fmaf(__uint_as_float(r[i + 3]), s.w, acc[c + i + 3]);
                    }
                }
            }
            if (!ok) fail();
            // this CTA's sums, [row of x][row of w], over the ring's first stages: the last MMA has read them (sum_bar)
            const uint32_t sums = base + (q * 32 + lane) * 4;
#pragma unroll
            for (int i = 0; i < kTok; ++i)
                if (i < p.m && ok) asm volatile("st.shared.f32 [%0], %1;" ::"r"(sums + i * kBM * 4), "f"(acc[i]) : "memory");
        }
    }

    tc_fence_before();
    if (split > 1)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.tmem_cols) : "memory");
    } else if (warp > 1) {
        // the cluster's warps share out the outputs, 32 rows of w of one row of x at a time
        for (int u = static_cast<int>(rank) * kXWarps + warp - 2; u < p.m * 4; u += static_cast<int>(split) * kXWarps) {
            const int r = u >> 2, o = (u & 3) * 32 + lane;
            const uint32_t at = base + (r * kBM + o) * 4;
            float v = 0.0f;
            if (split > 1) {
                for (uint32_t c = 0; c < split; ++c) v += remote_f32(at, c);
            } else {
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
            }
            const int64_t col = static_cast<int64_t>(tile) * kBM + o;
            if (col >= p.n) continue;
            if (p.bias) v += __ldg(p.bias + col);
            static_cast<T *>(p.y)[r * p.ldy + col] = from_f32<T>(apply_act_t<kAct>(v));
        }
    }
    if (split > 1) cluster_sync();  // a CTA's sums stay until its peers have read them
}

template <int kTok, typename TX, typename T, int kAct>
struct kernel_tag;

template <int kTok, typename TX, typename T, int kAct>
cudaError_t launch_form(const convrot_fp8_linear_args &a, int split, cudaStream_t stream)
{
    CUtensorMap tmX{}, tmW;
    if (!make_map_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, a.n, a.k, a.ldw, kBK, kBM)) return cudaErrorInvalidValue;
    if constexpr (std::is_void_v<TX>)
        if (!make_map_2d(&tmX, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.x, a.m, a.k, a.ldx, kBK, kTok)) return cudaErrorInvalidValue;
    FewParams p{};
    p.m = static_cast<int32_t>(a.m);
    p.n = static_cast<int32_t>(a.n);
    p.k = static_cast<int32_t>(a.k);
    p.blocks = static_cast<int32_t>((a.k + kBK - 1) / kBK);
    p.split = split;
    p.x = a.x;
    p.ldx = a.ldx;
    if constexpr (!std::is_void_v<TX>)
        p.wide_x = aligned_to(a.x, 4 * sizeof(TX)) && (a.m <= 1 || a.ldx % 4 == 0);
    p.x_scale = a.x_scale;
    p.ld_x_scale = a.ld_x_scale;
    p.w_scale = a.w_scale;
    p.ld_w_scale = a.ld_w_scale;
    p.bias = a.bias;
    p.y = a.y;
    p.ldy = a.ldy;
    p.dev_status = a.dev_status;
    const int share = (p.blocks + split - 1) / split;
    p.tmem_cols = 32;
    while (static_cast<int>(p.tmem_cols) < share * kTok) p.tmem_cols *= 2;
    // An allocation of tensor memory waits until there is room, and CTAs of two clusters that wait for each other's
    // room on two SMs would wait for ever. So a CTA takes at least the part of an SM's shared memory (228 KB) that it
    // takes of its 512 columns, less 4 KB: of such CTAs, each of 64 KB at least and of a multiple of 32 columns, three
    // at most fit side by side, and their columns would need 544 x 456 B - 3 x 4 KB > 228 KB to be too many.
    int bytes = 1024 + kStages * kStageBytes + share * kTok * kBK;
    const int part = static_cast<int>(p.tmem_cols) * (228 * 1024 / 512) - 4096;
    if (bytes < part) bytes = part;
    auto kernel = fp8_few_kernel<kTok, TX, T, kAct>;
    cudaError_t e = allow_shared<kernel_tag<kTok, TX, T, kAct>>(kernel);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t config{};
    config.gridDim = dim3(static_cast<unsigned>((a.n + kBM - 1) / kBM * split));
    config.blockDim = dim3(kThreads);
    config.dynamicSmemBytes = bytes;
    config.stream = stream;
    cudaLaunchAttribute attrs[2]{};
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim = {static_cast<unsigned>(split), 1, 1};
    config.attrs = attrs;
    config.numAttrs = split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&config, kernel, tmX, tmW, p);
}

// CTAs that share k: the widest cluster (1, 2, 4 or 8) that still lets every CTA be resident, two an SM, and keeps
// two blocks for each; more where a CTA's blocks would not have an accumulator each. 0: no split does.
int choose_split(int64_t n, int64_t blocks, int tok)
{
    const int64_t tiles = (n + kBM - 1) / kBM;
    const int64_t most = 512 / tok < kMaxBlocks ? 512 / tok : kMaxBlocks;
    int split = 1;
    while (split < kMaxSplit && ((tiles * 2 * split <= 2 * kSms && blocks >= 4 * split) || (blocks + split - 1) / split > most)) split *= 2;
    return (blocks + split - 1) / split <= most ? split : 0;
}

template <int kTok, typename TX>
cudaError_t launch_types(const convrot_fp8_linear_args &a, int split, cudaStream_t stream)
{
    return with_dtype(a.y_dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        if (a.act == CONVROT_ACT_GELU_ERF) return launch_form<kTok, TX, T, 1>(a, split, stream);
        if (a.act == CONVROT_ACT_GELU_TANH) return launch_form<kTok, TX, T, 2>(a, split, stream);
        return launch_form<kTok, TX, T, 0>(a, split, stream);
    });
}

int tokens_of(int64_t m) { return m <= 16 ? 16 : m <= 32 ? 32 : 64; }

}  // namespace

bool fp8_few_takes(int64_t m, int64_t n, int64_t k)
{
    return m <= 64 && choose_split(n, (k + kBK - 1) / kBK, tokens_of(m)) > 0;
}

bool fp8_few_quantizes(int64_t m, int64_t n, int64_t k) { return m <= 16 && fp8_few_takes(m, n, k); }

cudaError_t launch_fp8_few(const convrot_fp8_linear_args &a, cudaStream_t stream)
{
    const int tok = tokens_of(a.m), split = choose_split(a.n, (a.k + kBK - 1) / kBK, tok);
    if (tok == 16) return launch_types<16, void>(a, split, stream);
    if (tok == 32) return launch_types<32, void>(a, split, stream);
    return launch_types<64, void>(a, split, stream);
}

cudaError_t launch_fp8_few_quantize(const convrot_fp8_linear_args &a, cudaStream_t stream)
{
    const int split = choose_split(a.n, (a.k + kBK - 1) / kBK, 16);
    return with_dtype(a.x_dtype, [&](auto *tag) { return launch_types<16, std::remove_pointer_t<decltype(tag)>>(a, split, stream); });
}

}  // namespace convrot
