// The matrix products of the gated feed-forward's projections and of their
// gradient (include/convrot_block.h) on the 5th-generation tensor cores:
//
//   kForward  y = act(x w_gate^T + b_gate) * (x w_up^T + b_up)
//   kDx       dx = dg w_gate + du w_up        (one sum over both)
//   kDw       dw_gate = dg^T x, dw_up = du^T x
//
// A CTA pair (cluster of 2, cta_group::2), persistent over output tiles of 256
// rows and kBN accumulator columns, K in steps of 64:
//   warp 0      TMA producer of each CTA: its 128 rows of A and kBN / 2 of B
//   warp 1      tensor memory; in the even CTA one thread issues the MMAs
//   warps 4-11  drain: two warps a lane quadrant, half of the columns each
// Two accumulators of kBN columns, so that a tile's end runs under the next
// tile's products.
//
// kForward takes the gate's columns from the even CTA's rows of B and the up
// projection's from the odd one's: a tile is kBN / 2 columns of y, and a drain
// thread has both values of its outputs in its own lane, so that nothing of g
// and u leaves the SM. The gradients need no transposed copies: what is
// contracted over rows (w in kDx, both operands in kDw) is read MN-major from
// boxes of 64 x 64.
//
// Bound by the tensor cores: 32760 x 5120 x 13824 in 5.2 to 5.3 ms (1740 to 1790
// TFLOP/s, over cuBLAS's sustained rate), 8190 rows' dx and dw in 1.29 and 1.28 ms
// (1795 and 1815).
#include "gated.h"
#include "mma16.cuh"

namespace convrot {
namespace {

using namespace mma16;

enum Mode { kForward, kDx, kDw };

constexpr int kMaxSplits = 8;

constexpr int kBK = 64;   // of K a step: one swizzle span, or 64 rows
constexpr int kBM = 128;  // rows of A (and of the accumulators) per CTA
constexpr int kDrainWarps = 8, kThreads = 128 + 32 * kDrainWarps;

template <int kBN>
struct Cfg {
    static constexpr int A_BYTES = kBM * kBK * 2, B_BYTES = kBN / 2 * kBK * 2, STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int BUFS = 2;
    static constexpr int BAR_BYTES = 256;
    static constexpr int FIT = (kMaxShared - 1024 - kDrainWarps * kStageBytes - BAR_BYTES) / STAGE_BYTES;
    static constexpr int STAGES = FIT < 8 ? FIT : 8;
    static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + kDrainWarps * kStageBytes + BAR_BYTES;
    static_assert(SMEM > kTmemAlone, "no other tensor memory on this SM");
    static_assert(8 * (2 * STAGES + 2 * BUFS + 1) + 8 <= BAR_BYTES, "barriers fit");
    static_assert(BUFS * kBN <= 512, "accumulators fit");
};

struct Params {
    int32_t rows, cols;   // of an output (kForward: of y)
    int32_t tiles_m, tiles_n;
    int32_t steps;        // of K, in one operand pair
    int32_t parts;        // operand pairs that one sum runs over (kDx: 2)
    int32_t sections;     // outputs one above the other (kDw: 2)
    int32_t splits;       // CTA pairs that share the steps of a tile
    float *partial;       // splits > 1: [splits][rows][ld_partial]
    int64_t ld_partial;
    void *out[2];         // kForward: y; kDw: dw_gate, dw_up
    int64_t ld[2];
    void *keep[2];        // kForward: gate and up, or null
    int64_t ldkeep[2];
    const float *bias[2];
    int32_t wide_out[2], wide_keep[2];
    int32_t *dev_status;
};

// Tiles in bands of kBand row blocks, columns fastest between bands: the tiles
// in flight share a few panels of A and of B that stay in L2.
constexpr uint32_t kBand = 16;

__device__ __forceinline__ void tile_at(uint32_t t, uint32_t tiles_m, uint32_t tiles_n, uint32_t &mt, uint32_t &nt)
{
    const uint32_t per_band = kBand * tiles_n, band = t / per_band, first = band * kBand;
    const uint32_t rows = tiles_m - first < kBand ? tiles_m - first : kBand;
    const uint32_t local = t - band * per_band;
    mt = first + local % rows;
    nt = local / rows;
}

template <int kMode, int kBN, typename T, int kAct>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gated_gemm_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1, const __grid_constant__ CUtensorMap tmB0,
                      const __grid_constant__ CUtensorMap tmB1, const __grid_constant__ Params p)
{
    using C = Cfg<kBN>;
    constexpr bool kAmn = kMode == kDw, kBmn = kMode != kForward;
    constexpr uint32_t kId = idesc<T>(256, kBN, kAmn, kBmn);
    constexpr uint32_t kBox = kBoxElems * kBK * 2;  // bytes of an MN-major box
    constexpr int kOutCols = kMode == kForward ? kBN / 2 : kBN;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw));
    const uint32_t base = (raw + 1023u) & ~1023u;  // swizzle atoms are 1024-byte aligned
    uint8_t *gbase = smem_raw + (base - raw);
    constexpr int kOut = C::STAGES * C::STAGE_BYTES, kBars = kOut + kDrainWarps * kStageBytes;
    const uint32_t bars = base + kBars;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (C::STAGES + s); };
    auto sum_bar = [&](int b) { return bars + 8u * (2 * C::STAGES + b); };               // an accumulator is finished
    auto drained_bar = [&](int b) { return bars + 8u * (2 * C::STAGES + C::BUFS + b); };  // and free again
    const uint32_t done_bar = bars + 8u * (2 * C::STAGES + 2 * C::BUFS);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + kBars + 8 * (2 * C::STAGES + 2 * C::BUFS + 1));
    const Waits wait{reinterpret_cast<volatile int *>(tmem_slot + 1), p.dev_status};

    const uint32_t rank = cluster_rank();
    const bool leader = rank == 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t tiles_m = static_cast<uint32_t>(p.tiles_m) * p.sections;
    const uint32_t tiles = tiles_m * p.tiles_n, items = tiles * p.splits, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    // item -> tile, and its share of the steps (over all parts)
    const int all_steps = p.steps * p.parts;
    auto first_step = [&](uint32_t share) { return static_cast<int>(static_cast<int64_t>(all_steps) * share / p.splits); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < C::BUFS; ++b) {
            mbar_init(sum_bar(b), 1);
            mbar_init(drained_bar(b), 2 * kDrainWarps);
        }
        mbar_init(done_bar, 1);
        *wait.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&tmA0);
        prefetch_map(&tmA1);
        prefetch_map(&tmB0);
        prefetch_map(&tmB1);
    }
    if (warp == 1) tmem_alloc<2>(tmem_slot, 512u);
    tc_fence_before();
    cluster_sync();  // both CTAs' barriers and tensor memory are there before any remote use
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    after_previous();
    let_next_start();

    if (warp == 0 && lane == 0) {
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (uint32_t t = pair; t < items && ok; t += pairs) {
            uint32_t mt, nt;
            const uint32_t share = t / tiles;
            tile_at(t - share * tiles, tiles_m, p.tiles_n, mt, nt);
            const bool second = kMode == kDw && mt >= static_cast<uint32_t>(p.tiles_m);
            if (second) mt -= p.tiles_m;
            const int row = static_cast<int>(mt * 2 * kBM + rank * kBM);
            // kForward: each CTA's rows of its own weight; else its half of the tile's columns
            const int col = static_cast<int>(kMode == kForward ? nt * (kBN / 2) : nt * kBN + rank * (kBN / 2));
            const int end = first_step(share + 1);
            for (int step = first_step(share); step < end;) {
                const int part = step >= p.steps, j0 = step - part * p.steps, j1 = end - part * p.steps < p.steps ? end - part * p.steps : p.steps;
                const CUtensorMap *ma = (kMode == kDx ? part : second) ? &tmA1 : &tmA0;
                const CUtensorMap *mb = (kMode == kForward ? rank != 0 : kMode == kDx && part) ? &tmB1 : &tmB0;
                for (int j = j0; j < j1; ++j) {
                    if (!wait(empty_bar(stage), phase ^ 1u)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sa = base + stage * C::STAGE_BYTES, sb = sa + C::A_BYTES;
                    if (leader) mbar_arrive_expect_tx(full_bar(stage), 2u * C::STAGE_BYTES);
                    const uint32_t bar = map_to_rank(full_bar(stage), 0);
                    if constexpr (kAmn) {
#pragma unroll
                        for (int i = 0; i < kBM / kBoxElems; ++i) tma_load_pair(sa + i * kBox, ma, row + i * kBoxElems, j * kBK, bar);
                    } else {
                        tma_load_pair(sa, ma, j * kBK, row, bar);
                    }
                    if constexpr (kBmn) {
#pragma unroll
                        for (int i = 0; i < kBN / 2 / kBoxElems; ++i) tma_load_pair(sb + i * kBox, mb, col + i * kBoxElems, j * kBK, bar);
                    } else {
                        tma_load_pair(sb, mb, j * kBK, col, bar);
                    }
                    ++issued;
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                step += j1 - j0;
            }
        }
        if (!ok) {
            wait.fail();
            if (leader) {
                // both CTAs' copies for the stages armed here land before shared memory goes away
                for (int i = 0; i < C::STAGES && i < issued; ++i) {
                    if (--stage < 0) {
                        stage = C::STAGES - 1;
                        phase ^= 1u;
                    }
                    mbar_wait(full_bar(stage), phase);
                }
            }
        }
    } else if (warp == 1 && leader && lane == 0) {
        int stage = 0;
        uint32_t phase = 0, buf = 0, buf_phase = 0;
        bool ok = true;
        for (uint32_t t = pair; t < items && ok; t += pairs) {
            const uint32_t share = t / tiles;
            const int steps = first_step(share + 1) - first_step(share);
            if (!wait(drained_bar(buf), buf_phase ^ 1u)) {
                ok = false;
                break;
            }
            const uint32_t d = tmem + buf * kBN;
            for (int j = 0; j < steps; ++j) {
                if (!wait(full_bar(stage), phase)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sa = base + stage * C::STAGE_BYTES, sb = sa + C::A_BYTES;
                const uint64_t da = kAmn ? desc_mn(sa, kBox) : desc_k(sa), db = kBmn ? desc_mn(sb, kBox) : desc_k(sb);
#pragma unroll
                for (int kk = 0; kk < kBK / kMmaK; ++kk)
                    mma_ss<2>(d, da + (kAmn ? kStepMN : kStepK) * kk, db + (kBmn ? kStepMN : kStepK) * kk, kId, j > 0 || kk > 0 ? 1u : 0u);
                commit_both(empty_bar(stage));
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) break;
            commit_both(sum_bar(buf));
            if (++buf == C::BUFS) {
                buf = 0;
                buf_phase ^= 1u;
            }
        }
        if (!ok) wait.fail();
        commit_pair_local(done_bar);
        mbar_wait(done_bar, 0);
    } else if (warp >= 4) {
        const int q = warp & 3, part = (warp - 4) >> 2;  // lane quadrant, half of the columns
        const uint32_t stage = base + kOut + (warp - 4) * kStageBytes;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
        const uint32_t drained0 = map_to_rank(drained_bar(0), 0);
        uint32_t buf = 0, buf_phase = 0;
        bool ok = true;
        for (uint32_t t = pair; t < items; t += pairs) {
            uint32_t mt, nt;
            const uint32_t share = t / tiles;
            tile_at(t - share * tiles, tiles_m, p.tiles_n, mt, nt);
            const int second = kMode == kDw && mt >= static_cast<uint32_t>(p.tiles_m);
            if (second) mt -= p.tiles_m;
            const int64_t row0 = static_cast<int64_t>(mt) * 2 * kBM + rank * kBM + q * 32;
            const int rows = p.rows - row0 < 32 ? static_cast<int>(p.rows - row0) : 32;
            if (!wait.together(sum_bar(buf), buf_phase)) {
                ok = false;
                break;
            }
            tc_fence_after();
            constexpr int kPart = kOutCols / 2;  // output columns of this warp
#pragma unroll 1
            for (int c = 0; c < kPart; c += 32) {
                const int64_t col0 = static_cast<int64_t>(nt) * kOutCols + part * kPart + c;
                const int cols = p.cols - col0 < 32 ? static_cast<int>(p.cols - col0) : 32;
                const uint32_t at = lanes + buf * kBN + part * kPart + c;
                float v[32];
                if constexpr (kMode == kForward) {
                    uint32_t g[32], u[32];
                    tmem_ld32_async(at, g);
                    tmem_ld32_async(at + kBN / 2, u);
                    // lane i has the biases of column i
                    const float bg = p.bias[0] && lane < cols ? load_f32(p.bias[0] + col0 + lane) : 0.0f;
                    const float bu = p.bias[1] && lane < cols ? load_f32(p.bias[1] + col0 + lane) : 0.0f;
                    tmem_ld_wait(g);
                    tmem_ld_wait(u);
                    if (c + 32 == kPart) {  // read to the end: the buffer is free
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_remote(drained0 + 8u * buf);
                    }
                    float fg[32], fu[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        fg[i] = __uint_as_float(g[i]);
                        fu[i] = __uint_as_float(u[i]);
                    }
                    if (p.bias[0] || p.bias[1]) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            fg[i] += __shfl_sync(0xffffffffu, bg, i);
                            fu[i] += __shfl_sync(0xffffffffu, bu, i);
                        }
                    }
                    if (p.keep[0] && rows > 0 && cols > 0) {
                        store_rows<T>(static_cast<T *>(p.keep[0]) + row0 * p.ldkeep[0] + col0, p.ldkeep[0], rows, cols, p.wide_keep[0], stage, lane, fg);
                        store_rows<T>(static_cast<T *>(p.keep[1]) + row0 * p.ldkeep[1] + col0, p.ldkeep[1], rows, cols, p.wide_keep[1], stage, lane, fu);
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const F2 y = gate_act2<kAct>(F2(fg[i], fg[i + 1])) * F2(fu[i], fu[i + 1]);
                        v[i] = y.lo();
                        v[i + 1] = y.hi();
                    }
                } else {
                    uint32_t r[32];
                    tmem_ld32_async(at, r);
                    tmem_ld_wait(r);
                    if (c + 32 == kPart) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_remote(drained0 + 8u * buf);
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
                }
                if (kMode == kDx && p.partial) {
                    // (columns to the end of a group of four are there)
                    float *to = p.partial + (static_cast<int64_t>(share) * p.rows + row0 + lane) * p.ld_partial + col0;
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        if (lane < rows && i < cols) *reinterpret_cast<float4 *>(to + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                } else if (rows > 0 && cols > 0) {
                    T *y = static_cast<T *>(p.out[second]) + row0 * p.ld[second] + col0;
                    store_rows<T>(y, p.ld[second], rows, cols, p.wide_out[second], stage, lane, v);
                }
            }
            if (++buf == C::BUFS) {
                buf = 0;
                buf_phase ^= 1u;
            }
        }
        if (!ok) wait.fail();
    }
    __syncwarp();

    tc_fence_before();
    cluster_sync();  // neither CTA's shared or tensor memory goes away under the other's use
    tc_fence_after();
    if (warp == 1) tmem_free<2>(tmem, 512u);
}

// The shares of a split sum, added up in order, four columns a thread.
template <typename T>
__global__ void __launch_bounds__(256) join_shares_kernel(const float *partial, int64_t ld, int shares, int64_t rows, int64_t cols, T *out, int64_t ldo, int wide)
{
    after_previous();
    let_next_start();
    const int64_t per_row = ld / 4, at = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (at >= rows * per_row) return;
    const int64_t row = at / per_row, col = (at - row * per_row) * 4;
    const float *from = partial + row * ld + col;
    float4 w[kMaxSplits], sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kMaxSplits; ++i)
        if (i < shares) w[i] = __ldcg(reinterpret_cast<const float4 *>(from + i * rows * ld));
#pragma unroll
    for (int i = 0; i < kMaxSplits; ++i) {
        if (i >= shares) break;
        sum.x += w[i].x;
        sum.y += w[i].y;
        sum.z += w[i].z;
        sum.w += w[i].w;
    }
    T *to = out + row * ldo + col;
    if (wide && col + 4 <= cols) {
        *reinterpret_cast<uint2 *>(to) = make_uint2(pack2<T>(sum.x, sum.y), pack2<T>(sum.z, sum.w));
    } else {
        const float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (col + e < cols) to[e] = from_f32<T>(v[e]);
    }
}

// How a product is cut: accumulator columns of a tile, and pairs that share a tile's steps.
struct Cut {
    int bn, splits;
};

// By the time of the rounds that the 76 pairs take over the items, in steps of a wide tile (0.27 us): a narrow tile's
// step costs 3/4 of a wide one's (its operands are 3/4 of the bytes, and L2 feeds the tensor cores at their limit), an
// item's end 8, and a split the second kernel's start (3 us) and the trip of its fp32 shares.
Cut cut_of(int64_t rows, int64_t cols, int64_t out_cols, int64_t sections, int64_t steps, bool may_split)
{
    const int64_t pairs = kSms / 2;
    Cut best{256, 1};
    double least = 0.0;
    for (int bn : {256, 128}) {
        const int64_t width = out_cols * bn / 256, tiles = (rows + 255) / 256 * sections * ((cols + width - 1) / width);
        for (int splits = 1; splits <= (may_split ? kMaxSplits : 1); ++splits) {
            if (splits > 1 && steps / splits < 16) break;
            const int64_t rounds = (tiles * splits + pairs - 1) / pairs;
            double cost = static_cast<double>(rounds) * (static_cast<double>((steps + splits - 1) / splits) * (bn == 256 ? 1.0 : 0.75) + 8.0);
            if (splits > 1) cost += 11.0 + static_cast<double>(splits) * rows * cols * 8.0 / 1.6e6;
            if (least == 0.0 || cost < least) {
                least = cost;
                best = {bn, splits};
            }
        }
    }
    return best;
}

Cut cut_of_dx(int64_t m, int64_t n, int64_t k) { return cut_of(m, k, 256, 1, 2 * ((n + kBK - 1) / kBK), true); }

int64_t partial_pitch(int64_t cols) { return (cols + 3) / 4 * 4; }

template <int kMode, int kBN, typename T, int kAct>
struct gemm_tag;

template <int kMode, int kBN, typename T, int kAct>
cudaError_t launch(const CUtensorMap &a0, const CUtensorMap &a1, const CUtensorMap &b0, const CUtensorMap &b1, Params &p, cudaStream_t stream)
{
    using C = Cfg<kBN>;
    constexpr int kOutCols = kMode == kForward ? kBN / 2 : kBN;
    p.tiles_m = (p.rows + 2 * kBM - 1) / (2 * kBM);
    p.tiles_n = (p.cols + kOutCols - 1) / kOutCols;
    auto kernel = gated_gemm_kernel<kMode, kBN, T, kAct>;
    cudaError_t e = allow_shared<gemm_tag<kMode, kBN, T, kAct>>(kernel);
    if (e != cudaSuccess) return e;
    const int64_t items = static_cast<int64_t>(p.tiles_m) * p.sections * p.tiles_n * p.splits;
    if (items > INT32_MAX) return cudaErrorInvalidValue;
    const int64_t pairs = items < kSms / 2 ? items : kSms / 2;
    return launch_after(kernel, dim3(static_cast<unsigned>(2 * pairs)), kThreads, C::SMEM, stream, 1, a0, a1, b0, b1, p);
}

template <typename F>
auto with_16bit(int dtype, F f)
{
    return dtype == CONVROT_BF16 ? f(static_cast<__nv_bfloat16 *>(nullptr)) : f(static_cast<__half *>(nullptr));
}

int32_t wide(const void *p, int64_t ld) { return aligned_to(p, 16) && ld % 8 == 0; }

}  // namespace

cudaError_t launch_gated_gemm(const convrot_gated_linear_args &a, cudaStream_t stream)
{
    return with_16bit(a.dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        const Cut cut = cut_of(a.m, a.n, 128, 1, (a.k + kBK - 1) / kBK, false);
        CUtensorMap x, wg, wu;
        if (!matrix_map<T>(&x, a.x, a.m, a.k, a.ldx, kBM) || !matrix_map<T>(&wg, a.w_gate, a.n, a.k, a.ldw_gate, cut.bn / 2) ||
            !matrix_map<T>(&wu, a.w_up, a.n, a.k, a.ldw_up, cut.bn / 2))
            return cudaErrorInvalidValue;
        Params p{};
        p.rows = static_cast<int32_t>(a.m);
        p.cols = static_cast<int32_t>(a.n);
        p.steps = static_cast<int32_t>((a.k + kBK - 1) / kBK);
        p.parts = p.sections = p.splits = 1;
        p.out[0] = a.y;
        p.ld[0] = a.ldy;
        p.wide_out[0] = wide(a.y, a.ldy);
        p.keep[0] = a.gate;
        p.keep[1] = a.up;
        p.ldkeep[0] = a.ldgate;
        p.ldkeep[1] = a.ldup;
        p.wide_keep[0] = wide(a.gate, a.ldgate);
        p.wide_keep[1] = wide(a.up, a.ldup);
        p.bias[0] = a.b_gate;
        p.bias[1] = a.b_up;
        p.dev_status = a.dev_status;
        auto run = [&](auto act) {
            constexpr int kAct = decltype(act)::value;
            return cut.bn == 256 ? launch<kForward, 256, T, kAct>(x, x, wg, wu, p, stream) : launch<kForward, 128, T, kAct>(x, x, wg, wu, p, stream);
        };
        if (a.act == CONVROT_ACT_SILU) return run(std::integral_constant<int, 3>());
        if (a.act == CONVROT_ACT_GELU_TANH) return run(std::integral_constant<int, 2>());
        if (a.act == CONVROT_ACT_GELU_ERF) return run(std::integral_constant<int, 1>());
        return run(std::integral_constant<int, 0>());
    });
}

int64_t gated_dx_partial_bytes(int64_t m, int64_t n, int64_t k)
{
    const Cut cut = cut_of_dx(m, n, k);
    return cut.splits > 1 ? cut.splits * m * partial_pitch(k) * 4 : 0;
}

cudaError_t launch_gated_dx(const convrot_gated_linear_backward_args &a, const void *dg, const void *du, int64_t ldd, float *partial, cudaStream_t stream)
{
    return with_16bit(a.dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        CUtensorMap mg, mu, wg, wu;
        if (!matrix_map<T>(&mg, dg, a.m, a.n, ldd, kBM) || !matrix_map<T>(&mu, du, a.m, a.n, ldd, kBM) ||
            !matrix_map<T>(&wg, a.w_gate, a.n, a.k, a.ldw_gate, kBK) || !matrix_map<T>(&wu, a.w_up, a.n, a.k, a.ldw_up, kBK))
            return cudaErrorInvalidValue;
        Params p{};
        p.rows = static_cast<int32_t>(a.m);
        p.cols = static_cast<int32_t>(a.k);
        p.steps = static_cast<int32_t>((a.n + kBK - 1) / kBK);
        p.parts = 2;
        p.sections = 1;
        p.out[0] = a.dx;
        p.ld[0] = a.lddx;
        p.wide_out[0] = wide(a.dx, a.lddx);
        p.dev_status = a.dev_status;
        const Cut cut = cut_of_dx(a.m, a.n, a.k);
        p.splits = cut.splits;
        p.partial = cut.splits > 1 ? partial : nullptr;
        p.ld_partial = partial_pitch(a.k);
        const cudaError_t e = cut.bn == 256 ? launch<kDx, 256, T, 0>(mg, mu, wg, wu, p, stream) : launch<kDx, 128, T, 0>(mg, mu, wg, wu, p, stream);
        if (e != cudaSuccess || cut.splits == 1) return e;
        const int64_t threads = a.m * (p.ld_partial / 4);
        return launch_after(join_shares_kernel<T>, dim3(static_cast<unsigned>((threads + 255) / 256)), 256, 0, stream, 1,
                            static_cast<const float *>(partial), p.ld_partial, cut.splits, a.m, a.k, static_cast<T *>(a.dx), a.lddx,
                            aligned_to(a.dx, 8) && a.lddx % 4 == 0);
    });
}

cudaError_t launch_gated_dw(const convrot_gated_linear_backward_args &a, const void *dg, const void *du, int64_t ldd, cudaStream_t stream)
{
    return with_16bit(a.dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        CUtensorMap mg, mu, x;
        if (!matrix_map<T>(&mg, dg, a.m, a.n, ldd, kBK) || !matrix_map<T>(&mu, du, a.m, a.n, ldd, kBK) ||
            !matrix_map<T>(&x, a.x, a.m, a.k, a.ldx, kBK))
            return cudaErrorInvalidValue;
        Params p{};
        p.rows = static_cast<int32_t>(a.n);
        p.cols = static_cast<int32_t>(a.k);
        p.steps = static_cast<int32_t>((a.m + kBK - 1) / kBK);
        p.parts = p.splits = 1;
        p.sections = 2;
        p.out[0] = a.dw_gate;
        p.out[1] = a.dw_up;
        p.ld[0] = a.lddw_gate;
        p.ld[1] = a.lddw_up;
        p.wide_out[0] = wide(a.dw_gate, a.lddw_gate);
        p.wide_out[1] = wide(a.dw_up, a.lddw_up);
        p.dev_status = a.dev_status;
        const Cut cut = cut_of(a.n, a.k, 256, 2, (a.m + kBK - 1) / kBK, false);
        return cut.bn == 256 ? launch<kDw, 256, T, 0>(mg, mu, x, x, p, stream) : launch<kDw, 128, T, 0>(mg, mu, x, x, p, stream);
    });
}

int gated_gemm_shared(int form, int *columns)
{
    *columns = 512;
    return form == 0 ? Cfg<256>::SMEM : form == 1 ? Cfg<128>::SMEM : 0;
}

}  // namespace convrot
