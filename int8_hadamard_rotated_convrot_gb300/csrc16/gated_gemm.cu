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
#include "gated.h"
#include "mma16.cuh"

namespace convrot {
namespace {

using namespace mma16;

enum Mode { kForward, kDx, kDw };

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
    const uint32_t tiles = tiles_m * p.tiles_n, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

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

    if (warp == 0 && lane == 0) {
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (uint32_t t = pair; t < tiles && ok; t += pairs) {
            uint32_t mt, nt;
            tile_at(t, tiles_m, p.tiles_n, mt, nt);
            const bool second = kMode == kDw && mt >= static_cast<uint32_t>(p.tiles_m);
            if (second) mt -= p.tiles_m;
            const int row = static_cast<int>(mt * 2 * kBM + rank * kBM);
            // kForward: each CTA's rows of its own weight; else its half of the tile's columns
            const int col = static_cast<int>(kMode == kForward ? nt * (kBN / 2) : nt * kBN + rank * (kBN / 2));
            for (int part = 0; part < p.parts && ok; ++part) {
                const CUtensorMap *ma = (kMode == kDx ? part : second) ? &tmA1 : &tmA0;
                const CUtensorMap *mb = (kMode == kForward ? rank != 0 : kMode == kDx && part) ? &tmB1 : &tmB0;
                for (int j = 0; j < p.steps; ++j) {
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
        const int steps = p.steps * p.parts;
        for (uint32_t t = pair; t < tiles && ok; t += pairs) {
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
        for (uint32_t t = pair; t < tiles; t += pairs) {
            uint32_t mt, nt;
            tile_at(t, tiles_m, p.tiles_n, mt, nt);
            const int second = kMode == kDw && mt >= static_cast<uint32_t>(p.tiles_m);
            if (second) mt -= p.tiles_m;
            const int64_t row0 = static_cast<int64_t>(mt) * 2 * kBM + rank * kBM + q * 32;
            const int rows = p.rows - row0 < 32 ? static_cast<int>(p.rows - row0) : 32;
            if (!wait(sum_bar(buf), buf_phase)) {
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
                if (rows > 0 && cols > 0) {
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
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.sections * p.tiles_n;
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;
    const int64_t pairs = tiles < kSms / 2 ? tiles : kSms / 2;
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
        constexpr int kBN = 256;
        CUtensorMap x, wg, wu;
        if (!matrix_map<T>(&x, a.x, a.m, a.k, a.ldx, kBM) || !matrix_map<T>(&wg, a.w_gate, a.n, a.k, a.ldw_gate, kBN / 2) ||
            !matrix_map<T>(&wu, a.w_up, a.n, a.k, a.ldw_up, kBN / 2))
            return cudaErrorInvalidValue;
        Params p{};
        p.rows = static_cast<int32_t>(a.m);
        p.cols = static_cast<int32_t>(a.n);
        p.steps = static_cast<int32_t>((a.k + kBK - 1) / kBK);
        p.parts = p.sections = 1;
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
        if (a.act == CONVROT_ACT_SILU) return launch<kForward, kBN, T, 3>(x, x, wg, wu, p, stream);
        if (a.act == CONVROT_ACT_GELU_TANH) return launch<kForward, kBN, T, 2>(x, x, wg, wu, p, stream);
        if (a.act == CONVROT_ACT_GELU_ERF) return launch<kForward, kBN, T, 1>(x, x, wg, wu, p, stream);
        return launch<kForward, kBN, T, 0>(x, x, wg, wu, p, stream);
    });
}

cudaError_t launch_gated_dx(const convrot_gated_linear_backward_args &a, const void *dg, const void *du, int64_t ldd, cudaStream_t stream)
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
        return launch<kDx, 256, T, 0>(mg, mu, wg, wu, p, stream);
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
        p.parts = 1;
        p.sections = 2;
        p.out[0] = a.dw_gate;
        p.out[1] = a.dw_up;
        p.ld[0] = a.lddw_gate;
        p.ld[1] = a.lddw_up;
        p.wide_out[0] = wide(a.dw_gate, a.lddw_gate);
        p.wide_out[1] = wide(a.dw_up, a.lddw_up);
        p.dev_status = a.dev_status;
        return launch<kDw, 256, T, 0>(mg, mu, x, x, p, stream);
    });
}

int gated_gemm_shared(int form, int *columns)
{
    *columns = 512;
    return form == 0 ? Cfg<256>::SMEM : 0;
}

}  // namespace convrot
