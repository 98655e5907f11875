// The gated feed-forward's projections for few rows (include/convrot_block.h),
// where reading the weights counts, not the arithmetic.
//
// The weights are the MMA's M side: a CTA takes 64 rows of w_gate and the same
// 64 of w_up as its 128 lanes, and up to 256 rows of x as the N side, so that
// the weights are read once and no tensor-core row is wasted. k is split over a
// cluster of up to eight CTAs where there are few columns of y; the partial
// sums meet in distributed shared memory, added in a fixed order, and there the
// gate's sums meet the up projection's.
//   warp 0      TMA producer: 64 of k a stage (16 KB of weights, and x)
//   warp 1      tensor memory; one thread issues the MMAs
//   warps 2-5   drain: lane = row of a weight
//   warps 2-9   the activation and the product, a row of x at a time
//
// Bound by HBM: a row by 5120 x 13824 in 44.8 us, 6.3 TB/s of weights, 93 % of a copy.
#include "gated.h"
#include "mma16.cuh"

namespace convrot {
namespace {

using namespace mma16;

constexpr int kBK = 64, kRows = 64;  // of k a stage; of each weight a CTA
constexpr int kWeightBytes = 2 * kRows * kBK * 2;
constexpr int kWarps = 8, kThreads = 64 + 32 * kWarps;
constexpr int kMaxSplit = 8;

template <int kTok>
struct Shape {
    static constexpr int STAGE = kWeightBytes + kTok * kBK * 2;
    static constexpr int COLS = kTok <= 128 ? 128 : 256;  // of tensor memory
    static constexpr int PER_SM = kTok <= 128 ? 2 : 1;
    static constexpr int BARS = 256;
    static constexpr int FIT = (kMaxShared / PER_SM - 2048 - BARS) / STAGE;
    static constexpr int STAGES = FIT < 8 ? FIT : 8;
    static constexpr int USED = 1024 + STAGES * STAGE + BARS;
    static constexpr int SMEM = USED > tmem_share(COLS) ? USED : tmem_share(COLS);
    static_assert(STAGES * STAGE >= kTok * 2 * kRows * 4, "the sums fit over the stages");
    static_assert(8 * (2 * STAGES + 1) + 8 <= BARS, "barriers fit");
    static_assert(PER_SM * (SMEM + 1024) <= kSmShared && SMEM <= kMaxShared, "resident");
};

struct FewParams {
    int32_t m, n, steps, split;
    const float *bias[2];
    void *y, *keep[2];
    int64_t ldy, ldkeep[2];
    int32_t act;
    int32_t two_y, two_keep[2];  // rows start on 4 bytes
    int32_t *dev_status;
};

__device__ __forceinline__ float2 remote8(uint32_t local, uint32_t rank)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(map_to_rank(local, rank)) : "memory");
    return v;
}

template <typename T>
__device__ __forceinline__ void store2(T *to, float a, float b, int cols, bool two)
{
    if (two && cols >= 2) {
        *reinterpret_cast<uint32_t *>(to) = pack2<T>(a, b);
    } else {
        if (cols > 0) to[0] = from_f32<T>(a);
        if (cols > 1) to[1] = from_f32<T>(b);
    }
}

template <int kTok, typename T>
__global__ void __launch_bounds__(kThreads, Shape<kTok>::PER_SM)
    gated_few_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmG, const __grid_constant__ CUtensorMap tmU,
                     const __grid_constant__ FewParams p)
{
    using S = Shape<kTok>;
    constexpr uint32_t kId = idesc<T>(128, kTok, false, false);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw));
    const uint32_t base = (raw + 1023u) & ~1023u;  // swizzle atoms are 1024-byte aligned
    constexpr int kBars = S::STAGES * S::STAGE;
    const uint32_t bars = base + kBars;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (S::STAGES + s); };
    const uint32_t done_bar = bars + 8u * (2 * S::STAGES);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + (base - raw) + kBars + 8 * (2 * S::STAGES + 1));
    const Waits wait{reinterpret_cast<volatile int *>(tmem_slot + 1), p.dev_status};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t split = static_cast<uint32_t>(p.split), rank = split > 1 ? cluster_rank() : 0;
    const int col0 = static_cast<int>(blockIdx.x / split) * kRows;
    const int j0 = static_cast<int>(static_cast<int64_t>(p.steps) * rank / split), j1 = static_cast<int>(static_cast<int64_t>(p.steps) * (rank + 1) / split);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(done_bar, 1);
        *wait.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&tmX);
        prefetch_map(&tmG);
        prefetch_map(&tmU);
    }
    if (warp == 1) tmem_alloc<1>(tmem_slot, S::COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    after_previous();
    let_next_start();

    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            int issued = 0;
            for (int j = j0; j < j1; ++j, ++issued) {
                const int s = issued % S::STAGES;
                if (!wait(empty_bar(s), (issued / S::STAGES + 1) & 1)) {
                    ok = false;
                    break;
                }
                const uint32_t sa = base + s * S::STAGE;
                mbar_arrive_expect_tx(full_bar(s), S::STAGE);
                tma_load_2d(sa, &tmG, j * kBK, col0, full_bar(s));
                tma_load_2d(sa + kWeightBytes / 2, &tmU, j * kBK, col0, full_bar(s));
                tma_load_2d(sa + kWeightBytes, &tmX, j * kBK, 0, full_bar(s));
            }
            if (!ok) {
                wait.fail();
                // copies in flight land before shared memory goes away
                for (int i = issued > S::STAGES ? issued - S::STAGES : 0; i < issued; ++i) mbar_wait(full_bar(i % S::STAGES), (i / S::STAGES) & 1);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            for (int j = 0; j < j1 - j0; ++j) {
                const int s = j % S::STAGES;
                if (!wait(full_bar(s), (j / S::STAGES) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sa = base + s * S::STAGE;
                const uint64_t da = desc_k(sa), db = desc_k(sa + kWeightBytes);
#pragma unroll
                for (int kk = 0; kk < kBK / kMmaK; ++kk) mma_ss<1>(tmem, da + kStepK * kk, db + kStepK * kk, kId, j > 0 || kk > 0 ? 1u : 0u);
                mma_commit(empty_bar(s));
            }
            if (!ok) wait.fail();
            mma_commit(done_bar);
            mbar_wait(done_bar, 0);
        }
    } else if (warp < 6) {
        const int q = warp & 3;  // tensor-memory lanes of this warp
        ok = wait.together(done_bar, 0);
        tc_fence_after();
        if (!ok) wait.fail();
        // this CTA's sums, [row of x][row of the weights], over the ring's stages: every MMA has read them
        const uint32_t sums = base + (q * 32 + lane) * 4;
#pragma unroll
        for (int c = 0; c < kTok; c += 16) {
            if (c >= p.m || !ok) break;
            uint32_t r[16];
            tmem_ld16(tmem + (static_cast<uint32_t>(q * 32) << 16) + c, r);
#pragma unroll
            for (int i = 0; i < 16; ++i) asm volatile("st.shared.b32 [%0], %1;" ::"r"(sums + (c + i) * 2 * kRows * 4), "r"(r[i]) : "memory");
        }
    }
    __syncwarp();

    tc_fence_before();
    if (split > 1)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        tmem_free<1>(tmem, S::COLS);
    } else if (warp > 1) {
        // the cluster's warps share out the rows of x, two columns of y a lane
        const int64_t col = col0 + lane * 2;
        const int cols = static_cast<int>(p.n - col);
        float bias[2][2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) bias[t][e] = p.bias[t] && e < cols ? load_f32(p.bias[t] + col + e) : 0.0f;
        for (int r = static_cast<int>(rank) * kWarps + warp - 2; r < p.m; r += static_cast<int>(split) * kWarps) {
            const uint32_t at = base + (r * 2 * kRows + lane * 2) * 4;
            float2 g[kMaxSplit], u[kMaxSplit];
#pragma unroll
            for (uint32_t c = 0; c < kMaxSplit; ++c) {
                if (c >= split) break;
                g[c] = remote8(at, split > 1 ? c : 0);
                u[c] = remote8(at + kRows * 4, split > 1 ? c : 0);
            }
            F2 sg(0.0f), su(0.0f);
#pragma unroll
            for (uint32_t c = 0; c < kMaxSplit; ++c) {
                if (c >= split) break;
                sg = sg + F2(g[c].x, g[c].y);
                su = su + F2(u[c].x, u[c].y);
            }
            sg = sg + F2(bias[0][0], bias[0][1]);
            su = su + F2(bias[1][0], bias[1][1]);
            if (p.keep[0]) {
                store2(static_cast<T *>(p.keep[0]) + r * p.ldkeep[0] + col, sg.lo(), sg.hi(), cols, p.two_keep[0]);
                store2(static_cast<T *>(p.keep[1]) + r * p.ldkeep[1] + col, su.lo(), su.hi(), cols, p.two_keep[1]);
            }
            F2 a;
            if (p.act == CONVROT_ACT_SILU)
                a = gate_act2<CONVROT_ACT_SILU>(sg);
            else if (p.act == CONVROT_ACT_GELU_TANH)
                a = gate_act2<CONVROT_ACT_GELU_TANH>(sg);
            else if (p.act == CONVROT_ACT_GELU_ERF)
                a = gate_act2<CONVROT_ACT_GELU_ERF>(sg);
            else
                a = sg;
            a = a * su;
            store2(static_cast<T *>(p.y) + r * p.ldy + col, a.lo(), a.hi(), cols, p.two_y);
        }
    }
    if (split > 1) cluster_sync();  // a CTA's sums stay until its peers have read them
}

template <int kTok, typename T>
struct few_tag;

// Columns of the products (the stages of 80 are four instead of three: 66 to 80 rows of 1280 x 5120 take 9.3 us with them and
// 10.0 with 128, of 2056 x 3080 10.9 and 11.6; 96, three stages again, gained 1 %).
int tokens_of(int64_t m) { return m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : m <= 80 ? 80 : m <= 128 ? 128 : 256; }

template <int kTok>
int split_of(int64_t n, int64_t k)
{
    // The widest cluster (1, 2, 4 or 8) with which every CTA is still resident and has four steps of k or more: clusters
    // of 4 and 8 leave some SMs of a GPC over (36 and 15 of them fit at one CTA an SM).
    using S = Shape<kTok>;
    const int64_t units = (n + kRows - 1) / kRows, steps = (k + kBK - 1) / kBK;
    const int room[4] = {kSms, kSms, 36 * 4, 15 * 8};
    int split = 1;
    for (int i = 1; i < 4; ++i) {
        const int next = 1 << i;
        if (units * next > S::PER_SM * room[i] || steps < 4 * next) break;
        split = next;
    }
    return split;
}

template <int kTok, typename T>
cudaError_t launch(const convrot_gated_linear_args &a, cudaStream_t stream)
{
    using S = Shape<kTok>;
    CUtensorMap x, g, u;
    if (!matrix_map<T>(&x, a.x, a.m, a.k, a.ldx, kTok) || !matrix_map<T>(&g, a.w_gate, a.n, a.k, a.ldw_gate, kRows) ||
        !matrix_map<T>(&u, a.w_up, a.n, a.k, a.ldw_up, kRows))
        return cudaErrorInvalidValue;
    FewParams p{};
    p.m = static_cast<int32_t>(a.m);
    p.n = static_cast<int32_t>(a.n);
    p.steps = static_cast<int32_t>((a.k + kBK - 1) / kBK);
    p.split = split_of<kTok>(a.n, a.k);
    p.bias[0] = a.b_gate;
    p.bias[1] = a.b_up;
    p.y = a.y;
    p.ldy = a.ldy;
    p.keep[0] = a.gate;
    p.keep[1] = a.up;
    p.ldkeep[0] = a.ldgate;
    p.ldkeep[1] = a.ldup;
    auto two = [&](const void *q, int64_t ld) { return aligned_to(q, 4) && (a.m <= 1 || ld % 2 == 0); };
    p.two_y = two(a.y, a.ldy);
    p.two_keep[0] = two(a.gate, a.ldgate);
    p.two_keep[1] = two(a.up, a.ldup);
    p.act = a.act;
    p.dev_status = a.dev_status;
    auto kernel = gated_few_kernel<kTok, T>;
    cudaError_t e = allow_shared<few_tag<kTok, T>>(kernel);
    if (e != cudaSuccess) return e;
    const int64_t units = (a.n + kRows - 1) / kRows;
    return launch_after(kernel, dim3(static_cast<unsigned>(units * p.split)), kThreads, S::SMEM, stream, static_cast<unsigned>(p.split), x, g, u, p);
}

template <typename T>
cudaError_t launch_type(const convrot_gated_linear_args &a, cudaStream_t stream)
{
    switch (tokens_of(a.m)) {
    case 16: return launch<16, T>(a, stream);
    case 32: return launch<32, T>(a, stream);
    case 64: return launch<64, T>(a, stream);
    case 80: return launch<80, T>(a, stream);
    case 128: return launch<128, T>(a, stream);
    default: return launch<256, T>(a, stream);
    }
}

}  // namespace

// Up to 128 rows always: 128 of 5120 x 13824 take 51 us here and 60 in the many-row kernel, of 1280 x 5120 11.0 and 12.4, of
// 4096 x 11008 37 and 49. 129 to 256 rows, whose products have an SM's tensor memory to themselves, where sharing k out saves
// a CTA fifteen steps or more: the many-row kernel has as few tiles then, does not share k, and takes 0.28 us a step. (129 to
// 256 rows, here and there: 13824 x 640 16 to 18 us and 62, 5120 x 3840 22 to 25 and 27, 2560 x 3840 14 to 17 and 16, all with
// 20 steps saved or more; 1280 x 1920, 15 saved, 7.6 to 9.7 and 10.2. 1280 x 2560, 10 saved, 9.8 to 12.4 and 10.5; 640 x 2560,
// 5 saved, 7.7 to 10.3 and 7.5; none: 5120 x 13824 70 to 83 and 62, 1280 x 5120 12.6 to 15 and 12.3.)
bool gated_few_takes(int64_t m, int64_t n, int64_t k)
{
    if (m <= 128) return true;
    const int64_t steps = (k + kBK - 1) / kBK, split = split_of<256>(n, k);
    return m <= 256 && steps - (steps + split - 1) / split >= 15;
}

cudaError_t launch_gated_few(const convrot_gated_linear_args &a, cudaStream_t stream)
{
    return a.dtype == CONVROT_BF16 ? launch_type<__nv_bfloat16>(a, stream) : launch_type<__half>(a, stream);
}

int gated_few_shared(int form, int *columns)
{
    const int bytes[6] = {Shape<16>::SMEM, Shape<32>::SMEM, Shape<64>::SMEM, Shape<80>::SMEM, Shape<128>::SMEM, Shape<256>::SMEM};
    *columns = form < 5 ? Shape<128>::COLS : Shape<256>::COLS;
    return form < 6 ? bytes[form] : 0;
}

}  // namespace convrot
