// The block-scaled linear on the 5th-generation tensor cores
// (include/convrot_block.h):
//
//   Y[r, o] = act(sum_j s_x[r, j] s_w[o / 128, j] sum_{i in block j} q_x[r, i] q_w[o, i] + b[o])
//
// tcgen05.mma kind::f8f6f4 multiplies the e4m3 codes at twice the bf16 rate
// with fp32 accumulators in tensor memory. The scales are general fp32 numbers,
// so each block of 128 features is one accumulation of its own (four K = 32
// instructions) whose sums are drained, multiplied by the row's and the
// block's scale and added up in fp32 registers.
//
// fp8_pair_kernel (the calls that block_fp8_few.cu leaves: more than 64 rows,
// and more tiles than it has resident at once): a CTA pair (cluster of 2,
// cta_group::2), persistent over 256 x kBN output tiles, with the roles and the
// ring of the int8 GEMM:
//   warp 0      TMA producer of each CTA: a block's codes of its 128 rows of x
//               and kBN / 2 rows of w, 128 bytes a row, 128-byte swizzled
//   warp 1      tensor memory; in the even CTA one thread issues the MMAs
//   warps 4-11  drain: two warps a lane quadrant, kBN / 2 columns each
// What bounds it is the turn of the two accumulators: a block's MMAs take 512
// cycles, and then its sums are announced, read (two 64-column loads a warp),
// scaled (128 fmas a thread) and the buffer handed back, ~1600 cycles in all.
// Measured on one GB300: 1070 cycles a block and pair, 2.3 PFLOP/s without the
// activation and 2.05 with the tanh form of GELU (M32760 K5120 N13824, 2.10 and
// 2.35 ms with the pack), at 1380 W of 1400; the MMAs and copies alone would
// take 800 cycles, where L2 feeds 12.6 TB/s. Not faster: sixteen drain warps
// (more loads of fewer columns; 2.48 ms), slices of 128 columns with four
// accumulators (x's codes read twice; 3.46), one CTA on its own (half as much
// again from L2; 2.90), 16-column loads (2.87), scales through shared memory
// (2.70), scales fetched two or four blocks ahead (2.37, 2.44).
// A TMA map ends at column k, so a short last block is filled with zeros.
// Every wait is bounded: one that runs out writes CONVROT_ERR_TIMEOUT to the
// status word and the CTA winds down (copies and MMAs in flight are waited
// for, tensor memory is freed).
#include <cuda.h>
#include <cudaTypedefs.h>

#include "block.h"
#include "tc_common.cuh"

namespace convrot {
namespace {

using namespace tc;

constexpr int kBK = 128;             // codes of one block: 128 bytes, one swizzle span
constexpr int kBM = 128;             // rows of x (and of the accumulators) per CTA
constexpr int kMmaK = 32;
constexpr int kDrainWarps = 8;
constexpr int kPairThreads = 128 + kDrainWarps * 32;
// Registers a thread: launched at 168, warpgroup 0 leaves most of its own to the
// drain warps (128 sums, 64 values on the way): 4 x 32 x 40 + 8 x 32 x 232 = 384 x 168.
constexpr int kRegsWg0 = 40, kRegsDrain = 232;
static_assert(4 * 32 * kRegsWg0 + kDrainWarps * 32 * kRegsDrain <= kPairThreads * 168, "register split");

template <int kBN>
struct Cfg {
    static constexpr int A_BYTES = kBM * kBK, B_BYTES = kBN / 2 * kBK, STAGE_BYTES = A_BYTES + B_BYTES;
    // staging of the outputs: 32 rows of 64 bytes a warp, 80 bytes apart (16-byte accesses of eight rows meet all banks)
    static constexpr int OUT_WARP = 32 * 80;
    static constexpr int BUFS = 512 / kBN;  // accumulators of a block in tensor memory
    static constexpr int BAR_BYTES = 256;
    static constexpr int FIT = (232448 - 1024 - kDrainWarps * OUT_WARP - BAR_BYTES) / STAGE_BYTES;
    static constexpr int STAGES = FIT < 8 ? FIT : 8;
    static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + kDrainWarps * OUT_WARP + BAR_BYTES;
    // kind::f8f6f4: D fp32, A and B e4m3, K-major, M = 256 over both CTAs, N = kBN
    static constexpr uint32_t IDESC = (1u << 4) | (uint32_t(kBN >> 3) << 17) | (uint32_t(256 >> 4) << 24);
    static_assert(SMEM > kTmemAlone, "no other tensor memory on this SM");
    static_assert(8 * (2 * STAGES + BUFS + 1) + 8 <= BAR_BYTES, "barriers fit");
    // a drain warp reads a block's end off its stage's barrier: that may not come round again before every warp has
    // seen it, and block j + STAGES waits for the drains of block j + STAGES - BUFS
    static_assert(STAGES >= BUFS, "stages outlast accumulators");
};

struct Fp8Params {
    int32_t m, n, blocks;  // blocks of k
    int32_t tiles_m, tiles_n;
    const float *x_scale, *w_scale, *bias;
    int64_t ld_x_scale, ld_w_scale;
    void *y;
    int64_t ldy;
    int32_t *dev_status;
    int32_t vec_y;    // rows of y start on 16 bytes
};

__device__ __forceinline__ uint32_t map_to_rank(uint32_t local, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}

__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t leader_bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
        "{%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(leader_bar)
        : "memory");
}

__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrives on the barrier at this offset in both CTAs once the issued MMAs are done.
__device__ __forceinline__ void commit_both(uint32_t bar)
{
    const uint16_t mask = 0x3;
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(mask)
        : "memory");
}

__device__ __forceinline__ void commit_local(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// A drained buffer is handed back without a release: this warp wrote nothing
// that the MMA thread reads, and its tensor-memory loads have completed
// (wait::ld) and are fenced (before_thread_sync) before it arrives: the three
// stay together. (With a release at cluster scope, which waits for everything
// this thread has in flight: 4.70 ms instead of 2.63.)
__device__ __forceinline__ void arrive_remote(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// Tiles in bands of kBand row blocks, columns fastest between bands: the tiles
// in flight share a few panels of x and of w that stay in L2.
constexpr uint32_t kBand = 16;

__device__ __forceinline__ void tile_at(uint32_t t, uint32_t tiles_m, uint32_t tiles_n, uint32_t &mt, uint32_t &nt)
{
    const uint32_t per_band = kBand * tiles_n, band = t / per_band, first = band * kBand;
    const uint32_t rows = tiles_m - first < kBand ? tiles_m - first : kBand;
    const uint32_t local = t - band * per_band;
    mt = first + local % rows;
    nt = local / rows;
}

// 32 lanes x 64 consecutive 32-bit columns; thread i of the warp gets lane (base + i).
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,"
        "%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,"
        "%60,%61,%62,%63}, [%64];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]),
        "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]),
        "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
        "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
        "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// One warp's 32 rows of finished sums (lane: row), 64 bytes of each,
// activated and stored: staged in shared memory and written four lanes a row.
// Lane i has the bias of the slice's columns 4 i .. 4 i + 3; the box starts at
// its column `first`.
template <typename T, int kAct>
__device__ __forceinline__ void store_box(const Fp8Params &p, uint32_t out, int lane, int64_t row0, int64_t col0, const float *acc,
                                          const float (&bias)[4], int first)
{
    constexpr int kBox = 64 / sizeof(T);
    float v[kBox];
#pragma unroll
    for (int i = 0; i < kBox; ++i) v[i] = acc[i];
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < kBox; ++i) v[i] += __shfl_sync(0xffffffffu, bias[i % 4], (first + i) / 4);
    }
    if constexpr (kAct != 0) {
#pragma unroll
        for (int i = 0; i < kBox; i += 2) {
            const F2 two = act2<kAct>(F2(v[i], v[i + 1]));
            v[i] = two.lo();
            v[i + 1] = two.hi();
        }
    }
    Raw<T, kBox> raw;
    raw.pack(v);
    __syncwarp();  // the last box has been read
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(out + lane * 80 + 16 * i), "r"(raw.bits[i].x),
                     "r"(raw.bits[i].y), "r"(raw.bits[i].z), "r"(raw.bits[i].w)
                     : "memory");
    __syncwarp();
    T *y = static_cast<T *>(p.y) + row0 * p.ldy + col0;
    const int rows = p.m - row0 < 32 ? static_cast<int>(p.m - row0) : 32;
    if (p.vec_y && col0 + kBox <= p.n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + lane / 4;
            const uint4 u = shared16(out + r * 80 + lane % 4 * 16);
            if (r < rows) *(reinterpret_cast<uint4 *>(y + r * p.ldy) + lane % 4) = u;
        }
    } else if (lane < kBox && col0 + lane < p.n) {
#pragma unroll 4
        for (int r = 0; r < rows; ++r) {
            if constexpr (sizeof(T) == 4) {
                float u;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(u) : "r"(out + r * 80 + lane * 4) : "memory");
                y[r * p.ldy + lane] = u;
            } else {
                unsigned short u;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(u) : "r"(out + r * 80 + lane * 2) : "memory");
                reinterpret_cast<unsigned short *>(y)[r * p.ldy + lane] = u;
            }
        }
    }
}

template <int kBN, typename T, int kAct>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, const __grid_constant__ Fp8Params p)
{
    using C = Cfg<kBN>;
    constexpr int kCols = kBN / 2, kBox = 64 / sizeof(T);  // columns of a drain warp, and of a staged box
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw));
    const uint32_t base = (raw + 1023u) & ~1023u;  // swizzle atoms are 1024-byte aligned
    uint8_t *gbase = smem_raw + (base - raw);
    constexpr int kOut = C::STAGES * C::STAGE_BYTES, kBars = kOut + kDrainWarps * C::OUT_WARP;
    const uint32_t bars = base + kBars;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (C::STAGES + s); };
    auto acce_bar = [&](int b) { return bars + 8u * (2 * C::STAGES + b); };
    const uint32_t done_bar = bars + 8u * (2 * C::STAGES + C::BUFS);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + kBars + 8 * (2 * C::STAGES + C::BUFS + 1));
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const uint32_t rank = cluster_rank();
    const bool leader = rank == 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t tiles = static_cast<uint32_t>(p.tiles_m) * p.tiles_n, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < C::BUFS; ++b) mbar_init(acce_bar(b), 2 * kDrainWarps);
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmX)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmW)) : "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         static_cast<uint32_t>(__cvta_generic_to_shared(tmem_slot))),
                     "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_sync();  // both CTAs' barriers and tensor memory are there before any remote use
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    after_previous();  // x's codes and scales are the pack's

    // Bounded; gives up early once another role has.
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = globaltimer();
        for (;;) {
#pragma unroll 1
            for (int i = 0; i < 16; ++i)
                if (mbar_try_wait(bar, parity)) return true;
            if (*abort_flag || globaltimer() - t0 > kTimeoutNs) return false;
        }
    };
    auto fail = [&]() {
        *abort_flag = 1;
        if (p.dev_status) atomicExch(p.dev_status, static_cast<int32_t>(CONVROT_ERR_TIMEOUT));
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsWg0));
        if (warp == 0 && lane == 0) {
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (uint32_t t = pair; t < tiles && ok; t += pairs) {
                uint32_t mt, nt;
                tile_at(t, p.tiles_m, p.tiles_n, mt, nt);
                const int xrow = static_cast<int>(mt * 2 * kBM + rank * kBM), wrow = static_cast<int>(nt * kBN + rank * (kBN / 2));
                for (int j = 0; j < p.blocks; ++j) {
                    if (!wait(empty_bar(stage), phase ^ 1u)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sa = base + stage * C::STAGE_BYTES;
                    if (leader) mbar_arrive_expect_tx(full_bar(stage), 2u * C::STAGE_BYTES);
                    const uint32_t bar = map_to_rank(full_bar(stage), 0);
                    tma_load_pair(sa, &tmX, j * kBK, xrow, bar);
                    tma_load_pair(sa + C::A_BYTES, &tmW, j * kBK, wrow, bar);
                    ++issued;
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) {
                fail();
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
            for (uint32_t t = pair; t < tiles && ok; t += pairs) {
                for (int j = 0; j < p.blocks; ++j) {
                    if ((!wait(acce_bar(buf), buf_phase ^ 1u)) || !wait(full_bar(stage), phase)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = base + stage * C::STAGE_BYTES, d = tmem + buf * kBN;
                    const uint64_t da = smem_desc(sa), db = smem_desc(sa + C::A_BYTES);
#pragma unroll
                    for (int kk = 0; kk < kBK / kMmaK; ++kk)  // 32 bytes along K inside the swizzle span
                        mma_pair(d, da + 2u * kk, db + 2u * kk, C::IDESC, kk > 0 ? 1u : 0u);
                    commit_both(empty_bar(stage));  // the stage is free, and the block's sums are there
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (++buf == C::BUFS) {
                        buf = 0;
                        buf_phase ^= 1u;
                    }
                }
            }
            if (!ok) fail();
            commit_local(done_bar);
            mbar_wait(done_bar, 0);
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsDrain));
        const int q = warp & 3, part = (warp - 4) >> 2;  // lane quadrant, column slice
        const uint32_t out = base + kOut + (warp - 4) * C::OUT_WARP;
        const uint32_t taddr0 = tmem + (static_cast<uint32_t>(q * 32) << 16) + part * kCols;
        uint32_t buf = 0, stage = 0, phase = 0;
        const uint32_t acce0 = map_to_rank(acce_bar(0), 0);
        bool ok = true;
        for (uint32_t t = pair; t < tiles && ok; t += pairs) {
            uint32_t mt, nt;
            tile_at(t, p.tiles_m, p.tiles_n, mt, nt);
            const int64_t row0 = static_cast<int64_t>(mt) * 2 * kBM + rank * kBM + q * 32, col0 = static_cast<int64_t>(nt) * kBN + part * kCols;
            // this lane's row and this slice's columns share one scale in each block of k
            const bool row_in = row0 + lane < p.m, col_in = col0 < p.n;
            const float *sx = p.x_scale + (row_in ? row0 + lane : 0), *sw = p.w_scale + (col_in ? col0 / 128 * p.ld_w_scale : 0);
            float bias[4];  // read now, used after the tile's last block
#pragma unroll
            for (int e = 0; e < 4; ++e) bias[e] = p.bias && lane * 4 < kCols && col0 + lane * 4 + e < p.n ? load_f32(p.bias + col0 + lane * 4 + e) : 0.0f;
            float acc[kCols];
#pragma unroll
            for (int i = 0; i < kCols; ++i) acc[i] = 0.0f;
            float next_x = load_f32(sx), next_w = load_f32(sw);
            for (int j = 0; j < p.blocks; ++j) {
                const float scale = next_x * next_w;
                if (j + 1 < p.blocks) {  // the next block's scales arrive under this block's wait
                    sx += p.ld_x_scale;
                    next_x = load_f32(sx);
                    next_w = load_f32(++sw);
                }
                if (!all_lanes(wait(empty_bar(stage), phase))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t taddr = taddr0 + buf * kBN;
#pragma unroll
                for (int c = 0; c < kCols / 64; ++c) {
                    uint32_t r[64];
                    tmem_ld64(taddr + c * 64, r);
                    if (c == kCols / 64 - 1) {  // read to the end: the buffer is free
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_remote(acce0 + 8u * buf);
                    }
#pragma unroll
                    for (int i = 0; i < 64; ++i) acc[c * 64 + i] = fmaf(__uint_as_float(r[i]), scale, acc[c * 64 + i]);
                }
                if (++buf == C::BUFS) buf = 0;
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) break;
            if (row0 < p.m) {
#pragma unroll
                for (int c = 0; c < kCols / kBox; ++c)
                    if (col0 + c * kBox < p.n) store_box<T, kAct>(p, out, lane, row0, col0 + c * kBox, acc + c * kBox, bias, c * kBox);
            }
        }
        if (!ok) fail();
    }

    tc_fence_before();
    cluster_sync();  // neither CTA's shared or tensor memory goes away under the other's use
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

template <int kBN, typename T, int kAct>
struct pair_tag;

template <int kBN, typename T, int kAct>
cudaError_t launch_pair(const convrot_fp8_linear_args &a, cudaStream_t stream)
{
    using C = Cfg<kBN>;
    CUtensorMap tmX, tmW;
    if (!make_map_2d(&tmX, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.x, a.m, a.k, a.ldx, kBK, kBM) ||
        !make_map_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, a.n, a.k, a.ldw, kBK, kBN / 2))
        return cudaErrorInvalidValue;
    Fp8Params p{};
    p.m = static_cast<int32_t>(a.m);
    p.n = static_cast<int32_t>(a.n);
    p.blocks = static_cast<int32_t>((a.k + kBK - 1) / kBK);
    p.tiles_m = static_cast<int32_t>((a.m + 2 * kBM - 1) / (2 * kBM));
    p.tiles_n = static_cast<int32_t>((a.n + kBN - 1) / kBN);
    p.x_scale = a.x_scale;
    p.w_scale = a.w_scale;
    p.bias = a.bias;
    p.ld_x_scale = a.ld_x_scale;
    p.ld_w_scale = a.ld_w_scale;
    p.y = a.y;
    p.ldy = a.ldy;
    p.dev_status = a.dev_status;
    p.vec_y = aligned_to(a.y, 16) && a.ldy * sizeof(T) % 16 == 0;
    auto kernel = fp8_pair_kernel<kBN, T, kAct>;
    cudaError_t e = allow_shared<pair_tag<kBN, T, kAct>>(kernel);
    if (e != cudaSuccess) return e;
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    const int64_t pairs = tiles < kSms / 2 ? tiles : kSms / 2;
    return launch_after(kernel, dim3(static_cast<unsigned>(2 * pairs)), kPairThreads, C::SMEM, stream, 1, tmX, tmW, p);
}

}  // namespace

cudaError_t launch_fp8_gemm(const convrot_fp8_linear_args &a, cudaStream_t stream)
{
    return with_dtype(a.y_dtype, [&](auto *tag) {
        using T = std::remove_pointer_t<decltype(tag)>;
        // Tiles of 256 or 128 columns, by the rounds that the 76 pairs take over them: a block of k costs 0.59 us in a
        // wide tile and 0.48 us in a narrow one (M32760 K5120 N13824 and M256 K5120 N13824), so narrow ones pay only
        // where they save a round in five or spread a lone round over idle pairs.
        const int64_t rows = (a.m + 255) / 256, pairs = kSms / 2;
        const int64_t rounds_wide = (rows * ((a.n + 255) / 256) + pairs - 1) / pairs;
        const int64_t rounds_narrow = (rows * ((a.n + 127) / 128) + pairs - 1) / pairs;
        const bool wide = rounds_wide * 59 <= rounds_narrow * 48;
        if (a.act == CONVROT_ACT_GELU_ERF) return wide ? launch_pair<256, T, 1>(a, stream) : launch_pair<128, T, 1>(a, stream);
        if (a.act == CONVROT_ACT_GELU_TANH) return wide ? launch_pair<256, T, 2>(a, stream) : launch_pair<128, T, 2>(a, stream);
        return wide ? launch_pair<256, T, 0>(a, stream) : launch_pair<128, T, 0>(a, stream);
    });
}

}  // namespace convrot
