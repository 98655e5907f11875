// 16-bit matrix products on the 5th-generation tensor cores, for the kernels of
// this folder: tcgen05.mma kind::f16 (bf16 x bf16 or f16 x f16, fp32 sums in
// tensor memory) with operands that are K-major or MN-major in shared memory,
// or, for A, in tensor memory. (PTX ISA: tcgen05, cp.async.bulk.tensor.)
//
// Shared-memory tiles are what a TMA box of 64 elements (128 bytes) times some
// rows leaves with the 128-byte swizzle. The same bytes serve as both majors:
//   K-major   a row is an M (or N) index, its 64 elements are K: 8-row groups
//             1024 bytes apart, 16 elements of K are 32 bytes further
//   MN-major  a row is a K index, its 64 elements are M (or N): 8-row groups of
//             K 1024 bytes apart, 16 of K are 2048 bytes further, and the next
//             64 of M (or N) are the next box, `box` bytes on
#pragma once

#include "../csrc/block.h"
#include "../csrc/tc_common.cuh"

namespace convrot {
namespace mma16 {

using namespace tc;

constexpr int kBoxElems = 64;  // of a box's rows: 128 bytes, one swizzle span
constexpr int kMmaK = 16;

// Steps of the descriptors (16-byte units) for the next 16 elements of K.
constexpr uint32_t kStepK = 32 / 16, kStepMN = 2048 / 16;

__device__ __forceinline__ uint64_t desc_k(uint32_t addr) { return smem_desc(addr); }
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t box)
{
    return uint64_t((addr >> 4) & 0x3fff) | (uint64_t((box >> 4) & 0x3fff) << 16) | (uint64_t(1024 >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// Instruction descriptor: D fp32, A and B of T, M x N, either operand MN-major.
template <typename T>
__host__ __device__ constexpr uint32_t idesc(int m, int n, bool a_mn, bool b_mn)
{
    const uint32_t type = std::is_same_v<T, __nv_bfloat16> ? 1u : 0u;
    return (1u << 4) | (type << 7) | (type << 10) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// kGroup: CTAs that the product spans (the leader's thread issues for both).
template <int kGroup>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate)
{
    if constexpr (kGroup == 2)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(accumulate)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(accumulate)
                     : "memory");
}

// The same as parts of a longer sum, for tiles of 128 x 128, whose issue counts: an instruction takes the tensor cores 64
// cycles, and one thread that computes its operands in a branch of its own took 80 to 140 for its issue. So the issuing
// warp stays together up to the instruction itself (one_thread), which lets its operands live in uniform registers; the
// flag is an immediate, the descriptor's upper half is fixed, and the loops that call these are unrolled.
__device__ __forceinline__ bool one_thread()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
// The number of this thread's warp, the same for all its lanes as far as the compiler sees.
__device__ __forceinline__ int warp_number() { return __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0); }
struct Desc {
    uint32_t lo, hi;
    __device__ __forceinline__ explicit Desc(uint64_t d) : lo(static_cast<uint32_t>(d)), hi(static_cast<uint32_t>(d >> 32)) {}
};

template <bool kAccumulate>
__device__ __forceinline__ void mma_ss_step(uint32_t d, Desc a, uint32_t a_step, Desc b, uint32_t b_step, uint32_t id)
{
    if constexpr (kAccumulate)
        asm volatile("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, 1;\n\t}" ::"r"(d), "r"(a.lo + a_step), "r"(a.hi), "r"(b.lo + b_step), "r"(b.hi), "r"(id)
                     : "memory");
    else
        asm volatile("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, 0;\n\t}" ::"r"(d), "r"(a.lo + a_step), "r"(a.hi), "r"(b.lo + b_step), "r"(b.hi), "r"(id)
                     : "memory");
}

// A in tensor memory: lane = row, two elements of K a column.
template <bool kAccumulate>
__device__ __forceinline__ void mma_ts_step(uint32_t d, uint32_t a, Desc b, uint32_t b_step, uint32_t id)
{
    if constexpr (kAccumulate)
        asm volatile("{\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, 1;\n\t}" ::"r"(d), "r"(a), "r"(b.lo + b_step), "r"(b.hi), "r"(id)
                     : "memory");
    else
        asm volatile("{\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, 0;\n\t}" ::"r"(d), "r"(a), "r"(b.lo + b_step), "r"(b.hi), "r"(id)
                     : "memory");
}

// All of an SM's columns, or a part (a multiple of 128): a launch asks for the
// shared memory that goes with them (tc_common.cuh).
template <int kGroup>
__device__ __forceinline__ void tmem_alloc(uint32_t *slot, uint32_t columns)
{
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(slot));
    if constexpr (kGroup == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(at), "r"(columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(at), "r"(columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
}

template <int kGroup>
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t columns)
{
    if constexpr (kGroup == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns) : "memory");
}

__device__ __forceinline__ uint32_t map_to_rank(uint32_t local, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}

// Into this CTA's shared memory, counted at the barrier of the pair's leader.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t leader_bar)
{
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(leader_bar)
                 : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Arrives on the barrier at this offset in both CTAs of the pair once the issued MMAs are done.
__device__ __forceinline__ void commit_both(uint32_t bar)
{
    const uint16_t mask = 0x3;
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar), "h"(mask) : "memory");
}

__device__ __forceinline__ void commit_pair_local(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// For a buffer that was read from tensor memory: nothing that this thread wrote is read behind the barrier.
__device__ __forceinline__ void arrive_remote(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// 32 lanes x 32 columns, without the wait: r is there after tmem_ld_wait.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
          "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, uint32_t *r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
                   "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}
// The values pass through, so that nothing reads them before the wait.
template <int N>
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[N])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *v)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]),
                 "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two values rounded to T, the first in the low half.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}

// act of two values: GELU as in block.h, SiLU through one exponential and one reciprocal.
template <int kAct>
__device__ __forceinline__ F2 gate_act2(F2 v)
{
    if constexpr (kAct == CONVROT_ACT_SILU) {
        const F2 z = v * F2(-1.4426950f);
        const F2 e = F2(ex2(z.lo()), ex2(z.hi())) + F2(1.0f);
        return v * F2(rcp(e.lo()), rcp(e.hi()));
    } else {
        return act2<kAct>(v);
    }
}

// The kernels' bounded wait: gives up early once another role of the block has. It is one thread's; a warp that goes on to an
// instruction that all its lanes have to reach (tcgen05.ld, a shuffle, a barrier) waits together, since each lane reads the
// timer for itself.
struct Waits {
    volatile int *abort_flag;
    int32_t *dev_status;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const
    {
        if (mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = globaltimer();
        for (;;) {
            if (try_long(bar, parity)) return true;
            if (*abort_flag || globaltimer() - t0 > kTimeoutNs) return false;
        }
    }
    // A try that may sleep for 0.1 ms: warps that come back to try again take issue slots from those that compute.
    static __device__ __forceinline__ bool try_long(uint32_t bar, uint32_t parity)
    {
        uint32_t ok;
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 100000;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
        return ok != 0;
    }
    // by a whole warp: true for all lanes or for none, so that it leaves as a whole or not at all
    __device__ __forceinline__ bool together(uint32_t bar, uint32_t parity) const { return all_lanes((*this)(bar, parity)); }
    // whether it is there now
    __device__ __forceinline__ bool now(uint32_t bar, uint32_t parity) const
    {
        uint32_t ok;
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
        return __all_sync(0xffffffffu, ok != 0);
    }
    __device__ __forceinline__ void fail() const
    {
        *abort_flag = 1;
        if (dev_status) atomicExch(dev_status, static_cast<int32_t>(CONVROT_ERR_TIMEOUT));
    }
};

// Eight 16-bit elements from any address, of which the first n (1 to 8) are wanted and the others become 0. The one or two
// aligned 16-byte blocks that hold wanted elements are read whole, whoever's the rest of them is, and shifted. (A block is in
// one page, so its rest is there too; the header tells callers.)
__device__ __forceinline__ uint4 load8_any(const void *p, int n)
{
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    const int skip = static_cast<int>(at & 15) / 2;
    const uint4 *block = reinterpret_cast<const uint4 *>(at & ~uintptr_t{15});
    auto load = [](const uint4 *from) {
        uint4 v;
        asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(from));
        return v;
    };
    uint4 lo = load(block), hi = make_uint4(0, 0, 0, 0);
    if (skip + n > 8) hi = load(block + 1);
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = skip & 4 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = skip & 2 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = skip & 1 ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = 2 * i + 1 < n ? w[i] : 2 * i < n ? w[i] & 0xffffu : 0u;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Its counterpart: the first n of eight elements, in the widest pieces that the address allows.
__device__ __forceinline__ void store8_any(void *p, uint4 v, int n)
{
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (n >= 8 && at % 16 == 0) {
        *static_cast<uint4 *>(p) = v;
    } else if (n >= 4 && n % 4 == 0 && at % 8 == 0) {
        static_cast<uint2 *>(p)[0] = make_uint2(w[0], w[1]);
        if (n >= 8) static_cast<uint2 *>(p)[1] = make_uint2(w[2], w[3]);
    } else {
        unsigned short *to = static_cast<unsigned short *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (2 * i + 1 < n && at % 4 == 0) {
                reinterpret_cast<uint32_t *>(to)[i] = w[i];
            } else {
                if (2 * i < n) to[2 * i] = static_cast<unsigned short>(w[i] & 0xffffu);
                if (2 * i + 1 < n) to[2 * i + 1] = static_cast<unsigned short>(w[i] >> 16);
            }
        }
    }
}

__device__ __forceinline__ int64_t load_i32(const int32_t *p) { return *reinterpret_cast<const volatile int32_t *>(p); }

// One warp's 32 rows (lane: row) of 32 values each, rounded to T and stored:
// staged in shared memory (`stage`, kStageBytes of this warp's own: with 80
// bytes a row, 16-byte accesses of eight rows meet all banks) and written four
// lanes a row, 64 bytes of each. `rows` and `cols` of them exist; wide: rows
// start on 16 bytes.
constexpr int kStagePitch = 80, kStageBytes = 32 * kStagePitch;

template <typename T>
__device__ __forceinline__ void store_rows(T *y, int64_t ld, int rows, int cols, bool wide, uint32_t stage, int lane, const float (&v)[32])
{
    static_assert(sizeof(T) == 2, "16-bit elements");
    __syncwarp();  // the last box has been read
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * kStagePitch + 16 * i), "r"(pack2<T>(v[8 * i], v[8 * i + 1])),
                     "r"(pack2<T>(v[8 * i + 2], v[8 * i + 3])), "r"(pack2<T>(v[8 * i + 4], v[8 * i + 5])), "r"(pack2<T>(v[8 * i + 6], v[8 * i + 7]))
                     : "memory");
    __syncwarp();
    if (wide && cols >= 32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + lane / 4;
            const uint4 u = shared16(stage + r * kStagePitch + lane % 4 * 16);
            if (r < rows) *(reinterpret_cast<uint4 *>(y + r * ld) + lane % 4) = u;
        }
    } else if (lane < cols) {
#pragma unroll 4
        for (int r = 0; r < rows && r < 32; ++r) {
            unsigned short u;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(u) : "r"(stage + r * kStagePitch + lane * 2) : "memory");
            reinterpret_cast<unsigned short *>(y)[r * ld + lane] = u;
        }
    }
}

// The same without shared memory: four lanes trade their 16-byte pieces until each has one of each one's row.
template <typename T>
__device__ __forceinline__ void store_rows_traded(T *y, int64_t ld, int rows, int cols, bool wide, int lane, const float (&v)[32])
{
    uint32_t w[4][4];  // pieces of this lane's row
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) w[i][e] = pack2<T>(v[8 * i + 2 * e], v[8 * i + 2 * e + 1]);
    if (wide && cols >= 32) {
        // w[i] of lane l becomes piece l % 4 of the row of lane l / 4 * 4 + i
#pragma unroll
        for (int bit = 1; bit <= 2; bit <<= 1) {
            const bool high = lane & bit;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i & bit) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? w[i][e] : w[i | bit][e], bit);
                    if (high)
                        w[i][e] = got;
                    else
                        w[i | bit][e] = got;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = lane / 4 * 4 + i;
            if (r < rows) *(reinterpret_cast<uint4 *>(y + r * ld) + lane % 4) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
        }
    } else if (lane < rows) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i * 8 < cols) store8_any(y + lane * ld + i * 8, make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]), cols - i * 8);
    }
}

// What a tensor map can describe: rows that start on 16 bytes.
inline bool tma_rows(const void *p, int64_t ld, int64_t rows) { return aligned_to(p, 16) && (rows <= 1 || ld % 8 == 0); }

template <typename T>
constexpr CUtensorMapDataType map_type()
{
    return std::is_same_v<T, __nv_bfloat16> ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// A matrix [rows, cols] of T with rows that start on 16 bytes, in boxes of 64 columns.
template <typename T>
bool matrix_map(CUtensorMap *map, const void *p, int64_t rows, int64_t cols, int64_t ld, uint32_t box_rows)
{
    const int64_t pitch = rows > 1 ? ld : (cols + 7) / 8 * 8;
    return make_map_2d(map, map_type<T>(), p, rows, cols, pitch * 2, kBoxElems, box_rows);
}

}  // namespace mma16
}  // namespace convrot
