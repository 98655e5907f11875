// The keys' and values' gradients of attention (include/convrot_block.h), on
// the 5th-generation tensor cores:
//
//   dv_j = sum_i P_ij dout_i,  dk_j = scale sum_i dS_ij q_i
//   P = 2^(c s + base2),  dS = P (dP + delta),  dP = dout V^T
//
// A unit is 128 keys of one head: all queries of the heads that share it pass
// by, 128 at a time, and dV and dK stay in tensor memory. Everything is made
// transposed, a key a lane, so that P^T and dS^T are A operands straight from
// tensor memory and dout and q are read MN-major from the bytes that S^T = K Q^T
// and dP^T = V dout^T read K-major.
//   warp 0       TMA producer: the unit's keys and values, then tiles of queries,
//                their statistics and dout, a ring each: a tile of queries is
//                needed to its end, so its ring is one longer (with two of each,
//                the next S^T waited 1200 cycles a tile for its queries)
//   warp 1       tensor memory; one thread issues the MMAs: while P^T is made
//                from S^T the tensor cores do the tile before's dK and the next
//                dP^T, and while dS^T is made, dV and the next S^T
//   warps 4-19   P^T and dS^T: four threads a key, 32 of the tile's queries each
//
// kAll: where one tile holds all keys and the heads are narrow, dQ = scale dS K is
// made here too, from dS^T that the same threads leave in shared memory (an
// MN-major A operand), into one of two places in tensor memory; the threads read
// it, 16 elements of a query each, while the next tile's products run. Masked
// keys have zeros in K for it (warps 2 and 3), and in dS^T.
//
// The work of all units, laid end to end, is cut into equal runs of tiles, one a
// CTA, whatever the number of units: a unit that a cut goes through is left as
// partial sums in fp32 and added up by a second kernel in the order of the
// cuts, which depends on the sizes alone.
//
// 8190 queries, 512 keys, 40 heads of 128: 123 us and 11 for the joined sums, the
// tensor cores busy for 63 % of it; with kAll, 2 x 4096 queries, 77 keys, 10 heads of
// 64: 21 us and 5.
#include "attention.cuh"

namespace convrot {
namespace {

using namespace mma16;

constexpr int kMathWarps = 16, kThreads = 128 + 32 * kMathWarps;
// Registers a thread: launched at 96, warpgroup 0 leaves some of its own to the others.
constexpr int kRegsWg0 = 64, kRegsMath = 104;
static_assert(4 * 32 * kRegsWg0 + 32 * kMathWarps * kRegsMath <= kThreads * 96, "register split");
constexpr int kPart = 32;  // columns of a tile that a thread has

template <int kD, bool kAll>
struct Cfg {
    static_assert(!kAll || kD == 64, "tensor memory");
    static constexpr int HALVES = kD / 64, TILE = HALVES * kTileBox;
    static constexpr int QS = kD == 128 ? 3 : kAll ? 4 : 5, DS = kD == 128 ? 2 : kAll ? 3 : 4;  // tiles of queries, and of dout
    static constexpr int STATS = 2 * kTileQueries * 4;  // base2 and delta of a tile: DS of them, too
    static constexpr int DST = kAll ? 2 * kTileBox : 0;  // dS^T of a tile: two of them
    static constexpr int BARS = 2 * QS + 4 * DS + 11;
    static constexpr int BAR_BYTES = 384;
    static constexpr int SMEM = (2 + QS + DS) * TILE + 2 * DST + DS * STATS + BAR_BYTES;
    static constexpr uint32_t S_COL = 0, DP_COL = 128, DV_COL = 256, DK_COL = 384, DQ_COL = 320;  // dQ: + 128 for every other tile
    static_assert(SMEM > kTmemAlone && SMEM <= kMaxShared, "no other tensor memory on this SM");
    static_assert(8 * BARS + 8 <= BAR_BYTES, "barriers fit");
};

// How the tiles of all units are cut.
struct Cut {
    int64_t units, per_unit, work;
    int32_t runs;
    __host__ __device__ int64_t start(int64_t run) const { return run * work / runs; }
    // the run that a tile is in
    __host__ __device__ int64_t run_of(int64_t tile) const { return ((tile + 1) * runs - 1) / work; }
};

struct Params {
    HeadsMap q, dout, k, v;
    const int32_t *counts, *index;
    int64_t index_rows;
    const uint8_t *mask;  // applied here: gradients of keys that are not there are 0 (their rows of S^T and dP^T are theirs alone)
    int64_t mask_stride;
    const float *base2, *delta, *amax;
    int64_t amax_blocks, stat_rows;
    float *partial;  // [runs][2][2][128][kD]: a run's first and last unit where they are cut, dV and dK
    void *dk, *dv, *dq;
    int32_t *dev_status;
    Cut cut;
    int32_t q_tokens, kv_tokens, kv_heads, q_heads, group, q_tiles, key_tiles;
    int32_t d, wide;
    float scale, scale_log2;
};

// One unit: sample, head, tile of keys.
struct Unit {
    int b, h, tile, keys;  // keys of the sample
    int64_t row;           // of the first key in dk and dv, or in the index
};

template <typename P>
__device__ __forceinline__ Unit unit_at(const P &p, int64_t u)
{
    Unit r;
    const int64_t bh = u / p.key_tiles;
    r.tile = static_cast<int>(u - bh * p.key_tiles);
    r.b = static_cast<int>(bh / p.kv_heads);
    r.h = static_cast<int>(bh - static_cast<int64_t>(r.b) * p.kv_heads);
    r.keys = p.counts ? static_cast<int>(load_i32(p.counts + r.b)) : p.kv_tokens;
    return r;
}

// Where a key's row of a gradient is.
template <typename T>
__device__ __forceinline__ T *key_row(const Params &p, const Unit &u, void *to, int key)
{
    const int64_t token = p.index ? load_i32(p.index + u.b * p.index_rows + key) : key;
    return static_cast<T *>(to) + ((static_cast<int64_t>(u.b) * p.kv_tokens + token) * p.kv_heads + u.h) * p.d;
}

__device__ __forceinline__ bool key_masked(const Params &p, const Unit &u, int key)
{
    return p.mask && *reinterpret_cast<const volatile uint8_t *>(p.mask + u.b * p.mask_stride + key) == 0;
}

template <typename T, int kD, bool kAll>
__global__ void __launch_bounds__(kThreads, 1) attention_grad_kv_kernel(const __grid_constant__ Params p)
{
    using C = Cfg<kD, kAll>;
    constexpr bool kHalf = std::is_same_v<T, __half>;
    extern __shared__ __align__(1024) uint8_t smem_tiles[];  // swizzle atoms are 1024-byte aligned
    uint8_t *gbase = smem_tiles;
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem_tiles));
    constexpr int kQueries = 2 * C::TILE, kDouts = kQueries + C::QS * C::TILE, kDst = kDouts + C::DS * C::TILE, kStats = kDst + 2 * C::DST, kBars = kStats + C::DS * C::STATS;
    const uint32_t bars = base + kBars;
    auto q_full = [&](int s) { return bars + 8u * s; };
    auto q_empty = [&](int s) { return bars + 8u * (C::QS + s); };
    auto do_full = [&](int s) { return bars + 8u * (2 * C::QS + s); };
    auto do_empty = [&](int s) { return bars + 8u * (2 * C::QS + C::DS + s); };
    auto st_full = [&](int s) { return bars + 8u * (2 * C::QS + 2 * C::DS + s); };
    auto st_empty = [&](int s) { return bars + 8u * (2 * C::QS + 3 * C::DS + s); };
    const uint32_t kv_full = bars + 8u * (2 * C::QS + 4 * C::DS), kv_empty = kv_full + 8, s_full = kv_full + 16, dp_full = kv_full + 24;
    const uint32_t p_ready = kv_full + 32, ds_ready = kv_full + 40;
    const uint32_t sums_full = kv_full + 48, done_bar = kv_full + 56, kv_clean = kv_full + 64;
    auto dq_full = [&](int n) { return kv_full + 72 + 8u * (n & 1); };
    // the places of tile t, counted over all units of this run, and the parity of their n-th use
    auto q_at = [&](int t) { return base + kQueries + t % C::QS * C::TILE; };
    auto do_at = [&](int t) { return base + kDouts + t % C::DS * C::TILE; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + kBars + 8 * C::BARS);
    const Waits wait{reinterpret_cast<volatile int *>(tmem_slot + 1), p.dev_status};
    const int warp = warp_number(), lane = threadIdx.x & 31;

    if (base & 1023u) {  // (no room to align it here: what the compiler was asked for above)
        if (threadIdx.x == 0 && p.dev_status) atomicExch(p.dev_status, static_cast<int32_t>(CONVROT_ERR_ALIGNMENT));
        return;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::QS; ++s) {
            mbar_init(q_full(s), 1);
            mbar_init(q_empty(s), 1);
        }
        for (int s = 0; s < C::DS; ++s) {
            mbar_init(do_full(s), 1);
            mbar_init(do_empty(s), 1);
            mbar_init(st_full(s), 1);
            mbar_init(st_empty(s), kMathWarps);
        }
        mbar_init(kv_full, 1);
        mbar_init(kv_empty, 1);
        mbar_init(s_full, 1);
        mbar_init(dp_full, 1);
        mbar_init(p_ready, kMathWarps);
        mbar_init(ds_ready, kMathWarps);
        mbar_init(sums_full, 1);
        mbar_init(done_bar, 1);
        mbar_init(kv_clean, 2);
        mbar_init(dq_full(0), 1);
        mbar_init(dq_full(1), 1);
        *wait.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&p.q.map);
        prefetch_map(&p.dout.map);
        prefetch_map(&p.k.map);
        prefetch_map(&p.v.map);
    }
    if (warp == 1) tmem_alloc<1>(tmem_slot, 512u);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    after_previous();
    let_next_start();

    const int64_t first = p.cut.start(blockIdx.x), last = p.cut.start(blockIdx.x + 1);
    // calls f(unit, its number, first and last tile of it here) for the units of this run that have keys
    auto each_unit = [&](auto f) {
        for (int64_t w = first; w < last;) {
            const int64_t n = w / p.cut.per_unit, begin = n * p.cut.per_unit, end = begin + p.cut.per_unit;
            const int64_t to = end < last ? end : last;
            const Unit u = unit_at(p, n);
            if (u.tile * kTileKeys < u.keys)
                if (!f(u, static_cast<int>(w - begin), static_cast<int>(to - begin))) return false;
            w = to;
        }
        return true;
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsWg0));
        if (warp == 0 && lane == 0) {
            int n = 0, loaded_q = 0, loaded_st = 0, loaded_do = 0;  // tiles, over all units
            uint32_t kv_phase = 0;
            bool kv = false;
            const bool ok = each_unit([&](const Unit &u, int t0, int t1) {
                if (!wait(kv_empty, kv_phase ^ 1u)) return false;
                kv_phase ^= 1u;
                mbar_arrive_expect_tx(kv_full, 2 * C::TILE);
                load_tile<C::HALVES>(base, p.k, u.tile * kTileKeys, u.h, u.b, kv_full);
                load_tile<C::HALVES>(base + C::TILE, p.v, u.tile * kTileKeys, u.h, u.b, kv_full);
                kv = true;
                for (int t = t0; t < t1; ++t, ++n) {
                    const int h = u.h * p.group + t / p.q_tiles, q0 = t % p.q_tiles * kTileQueries, qs = n % C::QS, ds = n % C::DS;
                    const int64_t row = (static_cast<int64_t>(u.b) * p.q_heads + h) * p.stat_rows + q0;
                    if (!wait(q_empty(qs), (n / C::QS + 1) & 1)) return false;
                    mbar_arrive_expect_tx(q_full(qs), C::TILE);
                    load_tile<C::HALVES>(q_at(n), p.q, q0, h, u.b, q_full(qs));
                    ++loaded_q;
                    if (!wait(st_empty(ds), (n / C::DS + 1) & 1)) return false;
                    const uint32_t stats = base + kStats + ds * C::STATS;
                    mbar_arrive_expect_tx(st_full(ds), C::STATS);
                    bulk_load(stats, p.base2 + row, kTileQueries * 4, st_full(ds));
                    bulk_load(stats + kTileQueries * 4, p.delta + row, kTileQueries * 4, st_full(ds));
                    ++loaded_st;
                    if (!wait(do_empty(ds), (n / C::DS + 1) & 1)) return false;
                    mbar_arrive_expect_tx(do_full(ds), C::TILE);
                    load_tile<C::HALVES>(do_at(n), p.dout, q0, h, u.b, do_full(ds));
                    ++loaded_do;
                }
                return true;
            });
            if (!ok) {
                wait.fail();
                // copies in flight land before shared memory goes away
                for (int i = loaded_q > C::QS ? loaded_q - C::QS : 0; i < loaded_q; ++i) mbar_wait(q_full(i % C::QS), (i / C::QS) & 1);
                for (int i = loaded_st > C::DS ? loaded_st - C::DS : 0; i < loaded_st; ++i) mbar_wait(st_full(i % C::DS), (i / C::DS) & 1);
                for (int i = loaded_do > C::DS ? loaded_do - C::DS : 0; i < loaded_do; ++i) mbar_wait(do_full(i % C::DS), (i / C::DS) & 1);
                if (kv) mbar_wait(kv_full, kv_phase ^ 1u);
            }
        } else if (warp == 1) {
            const uint32_t id_s = idesc<T>(128, 128, false, false);
            const int n_o = (p.d + 15) / 16 * 16, steps = (p.d + kMmaK - 1) / kMmaK;
            const uint32_t id_o = idesc<T>(128, n_o, false, true);
            const uint32_t id_q = idesc<T>(128, n_o, true, true);
            int n = 0;  // tiles, over all units
            uint32_t kv_phase = 0;
            auto product = [&](uint32_t to, uint32_t rows, uint32_t cols) { tile_product<kD>(to, rows, cols, id_s, steps); };
            // sums += (what a region's quarters hold in 16 bits) x a tile, over the queries
            auto add = [&](uint32_t sums, uint32_t region, uint32_t tile, bool fresh) { tile_add<4>(sums, region, tile, id_o, fresh); };
            auto q_there = [&](int t) { return wait.together(q_full(t % C::QS), (t / C::QS) & 1); };
            auto do_there = [&](int t) { return wait.together(do_full(t % C::DS), (t / C::DS) & 1); };
            const bool ok = each_unit([&](const Unit &, int t0, int t1) {
                if (!wait.together(kv_full, kv_phase) || !q_there(n) || !do_there(n)) return false;
                if (kAll && p.mask && !wait.together(kv_clean, kv_phase)) return false;
                kv_phase ^= 1u;
                tc_fence_after();
                if (one_thread()) {
                    product(tmem + C::S_COL, base, q_at(n));
                    mma_commit(s_full);
                    product(tmem + C::DP_COL, base + C::TILE, do_at(n));
                    mma_commit(dp_full);
                }
                __syncwarp();
                for (int t = t0; t < t1; ++t, ++n) {
                    const bool more = t + 1 < t1;
                    // (what the ring brings is waited for ahead of what the threads make: the tensor cores idle meanwhile)
                    if ((more && !q_there(n + 1)) || !wait.together(p_ready, n & 1)) return false;
                    tc_fence_after();
                    if (one_thread()) {
                        add(tmem + C::DV_COL, tmem + C::S_COL, do_at(n), t == t0);
                        if (more) {
                            product(tmem + C::S_COL, base, q_at(n + 1));
                            mma_commit(s_full);
                        }
                        mma_commit(do_empty(n % C::DS));  // (the tile's dP^T came before)
                    }
                    __syncwarp();
                    if ((more && !do_there(n + 1)) || !wait.together(ds_ready, n & 1)) return false;
                    tc_fence_after();
                    if (one_thread()) {
                        add(tmem + C::DK_COL, tmem + C::DP_COL, q_at(n), t == t0);
                        if (more) {
                            product(tmem + C::DP_COL, base + C::TILE, do_at(n + 1));
                            mma_commit(dp_full);
                        }
                        mma_commit(q_empty(n % C::QS));
                        if constexpr (kAll) {  // dQ = dS K, over the keys
                            const Desc a(desc_mn(base + kDst + (n & 1) * C::DST, kTileBox)), b(desc_mn(base, kTileBox));
                            const uint32_t dq = tmem + C::DQ_COL + 128 * (n & 1);
                            mma_ss_step<false>(dq, a, 0, b, 0, id_q);
#pragma unroll
                            for (int kk = 1; kk < kTileKeys / kMmaK; ++kk) mma_ss_step<true>(dq, a, kStepMN * kk, b, kStepMN * kk, id_q);
                            mma_commit(dq_full(n));
                        }
                        if (!more) {
                            mma_commit(kv_empty);
                            mma_commit(sums_full);
                        }
                    }
                    __syncwarp();
                }
                return true;
            });
            if (!ok) wait.fail();
            if (one_thread()) {
                mma_commit(done_bar);
                mbar_wait(done_bar, 0);
            }
        } else if (kAll && warp >= 2 && p.mask) {
            uint32_t kv_phase = 0;
            MaskedRows rows;
            const bool ok = each_unit([&](const Unit &u, int, int) {
                rows.of(p.mask, p.mask_stride, u.b, u.keys, warp - 2, lane);
                if (!wait.together(kv_full, kv_phase)) return false;
                kv_phase ^= 1u;
                clean_rows<C::HALVES>(base, rows.there, warp - 2, lane);
                if (lane == 0) mbar_arrive(kv_clean);
                return true;
            });
            if (!ok) wait.fail();
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMath));
        const int part = (warp - 4) >> 2, quad = warp & 3;  // of the tile's queries; of the keys
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        const F2 c2(p.scale_log2);
        int n = 0;  // tiles, over all units
        uint32_t sums_phase = 0;
        const bool ok = each_unit([&](const Unit &u, int t0, int t1) {
            int exponent = 0;
            if constexpr (kHalf)
                exponent = grad_exponent(p.amax + (static_cast<int64_t>(u.b) * p.kv_heads + u.h) * p.amax_blocks, p.amax_blocks, lane);
            const F2 up(kHalf ? exp2i(exponent) * exp2i(-15) : 1.0f);
            const int key = u.tile * kTileKeys + quad * 32 + lane;
            const bool there = key < u.keys, masked = there && key_masked(p, u, key);
            // dQ of tile t of this unit, the m-th of this run: 16 elements of a query
            auto read_dq = [&](int t, int m) {
                if (!wait.together(dq_full(m), (m >> 1) & 1)) return false;
                tc_fence_after();
                const int h = u.h * p.group + t / p.q_tiles, row = t % p.q_tiles * kTileQueries + quad * 32 + lane, col = part * 16;
                if (col >= p.d) return true;
                uint32_t o[16];
                tmem_ld16_async(lanes + C::DQ_COL + 128 * (m & 1) + col, o);
                tmem_ld_wait(o);
                tc_fence_before();
                if (row >= p.q_tokens) return true;
                const float down = p.scale * (kHalf ? exp2i(-exponent) : 1.0f);
                T *to = static_cast<T *>(p.dq) + ((static_cast<int64_t>(u.b) * p.q_tokens + row) * p.q_heads + h) * p.d + col;
                float v[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(o[e]) * down;
#pragma unroll
                for (int e = 0; e < 16; e += 8)
                    if (col + e < p.d)
                        store8_any(to + e, make_uint4(pack2<T>(v[e], v[e + 1]), pack2<T>(v[e + 2], v[e + 3]), pack2<T>(v[e + 4], v[e + 5]), pack2<T>(v[e + 6], v[e + 7])),
                                   p.d - col - e);
                return true;
            };
            for (int t = t0; t < t1; ++t, ++n) {
                const int ds = n % C::DS;
                if (!wait.together(st_full(ds), (n / C::DS) & 1) || !wait.together(s_full, n & 1)) return false;
                tc_fence_after();
                const uint32_t stats = base + kStats + ds * C::STATS + part * kPart * 4;
                uint32_t s[kPart], g[kPart], pk[kPart / 2];
                tmem_ld32_async(lanes + C::S_COL + kPart * part, s);
                tmem_ld_wait(s);
#pragma unroll
                for (int k = 0; k < kPart; k += 4) {
                    const uint4 w = shared16(stats + k * 4);
                    const F2 x0 = fma2(F2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), c2, F2(__uint_as_float(w.x), __uint_as_float(w.y)));
                    const F2 x1 = fma2(F2(__uint_as_float(s[k + 2]), __uint_as_float(s[k + 3])), c2, F2(__uint_as_float(w.z), __uint_as_float(w.w)));
                    s[k] = __float_as_uint(ex2(x0.lo()));
                    s[k + 1] = __float_as_uint(ex2(x0.hi()));
                    s[k + 2] = __float_as_uint(ex2(x1.lo()));
                    s[k + 3] = __float_as_uint(ex2(x1.hi()));
                    pk[k / 2] = pack2<T>(__uint_as_float(s[k]), __uint_as_float(s[k + 1]));
                    pk[k / 2 + 1] = pack2<T>(__uint_as_float(s[k + 2]), __uint_as_float(s[k + 3]));
                }
                tmem_st16(lanes + C::S_COL + kPart * part, pk);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_ready);
                if (!wait.together(dp_full, n & 1)) return false;
                tc_fence_after();
                tmem_ld32_async(lanes + C::DP_COL + kPart * part, g);
                tmem_ld_wait(g);
#pragma unroll
                for (int k = 0; k < kPart; k += 4) {
                    const uint4 w = shared16(stats + kTileQueries * 4 + k * 4);
                    F2 x0 = F2(__uint_as_float(g[k]), __uint_as_float(g[k + 1])) + F2(__uint_as_float(w.x), __uint_as_float(w.y));
                    F2 x1 = F2(__uint_as_float(g[k + 2]), __uint_as_float(g[k + 3])) + F2(__uint_as_float(w.z), __uint_as_float(w.w));
                    x0 = x0 * F2(__uint_as_float(s[k]), __uint_as_float(s[k + 1]));
                    x1 = x1 * F2(__uint_as_float(s[k + 2]), __uint_as_float(s[k + 3]));
                    if constexpr (kHalf) {
                        x0 = x0 * up;
                        x1 = x1 * up;
                    }
                    pk[k / 2] = pack2<T>(x0.lo(), x0.hi());
                    pk[k / 2 + 1] = pack2<T>(x1.lo(), x1.hi());
                }
                if constexpr (kAll) {
                    if (!there || masked) {
#pragma unroll
                        for (int k = 0; k < kPart / 2; ++k) pk[k] = 0;
                    }
                    // row: key; 16-byte piece c of it at c ^ (key & 7), as the descriptor's swizzle has it
                    const uint32_t row = base + kDst + (n & 1) * C::DST + part / 2 * kTileBox + (quad * 32 + lane) * 128;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + ((part % 2 * 4 + c) ^ (lane & 7)) * 16), "r"(pk[4 * c]), "r"(pk[4 * c + 1]),
                                     "r"(pk[4 * c + 2]), "r"(pk[4 * c + 3])
                                     : "memory");
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                tmem_st16(lanes + C::DP_COL + kPart * part, pk);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(ds_ready);
                    mbar_arrive(st_empty(ds));
                }
                if (kAll && t > t0 && !read_dq(t - 1, n - 1)) return false;
            }
            if (kAll && !read_dq(t1 - 1, n - 1)) return false;
            if (!wait.together(sums_full, sums_phase)) return false;
            sums_phase ^= 1u;
            tc_fence_after();
            // the first eight warps have dV, the others dK
            const int half = part >> 1;
            const bool whole = t1 - t0 == p.cut.per_unit;
            const float down = half == 0 ? (kHalf ? exp2i(-15) : 1.0f) : p.scale * (kHalf ? exp2i(-exponent) : 1.0f);
            T *row = whole && there ? key_row<T>(p, u, half == 0 ? p.dv : p.dk, key) : nullptr;
            // a run's first unit may start inside, and its last one end inside
            float *shares = p.partial + (((static_cast<int64_t>(blockIdx.x) * 2 + (t0 == 0)) * 2 + half) * kTileKeys + quad * 32 + lane) * kD;
#pragma unroll 1
            for (int k = (part & 1) * 32; k < p.d; k += 64) {
                uint32_t o[32];
                tmem_ld32_async(lanes + (half == 0 ? C::DV_COL : C::DK_COL) + k, o);
                tmem_ld_wait(o);
                float v[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = masked ? 0.0f : __uint_as_float(o[e]) * down;
                // (each lane its own row: these are few bytes beside the queries')
                if (!whole) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4 *>(shares + k + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                } else if (there) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        if (k + e < p.d)
                            store8_any(row + k + e, make_uint4(pack2<T>(v[e], v[e + 1]), pack2<T>(v[e + 2], v[e + 3]), pack2<T>(v[e + 4], v[e + 5]), pack2<T>(v[e + 6], v[e + 7])),
                                       p.d - k - e);
                }
            }
            tc_fence_before();  // the sums are read before the next unit's first P is announced
            return true;
        });
        if (!ok) wait.fail();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_free<1>(tmem, 512u);
}

// Units that a cut goes through: the blocks of column r add up the one in which run r's end is the first cut (or unit r), four
// elements of dV or dK a thread.
template <typename T, int kD, int kRounds>
__global__ void __launch_bounds__(256) attention_grad_join_kernel(const __grid_constant__ Params p)
{
    after_previous();
    let_next_start();
    // (a column a unit, where there are fewer of them than cuts)
    const bool by_cut = p.cut.units >= p.cut.runs;
    const int64_t cut_at = by_cut ? p.cut.start(blockIdx.x + 1) : 0, n = by_cut ? cut_at / p.cut.per_unit : blockIdx.x, begin = n * p.cut.per_unit;
    if (by_cut && cut_at == begin) return;           // between units
    const int64_t r0 = p.cut.run_of(begin), r1 = p.cut.run_of(begin + p.cut.per_unit - 1);
    if (by_cut ? r0 != blockIdx.x : r0 == r1) return;  // an earlier column's; not cut
    const Unit u = unit_at(p, n);
    const int count = static_cast<int>(r1 - r0);
    // the unit starts in run r0, as its last unit or its only one, and before all others, whose first one it is
    const float *first = p.partial + (r0 * 2 + 1) * 2 * kTileKeys * kD, *other = p.partial + (r0 + 1) * 4 * kTileKeys * kD;
    int at[kRounds], key[kRounds];
    bool here[kRounds];
    float4 sum[kRounds];
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        at[i] = ((blockIdx.y * kRounds + i) * 256 + threadIdx.x) * 4;
        key[i] = u.tile * kTileKeys + at[i] / kD % kTileKeys;
        here[i] = key[i] < u.keys && at[i] % kD < p.d;
        if (here[i]) sum[i] = __ldcg(reinterpret_cast<const float4 *>(first + at[i]));
    }
    constexpr int kBatch = 8 / kRounds;  // of the others at a time, all rounds together: 8 loads in flight
    for (int r = 0; r < count; r += kBatch) {
        float4 w[kBatch][kRounds];
#pragma unroll
        for (int e = 0; e < kBatch; ++e)
#pragma unroll
            for (int i = 0; i < kRounds; ++i)
                if (r + e < count && here[i]) w[e][i] = __ldcg(reinterpret_cast<const float4 *>(other + static_cast<int64_t>(r + e) * 4 * kTileKeys * kD + at[i]));
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            if (r + e >= count) break;
#pragma unroll
            for (int i = 0; i < kRounds; ++i) {
                sum[i].x += w[e][i].x;
                sum[i].y += w[e][i].y;
                sum[i].z += w[e][i].z;
                sum[i].w += w[e][i].w;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        if (!here[i]) continue;
        if (key_masked(p, u, key[i])) sum[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const int col = at[i] % kD;
        T *to = key_row<T>(p, u, at[i] / (kTileKeys * kD) == 0 ? p.dv : p.dk, key[i]) + col;
        if (p.wide) {
            *reinterpret_cast<uint2 *>(to) = make_uint2(pack2<T>(sum[i].x, sum[i].y), pack2<T>(sum[i].z, sum[i].w));
        } else {
            const float v[4] = {sum[i].x, sum[i].y, sum[i].z, sum[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < p.d) to[e] = from_f32<T>(v[e]);
        }
    }
}

Cut cut_of(int64_t batch, int64_t q_tokens, int64_t kv_tokens, int64_t q_heads, int64_t kv_heads)
{
    Cut c{};
    c.units = batch * kv_heads * ((kv_tokens + kTileKeys - 1) / kTileKeys);
    c.per_unit = q_heads / kv_heads * ((q_tokens + kTileQueries - 1) / kTileQueries);
    c.work = c.units * c.per_unit;
    c.runs = static_cast<int32_t>(c.work < kSms ? c.work : kSms);
    return c;
}

template <typename T, int kD, bool kAll>
struct grad_kv_tag;

template <typename T, int kD, bool kAll>
cudaError_t launch_form(const AttentionGradArgs &a, cudaStream_t stream)
{
    using C = Cfg<kD, kAll>;
    Params p{};
    p.cut = cut_of(a.batch, a.q.tokens, a.kv_tokens, a.q.heads, a.k.heads);
    if (p.cut.work == 0) return cudaSuccess;
    if (!heads_map<T>(&p.q, a.q, a.batch, a.d, kTileQueries) || !heads_map<T>(&p.dout, a.dout, a.batch, a.d, kTileQueries) ||
        !heads_map<T>(&p.k, a.k, a.batch, a.d, kTileKeys) || !heads_map<T>(&p.v, a.v, a.batch, a.d, kTileKeys))
        return cudaErrorInvalidValue;
    if (p.cut.per_unit > INT32_MAX || p.cut.work > INT64_MAX / 1024) return cudaErrorInvalidValue;
    p.counts = a.counts;
    p.index = a.index;
    p.index_rows = a.index_rows;
    p.mask = a.mask;
    p.mask_stride = a.mask_stride;
    p.base2 = a.base2;
    p.delta = a.delta;
    p.amax = a.amax;
    p.stat_rows = stat_rows(a.q.tokens);
    p.amax_blocks = a.q.heads / a.k.heads * stat_blocks(a.q.tokens, a.q.heads / a.k.heads);
    p.partial = a.partial;
    p.dk = a.dk;
    p.dv = a.dv;
    p.dq = a.dq;
    p.dev_status = a.dev_status;
    p.q_tokens = static_cast<int32_t>(a.q.tokens);
    p.kv_tokens = static_cast<int32_t>(a.kv_tokens);
    p.kv_heads = static_cast<int32_t>(a.k.heads);
    p.q_heads = static_cast<int32_t>(a.q.heads);
    p.group = p.q_heads / p.kv_heads;
    p.q_tiles = static_cast<int32_t>((a.q.tokens + kTileQueries - 1) / kTileQueries);
    p.key_tiles = static_cast<int32_t>((a.kv_tokens + kTileKeys - 1) / kTileKeys);
    p.d = a.d;
    p.wide = aligned_to(a.dk, 8) && aligned_to(a.dv, 8) && a.d % 4 == 0;  // four elements of the second kernel
    p.scale = a.scale;
    p.scale_log2 = a.scale * kLog2e;
    auto kernel = attention_grad_kv_kernel<T, kD, kAll>;
    cudaError_t e = allow_shared<grad_kv_tag<T, kD, kAll>>(kernel);
    if (e == cudaSuccess) e = launch_after(kernel, dim3(static_cast<unsigned>(p.cut.runs)), kThreads, C::SMEM, stream, 1, p);
    if (e != cudaSuccess || p.cut.runs == 1) return e;
    // Four rounds a block, since what it computes of the cuts costs more than a round (40 heads of 128, 4 tiles of keys: 16 us
    // one after the other, 11 together); one where few units are cut, each many times (4 units in 152 runs, heads of 80: 17 us
    // with four and a column a cut, 7 so).
    const unsigned columns = static_cast<unsigned>(p.cut.units < p.cut.runs ? p.cut.units : p.cut.runs - 1), rounds = 2 * kTileKeys * kD / 1024;
    if (columns >= kSms / 2)
        return launch_after(attention_grad_join_kernel<T, kD, 4>, dim3(columns, rounds / 4), 256, 0, stream, 1, p);
    return launch_after(attention_grad_join_kernel<T, kD, 1>, dim3(columns, rounds), 256, 0, stream, 1, p);
}

template <typename T, int kD>
cudaError_t launch(const AttentionGradArgs &a, cudaStream_t stream)
{
    if constexpr (kD == 64)
        if (grad_kv_makes_dq(a.kv_tokens, a.d)) return launch_form<T, kD, true>(a, stream);
    return launch_form<T, kD, false>(a, stream);
}

}  // namespace

// (2 x 4096 queries, 77 keys, 10 heads of 64: the other kernel took 15 us for it, 26 with a mask)
bool grad_kv_makes_dq(int64_t kv_tokens, int d) { return kv_tokens <= kTileKeys && d <= 64; }

int64_t grad_kv_partial_bytes(int64_t batch, int64_t q_tokens, int64_t kv_tokens, int64_t q_heads, int64_t kv_heads, int d)
{
    const Cut c = cut_of(batch, q_tokens, kv_tokens, q_heads, kv_heads);
    return int64_t{c.runs} * 2 * 2 * kTileKeys * (d <= 64 ? 64 : 128) * 4;
}

cudaError_t launch_attention_grad_kv(const AttentionGradArgs &a, cudaStream_t stream)
{
    if (a.dtype == CONVROT_BF16) return a.d <= 64 ? launch<__nv_bfloat16, 64>(a, stream) : launch<__nv_bfloat16, 128>(a, stream);
    return a.d <= 64 ? launch<__half, 64>(a, stream) : launch<__half, 128>(a, stream);
}

int attention_grad_kv_shared(int form, int *columns)
{
    *columns = 512;
    return form == 0 ? Cfg<64, false>::SMEM : form == 1 ? Cfg<128, false>::SMEM : form == 2 ? Cfg<64, true>::SMEM : 0;
}

}  // namespace convrot
