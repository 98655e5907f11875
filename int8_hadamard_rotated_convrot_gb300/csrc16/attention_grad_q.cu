// The queries' gradient of attention (include/convrot_block.h), on the
// 5th-generation tensor cores:
//
//   dq_i = scale sum_j dS_ij k_j,  dS = P (dP + delta),  P = 2^(c s + base2),  dP = dout V^T
//
// A CTA takes 128 queries of a head and goes over the keys in tiles of 128;
// it is persistent over such items. No sums of a softmax are needed any more,
// so a tile's dS depends on nothing before it.
//   warp 0       TMA producer: the item's queries and dout, then tiles of keys
//                and values in turn, through one ring; where one tile holds
//                all keys and a head has several items (kStay), the keys and
//                values stay, and the ring is the queries' and dout's (each
//                CTA has a run of items, so that it meets few heads)
//   warp 1       tensor memory; one thread issues the MMAs
//   warps 4-19   dS: four threads a row, 32 of the tile's keys each
// Tensor memory: two tiles of S = Q K^T in turn, so that the next one is
// multiplied while dS is made, dP, whose columns then hold dS (16 bits, the A
// operand of dS K), and the sums dQ. The tile of keys is read K-major for S
// and MN-major for dQ from the same bytes.
//
// Few items and long keys: shares of the keys as in the forward pass, added up in
// order by a second kernel (64 queries, 8 heads of 128, 77000 keys: the gradient
// took 937 us, 290 so).
//
// 8190 queries, 512 keys, 40 heads of 128: 116 us, 47 % of it products; each tile's dS
// stands between its dP and its dQ. The last tile of an item has code of its own,
// since conditions for it in the loop cost the issuing warp 5 % of the time of all.
#include "attention.cuh"

namespace convrot {
namespace {

using namespace mma16;

constexpr int kMathWarps = 16, kThreads = 128 + 32 * kMathWarps;
// Registers a thread: launched at 96, warpgroup 0 leaves some of its own to the others.
constexpr int kRegsWg0 = 64, kRegsMath = 104;
static_assert(4 * 32 * kRegsWg0 + 32 * kMathWarps * kRegsMath <= kThreads * 96, "register split");
constexpr int kPart = 32;  // columns of a tile that a thread has

template <int kD>
struct Cfg {
    static constexpr int HALVES = kD / 64, TILE = HALVES * kTileBox;
    static constexpr int STAGES = kD == 64 ? 10 : 5;
    static constexpr int BARS = 3 * STAGES + 10;
    static constexpr int BAR_BYTES = 384;
    static constexpr int SMEM = 1024 + (2 + STAGES) * TILE + BAR_BYTES;
    static constexpr uint32_t S_COL = 0, DP_COL = 256, DQ_COL = 384;  // S: + 128 for every other tile
    static_assert(SMEM > kTmemAlone && SMEM <= kMaxShared, "no other tensor memory on this SM");
    static_assert(8 * BARS + 8 <= BAR_BYTES, "barriers fit");
};

struct Params {
    HeadsMap q, dout, k, v;
    const int32_t *counts;
    const uint8_t *mask;
    int64_t mask_stride;
    const float *base2, *delta, *amax;
    int64_t amax_blocks;
    void *dq;
    int32_t *dev_status;
    int32_t q_tokens, stat_rows, kv_tokens, q_heads, group;
    int32_t q_tiles, items;
    int32_t d, wide;
    float scale, scale_log2;
    int32_t splits;
    float *partial;  // [splits][rows of dq][pitch]: what a share of the keys gives, where there are several
    int64_t rows;
    int32_t pitch;
};

template <typename T, int kD, KeyForm kForm>
__global__ void __launch_bounds__(kThreads, 1) attention_grad_q_kernel(const __grid_constant__ Params p)
{
    constexpr bool kStay = kForm == kStays, kShares = kForm == kShared;
    using C = Cfg<kD>;
    constexpr bool kHalf = std::is_same_v<T, __half>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw));
    const uint32_t base = (raw + 1023u) & ~1023u;  // swizzle atoms are 1024-byte aligned
    uint8_t *gbase = smem_raw + (base - raw);
    constexpr int kRing = 2 * C::TILE, kBars = kRing + C::STAGES * C::TILE;
    const uint32_t bars = base + kBars;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (C::STAGES + s); };
    auto s_full = [&](int i) { return bars + 8u * (2 * C::STAGES + i); };
    // What is not in the ring, at `base`: an item's queries and, with barriers of their own, dout; or with kStay a head's keys and
    // values.
    const uint32_t q_full = bars + 8u * (2 * C::STAGES + 2), q_empty = q_full + 8, dp_full = q_full + 16, ds_ready = q_full + 24;
    const uint32_t dq_full = q_full + 32, done_bar = q_full + 40, dout_full = q_full + 48, dout_empty = q_full + 56;
    auto clean_bar = [&](int s) { return q_full + 64 + 8u * s; };  // a masked tile of keys, the i-th, has its zeros: i % STAGES
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + kBars + 8 * C::BARS);
    const Waits wait{reinterpret_cast<volatile int *>(tmem_slot + 1), p.dev_status};
    const int warp = warp_number(), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
            mbar_init(clean_bar(s), 2);
        }
        mbar_init(s_full(0), 1);
        mbar_init(s_full(1), 1);
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(dp_full, 1);
        mbar_init(ds_ready, kMathWarps);
        mbar_init(dq_full, 1);
        mbar_init(done_bar, 1);
        mbar_init(dout_full, 1);
        mbar_init(dout_empty, 1);
        *wait.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&p.q.map);
        prefetch_map(&p.dout.map);
        if (p.kv_tokens > 0) prefetch_map(&p.k.map);
        if (p.kv_tokens > 0) prefetch_map(&p.v.map);
    }
    if (warp == 1) tmem_alloc<1>(tmem_slot, 512u);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    after_previous();
    let_next_start();

    struct Item {
        int b, h, q0, keys, tiles;
        int head;  // of the keys
        int first_tile, share;
    };
    const int first = kStay ? static_cast<int>(static_cast<int64_t>(p.items) * blockIdx.x / gridDim.x) : blockIdx.x;
    const int end = kStay ? static_cast<int>(static_cast<int64_t>(p.items) * (blockIdx.x + 1) / gridDim.x) : p.items;
    const int step = kStay ? 1 : gridDim.x;
    auto item_at = [&](int i) {
        Item it;
        it.share = kShares ? i % p.splits : 0;
        if (kShares) i /= p.splits;
        const int bh = i / p.q_tiles;
        it.q0 = (i - bh * p.q_tiles) * kTileQueries;
        it.b = bh / p.q_heads;
        it.h = bh - it.b * p.q_heads;
        it.head = bh / p.group;
        it.keys = p.counts ? static_cast<int>(load_i32(p.counts + it.b)) : p.kv_tokens;
        it.tiles = (it.keys + kTileKeys - 1) / kTileKeys;
        it.first_tile = 0;
        if (kShares) {
            it.first_tile = static_cast<int>(static_cast<int64_t>(it.tiles) * it.share / p.splits);
            it.tiles = static_cast<int>(static_cast<int64_t>(it.tiles) * (it.share + 1) / p.splits) - it.first_tile;
        }
        return it;
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsWg0));
        if (warp == 0 && lane == 0) {
            int stage = 0, head = -1;
            uint32_t phase = 0, q_phase = 0, dout_phase = 0, armed = 0;
            bool ok = true;
            auto load = [&](const HeadsMap &m, int token, int head, int b) {
                if (!ok || !wait(empty_bar(stage), phase ^ 1u)) return void(ok = false);
                mbar_arrive_expect_tx(full_bar(stage), C::TILE);
                load_tile<C::HALVES>(base + kRing + stage * C::TILE, m, token, head, b, full_bar(stage));
                armed |= 1u << stage;
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            };
            for (int i = first; i < end && ok; i += step) {
                const Item it = item_at(i);
                if (it.tiles == 0) continue;
                if constexpr (kStay) {
                    if (it.head != head) {
                        head = it.head;
                        if (!(ok = wait(q_empty, q_phase ^ 1u))) break;
                        q_phase ^= 1u;
                        mbar_arrive_expect_tx(q_full, 2 * C::TILE);
                        load_tile<C::HALVES>(base, p.k, 0, it.h / p.group, it.b, q_full);
                        load_tile<C::HALVES>(base + C::TILE, p.v, 0, it.h / p.group, it.b, q_full);
                        armed |= 1u << 16;
                    }
                    load(p.q, it.q0, it.h, it.b);
                    load(p.dout, it.q0, it.h, it.b);
                } else {
                    load(p.k, it.first_tile * kTileKeys, it.h / p.group, it.b);
                    if (!ok || !(ok = wait(q_empty, q_phase ^ 1u))) break;
                    mbar_arrive_expect_tx(q_full, C::TILE);
                    load_tile<C::HALVES>(base, p.q, it.q0, it.h, it.b, q_full);
                    armed |= 1u << 16;
                    q_phase ^= 1u;
                    load(p.v, it.first_tile * kTileKeys, it.h / p.group, it.b);
                    if (!ok || !(ok = wait(dout_empty, dout_phase ^ 1u))) break;
                    mbar_arrive_expect_tx(dout_full, C::TILE);
                    load_tile<C::HALVES>(base + C::TILE, p.dout, it.q0, it.h, it.b, dout_full);
                    armed |= 1u << 17;
                    dout_phase ^= 1u;
                    for (int j = 1; j < it.tiles && ok; ++j) {
                        load(p.k, (it.first_tile + j) * kTileKeys, it.h / p.group, it.b);
                        load(p.v, (it.first_tile + j) * kTileKeys, it.h / p.group, it.b);
                    }
                }
            }
            if (!ok) {
                wait.fail();
                for (int s = 0; s < C::STAGES; ++s)  // copies in flight land before shared memory goes away
                    if (armed >> s & 1u) mbar_wait(full_bar(s), s < stage ? phase : phase ^ 1u);
                if (armed >> 16 & 1u) mbar_wait(q_full, q_phase ^ 1u);
                if (armed >> 17 & 1u) mbar_wait(dout_full, dout_phase ^ 1u);
            }
        } else if (warp == 1) {
            const uint32_t id_s = idesc<T>(128, 128, false, false);
            const int n_o = (p.d + 15) / 16 * 16, steps = (p.d + kMmaK - 1) / kMmaK;
            const uint32_t id_o = idesc<T>(128, n_o, false, true);
            int stage = 0;
            uint32_t phase = 0, q_phase = 0, ds_phase = 0;
            int tile_no = 0;  // over all items: which of the two S
            bool ok = true;
            int cleaned = 0;  // masked tiles of keys (which are not always those of a stage)
            auto take = [&](int &at, bool clean = false) {  // the next stage of the ring, once it is there
                ok = clean ? wait.together(clean_bar(cleaned % C::STAGES), (cleaned / C::STAGES) & 1) : wait.together(full_bar(stage), phase);
                cleaned += clean;
                at = stage;
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
                return ok;
            };
            if constexpr (kStay) {
                // S of an item while dS of the one before is made, where they have the same keys
                int head = -1;
                auto s_of = [&](int at) {  // Q of an item by the keys
                    tc_fence_after();
                    if (one_thread()) {
                        tile_product<kD>(tmem + C::S_COL + 128 * (tile_no & 1), base + kRing + at * C::TILE, base, id_s, steps);
                        mma_commit(s_full(tile_no & 1));
                        mma_commit(empty_bar(at));
                    }
                    __syncwarp();
                    ++tile_no;
                };
                auto dp_of = [&](int at) {  // (one thread) dout of an item by the values
                    tile_product<kD>(tmem + C::DP_COL, base + kRing + at * C::TILE, base + C::TILE, id_s, steps);
                    mma_commit(dp_full);
                    mma_commit(empty_bar(at));
                };
                for (int i = first; i < end && ok; ++i) {
                    int at;
                    const int now = item_at(i).head;
                    if (now != head) {
                        head = now;
                        ok = wait.together(q_full, q_phase) && (!p.mask || wait.together(clean_bar(cleaned % C::STAGES), (cleaned / C::STAGES) & 1));
                        if (!ok) break;
                        q_phase ^= 1u;
                        ++cleaned;
                        if (!take(at)) break;
                        s_of(at);
                        if (!take(at)) break;
                        tc_fence_after();
                        if (one_thread()) dp_of(at);
                        __syncwarp();
                    }
                    const bool more = i + 1 < end && item_at(i + 1).head == head;
                    if (more) {
                        if (!take(at)) break;
                        s_of(at);
                        if (!take(at)) break;
                    }
                    if (!(ok = wait.together(ds_ready, ds_phase))) break;
                    ds_phase ^= 1u;
                    tc_fence_after();
                    if (one_thread()) {
                        tile_add<4>(tmem + C::DQ_COL, tmem + C::DP_COL, base, id_o, true);
                        mma_commit(dq_full);
                        if (more)
                            dp_of(at);
                        else
                            mma_commit(q_empty);
                    }
                    __syncwarp();
                }
            } else {
                uint32_t dout_phase = 0;
                auto s_of = [&](int at) {  // (one thread) the item's queries by a tile of keys
                    tile_product<kD>(tmem + C::S_COL + 128 * (tile_no & 1), base, base + kRing + at * C::TILE, id_s, steps);
                    mma_commit(s_full(tile_no & 1));
                };
                auto dp_of = [&](int at, bool last) {  // (one thread) its dout by the values; last: of the item
                    tile_product<kD>(tmem + C::DP_COL, base + C::TILE, base + kRing + at * C::TILE, id_s, steps);
                    mma_commit(dp_full);
                    mma_commit(empty_bar(at));
                    if (last) mma_commit(dout_empty);
                };
                int i = first - step;
                auto item_after = [&]() {  // the next item that has keys; without one, tiles is 0
                    Item it{};
                    for (i += step; i < end; i += step) {
                        it = item_at(i);
                        if (it.tiles > 0) break;
                    }
                    if (i >= end) it.tiles = 0;
                    return it;
                };
                Item it = item_after();
                int k_at = 0, v_at = 0;
                if (it.tiles > 0 && (ok = wait.together(q_full, q_phase)) && take(k_at, p.mask)) {
                    q_phase ^= 1u;
                    tc_fence_after();
                    if (one_thread()) {
                        s_of(k_at);
                        if (it.tiles == 1) mma_commit(q_empty);
                    }
                    __syncwarp();
                    ++tile_no;
                    if ((ok = wait.together(dout_full, dout_phase)) && take(v_at)) {
                        dout_phase ^= 1u;
                        tc_fence_after();
                        if (one_thread()) dp_of(v_at, it.tiles == 1);
                        __syncwarp();
                    }
                }
                while (ok && it.tiles > 0) {
                    const Item then = item_after();
                    for (int j = 0; j + 1 < it.tiles; ++j) {
                        const int left = it.tiles - j - 1;  // tiles of the item after this one
                        int k_next = 0;
                        if (!take(k_next)) break;
                        tc_fence_after();
                        if (one_thread()) {
                            s_of(k_next);
                            if (left == 1) mma_commit(q_empty);
                        }
                        __syncwarp();
                        ++tile_no;
                        // dQ of this tile and dP of the next, together where its values are there (their place in the ring became
                        // free with the last dQ)
                        bool both = wait.now(full_bar(stage), phase);
                        if (!(ok = wait.together(ds_ready, ds_phase))) break;
                        ds_phase ^= 1u;
                        if (!both) both = wait.now(full_bar(stage), phase);
                        tc_fence_after();
                        v_at = stage;
                        if (one_thread()) {
                            // (each quarter of the keys has its own quarter of dP's columns)
                            tile_add<4>(tmem + C::DQ_COL, tmem + C::DP_COL, base + kRing + k_at * C::TILE, id_o, j == 0);
                            if (both) dp_of(v_at, left == 1);
                            mma_commit(empty_bar(k_at));
                        }
                        __syncwarp();
                        if (!take(v_at)) break;
                        if (!both) {
                            tc_fence_after();
                            if (one_thread()) dp_of(v_at, left == 1);
                            __syncwarp();
                        }
                        k_at = k_next;
                    }
                    if (!ok) break;
                    // After the last tile, S and dP of the next item's first: its queries came since the last S, its dout since
                    // the last dP.
                    const bool more = then.tiles > 0;
                    int k_next = 0;
                    auto next_s = [&]() {
                        if (!(ok = wait.together(q_full, q_phase)) || !take(k_next, p.mask)) return false;
                        q_phase ^= 1u;
                        tc_fence_after();
                        if (one_thread()) {
                            s_of(k_next);
                            if (then.tiles == 1) mma_commit(q_empty);
                        }
                        __syncwarp();
                        ++tile_no;
                        return true;
                    };
                    const bool early = more && !p.mask && wait.now(q_full, q_phase) && wait.now(full_bar(stage), phase);
                    if (early && !next_s()) break;
                    if (!(ok = wait.together(ds_ready, ds_phase))) break;
                    ds_phase ^= 1u;
                    tc_fence_after();
                    if (one_thread()) {
                        tile_add<4>(tmem + C::DQ_COL, tmem + C::DP_COL, base + kRing + k_at * C::TILE, id_o, it.tiles == 1);
                        mma_commit(dq_full);
                        mma_commit(empty_bar(k_at));
                    }
                    __syncwarp();
                    if (more) {
                        if (!early && !next_s()) break;
                        if (!(ok = wait.together(dout_full, dout_phase)) || !take(v_at)) break;
                        dout_phase ^= 1u;
                        tc_fence_after();
                        if (one_thread()) dp_of(v_at, then.tiles == 1);
                        __syncwarp();
                    }
                    k_at = k_next;
                    it = then;
                }
            }
            if (!ok) wait.fail();
            if (one_thread()) {
                mma_commit(done_bar);
                mbar_wait(done_bar, 0);
            }
        } else if (kStay && warp >= 2 && p.mask) {
            bool ok = true;
            int head = -1, cleaned = 0;
            MaskedRows rows;
            for (int i = first; i < end && ok; ++i) {
                const Item it = item_at(i);
                if (it.head == head) continue;
                head = it.head;
                rows.of(p.mask, p.mask_stride, it.b, p.kv_tokens, warp - 2, lane);
                if (!(ok = wait.together(q_full, cleaned & 1))) break;
                clean_rows<C::HALVES>(base, rows.there, warp - 2, lane);
                if (lane == 0) mbar_arrive(clean_bar(cleaned % C::STAGES));
                ++cleaned;
            }
            if (!ok) wait.fail();
        } else if (!kStay && warp >= 2 && p.mask) {  // (one tile an item: keys, then values)
            bool ok = true;
            int entry = 0, cleaned = 0;
            MaskedRows rows;
            for (int i = first; i < end && ok; i += step, entry += 2, ++cleaned) {
                const int s = entry % C::STAGES;
                rows.of(p.mask, p.mask_stride, item_at(i).b, p.kv_tokens, warp - 2, lane);
                if (!(ok = wait.together(full_bar(s), (entry / C::STAGES) & 1))) break;
                clean_rows<C::HALVES>(base + kRing + s * C::TILE, rows.there, warp - 2, lane);
                if (lane == 0) mbar_arrive(clean_bar(cleaned % C::STAGES));
            }
            if (!ok) wait.fail();
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMath));
        const int part = (warp - 4) >> 2, quad = warp & 3;  // of the tile's keys; of the rows
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        const F2 c2(p.scale_log2);
        uint32_t dp_phase = 0, dq_phase = 0;
        uint32_t there = 0;  // a mask's keys of this thread
        int masked = -1;     // its sample
        int tile_no = 0;
        bool ok = true;
        for (int i = first; i < end && ok; i += step) {
            const Item it = item_at(i);
            const int row0 = it.q0 + quad * 32, rows = p.q_tokens - row0 < 32 ? p.q_tokens - row0 : 32;
            const int64_t at = (static_cast<int64_t>(it.b) * p.q_heads + it.h) * p.stat_rows + row0 + lane;
            const float base2 = load_f32(p.base2 + at), delta = load_f32(p.delta + at);
            int exponent = 0;
            if constexpr (kHalf) {
                const int64_t head = static_cast<int64_t>(it.b) * (p.q_heads / p.group) + it.h / p.group;
                exponent = grad_exponent(p.amax + head * p.amax_blocks, p.amax_blocks, lane);
            }
            // what dS is multiplied by: P is 2^15 times as large
            const F2 up(kHalf ? exp2i(exponent) * exp2i(-15) : 1.0f), off2(base2), delta2(delta);
            if (p.mask && it.b != masked) {
                masked = it.b;
                there = keys_there(p.mask + it.b * p.mask_stride, part * kPart + lane, p.kv_tokens);
            }
            for (int j = 0; j < it.tiles; ++j, ++tile_no) {
                const int b = tile_no & 1;
                if (!wait.together(s_full(b), (tile_no >> 1) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t s[kPart], g[kPart];
                tmem_ld32_async(lanes + C::S_COL + 128 * b + kPart * part, s);
                tmem_ld_wait(s);
                const int keys = it.keys - (it.first_tile + j) * kTileKeys - part * kPart;
#pragma unroll
                for (int k = 0; k < kPart; k += 2) {
                    const F2 x = fma2(F2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), c2, off2);
                    s[k] = __float_as_uint(ex2(x.lo()));
                    s[k + 1] = __float_as_uint(ex2(x.hi()));
                }
                if (keys < kPart) {
#pragma unroll
                    for (int k = 0; k < kPart; ++k)
                        if (k >= keys) s[k] = 0u;
                }
                if (!wait.together(dp_full, dp_phase)) {
                    ok = false;
                    break;
                }
                dp_phase ^= 1u;
                tc_fence_after();
                tmem_ld32_async(lanes + C::DP_COL + kPart * part, g);
                tmem_ld_wait(g);
                uint32_t pk[kPart / 2];
#pragma unroll
                for (int k = 0; k < kPart; k += 2) {
                    F2 x = F2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])) * (F2(__uint_as_float(g[k]), __uint_as_float(g[k + 1])) + delta2);
                    if constexpr (kHalf) x = x * up;
                    pk[k / 2] = pack2<T>(x.lo(), x.hi());
                }
                if (p.mask) {  // (a masked value may have made dP NaN)
#pragma unroll
                    for (int k = 0; k < kPart; k += 2) pk[k / 2] &= (there & 1u << k ? 0xffffu : 0u) | (there & 2u << k ? 0xffff0000u : 0u);
                }
                tmem_st16(lanes + C::DP_COL + kPart * part, pk);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ds_ready);
            }
            if (!ok) break;
            if (it.tiles > 0) {
                if (!wait.together(dq_full, dq_phase)) {
                    ok = false;
                    break;
                }
                dq_phase ^= 1u;
                tc_fence_after();
            }
            const float down = kHalf ? p.scale * exp2i(-exponent) : p.scale;
            T *dq = static_cast<T *>(p.dq) + ((static_cast<int64_t>(it.b) * p.q_tokens + row0) * p.q_heads + it.h) * p.d;
#pragma unroll 1
            for (int k = part * 32; k < p.d; k += 128) {
                uint32_t o[32];
                float v[32];
                if (it.tiles > 0) {
                    tmem_ld32_async(lanes + C::DQ_COL + k, o);
                    tmem_ld_wait(o);
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = it.tiles > 0 ? __uint_as_float(o[e]) * down : 0.0f;
                if (kShares) {
                    const int64_t row = it.share * p.rows + (static_cast<int64_t>(it.b) * p.q_tokens + row0 + lane) * p.q_heads + it.h;
                    if (lane < rows) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            if (k + e < p.pitch) *reinterpret_cast<float4 *>(p.partial + row * p.pitch + k + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                    }
                    continue;
                }
                if (rows > 0)
                    store_rows_traded<T>(dq + k, static_cast<int64_t>(p.q_heads) * p.d, rows, p.d - k < 32 ? p.d - k : 32, p.wide, lane, v);
            }
            tc_fence_before();  // dQ is read before the next item's first dS is announced
        }
        if (!ok) wait.fail();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_free<1>(tmem, 512u);
}

// dq from the shares, in their order, four elements a thread.
template <typename T>
__global__ void __launch_bounds__(256) attention_grad_q_join_kernel(const float *partial, int splits, int64_t rows, int pitch, int d, T *dq)
{
    after_previous();
    let_next_start();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, row = i / (pitch / 4);
    const int e0 = static_cast<int>(i - row * (pitch / 4)) * 4;
    if (row >= rows) return;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(partial + (s * rows + row) * pitch + e0));
        sum.x += v.x;
        sum.y += v.y;
        sum.z += v.z;
        sum.w += v.w;
    }
    const float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e0 + e < d) dq[row * d + e0 + e] = from_f32<T>(v[e]);
}

int32_t splits_of(int64_t batch, int64_t q_tokens, int64_t kv_tokens, int64_t q_heads)
{
    return key_shares(batch * q_heads * ((q_tokens + kTileQueries - 1) / kTileQueries), kv_tokens);
}

template <typename T, int kD, KeyForm kForm>
struct grad_q_tag;

template <typename T, int kD, KeyForm kForm>
cudaError_t launch_form(const AttentionGradArgs &a, cudaStream_t stream)
{
    using C = Cfg<kD>;
    Params p{};
    if (!heads_map<T>(&p.q, a.q, a.batch, a.d, kTileQueries) || !heads_map<T>(&p.dout, a.dout, a.batch, a.d, kTileQueries))
        return cudaErrorInvalidValue;
    if (a.k.tokens > 0 && (!heads_map<T>(&p.k, a.k, a.batch, a.d, kTileKeys) || !heads_map<T>(&p.v, a.v, a.batch, a.d, kTileKeys)))
        return cudaErrorInvalidValue;
    p.counts = a.counts;
    p.mask = a.mask;
    p.mask_stride = a.mask_stride;
    p.base2 = a.base2;
    p.delta = a.delta;
    p.amax = a.amax;
    p.stat_rows = static_cast<int32_t>(stat_rows(a.q.tokens));
    p.amax_blocks = a.q.heads / a.k.heads * stat_blocks(a.q.tokens, a.q.heads / a.k.heads);
    p.dq = a.dq;
    p.dev_status = a.dev_status;
    p.q_tokens = static_cast<int32_t>(a.q.tokens);
    p.kv_tokens = static_cast<int32_t>(a.kv_tokens);
    p.q_heads = static_cast<int32_t>(a.q.heads);
    p.group = static_cast<int32_t>(a.q.heads / a.k.heads);
    p.q_tiles = static_cast<int32_t>((a.q.tokens + kTileQueries - 1) / kTileQueries);
    p.splits = kForm == kShared ? splits_of(a.batch, a.q.tokens, a.kv_tokens, a.q.heads) : 1;
    p.partial = a.partial_q;
    p.rows = a.batch * a.q.tokens * a.q.heads;
    p.pitch = (a.d + 3) / 4 * 4;
    const int64_t items = a.batch * a.q.heads * p.q_tiles * p.splits;
    if (items > INT32_MAX) return cudaErrorInvalidValue;
    p.items = static_cast<int32_t>(items);
    p.d = a.d;
    p.wide = aligned_to(a.dq, 16) && a.d % 8 == 0;
    p.scale = a.scale;
    p.scale_log2 = a.scale * kLog2e;
    auto kernel = attention_grad_q_kernel<T, kD, kForm>;
    cudaError_t e = allow_shared<grad_q_tag<T, kD, kForm>>(kernel);
    if (e != cudaSuccess) return e;
    e = launch_after(kernel, dim3(static_cast<unsigned>(items < kSms ? items : kSms)), kThreads, C::SMEM, stream, 1, p);
    if (e != cudaSuccess || p.splits == 1) return e;
    const int64_t blocks = (p.rows * (p.pitch / 4) + 255) / 256;
    return launch_after(attention_grad_q_join_kernel<T>, dim3(static_cast<unsigned>(blocks)), 256, 0, stream, 1, a.partial_q, p.splits, p.rows, p.pitch, p.d,
                        static_cast<T *>(a.dq));
}

// Keys that stay: as in the forward pass (4 x 1270 queries, 20 keys, 43 heads of 80 on one: 64 us with an item's queries,
// dout, keys and values read after the item before, 34 so). Heads of up to 64 with a tile of keys never come here (grad_kv_makes_dq).
template <typename T, int kD>
cudaError_t launch(const AttentionGradArgs &a, cudaStream_t stream)
{
    if constexpr (kD > 64) {
        const int64_t of_head = a.q.heads / a.k.heads * ((a.q.tokens + kTileQueries - 1) / kTileQueries);
        if (!a.counts && a.kv_tokens > 0 && a.kv_tokens <= kTileKeys && of_head >= 4) return launch_form<T, kD, kStays>(a, stream);
    }
    return splits_of(a.batch, a.q.tokens, a.kv_tokens, a.q.heads) > 1 ? launch_form<T, kD, kShared>(a, stream) : launch_form<T, kD, kPass>(a, stream);
}

}  // namespace

cudaError_t launch_attention_grad_q(const AttentionGradArgs &a, cudaStream_t stream)
{
    if (a.dtype == CONVROT_BF16) return a.d <= 64 ? launch<__nv_bfloat16, 64>(a, stream) : launch<__nv_bfloat16, 128>(a, stream);
    return a.d <= 64 ? launch<__half, 64>(a, stream) : launch<__half, 128>(a, stream);
}

int64_t grad_q_partial_bytes(int64_t batch, int64_t q_tokens, int64_t kv_tokens, int64_t q_heads, int d)
{
    const int32_t splits = splits_of(batch, q_tokens, kv_tokens, q_heads);
    return splits > 1 ? splits * batch * q_tokens * q_heads * ((d + 3) / 4 * 4) * 4 : 0;
}

int attention_grad_q_shared(int form, int *columns)
{
    *columns = 512;
    return form == 0 ? Cfg<64>::SMEM : form == 1 ? Cfg<128>::SMEM : 0;
}

}  // namespace convrot
