// Attention to other states on the 5th-generation tensor cores
// (include/convrot_block.h): one pass over the keys with the running maximum and
// sum of each row's softmax.
//
// A CTA takes 256 queries of a head, two groups of 128 that take turns: while
// the tensor cores multiply for one, the other's softmax runs. It is persistent
// over such items.
//   warp 0       TMA producer: the groups' queries, then the tiles of 128 keys
//                and values in turn, through one ring; where one tile holds
//                all keys and a head has several items (kStay), the keys and
//                values stay, and the ring is the queries' (each CTA has a
//                run of items, so that it meets few heads)
//   warp 1       tensor memory; one thread issues the MMAs
//   warps 4-11   the first group's softmax, warps 12-19 the second's: two threads a
//                row, 64 of the tile's keys each
// Tensor memory: for each group 128 columns of S = Q K^T, whose halves' first
// halves then hold P (16 bits, the A operand of P V, so that P never passes
// through shared memory), and the sums O.
//
// The maximum is a reference only: O and the sum are rescaled when a row's
// maximum has grown by more than 2^8 since, which is rare after the first tile
// (probabilities may be up to 2^8 meanwhile, the sums are fp32). float16 has few
// exponents below 1, so there P is 2^7 times as large, which the division by the
// sum takes back.
//
// Where the items are fewer than half the SMs and the keys long, the keys are
// shared out: an item is some queries and a share of their keys, its outputs stay
// fp32, and a second kernel weighs the shares by their lse (key_shares; 64 queries,
// 8 heads of 128, 77000 keys: 811 us whole, 62 so).
//
// 32760 queries, heads of 128: 1515 TFLOP/s at 4096 keys and 10 heads (453 us), 1145 to
// 1215 at 512 keys and 40 heads (283 to 300 us in different runs), where an item is four
// tiles. The products with
// their copies and waits, without a softmax, take 415 and 245 us of these, so the
// softmax is nearly hidden: half of the exponentials, the maxima and the exchange
// between a row's threads are 3 % together. Two CTAs that share each tile of keys
// (products of 256 x 128) were slower, 665 us: every turn waits for both. Issuing
// S of the next item before this one's outputs, or fetching its queries to L2
// ahead, changed nothing.
#include "attention.cuh"

namespace convrot {
namespace {

using namespace mma16;

constexpr int kGroupRows = 128, kItemRows = 2 * kGroupRows;
constexpr int kSoftmaxWarps = 16, kThreads = 128 + 32 * kSoftmaxWarps;
// Registers a thread: launched at 96, warpgroup 0 leaves some of its own to the softmax:
// 4 x 32 x 64 + 16 x 32 x 104 = 640 x 96.
constexpr int kRegsWg0 = 64, kRegsSoftmax = 104;
static_assert(4 * 32 * kRegsWg0 + 32 * kSoftmaxWarps * kRegsSoftmax <= kThreads * 96, "register split");
constexpr int kHalfKeys = kTileKeys / 2;
constexpr float kGrow = 8.0f;  // log2 of what a row's probabilities may grow to before O is rescaled

template <int kD>
struct Cfg {
    static constexpr int HALVES = kD / 64, TILE = HALVES * kTileBox;
    static constexpr int STAGES = kD == 64 ? 9 : 4;
    static constexpr int BARS = 3 * STAGES + 2 * 5 + 1;
    static constexpr int BAR_BYTES = 384;
    static constexpr int MEET = 2 * 2 * 4 * 2 * 32 * 4;  // maxima of the two threads of a row: in turn, group, quadrant, half
    static constexpr int SMEM = 1024 + (2 + STAGES) * TILE + MEET + BAR_BYTES;
    static constexpr uint32_t S_COL = 0, O_COL = 256;  // + 128 g and + kD g
    static_assert(SMEM > kTmemAlone && SMEM <= kMaxShared, "no other tensor memory on this SM");
    static_assert(8 * BARS + 8 <= BAR_BYTES, "barriers fit");
};

struct Params {
    HeadsMap q, k, v;
    const int32_t *counts;
    const uint8_t *mask;
    int64_t mask_stride;
    void *out;
    int64_t out_strides[3];
    float *lse;
    int32_t *dev_status;
    int32_t q_tokens, kv_tokens, q_heads, group;  // query heads that share a head
    int32_t q_tiles, items;
    int32_t d, wide;
    float scale_log2;
    int32_t splits;
    float *partial;  // [splits][rows of all heads][pitch]: a share's outputs, and behind them [splits][rows] its lse
    int64_t rows;
    int32_t pitch;
};

template <typename T, int kD, KeyForm kForm>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(const __grid_constant__ Params p)
{
    constexpr bool kStay = kForm == kStays, kShares = kForm == kShared;
    using C = Cfg<kD>;
    constexpr float kShift = std::is_same_v<T, __half> ? 7.0f : 0.0f;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw));
    const uint32_t base = (raw + 1023u) & ~1023u;  // swizzle atoms are 1024-byte aligned
    uint8_t *gbase = smem_raw + (base - raw);
    constexpr int kRing = 2 * C::TILE, kMeet = kRing + C::STAGES * C::TILE, kBars = kMeet + C::MEET;
    const uint32_t bars = base + kBars;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (C::STAGES + s); };
    auto q_full = [&](int g) { return bars + 8u * (2 * C::STAGES + g); };
    auto q_empty = [&](int g) { return bars + 8u * (2 * C::STAGES + 2 + g); };
    auto s_full = [&](int g) { return bars + 8u * (2 * C::STAGES + 4 + g); };   // S is there (and P V of the tile before)
    auto p_ready = [&](int g) { return bars + 8u * (2 * C::STAGES + 6 + g); };  // P is there, and O rescaled
    auto o_full = [&](int g) { return bars + 8u * (2 * C::STAGES + 8 + g); };
    const uint32_t done_bar = bars + 8u * (2 * C::STAGES + 10);
    auto clean_bar = [&](int s) { return done_bar + 8u * (1 + s); };  // a masked tile of values, the i-th, has its zeros: i % STAGES
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + kBars + 8 * C::BARS);
    const Waits wait{reinterpret_cast<volatile int *>(tmem_slot + 1), p.dev_status};
    const int warp = warp_number(), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
            mbar_init(clean_bar(s), 2);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(q_full(g), 1);
            mbar_init(q_empty(g), 1);
            mbar_init(s_full(g), 1);
            mbar_init(p_ready(g), 8);
            mbar_init(o_full(g), 1);
        }
        mbar_init(done_bar, 1);
        *wait.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&p.q.map);
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

    // item -> (sample, head, first query); the tiles of one head follow each other and share its keys in L2
    struct Item {
        int b, h, q0, keys, tiles, groups;
        int first, share;  // tile; of the keys
    };
    auto item_at = [&](int i) {
        Item it;
        it.share = kShares ? i % p.splits : 0;
        if (kShares) i /= p.splits;
        const int bh = i / p.q_tiles;
        it.q0 = (i - bh * p.q_tiles) * kItemRows;
        it.b = bh / p.q_heads;
        it.h = bh - it.b * p.q_heads;
        it.keys = p.counts ? static_cast<int>(load_i32(p.counts + it.b)) : p.kv_tokens;
        it.tiles = (it.keys + kTileKeys - 1) / kTileKeys;
        it.first = 0;
        if (kShares) {
            it.first = static_cast<int>(static_cast<int64_t>(it.tiles) * it.share / p.splits);
            it.tiles = static_cast<int>(static_cast<int64_t>(it.tiles) * (it.share + 1) / p.splits) - it.first;
        }
        it.groups = p.q_tokens - it.q0 > kGroupRows ? 2 : 1;
        return it;
    };

    // this CTA's items: every so many, or, where the keys stay, a run of them
    const int begin = kStay ? static_cast<int>(static_cast<int64_t>(p.items) * blockIdx.x / gridDim.x) : static_cast<int>(blockIdx.x);
    const int end = kStay ? static_cast<int>(static_cast<int64_t>(p.items) * (blockIdx.x + 1) / gridDim.x) : p.items;
    const int step = kStay ? 1 : static_cast<int>(gridDim.x);
    // kStay: whether item i's keys are others than those of the item before
    auto other_keys = [&](const Item &it, const Item &before) { return it.b != before.b || it.h / p.group != before.h / p.group; };
    const uint32_t kv_full = q_full(0), kv_empty = q_empty(0);  // kStay

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsWg0));
        if (kStay && warp == 0 && lane == 0) {
            int entry = 0, heads = 0;  // tiles of queries, and of keys
            bool ok = true;
            Item it{}, before{};
            for (int i = begin; i < end && ok; ++i, before = it) {
                it = item_at(i);
                if (i == begin || other_keys(it, before)) {
                    if (!(ok = wait(kv_empty, (heads + 1) & 1))) break;
                    ++heads;
                    mbar_arrive_expect_tx(kv_full, 2 * C::TILE);
                    load_tile<C::HALVES>(base, p.k, 0, it.h / p.group, it.b, kv_full);
                    load_tile<C::HALVES>(base + C::TILE, p.v, 0, it.h / p.group, it.b, kv_full);
                }
                for (int g = 0; g < it.groups; ++g, ++entry) {
                    const int s = entry % C::STAGES;
                    if (!(ok = wait(empty_bar(s), (entry / C::STAGES + 1) & 1))) break;
                    mbar_arrive_expect_tx(full_bar(s), C::TILE);
                    load_tile<C::HALVES>(base + kRing + s * C::TILE, p.q, it.q0 + g * kGroupRows, it.h, it.b, full_bar(s));
                }
            }
            if (!ok) {
                wait.fail();
                // copies in flight land before shared memory goes away
                for (int e = entry > C::STAGES ? entry - C::STAGES : 0; e < entry; ++e) mbar_wait(full_bar(e % C::STAGES), (e / C::STAGES) & 1);
                if (heads > 0) mbar_wait(kv_full, (heads - 1) & 1);
            }
        } else if (kStay && warp == 1) {
            const uint32_t id_s = idesc<T>(128, 128, false, false);
            const int n_o = (p.d + 15) / 16 * 16, steps = (p.d + kMmaK - 1) / kMmaK;
            const uint32_t id_o = idesc<T>(128, n_o, false, true);
            int entry = 0, heads = 0;
            uint32_t p_phase[2] = {0, 0};
            bool ok = true;
            auto scores = [&](int g) {  // S = Q K^T, once the next tile of queries is there
                const int s = entry % C::STAGES;
                if (!(ok = wait.together(full_bar(s), (entry / C::STAGES) & 1))) return;
                ++entry;
                tc_fence_after();
                if (one_thread()) {
                    tile_product<kD>(tmem + C::S_COL + 128 * g, base + kRing + s * C::TILE, base, id_s, steps);
                    mma_commit(s_full(g));
                    mma_commit(empty_bar(s));
                }
                __syncwarp();
            };
            Item it{}, next{};
            if (begin < end) next = item_at(begin);
            for (int i = begin; i < end && ok; ++i) {
                it = next;
                const bool more = i + 1 < end;
                if (more) next = item_at(i + 1);
                const bool leave = more && other_keys(next, it);
                if (i == begin) {
                    if (!(ok = wait.together(kv_full, 0))) break;
                    for (int g = 0; g < it.groups && ok; ++g) scores(g);
                    if (!ok) break;
                }
                if (p.mask && !(ok = wait.together(clean_bar(0), heads & 1))) break;  // (done already, but for a head's first item)
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    if (g < it.groups) {
                        if (!(ok = wait.together(p_ready(g), p_phase[g]))) break;
                        p_phase[g] ^= 1u;
                        tc_fence_after();
                        if (one_thread()) {
                            tile_add<2>(tmem + C::O_COL + kD * g, tmem + C::S_COL + 128 * g, base + C::TILE, id_o, true);
                            mma_commit(o_full(g));
                        }
                        __syncwarp();
                    }
                    if (more && !leave && g < next.groups) {
                        scores(g);
                        if (!ok) break;
                    }
                }
                if (!ok) break;
                if (leave) {
                    if (one_thread()) mma_commit(kv_empty);
                    __syncwarp();
                    ++heads;
                    if (!(ok = wait.together(kv_full, heads & 1))) break;
                    for (int g = 0; g < next.groups && ok; ++g) scores(g);
                }
            }
            if (!ok) wait.fail();
            if (one_thread()) {
                mma_commit(done_bar);
                mbar_wait(done_bar, 0);
            }
        } else if (kStay && warp >= 2 && p.mask) {
            bool ok = true;
            int heads = 0;
            MaskedRows rows;
            Item it{}, before{};
            for (int i = begin; i < end; ++i, before = it) {
                it = item_at(i);
                if (i > begin && !other_keys(it, before)) continue;
                rows.of(p.mask, p.mask_stride, it.b, p.kv_tokens, warp - 2, lane);
                if (!(ok = wait.together(kv_full, heads & 1))) break;
                clean_rows<C::HALVES>(base + C::TILE, rows.there, warp - 2, lane);
                if (lane == 0) mbar_arrive(clean_bar(0));
                ++heads;
            }
            if (!ok) wait.fail();
        } else if (!kStay && warp == 0 && lane == 0) {
            int stage = 0;
            uint32_t phase = 0, q_phase[2] = {0, 0};
            uint32_t armed = 0;  // stages and groups whose copies may be in flight
            bool ok = true;
            auto load = [&](const HeadsMap &m, int tile, const Item &it) {
                if (!ok || !wait(empty_bar(stage), phase ^ 1u)) return void(ok = false);
                mbar_arrive_expect_tx(full_bar(stage), C::TILE);
                load_tile<C::HALVES>(base + kRing + stage * C::TILE, m, (it.first + tile) * kTileKeys, it.h / p.group, it.b, full_bar(stage));
                armed |= 1u << stage;
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            };
            for (int i = begin; i < end && ok; i += step) {
                const Item it = item_at(i);
                if (it.tiles == 0) continue;
                for (int g = 0; g < it.groups && ok; ++g) {
                    if (!wait(q_empty(g), q_phase[g] ^ 1u)) {
                        ok = false;
                        break;
                    }
                    q_phase[g] ^= 1u;
                    mbar_arrive_expect_tx(q_full(g), C::TILE);
                    load_tile<C::HALVES>(base + g * C::TILE, p.q, it.q0 + g * kGroupRows, it.h, it.b, q_full(g));
                    armed |= 1u << (16 + g);
                    if (g == 0) load(p.k, 0, it);
                }
                for (int j = 0; j < it.tiles && ok; ++j) {
                    load(p.v, j, it);
                    if (j + 1 < it.tiles) load(p.k, j + 1, it);
                }
            }
            if (!ok) {
                wait.fail();
                // copies in flight land before shared memory goes away: a stage's last phase, then the groups'
                for (int s = 0; s < C::STAGES; ++s)
                    if (armed >> s & 1u) mbar_wait(full_bar(s), s < stage ? phase : phase ^ 1u);
                for (int g = 0; g < 2; ++g)
                    if (armed >> (16 + g) & 1u) mbar_wait(q_full(g), q_phase[g] ^ 1u);
            }
        } else if (!kStay && warp == 1) {
            const uint32_t kIdS = idesc<T>(128, 128, false, false);
            const int n_o = (p.d + 15) / 16 * 16, steps = (p.d + kMmaK - 1) / kMmaK;
            const uint32_t id_o = idesc<T>(128, n_o, false, true);
            int stage = 0;
            uint32_t phase = 0, q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
            int cleaned = 0;  // masked tiles of values (which are not always those of a stage)
            bool ok = true;
            auto next = [&]() {
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            };
            auto scores = [&](int g, int at) {  // S = Q K^T
                tile_product<kD>(tmem + C::S_COL + 128 * g, base + g * C::TILE, base + kRing + at * C::TILE, kIdS, steps);
                mma_commit(s_full(g));
            };
            for (int i = begin; i < end && ok; i += step) {
                const Item it = item_at(i);
                if (it.tiles == 0) continue;
                if (!(ok = wait.together(full_bar(stage), phase))) break;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    if (g >= it.groups) break;
                    if (!(ok = wait.together(q_full(g), q_phase[g]))) break;
                    q_phase[g] ^= 1u;
                    tc_fence_after();
                    if (one_thread()) {
                        scores(g, stage);
                        if (it.tiles == 1) mma_commit(q_empty(g));
                        if (g + 1 == it.groups) mma_commit(empty_bar(stage));
                    }
                    __syncwarp();
                }
                if (!ok) break;
                next();
                for (int j = 0; j < it.tiles; ++j) {
                    const int v_stage = stage;
                    const bool last = j + 1 == it.tiles;
                    if (!(ok = p.mask ? wait.together(clean_bar(cleaned % C::STAGES), (cleaned / C::STAGES) & 1) : wait.together(full_bar(stage), phase))) break;
                    ++cleaned;
                    next();
                    if (!last && !(ok = wait.together(full_bar(stage), phase))) break;
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        if (g >= it.groups) break;
                        if (!(ok = wait.together(p_ready(g), p_phase[g]))) break;
                        p_phase[g] ^= 1u;
                        tc_fence_after();
                        if (one_thread()) {
                            tile_add<2>(tmem + C::O_COL + kD * g, tmem + C::S_COL + 128 * g, base + kRing + v_stage * C::TILE, id_o, j == 0);
                            if (last) {
                                mma_commit(o_full(g));
                            } else {
                                scores(g, stage);
                                if (j + 2 == it.tiles) mma_commit(q_empty(g));
                            }
                            if (g + 1 == it.groups) {
                                mma_commit(empty_bar(v_stage));
                                if (!last) mma_commit(empty_bar(stage));
                            }
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    if (!last) next();
                }
            }
            if (!ok) wait.fail();
            if (one_thread()) {
                mma_commit(done_bar);
                mbar_wait(done_bar, 0);
            }
        } else if (!kStay && warp >= 2 && p.mask) {  // (one tile an item: keys, then values)
            bool ok = true;
            int entry = 1, cleaned = 0;
            MaskedRows rows;
            for (int i = begin; i < end && ok; i += step, entry += 2, ++cleaned) {
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
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        const int g = (warp - 4) >> 3, half = (warp >> 2) & 1 ^ 1, quad = warp & 3;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        const uint32_t s_at = lanes + C::S_COL + 128 * g + kHalfKeys * half, o_at = lanes + C::O_COL + kD * g;
        const float c = p.scale_log2;
        // What this thread and the one with the row's other keys tell each other. A warp whose wait ran out says so at the
        // next meeting (kGone, a NaN that no arithmetic gives), and both leave there: neither waits for one that has left.
        constexpr uint32_t kGone = 0x7fabcdefu;
        float *meet = reinterpret_cast<float *>(gbase + kMeet) + ((g * 4 + quad) * 2) * 32 + lane;
        constexpr int kTurn = 2 * 4 * 2 * 32;
        bool ok = true, gone = false;
        int turn = 0;  // a place is written again only after the other thread came to the meeting in between
        auto other = [&](float mine) {
            meet[turn * kTurn + half * 32] = ok ? mine : __uint_as_float(kGone);
            asm volatile("bar.sync %0, 64;" ::"r"(1 + g * 4 + quad) : "memory");
            const float theirs = *reinterpret_cast<volatile float *>(&meet[turn * kTurn + (half ^ 1) * 32]);
            gone = !ok || __float_as_uint(theirs) == kGone;
            turn ^= 1;
            return theirs;
        };
        uint32_t s_phase = 0, o_phase = 0;
        uint32_t there[2] = {0, 0};  // a mask's keys of this thread
        int masked = -1;             // its sample
        for (int i = begin; i < end && !gone; i += step) {
            const Item it = item_at(i);
            if (g >= it.groups) continue;
            if (p.mask && it.b != masked) {
                masked = it.b;
#pragma unroll
                for (int n = 0; n < 2; ++n) there[n] = keys_there(p.mask + it.b * p.mask_stride, half * kHalfKeys + n * 32 + lane, p.kv_tokens);
            }
            float top = neg_inf(), sum = 0.0f;  // the reference, and this thread's sum of 2^(c (s - top) + kShift)
            for (int j = 0; j < it.tiles; ++j) {
                ok = ok && wait.together(s_full(g), s_phase);
                s_phase ^= 1u;
                tc_fence_after();
                uint32_t r[kHalfKeys];
#pragma unroll
                for (int k = 0; k < kHalfKeys; k += 32) tmem_ld32_async(s_at + k, r + k);
                tmem_ld_wait(r);
                const int keys = it.keys - (it.first + j) * kTileKeys - half * kHalfKeys;
                if (p.mask) {
#pragma unroll
                    for (int k = 0; k < kHalfKeys; ++k)
                        if (!(there[k / 32] & 1u << k % 32)) r[k] = 0xff800000u;
                } else if (keys < kHalfKeys) {
#pragma unroll
                    for (int k = 0; k < kHalfKeys; ++k)
                        if (k >= keys) r[k] = 0xff800000u;
                }
                float m[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
                for (int k = 0; k < kHalfKeys; ++k) m[k % 4] = fmaxf(m[k % 4], __uint_as_float(r[k]));
                const float mine = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
                const float now = fmaxf(mine, other(mine));
                if (gone) break;
                if (j == 0) {
                    top = now;
                } else if (__any_sync(0xffffffffu, (now - top) * c > kGrow)) {
                    // P V of the tile before is complete: the same commit told of it
                    const float next = fmaxf(top, now), factor = next == neg_inf() ? 1.0f : ex2((top - next) * c);
                    top = next;
                    sum *= factor;
#pragma unroll 1
                    for (int k = half * 16; k < p.d; k += 32) {
                        uint32_t o[16];
                        tmem_ld16_async(o_at + k, o);
                        tmem_ld_wait(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * factor);
                        tmem_st16(o_at + k, o);
                    }
                }
                // (a row of scores that are all -infinity so far, also where c s is past the floats: no term at all)
                const float most = top * c, off = most == neg_inf() ? 0.0f : kShift - most;
                const F2 c2(c), off2(off);
                F2 add[2] = {F2(0.0f), F2(0.0f)};
#pragma unroll
                for (int k0 = 0; k0 < kHalfKeys; k0 += 32) {
                    uint32_t pk[16];
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        const F2 x = fma2(F2(__uint_as_float(r[k0 + k]), __uint_as_float(r[k0 + k + 1])), c2, off2);
                        const F2 e(ex2(x.lo()), ex2(x.hi()));
                        add[k / 2 % 2] = add[k / 2 % 2] + e;
                        pk[k / 2] = pack2<T>(e.lo(), e.hi());
                    }
                    tmem_st16(s_at + k0 / 2, pk);
                }
                sum += add[0].sum() + add[1].sum();
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_ready(g));
            }
            if (gone) break;
            const int row0 = it.q0 + g * kGroupRows + quad * 32, rows = p.q_tokens - row0 < 32 ? p.q_tokens - row0 : 32;
            const float theirs = other(sum);
            if (gone) break;
            sum = half == 0 ? sum + theirs : theirs + sum;
            if (top * c == -neg_inf()) sum = __uint_as_float(0x7fffffffu);  // infinity less itself, as for infinite S (no term was left)
            const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;  // NaN stays
            // (of this share, where there are several: the second kernel puts them together)
            const int64_t row = it.share * p.rows + (static_cast<int64_t>(it.b) * p.q_heads + it.h) * p.q_tokens + row0 + lane;
            if (half == 0 && lane < rows)
                (kShares ? p.partial + p.splits * p.rows * p.pitch : p.lse)[row] = sum == 0.0f ? neg_inf() : kLn2 * (top * c + (log2f(sum) - kShift));
            T *out = static_cast<T *>(p.out) + it.b * p.out_strides[0] + row0 * p.out_strides[1] + it.h * p.out_strides[2];
            if (it.tiles > 0) {
                ok = wait.together(o_full(g), o_phase);
                o_phase ^= 1u;
                tc_fence_after();
            }
#pragma unroll 1
            for (int k = half * 32; k < p.d; k += 64) {
                uint32_t o[32];
                float v[32];
                if (it.tiles > 0) {
                    tmem_ld32_async(o_at + k, o);
                    tmem_ld_wait(o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = sum == 0.0f ? 0.0f : __uint_as_float(o[e]) * inv;
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0.0f;
                }
                if (kShares) {
                    if (lane < rows && ok) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            if (k + e < p.pitch) *reinterpret_cast<float4 *>(p.partial + row * p.pitch + k + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                    }
                    continue;
                }
                if (rows > 0 && ok)
                    store_rows_traded<T>(out + k, p.out_strides[1], rows, p.d - k < 32 ? p.d - k : 32, p.wide, lane, v);
            }
            tc_fence_before();  // O is read before the next item's first P is announced
        }
        if (!ok) wait.fail();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_free<1>(tmem, 512u);
}

struct JoinParams {
    const float *partial;
    int32_t splits, pitch, d, q_heads;
    int64_t rows, q_tokens;
    void *out;
    int64_t out_strides[3];
    float *lse;
};

// A row of the outputs from its shares, weighted by e^(lse of the share - lse): a warp a row, four elements a lane.
template <typename T>
__global__ void __launch_bounds__(256) attention_join_kernel(const __grid_constant__ JoinParams p)
{
    after_previous();
    let_next_start();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;
    const int lane = threadIdx.x & 31, e0 = lane * 4;
    if (row >= p.rows) return;
    const float *lses = p.partial + p.splits * p.rows * p.pitch;
    const float mine = lane < p.splits ? load_f32(lses + lane * p.rows + row) : neg_inf();
    float top = mine;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    const float weight = top == neg_inf() && mine == top ? 0.0f : ex2((mine - top) * kLog2e);  // (NaN stays)
    float sum = weight;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s = 0; s < p.splits; ++s) {
        const float w = __shfl_sync(0xffffffffu, weight, s);
        if (e0 >= p.d) continue;
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.partial + (s * p.rows + row) * p.pitch + e0));
        o.x = fmaf(w, v.x, o.x);
        o.y = fmaf(w, v.y, o.y);
        o.z = fmaf(w, v.z, o.z);
        o.w = fmaf(w, v.w, o.w);
    }
    const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;
    if (lane == 0) p.lse[row] = sum == 0.0f ? neg_inf() : top + logf(sum);
    const int64_t bh = row / p.q_tokens, t = row - bh * p.q_tokens, b = bh / p.q_heads, h = bh - b * p.q_heads;
    T *out = static_cast<T *>(p.out) + b * p.out_strides[0] + t * p.out_strides[1] + h * p.out_strides[2] + e0;
    const float v[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e0 + e < p.d) out[e] = from_f32<T>(v[e]);
}

template <typename T, int kD, KeyForm kForm>
struct attention_tag;

template <typename T, int kD, KeyForm kForm>
cudaError_t launch_form(const AttentionArgs &a, cudaStream_t stream)
{
    using C = Cfg<kD>;
    Params p{};
    if (!heads_map<T>(&p.q, a.q, a.batch, a.d, kGroupRows)) return cudaErrorInvalidValue;
    if (a.k.tokens > 0 && (!heads_map<T>(&p.k, a.k, a.batch, a.d, kTileKeys) || !heads_map<T>(&p.v, a.v, a.batch, a.d, kTileKeys)))
        return cudaErrorInvalidValue;
    p.counts = a.counts;
    p.mask = a.mask;
    p.mask_stride = a.mask_stride;
    p.out = a.out;
    for (int i = 0; i < 3; ++i) p.out_strides[i] = a.out_strides[i];
    p.lse = a.lse;
    p.dev_status = a.dev_status;
    p.q_tokens = static_cast<int32_t>(a.q.tokens);
    p.kv_tokens = static_cast<int32_t>(a.kv_tokens);
    p.q_heads = static_cast<int32_t>(a.q.heads);
    p.group = static_cast<int32_t>(a.q.heads / a.k.heads);
    p.q_tiles = static_cast<int32_t>((a.q.tokens + kItemRows - 1) / kItemRows);
    p.splits = kForm == kShared ? a.splits : 1;
    p.partial = a.partial;
    p.rows = a.batch * a.q.heads * a.q.tokens;
    p.pitch = (a.d + 3) / 4 * 4;
    const int64_t items = a.batch * a.q.heads * p.q_tiles * p.splits;
    if (items > INT32_MAX) return cudaErrorInvalidValue;
    p.items = static_cast<int32_t>(items);
    p.d = a.d;
    p.wide = heads_wide(a.out, a.out_strides, a.batch, a.q.tokens, a.q.heads);
    p.scale_log2 = a.scale * kLog2e;
    auto kernel = attention_kernel<T, kD, kForm>;
    cudaError_t e = allow_shared<attention_tag<T, kD, kForm>>(kernel);
    if (e != cudaSuccess) return e;
    e = launch_after(kernel, dim3(static_cast<unsigned>(items < kSms ? items : kSms)), kThreads, C::SMEM, stream, 1, p);
    if (e != cudaSuccess || p.splits == 1) return e;
    JoinParams j{a.partial, p.splits, p.pitch, p.d, p.q_heads, p.rows, a.q.tokens, a.out, {a.out_strides[0], a.out_strides[1], a.out_strides[2]}, a.lse};
    return launch_after(attention_join_kernel<T>, dim3(static_cast<unsigned>((p.rows + 7) / 8)), 256, 0, stream, 1, j);
}

// Keys of one tile stay with a CTA where a key head has four items or more: changing heads stops it for a copy (1.5 us),
// and with a head an item that would be all the time (2 x 4096 queries, 77 keys, 10 heads of 64: 12.6 us through the ring).
template <typename T, int kD>
cudaError_t launch(const AttentionArgs &a, cudaStream_t stream)
{
    const int64_t of_head = a.q.heads / a.k.heads * ((a.q.tokens + kItemRows - 1) / kItemRows);
    const bool stay = !a.counts && a.kv_tokens > 0 && a.kv_tokens <= kTileKeys && of_head >= 4;
    if (stay) return launch_form<T, kD, kStays>(a, stream);
    return a.splits > 1 ? launch_form<T, kD, kShared>(a, stream) : launch_form<T, kD, kPass>(a, stream);
}

}  // namespace

cudaError_t launch_attention(const AttentionArgs &a, cudaStream_t stream)
{
    if (a.dtype == CONVROT_BF16) return a.d <= 64 ? launch<__nv_bfloat16, 64>(a, stream) : launch<__nv_bfloat16, 128>(a, stream);
    return a.d <= 64 ? launch<__half, 64>(a, stream) : launch<__half, 128>(a, stream);
}

int32_t attention_splits(int64_t batch, int64_t q_tokens, int64_t kv_tokens, int64_t q_heads)
{
    return key_shares(batch * q_heads * ((q_tokens + kItemRows - 1) / kItemRows), kv_tokens);
}

int64_t attention_partial_bytes(int64_t batch, int64_t q_tokens, int64_t kv_tokens, int64_t q_heads, int d)
{
    const int32_t splits = attention_splits(batch, q_tokens, kv_tokens, q_heads);
    return splits > 1 ? splits * batch * q_heads * q_tokens * ((d + 3) / 4 * 4 + 1) * 4 : 0;
}

int attention_shared(int form, int *columns)
{
    *columns = 512;
    return form == 0 ? Cfg<64>::SMEM : form == 1 ? Cfg<128>::SMEM : 0;
}

}  // namespace convrot
