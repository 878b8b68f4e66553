// Attention within packed prompts of different lengths.
//
// An item is 256 rows against one key head of one sequence: two query tiles of 128 rows, each as many
// tokens as fit with the G query heads that share the key head, so keys and values are loaded once for
// 256 rows.  A persistent CTA per SM takes items from a queue, the ones with the most keys first, and
// streams the sequence's keys and values past its two tiles in tiles of 128 tokens.  While one tile's
// scores go through the softmax, the tensor cores work for the other.
//
//   warps 0-7, 8-15  softmax and output of one query tile each: two threads per row, 64 of a key
//                    tile's tokens each; running maximum and sum in fp32, weights rounded to the
//                    inputs' type; at the end zeros for the tokens outside every sequence
//   warp 16          takes the items and loads (TMA) queries, keys and values
//   warps 17, 18     issue S = Q K^T and O += P V of one query tile each on tcgen05 (M = 128, fp32 in
//                    tensor memory; P replaces half of S)
//
// The running maximum is raised only when a tile exceeds it by 2^8 (O is then rescaled): weights up to
// 2^8 lose nothing in a floating type, and the rescaling leaves the common path.  In fp16 the exponentials'
// reference is 2^7 below it (kHeadroom).
//
// A row must not see what lies outside its limit, but 0 * infinity is not 0.  Values past the
// sequence's end are zeroed in shared memory before the product.  A query tile whose result is not
// finite is done again alone with the infinities and NaN taken out of every value tile and added to
// the rows that see them; nothing else changes then, so rows that do not see them come out bit for
// bit as without them.
//
// Meant to be bound by the tensor cores: a key tile's products of both query tiles take 2048 cycles (D = 128,
// 64 for each of 32 instructions).  8192 tokens of 32 heads of 128 on 8, causal, take 371 us (385 us in a long run,
// where the clock is lower): 1.48 PFLOP/s, 0.78 of what a large product reaches, 3000 cycles a key tile.  What is
// left is a chain: with D = 128 the two S and O fill tensor memory, so a tile's next S waits for its own P (768
// cycles of products), and its softmax (about 1500 cycles, half of them the exponential's unit) for S.  Measured on
// the way: a thread per row 522 us with a warp issuing for each query tile (they ran in step), 416 us with one warp
// issuing for both; two threads per row 416 us; the tiles taking turns, waits ahead of the turn and out of line
// 372 us.  Starting the second tile half a step late, and with D = 64 a P apart from S, made no difference.
#include "attention_common.cuh"
#include "host_common.h"

#include <algorithm>

namespace dspark {
namespace {

constexpr int kTile = 128;                 // key tokens per tile, and MMA rows
constexpr int kThreads = 608;
constexpr int kRowThreads = 256;           // softmax threads of a query tile: two to a row, 64 of a key tile's tokens each
constexpr float kRaise = 8.0f;             // log2 units
constexpr int kAhead = 4;                  // items between the loads and the results
constexpr int kRedo = 2 * kAhead;          // items of which a query tile waits to be done again: at most those under way
constexpr int kSlots = 2;                  // key tiles, and value tiles, in flight
constexpr int kOrdered = 256;              // up to so many sequences the items are put in order of their size
constexpr uint32_t kColS = 0, kColP = 64, kColO = 256, kTmemCols = 512;    // S and O of tile 1: + 128
// named barriers: + query tile; + 4 * query tile + quadrant, the two warps of the same rows; + query tile
constexpr uint32_t kWarpLoad = 16, kWarpMma = 17;
constexpr uint32_t kBarTile = 1, kBarRows = 3, kBarFirst = 11;
constexpr uint32_t kWaitLoad = 0x901, kWaitMma = 0x902, kWaitSoftmax = 0x903;

struct Plan {
    WsHeader header;
    int items;                             // without the heads
    unsigned int next;                     // of the queue, heads innermost
    int begin, end;                        // the tokens of all sequences
    int pad[60];
};
static_assert(sizeof(Plan) == 512, "the item list behind the plan is aligned");

struct PromptArgs {
    const int32_t* cu_seqlens;
    int causal, B, T, Hq, Hkv, group;
    int tile_tokens;                       // tokens of a query tile
    float scale;
    void* out;
    float* lse;
    Plan* plan;
    int4* items;                           // sequence begin, end, pair of query tiles, 0
    long long timeout_ns;
};

// An item as the roles see it.
struct Item {
    int begin, end;                        // the sequence
    int tok;                               // first token of tile 0, relative to the sequence
    int h;
    int n[2];                              // key tiles of each query tile
    int redo;                              // done again: infinities are moved
    int id, pair;
};

// Key tiles that query tile x of an item sees.
__device__ __forceinline__ int tiles_seen(const PromptArgs& a, int len, int tok, int x) {
    const int first = tok + x * a.tile_tokens;
    if (first >= len) return 0;
    const int last = a.causal ? min(len, first + a.tile_tokens) : len;
    return (last + kTile - 1) / kTile;
}

// ---------------------------------------------------------------------------
// Plan: one block.  Clears the status word and the queue, reads the sequences' bounds as their running
// maximum within [0, T], and lists the items.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kPlanThreads) prompt_plan_kernel(const __grid_constant__ PromptArgs a) {
    __shared__ int s_warp[kPlanThreads / 32], s_carry;
    __shared__ int s_end[kPlanThreads + 1];                // bounds of the sequences at hand
    __shared__ int s_first[kPlanThreads + 1];              // their first items
    Plan* p = a.plan;
    const int tid = threadIdx.x;
    grid_dependency_launch();                              // the attention kernel sets itself up meanwhile
    if (tid < 64) reinterpret_cast<uint32_t*>(&p->header)[tid] = 0u;
    // inclusive scan over the block, by maximum or sum, on top of `carry`
    auto scan = [&](int x, bool sum) {
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, x, d);
            if (lane_id() >= static_cast<uint32_t>(d)) x = sum ? x + y : max(x, y);
        }
        __syncthreads();
        if (lane_id() == 31) s_warp[warp_id()] = x;
        __syncthreads();
        int before = 0;
        for (uint32_t w = 0; w < warp_id(); ++w) before = sum ? before + s_warp[w] : max(before, s_warp[w]);
        return sum ? x + before : max(x, before);
    };
    const int pair = 2 * a.tile_tokens;
    int bound = min(max(a.cu_seqlens[0], 0), a.T), total = 0;
    __syncthreads();
    if (tid == 0) {
        p->begin = bound;
        if (a.cu_seqlens[0] != bound) flag_input_index(&p->header);
    }
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
        const int count = min(kPlanThreads, a.B - b0);
        const int raw = tid < count ? a.cu_seqlens[b0 + tid + 1] : 0;
        const int end = max(bound, scan(min(max(raw, 0), a.T), false));
        if (tid < count && raw != end) flag_input_index(&p->header);
        s_end[tid + 1] = end;
        if (tid == 0) s_end[0] = bound;
        __syncthreads();
        const int mine = tid < count ? (end - s_end[tid] + pair - 1) / pair : 0;
        const int last = total + scan(mine, true), first = last - mine;
        s_first[tid] = first;
        if (tid == kPlanThreads - 1) s_carry = last;
        __syncthreads();
        total = s_carry;
        bound = s_end[count];
        if (a.B > kOrdered) {
            // sequence by sequence, the later tokens first
            for (int x = 0; x < mine; ++x) a.items[first + x] = make_int4(s_end[tid], end, mine - 1 - x, 0);
            __syncthreads();
        }
    }
    if (a.B <= kOrdered) {
        // by the place in the sequence, the last first: that is the order of the work under the causal mask
        for (int e = tid; e < total; e += kPlanThreads) {
            int lo = 0, hi = a.B - 1;                      // the sequence of item e
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (s_first[mid] <= e) lo = mid; else hi = mid - 1;
            }
            const int x = e - s_first[lo];
            int at = 0;
            for (int b = 0; b < a.B; ++b) {
                const int n = (b + 1 < a.B ? s_first[b + 1] : total) - s_first[b];
                at += max(0, n - x - 1) + (b < lo && n > x ? 1 : 0);
            }
            a.items[at] = make_int4(s_end[lo], s_end[lo + 1], x, 0);
        }
    }
    if (tid == 0) {
        p->items = total;
        p->next = 0u;
        p->end = bound;
    }
}

template <int D>
struct PromptSmem {
    static constexpr int kHalves = D / 64;                        // 128-byte column blocks
    static constexpr uint32_t kBlockBytes = kTile * 128;
    static constexpr uint32_t kTileBytes = kHalves * kBlockBytes;
    alignas(1024) uint8_t q[2][kTileBytes];
    alignas(1024) uint8_t k[kSlots][kTileBytes];
    alignas(1024) uint8_t v[kSlots][kTileBytes];
    alignas(1024) uint4 stage[16][128];                           // 32 columns of a warp's rows; a row of values where a tile is done again
    Item item[kAhead];
    float half[2][2][kTile];                                      // by query tile and half of the key tiles: a row's largest score, at last its sum
    uint32_t masks[2][4];
    int redo[2][kRedo];                                           // items to be done again, by query tile
    unsigned int redo_count[2];                                   // entries written so far
    uint64_t item_full[kAhead], item_empty[kAhead];
    uint64_t q_full[2], q_empty[2];
    uint64_t k_full[kSlots], k_empty[kSlots], v_full[kSlots], v_empty[kSlots];
    uint64_t s_full[2], p_first[2], p_last[2], pv_done[2], o_empty[2], turn[2], drain;
    uint32_t tmem_base;
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
prompt_attention_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PromptArgs a) {
    using Smem = PromptSmem<D>;
    constexpr int kHalves = Smem::kHalves;
    constexpr uint32_t kBlockBytes = Smem::kBlockBytes, kTileBytes = Smem::kTileBytes;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem& s = *reinterpret_cast<Smem*>(smem_raw);
    const uint32_t warp = warp_id(), lane = lane_id();
    WsHeader* ws = &a.plan->header;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kAhead; ++i) {
            mbar_init(&s.item_full[i], 1);
            mbar_init(&s.item_empty[i], 2 * kRowThreads + 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.q_full[i], 1);
            mbar_init(&s.q_empty[i], 1);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.turn[i], 1);
            mbar_init(&s.p_first[i], kRowThreads);
            mbar_init(&s.p_last[i], kRowThreads);
            mbar_init(&s.pv_done[i], 1);
            mbar_init(&s.o_empty[i], kRowThreads);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&s.k_full[i], 1);
            mbar_init(&s.k_empty[i], 2);
            mbar_init(&s.v_full[i], 1);
            mbar_init(&s.v_empty[i], 2);
        }
        mbar_init(&s.drain, 2);
        s.redo_count[0] = s.redo_count[1] = 0u;
        fence_mbarrier_init();
        prefetch_tensormap(&tmQ);
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (warp == kWarpMma) {
        tmem_alloc(&s.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem_base;
    grid_dependency_wait();

    bool ok = true;
    auto all = [&](bool x) { return __all_sync(0xFFFFFFFFu, x); };
    auto wait = [&](uint64_t& bar, int use, uint32_t where) {            // use: how often it completed before
        return mbar_wait_short(&bar, static_cast<uint32_t>(use) & 1u, ws, a.timeout_ns, where);
    };

    if (warp == kWarpLoad) {
        // ---------------- items and loads ----------------
        if (lane == 0) {
            const uint64_t keep = l2_policy_evict_last();
            const int total = a.plan->items * a.Hkv;
            int kt = 0, qt[2] = {0, 0}, count = 0;        // key tiles, query tiles, items so far
            unsigned int redone[2] = {0, 0};
            // a query tile to be done again (item * 2 + tile), or -1
            auto pending = [&] {
                for (int x = 0; x < 2; ++x) {
                    if (redone[x] == *reinterpret_cast<volatile unsigned int*>(&s.redo_count[x])) continue;
                    __threadfence_block();
                    return s.redo[x][redone[x]++ % kRedo] * 2 + x;
                }
                return -1;
            };
            while (true) {
                Item it{};
                int again = pending();                    // else the queue's next item
                int id = again >= 0 ? again >> 1 : static_cast<int>(atomicAdd(&a.plan->next, 1u));
                if (again < 0 && id >= total) {
                    // the queue is empty: what is under way may still ask for a tile to be done again
                    for (int x = std::max(0, count - kAhead); ok && x < count; ++x)
                        ok = wait(s.item_empty[x % kAhead], x / kAhead, kWaitLoad);
                    if (ok) again = pending();
                    if (again < 0) break;
                    id = again >> 1;
                }
                const int entry = id / a.Hkv;
                const int4 e = a.items[entry];
                it.begin = e.x;
                it.end = e.y;
                it.h = id - entry * a.Hkv;
                it.tok = e.z * 2 * a.tile_tokens;
                it.id = id;
                it.redo = again >= 0 ? 1 : 0;
                for (int x = 0; x < 2; ++x)
                    it.n[x] = again >= 0 && (again & 1) != x ? 0 : tiles_seen(a, it.end - it.begin, it.tok, x);
                ok = wait(s.item_empty[count % kAhead], count / kAhead + 1, kWaitLoad);
                if (!ok) break;
                s.item[count % kAhead] = it;
                mbar_arrive(&s.item_full[count % kAhead]);
                ++count;
                for (int x = 0; ok && x < 2; ++x) {
                    if (it.n[x] == 0) continue;
                    ok = wait(s.q_empty[x], qt[x] + 1, kWaitLoad);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&s.q_full[x], static_cast<uint32_t>(a.tile_tokens * a.group) * 128u * kHalves);
                    for (int y = 0; y < kHalves; ++y)
                        tma_load_3d(s.q[x] + y * kBlockBytes, &tmQ, y * 64, it.h * a.group,
                                    it.begin + it.tok + x * a.tile_tokens, &s.q_full[x], keep);
                    ++qt[x];
                }
                const int n = std::max(it.n[0], it.n[1]);
                for (int t = 0; ok && t < n; ++t, ++kt) {
                    const int slot = kt % kSlots;
                    ok = wait(s.k_empty[slot], kt / kSlots + 1, kWaitLoad);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&s.k_full[slot], kTileBytes);
                    for (int y = 0; y < kHalves; ++y)
                        tma_load_3d(s.k[slot] + y * kBlockBytes, &tmK, y * 64, it.h, it.begin + t * kTile, &s.k_full[slot], keep);
                    ok = wait(s.v_empty[slot], kt / kSlots + 1, kWaitLoad);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&s.v_full[slot], kTileBytes);
                    for (int y = 0; y < kHalves; ++y)
                        tma_load_3d(s.v[slot] + y * kBlockBytes, &tmV, y * 64, it.h, it.begin + t * kTile, &s.v_full[slot], keep);
                }
                if (!ok) break;
            }
            if (ok) {
                // the end: an item without a head
                ok = wait(s.item_empty[count % kAhead], count / kAhead + 1, kWaitLoad);
                if (ok) {
                    s.item[count % kAhead].h = -1;
                    mbar_arrive(&s.item_full[count % kAhead]);
                }
            }
            if (!ok) {
                // give copies in flight time to land before the block exits
                const long long t0 = global_ns();
                while (global_ns() - t0 < a.timeout_ns) {
                }
            }
        }
    } else if (warp >= kWarpMma) {
        // ---------------- products of query tile w: the whole warp waits, one lane issues ----------------
        // The tensor cores run one tile's products in the order of issue, so S may be written as soon as the
        // product that read P (in S) has been issued.  The tiles take turns with the end of a product and the
        // next scores: then one tile's products run while the other is in its softmax (left alone, the two
        // ran in step and waited for each other's tensor work).  The waits of a turn are done before it, since
        // one takes about as long as the tensor cores' queue lasts.
        const int w = static_cast<int>(warp - kWarpMma);
        constexpr uint32_t kIdescS = attn_idesc<T, false>(kTile, kTile);
        constexpr uint32_t kIdescO = attn_idesc<T, true>(kTile, D);
        constexpr uint32_t kStep = kTileBytes >> 4;               // a tile, in descriptor units
        const uint64_t q_desc = sw128_kmajor_desc(smem_u32(s.q[w]));
        const uint64_t k_desc = sw128_kmajor_desc(smem_u32(s.k[0]));
        const uint64_t v_desc = sw128_token_rows_desc(smem_u32(s.v[0]), kBlockBytes);
        const uint32_t tS = tmem + kColS + w * 128u, tP = tmem + kColP + w * 128u, tO = tmem + kColO + w * 128u;
        int kt = 0, i = 0, used = 0, turn = 0;                    // key tiles, own key tiles, own query tiles, turns
        auto take_turn = [&] {
            const bool mine = w == 0 ? turn == 0 || wait(s.turn[0], turn - 1, kWaitMma) : wait(s.turn[1], turn, kWaitMma);
            ++turn;
            return all(mine);
        };
        for (int count = 0; ok; ++count) {
            ok = all(wait(s.item_full[count % kAhead], count / kAhead, kWaitMma));
            if (!ok) break;
            const Item& it = s.item[count % kAhead];
            const int h = __shfl_sync(0xFFFFFFFFu, it.h, 0);
            if (h < 0) break;
            const int n = __shfl_sync(0xFFFFFFFFu, it.n[w], 0), other = __shfl_sync(0xFFFFFFFFu, it.n[1 - w], 0);
            const int len = __shfl_sync(0xFFFFFFFFu, it.end - it.begin, 0);
            const int redo = __shfl_sync(0xFFFFFFFFu, it.redo, 0);
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.item_empty[count % kAhead]);
            const int most = max(n, other);
            if (most == 0) continue;
            // turn t: the end of the product of key tile t - 1 and the scores of key tile t
            for (int t = 0; t <= most; ++t) {
                const uint64_t v = v_desc + static_cast<uint32_t>((kt + t - 1) % kSlots) * kStep;
                const uint64_t k = k_desc + static_cast<uint32_t>((kt + t) % kSlots) * kStep;
                // what is usually there comes first, the weights last
                if (t < most) ok = all(wait(s.k_full[(kt + t) % kSlots], (kt + t) / kSlots, kWaitMma));
                if (ok && t == 0 && n > 0) ok = all(wait(s.q_full[w], used, kWaitMma));
                if (!ok) break;
                if (t > 0) {
                    const int slot = (kt + t - 1) % kSlots;
                    ok = all(wait(s.v_full[slot], (kt + t - 1) / kSlots, kWaitMma));
                    if (!ok) break;
                    if (t <= n) {
                        const int held = len - (t - 1) * kTile;
                        if (held < kTile) {                       // behind the sequence's end nothing may count
                            const int pieces = (kTile - held) * 8;    // of 16 bytes, per block
                            for (int y = 0; y < kHalves; ++y)
                                for (int x = static_cast<int>(lane); x < pieces; x += 32)
                                    *reinterpret_cast<uint4*>(s.v[slot] + y * kBlockBytes + held * 128 + x * 16) =
                                        make_uint4(0u, 0u, 0u, 0u);
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                        ok = all(wait(s.p_first[w], i, kWaitMma) && (t > 1 || used == 0 || wait(s.o_empty[w], used - 1, kWaitMma)));
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t onto = t == 1 && redo == 0 ? 0u : 1u;   // done again, O starts from what is there
                        // 16 tokens a product; of each half of the tile, the first 32 tokens' weights are ready first
                        if (elect_one()) {
#pragma unroll
                            for (int z = 0; z < 4; ++z) {
                                const int y = z + (z & 2);
                                mma_issue_ta(tO, tP + y * 8, v + y * 128, kIdescO, z == 0 ? onto : 1u);
                            }
                        }
                        __syncwarp();
                    }
                }
                ok = take_turn();
                if (ok && t > 0 && t <= n) ok = all(wait(s.p_last[w], i++, kWaitMma));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    if (t > 0 && t <= n) {
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const int y = 2 + z + (z & 2);
                            mma_issue_ta(tO, tP + y * 8, v + y * 128, kIdescO, 1u);
                        }
                        mma_commit(&s.pv_done[w]);
                    }
                    if (t < n) {
#pragma unroll
                        for (int d = 0; d < D / 16; ++d) {
                            const uint64_t off = (static_cast<uint32_t>(d / 4) * kBlockBytes + (d % 4) * 32) >> 4;
                            mma_issue<false>(tS, q_desc + off, k + off, kIdescS, d != 0 ? 1u : 0u);
                        }
                        mma_commit(&s.s_full[w]);
                    }
                    mbar_arrive(&s.turn[1 - w]);
                    if (t + 1 == n) mma_commit(&s.q_empty[w]);
                    if (t > 0) mma_commit(&s.v_empty[(kt + t - 1) % kSlots]);
                    if (t < most) mma_commit(&s.k_empty[(kt + t) % kSlots]);
                }
                __syncwarp();
            }
            if (!ok) break;
            kt += most;
            used += n > 0 ? 1 : 0;
        }
        if (elect_one()) mma_commit(&s.drain);
        __syncwarp();
        const long long t0 = global_ns();
        while (!mbar_try_wait(&s.drain, 0) && global_ns() - t0 < a.timeout_ns) {
        }
        __syncwarp();
    } else {
        // ---------------- softmax and output of query tile w ----------------
        const int w = static_cast<int>(warp >> 3);
        const int part = static_cast<int>(warp >> 2) & 1;  // 64 of the key tile's tokens, half of the output's columns
        const uint32_t quad = warp & 3u;
        const uint32_t bar_tile = kBarTile + static_cast<uint32_t>(w), bar_rows = kBarRows + 4u * static_cast<uint32_t>(w) + quad;
        const uint32_t lanes = (quad * 32u) << 16;
        const uint32_t tS = tmem + lanes + kColS + w * 128u + part * 64u, tP = tmem + lanes + kColP + w * 128u + part * 32u;
        const uint32_t tO = tmem + lanes + kColO + w * 128u + part * (D / 2u);
        const int row = static_cast<int>(quad * 32u + lane);
        const int row_tok = row / a.group;
        const bool row_used = row < a.tile_tokens * a.group;
        const float sl2 = a.scale * kLog2e;
        const bool falling = sl2 < 0.0f;                          // the largest score is the smallest product
        const float none = falling ? INFINITY : -INFINITY;
        int i = 0;                                                // own key tiles
        int kt = 0;                                               // key tiles
        for (int count = 0;; ++count) {
            ok = named_bar_and(bar_tile, kRowThreads, wait(s.item_full[count % kAhead], count / kAhead, kWaitSoftmax));
            if (!ok) break;
            const Item& it = s.item[count % kAhead];
            if (it.h < 0) break;
            const int n = it.n[w], len = it.end - it.begin;
            const bool redo = it.redo != 0;
            if (n == 0) {
                kt += it.n[1 - w];
                mbar_arrive(&s.item_empty[count % kAhead]);
                continue;
            }
            const int tok = it.tok + w * a.tile_tokens + row_tok;         // of this row, in its sequence
            const bool valid = row_used && tok < len;
            const int limit = valid && a.causal ? tok + 1 : len;
            float m2 = -INFINITY, l = 0.0f;
            for (int t = 0; t < n; ++t, ++i) {
                bool go = wait(s.s_full[w], i, kWaitSoftmax);
                if (redo) go = named_bar_and(bar_tile, kRowThreads, go);  // these meet in barriers below
                go = all(go);
                // 64 scores in registers
                uint32_t r[2][32];
                const int seen = limit - t * kTile - part * 64;
                const bool masked = __any_sync(0xFFFFFFFFu, seen < 64);
                tc_fence_after();
                tmem_ld32(tS, r[0]);
                tmem_ld32(tS + 32, r[1]);
                tmem_wait_ld32(r[0]);
                tmem_wait_ld32(r[1]);
                if (masked) {
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        if (c >= seen) r[c >> 5][c & 31] = __float_as_uint(none);
                }
                float best[4] = {none, none, none, none};
                if (!falling) {
#pragma unroll
                    for (int c = 0; c < 64; c += 8)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            best[e] = max3(best[e], __uint_as_float(r[c >> 5][(c & 31) + e]),
                                           __uint_as_float(r[c >> 5][(c & 31) + 4 + e]));
                } else {
#pragma unroll
                    for (int c = 0; c < 64; ++c) best[c & 3] = fminf(best[c & 3], __uint_as_float(r[c >> 5][c & 31]));
                }
                const float top = falling ? fminf(fminf(best[0], best[1]), fminf(best[2], best[3]))
                                          : fmaxf(fmaxf(best[0], best[1]), fmaxf(best[2], best[3]));
                float mt = top == none ? -INFINITY : top * sl2 - HalfType<T>::kHeadroom;
                // The two threads of a row meet: P may then replace the scores, and if either finds the maximum
                // too low (or has given up) they exchange theirs.
                bool raise = t == 0 || !go || (valid && mt > m2 + kRaise);
                if (t > 0) raise = !named_bar_and(bar_rows, 64, !raise);
                ok = go;
                if (raise) {
                    s.half[w][part][row] = mt;
                    if (t > 0) go = go && all(wait(s.pv_done[w], i - 1, kWaitSoftmax));
                    ok = named_bar_and(bar_rows, 64, go);
                    if (!ok && !redo) break;                              // else at the vote below
#ifdef DSPARK_LATE_PART                                                   // a test build: this half of the rows' threads reads late
                    if (part == (DSPARK_LATE_PART)) {
                        const long long t0 = global_ns();
                        while (global_ns() - t0 < 50000) {
                        }
                    }
#endif
                    mt = fmaxf(mt, s.half[w][1 - part][row]);
                    if (t == 0) {
                        m2 = mt;
                    } else if (ok) {
                        tc_fence_after();
                        const bool up = valid && mt > m2 + kRaise;
                        const float f = up ? exp2_approx(m2 - mt) : 1.0f;
                        if (up) {
                            l *= f;
                            m2 = mt;
                        }
#pragma unroll 1
                        for (uint32_t c = 0; c < D / 2; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(tO + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                            tmem_st16(tO + c, o);
                        }
                        tmem_wait_st();
                    }
                }
                const float ref = m2 == -INFINITY ? 0.0f : m2;
                float2 sum[2] = {};
                const float2 slope = make_float2(sl2, sl2), shift = make_float2(-ref, -ref);
                // 32 weights, to P.  Without a mask it is one straight piece of code, for which the compiler
                // finds an order that keeps the exponential's unit (4 cycles a warp) at work.
                auto weigh = [&](int x) {
                    uint32_t p[16];
                    if (!masked) {
#pragma unroll
                        for (int c = 0; c < 32; c += 2) {
                            const float2 y = __ffma2_rn(make_float2(__uint_as_float(r[x][c]), __uint_as_float(r[x][c + 1])), slope, shift);
                            const float2 e = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                            sum[(c >> 1) & 1] = __fadd2_rn(sum[(c >> 1) & 1], e);
                            p[c >> 1] = pack2(e.x, e.y, T{});
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 32; c += 2) {
                            const float2 y = __ffma2_rn(make_float2(__uint_as_float(r[x][c]), __uint_as_float(r[x][c + 1])), slope, shift);
                            const float2 e = make_float2(x * 32 + c < seen ? exp2_approx(y.x) : 0.0f,
                                                         x * 32 + c + 1 < seen ? exp2_approx(y.y) : 0.0f);
                            sum[(c >> 1) & 1] = __fadd2_rn(sum[(c >> 1) & 1], e);
                            p[c >> 1] = pack2(e.x, e.y, T{});
                        }
                    }
                    tmem_st16(tP + x * 16, p);
                    tmem_wait_st();
                };
                weigh(0);
                if (!redo) {
                    tc_fence_before();
                    mbar_arrive(&s.p_first[w]);
                }
                weigh(1);
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                if (redo) {
                    const int slot = (kt + t) % kSlots;
                    bool there = ok && wait(s.v_full[slot], (kt + t) / kSlots, kWaitSoftmax);
                    // O is about to be changed here: the products before must be complete
                    if (there && t > 0) there = wait(s.pv_done[w], i - 1, kWaitSoftmax);
                    there = all(there);
                    if (there && t == 0) {
                        uint32_t zero[16];
#pragma unroll
                        for (int c = 0; c < 16; ++c) zero[c] = 0u;
                        for (uint32_t c = 0; c < D / 2; c += 16) tmem_st16(tO + c, zero);
                        tmem_wait_st();
                    }
                    tc_fence_before();
                    ok = named_bar_and(bar_tile, kRowThreads, there);     // P and O of both halves are in place
                    if (!ok) break;
                    tc_fence_after();
                    if (part == 0) {
                        move_infinities<T>(s.v[slot], kBlockBytes, kHalves, row, len - t * kTile,
                                           [=](int x) { return x < min(limit - t * kTile, kTile); }, tP, tO,
                                           reinterpret_cast<float*>(s.stage[8 * w]), s.masks[w], kBarFirst + static_cast<uint32_t>(w));
                        fence_proxy_async_smem();
                    }
                    tc_fence_before();
                    mbar_arrive(&s.p_first[w]);
                }
                tc_fence_before();
                mbar_arrive(&s.p_last[w]);
            }
            kt += max(n, it.n[1 - w]);

            // ---------------- the query tile's rows ----------------
            if (ok) ok = all(wait(s.pv_done[w], i - 1, kWaitSoftmax));
            // The sum goes where this thread has read the other's maximum (the two sums are added, either way round): this
            // thread's own maximum may not have been read yet.
            s.half[w][1 - part][row] = l;
            ok = named_bar_and(bar_tile, kRowThreads, ok);                // the warps meet again: give up together
            if (!ok) break;
            {
                tc_fence_after();
                l = s.half[w][0][row] + s.half[w][1][row];
                const float f = l != 0.0f ? 1.0f / l : 0.0f;
                float check[4] = {l * 0.0f, 0.0f, 0.0f, 0.0f};            // 0, or NaN
                // 32 columns at a time through shared memory, so that four lanes write a row's piece together
                uint4* stage = s.stage[warp];
                const int piece = static_cast<int>(lane) & 3;             // eight columns
                const int first = it.tok + w * a.tile_tokens;
                const int rows = min(a.tile_tokens, len - first) * a.group;
                const long long row0 = static_cast<long long>(it.begin + first) * a.Hq + it.h * a.group;
                T* to[4];                                                 // this lane's four rows (null: none)
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int rr = static_cast<int>(quad) * 32 + y * 8 + (static_cast<int>(lane) >> 2);
                    const int rt = rr / a.group;
                    to[y] = rr >= rows ? nullptr
                                       : static_cast<T*>(a.out) + (row0 + static_cast<long long>(rt) * a.Hq + (rr - rt * a.group)) * D +
                                             part * (D / 2) + piece * 8;
                }
#pragma unroll
                for (int c = 0; c < D / 2; c += 32) {
                    float o[32];
                    tmem_ld32(tO + c, reinterpret_cast<uint32_t*>(o));
                    tmem_wait_ld32(reinterpret_cast<uint32_t*>(o));
                    if (c + 32 == D / 2) {
                        tc_fence_before();
                        mbar_arrive(&s.o_empty[w]);
                    }
                    __syncwarp();                                         // the columns before have been read
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            check[e & 3] = fmaf(o[8 * x + e], 0.0f, check[e & 3]);
                            o[8 * x + e] *= f;
                        }
                        stage[lane * 4 + (x ^ ((lane >> 1) & 3))] = pack8(o + 8 * x, T{});
                    }
                    __syncwarp();
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int from = y * 8 + (static_cast<int>(lane) >> 2);
                        if (to[y]) *reinterpret_cast<uint4*>(to[y] + c) = stage[from * 4 + (piece ^ ((from >> 1) & 3))];
                    }
                }
                if (valid && a.lse && part == 0)
                    a.lse[static_cast<long long>(it.begin + tok) * a.Hq + it.h * a.group + (row - row_tok * a.group)] = lse_of(m2, l);
                // a row that is not finite: the tile is done again (before the item is given up, so that the
                // loading warp learns of it in time)
                if (!redo) {
                    const bool fine = !valid || check[0] + check[1] + check[2] + check[3] == 0.0f;
                    if (!named_bar_and(bar_tile, kRowThreads, fine) && row == 0 && part == 0) {
                        const unsigned int at = s.redo_count[w];
                        s.redo[w][at % kRedo] = it.id;
                        __threadfence_block();
                        *reinterpret_cast<volatile unsigned int*>(&s.redo_count[w]) = at + 1;
                    }
                }
                mbar_arrive(&s.item_empty[count % kAhead]);
            }
        }
    }

    // ---------------- tokens outside every sequence ----------------
    if (warp < kWarpLoad) {
        const int begin = a.plan->begin, end = a.plan->end;
        const int outside = begin + (a.T - end);
        for (int x = blockIdx.x * static_cast<int>(kWarpLoad) + static_cast<int>(warp); x < outside; x += gridDim.x * static_cast<int>(kWarpLoad)) {
            const long long t = x < begin ? x : end + (x - begin);
            uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + t * a.Hq * D);
            for (int y = static_cast<int>(lane); y < a.Hq * (D / 8); y += 32) dst[y] = make_uint4(0u, 0u, 0u, 0u);
            if (a.lse)
                for (int y = static_cast<int>(lane); y < a.Hq; y += 32) a.lse[t * a.Hq + y] = -INFINITY;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
template <typename T, int D>
dspark_status launch_typed(const void* q, const void* k, const void* v, long long q_stride, long long k_stride,
                           long long v_stride, const PromptArgs& a, int grid, cudaStream_t stream) {
    const uint64_t e = sizeof(T);
    CUtensorMap mq, mk, mv;
    const uint64_t qd[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(a.Hq), static_cast<uint64_t>(a.T)};
    const uint64_t kd[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(a.Hkv), static_cast<uint64_t>(a.T)};
    const uint64_t qs[2] = {D * e, q_stride * e}, ks[2] = {D * e, k_stride * e}, vs[2] = {D * e, v_stride * e};
    const uint32_t qb[3] = {64, static_cast<uint32_t>(a.group), static_cast<uint32_t>(a.tile_tokens)};
    const uint32_t kb[3] = {64, 1, kTile};
    if (!make_tensor_map(&mq, HalfType<T>::kMapType, 3, q, qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tensor_map(&mk, HalfType<T>::kMapType, 3, k, kd, ks, kb, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tensor_map(&mv, HalfType<T>::kMapType, 3, v, kd, vs, kb, CU_TENSOR_MAP_SWIZZLE_128B))
        return DSPARK_ERR_CUDA;
    prompt_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return cuda_error(err, "launch(prompt_attention plan)");
    constexpr size_t kSmem = sizeof(PromptSmem<D>);
    static_assert(kSmem <= 227 * 1024, "shared memory of one SM");
    err = cudaFuncSetAttribute(prompt_attention_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(kSmem));
    if (err == cudaSuccess)
        err = launch_dependent(prompt_attention_kernel<T, D>, dim3(grid), dim3(kThreads), kSmem, stream, mq, mk, mv, a);
    if (err != cudaSuccess) return cuda_error(err, "launch(prompt_attention)");
    return DSPARK_OK;
}

// Items, without the heads, of T tokens in B sequences with at most `heads` query heads to a key head.
long long items_bound(int B, int T, int heads) {
    const int tokens = 2 * (kTile / std::min(heads, kTile));
    return static_cast<long long>(B) + T / tokens;
}

}  // namespace

size_t prompt_attention_workspace_bytes(int B, int T, int Hq) {
    if (B < 1 || T < 1 || Hq < 1) return 0;
    return sizeof(Plan) + static_cast<size_t>(items_bound(B, T, Hq)) * sizeof(int4);
}

dspark_status launch_prompt_attention(const void* q, const void* k, const void* v, dspark_dtype dtype,
                                      long long q_stride, long long k_stride, long long v_stride,
                                      const int32_t* cu_seqlens, float scale, int causal, int B, int T, int Hq,
                                      int Hkv, int D, void* out, float* lse, void* ws, cudaStream_t stream,
                                      const DeviceInfo& dev) {
    PromptArgs a{};
    a.cu_seqlens = cu_seqlens;
    a.causal = causal;
    a.B = B;
    a.T = T;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.group = Hq / Hkv;
    a.tile_tokens = kTile / a.group;
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    a.plan = static_cast<Plan*>(ws);
    a.items = reinterpret_cast<int4*>(static_cast<uint8_t*>(ws) + sizeof(Plan));
    a.timeout_ns = kDefaultTimeoutNs;
    if (items_bound(B, T, a.group) * Hkv >= (1ll << 30)) {
        set_error("prompt_attention: too much work for one call (B=%d T=%d Hq=%d Hkv=%d)", B, T, Hq, Hkv);
        return DSPARK_ERR_UNSUPPORTED;
    }
    if (dtype == DSPARK_BF16)
        return D == 64 ? launch_typed<__nv_bfloat16, 64>(q, k, v, q_stride, k_stride, v_stride, a, dev.sm_count, stream)
                       : launch_typed<__nv_bfloat16, 128>(q, k, v, q_stride, k_stride, v_stride, a, dev.sm_count, stream);
    return D == 64 ? launch_typed<__half, 64>(q, k, v, q_stride, k_stride, v_stride, a, dev.sm_count, stream)
                   : launch_typed<__half, 128>(q, k, v, q_stride, k_stride, v_stride, a, dev.sm_count, stream);
}

}  // namespace dspark
