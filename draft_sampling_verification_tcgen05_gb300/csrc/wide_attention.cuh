// Masked attention over a paged cache where the rows of a key head fill more than one tile (a tree of 64 nodes with four
// query heads to a key head, a chunk of a prompt): a unit is two row tiles of 128 rows, so keys and values are loaded
// once for 256 rows, and while one tile's scores go through the softmax, the tensor cores work for the other.  Units,
// runs, partial results, plan and join are those of paged_attention.cuh.
//
//   warps 0-7, 8-15  softmax and results of one row tile each: two threads per row, 64 of a key tile's tokens each
//   warp 16          walks the run's segments and loads (TMA) queries, and page by page keys
//   warp 19          loads the values (with pages of 16 a tile is 16 boxes, whose issue takes 1300 cycles: one warp for both
//                    loads was slower than the products, by 7 % for 16 trees of up to 64 nodes over 500 to 8000 tokens)
//   warps 17, 18     issue S = Q K^T and O += P V of one row tile each on tcgen05 (M = 128, fp32 in tensor memory; P
//                    replaces half of S)
//
// Maxima, rounding and infinities are handled as in paged_attention.cuh; where a result is not finite, the CTA goes
// through its run again, once for each row tile, as the values' infinities are taken out for its rows.
//
// Bound by the chain scores -> softmax -> product of a key tile, of which the two row tiles hide each other's: 1.8 us for
// both (the products alone are 1.0), and by a unit's ends, about 4 us: the last product, the results, the next unit's first scores.
// Two chunks of 4096 tokens with a window of 1024, 32 on 8 heads of 128 (140 GFLOP): 193 us, 0.72 PFLOP/s counted, the
// tensor pipe at 43 % of its cycles since the tiles at the windows' ends are computed whole; 186 where the output's memory
// is one that the call before has written too, and then 256 with one row tile at a time.  16 trees of 64 nodes over 500 to 8000
// tokens: 72, and 76 with one row tile at a time.  More sizes of both are in masked_attention.cu.
#pragma once

#include "paged_attention.cuh"

namespace dspark {
namespace {

namespace wide {

constexpr int kThreads = 640;
constexpr int kRowThreads = 256;           // softmax threads of a row tile: two to a row, 64 of a key tile's tokens each
constexpr int kAhead = 4;                  // segments between the loads and the results
constexpr int kSlots = 2;                  // key tiles, and value tiles, in flight
constexpr uint32_t kColS = 0, kColP = 64, kColO = 256, kTmemCols = 512;    // S and O of tile 1: + 128
constexpr uint32_t kWarpLoad = 16, kWarpMma = 17, kWarpValues = 19;
// named barriers: + row tile; + 4 * row tile + quadrant, the two warps of the same rows; + row tile
constexpr uint32_t kBarTile = 1, kBarRows = 3, kBarFirst = 11;
constexpr uint32_t kWaitLoad = 0x811, kWaitMma = 0x812, kWaitSoftmax = 0x813;

// A segment as the roles see it: n key tiles for each row tile that takes part (t0 = t1: the end of a pass).
struct Item {
    Segment<true> g;
    int n[2];
};

template <int D>
struct Smem {
    static constexpr int kHalves = D / 64;                        // 128-byte column blocks
    static constexpr uint32_t kBlockBytes = kTile * 128;
    static constexpr uint32_t kTileBytes = kHalves * kBlockBytes;
    alignas(1024) uint8_t q[2][kTileBytes];
    alignas(1024) uint8_t k[kSlots][kTileBytes];
    alignas(1024) uint8_t v[kSlots][kTileBytes];
    alignas(1024) uint4 stage[16][128];                           // 32 columns of a warp's rows; a row of values in a later pass
    Item item[kAhead];
    float half[2][2][kTile];                                      // by row tile and half of the key tiles: a row's largest score, at last its sum
    uint8_t token_of[kTile];                                      // of a row tile's rows
    uint32_t masks[2][4];
    PagedArgs args;                                               // for functions out of line: the kernel's own are slower to read through a reference
    uint32_t again, failed;                                       // further passes are needed / a wait gave up
    uint64_t item_full[kAhead], item_empty[kAhead];
    uint64_t q_full[2], q_empty[2];
    uint64_t k_full[kSlots], k_empty[kSlots], v_full[kSlots], v_empty[kSlots];
    uint64_t s_full[2], p_first[2], p_last[2], pv_done[2], o_empty[2], turn[2], drain;
    uint32_t tmem_base;
};

// 32 lanes x 32 bits, 8 consecutive columns from r[0..7].
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Which of the 64 tokens from j on row `tok` sees.  Out of line, and called where little else is alive: it is needed in few
// tiles, and the softmax has no registers to spare.
inline __device__ __noinline__ uint2 row_bits(const PagedArgs& a, const Segment<true>& g, int tok, bool valid, int j) {
    SeenBits<64> sees;
    RowMask<true>(a, g, tok, valid).get(a, j, sees);
    return make_uint2(sees.word[0], sees.word[1]);
}

}  // namespace wide

// The results of row tile w of a segment, to `out` or as a partial one, with m2 the rows' maxima and their sums in s.half; use:
// that of pv_done by the last product.  Returns 1 where a row is not finite, -1 where the wait gave up.  Out of line: it is run
// once per unit, and its registers would be missing in the loop over the key tiles.
template <typename T, int D>
__device__ __noinline__ int tile_results(const PagedArgs& a, wide::Smem<D>& s, const Segment<true>& g, int w, float m2, int use) {
    const uint32_t warp = warp_id(), lane = lane_id(), quad = warp & 3u;
    const int part = static_cast<int>(warp >> 2) & 1, row = static_cast<int>(quad * 32u + lane), row_tok = row / a.group;
    const uint32_t tO = s.tmem_base + ((quad * 32u) << 16) + wide::kColO + w * 128u + part * (D / 2u);
    const int first = g.rt * a.unit_tokens + w * a.tile_tokens;
    const bool valid = row < a.tile_tokens * a.group && first + row_tok < g.n;
    // What does not need O comes before the wait for its last product.
    const float l = s.half[w][0][row] + s.half[w][1][row];
    const bool whole = g.t0 == 0 && g.t1 == g.tiles;
    const float f = whole ? (l != 0.0f ? 1.0f / l : 0.0f) : 1.0f;
    float check[4] = {l * 0.0f, 0.0f, 0.0f, 0.0f};                        // 0, or NaN
    uint4* stage = s.stage[warp];
    const int rows = min(a.tile_tokens, g.n - first) * a.group;
    const long long row0 = (static_cast<long long>(g.b) * a.N + first) * a.Hq + g.h * a.group;
    const long long part_base = static_cast<long long>(2 * blockIdx.x + (g.t0 == 0 ? 1 : 0)) * a.rows_cap + w * a.tile_tokens * a.group;
    if (valid && part == 0) {
        if (!whole) reinterpret_cast<float2*>(a.part_ml)[part_base + row] = make_float2(m2, l);
        else if (a.lse) a.lse[row0 + static_cast<long long>(row_tok) * a.Hq + (row - row_tok * a.group)] = lse_of(m2, l);
    }
    const int at0 = static_cast<int>(lane) >> 2, piece = static_cast<int>(lane) & 3;
    int to_row[4];                                            // of this lane's rows of a store, from the tile's first
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int rr = static_cast<int>(quad) * 32 + at0 + 8 * x, rt = s.token_of[rr];
        to_row[x] = rr >= rows ? -1 : whole ? (rt * a.Hq + (rr - rt * a.group)) * D : rr * D;
    }
    if (!__all_sync(0xFFFFFFFFu, mbar_wait_short(&s.pv_done[w], static_cast<uint32_t>(use) & 1u, &a.plan->header, a.timeout_ns, wide::kWaitSoftmax)))
        return -1;
    tc_fence_after();
    // Through shared memory, 64 bytes of each row at a time, so that a store's lanes write whole pieces of eight rows.
    auto put = [&](int x, uint4 v) { stage[lane * 4 + (x ^ ((lane >> 1) & 3))] = v; };
    auto of = [&](int at) { return stage[at * 4 + (piece ^ ((at >> 1) & 3))]; };
    if (whole) {
        T* out = static_cast<T*>(a.out) + row0 * D + part * (D / 2) + piece * 8;
#pragma unroll 1
        for (int c = 0; c < D / 2; c += 32) {
            uint32_t o[32];
            tmem_ld32(tO + c, o);
            tmem_wait_ld32(o);
            if (c + 32 == D / 2) {
                tc_fence_before();
                mbar_arrive(&s.o_empty[w]);
            }
            __syncwarp();                                     // the columns before have been read
#pragma unroll
            for (int x = 0; x < 32; ++x) {
                check[x & 3] = fmaf(__uint_as_float(o[x]), 0.0f, check[x & 3]);
                o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) put(x, pack8(reinterpret_cast<const float*>(o) + 8 * x, T{}));
            __syncwarp();
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (to_row[x] >= 0) *reinterpret_cast<uint4*>(out + to_row[x] + c) = of(at0 + 8 * x);
        }
    } else {
        float* out = a.part_o + part_base * D + part * (D / 2) + piece * 4;
#pragma unroll 1
        for (int c = 0; c < D / 2; c += 16) {
            uint32_t o[16];
            tmem_ld16(tO + c, o);
            tmem_wait_ld();
            if (c + 16 == D / 2) {
                tc_fence_before();
                mbar_arrive(&s.o_empty[w]);
            }
            __syncwarp();
#pragma unroll
            for (int x = 0; x < 16; ++x) check[x & 3] = fmaf(__uint_as_float(o[x]), 0.0f, check[x & 3]);
#pragma unroll
            for (int x = 0; x < 4; ++x) put(x, make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]));
            __syncwarp();
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (to_row[x] >= 0) *reinterpret_cast<uint4*>(out + to_row[x] + c) = of(at0 + 8 * x);
        }
    }
    return valid && check[0] + check[1] + check[2] + check[3] != 0.0f ? 1 : 0;
}

template <typename T, int D>
__global__ void __launch_bounds__(wide::kThreads, 1)
wide_attention_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PagedArgs a) {
    using namespace wide;
    using Smem = wide::Smem<D>;
    constexpr int kHalves = Smem::kHalves;
    constexpr uint32_t kBlockBytes = Smem::kBlockBytes, kTileBytes = Smem::kTileBytes;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem& s = *reinterpret_cast<Smem*>(smem_raw);
    const uint32_t warp = warp_id(), lane = lane_id();
    WsHeader* ws = &a.plan->header;

    if (threadIdx.x == 0) {
        for (int i = 0; i < wide::kAhead; ++i) {
            mbar_init(&s.item_full[i], 1);
            mbar_init(&s.item_empty[i], 2 * wide::kRowThreads + 3);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.q_full[i], 1);
            mbar_init(&s.q_empty[i], 1);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.turn[i], 1);
            mbar_init(&s.p_first[i], wide::kRowThreads);
            mbar_init(&s.p_last[i], wide::kRowThreads);
            mbar_init(&s.pv_done[i], 1);
            mbar_init(&s.o_empty[i], wide::kRowThreads);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&s.k_full[i], 1);
            mbar_init(&s.k_empty[i], 2);
            mbar_init(&s.v_full[i], 1);
            mbar_init(&s.v_empty[i], 2);
        }
        mbar_init(&s.drain, 2);
        s.again = s.failed = 0u;
        fence_mbarrier_init();
        prefetch_tensormap(&tmQ);
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (threadIdx.x == 32) s.args = a;
    if (threadIdx.x < kTile) s.token_of[threadIdx.x] = static_cast<uint8_t>(threadIdx.x / a.group);
    if (warp == kWarpMma) {
        tmem_alloc(&s.tmem_base, wide::kTmemCols);
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
    // Carried from pass to pass, each role for itself: items, key tiles, own key tiles, own row tiles, turns.
    int count = 0, kt = 0, i = 0, used = 0, turn = 0, qt[2] = {0, 0};
    // Pass 0 is all there is, as a rule; passes 1 and 2 take one row tile each.
    for (int pass = 0;; ++pass) {
        if (warp == kWarpLoad || warp == kWarpValues) {
            // ---------------- segments and loads ----------------
            const bool keys = warp == kWarpLoad;
            const CUtensorMap* map = keys ? &tmK : &tmV;
            uint8_t* ring = keys ? s.k[0] : s.v[0];
            uint64_t* full = keys ? s.k_full : s.v_full;
            uint64_t* empty = keys ? s.k_empty : s.v_empty;
            const uint64_t keep = l2_policy_evict_last();
            const int page_bits = __ffs(a.page) - 1;
            const int boxes = kTile / a.box_rows * kHalves;
            const int box = static_cast<int>(lane) / kHalves, half = static_cast<int>(lane) % kHalves;
            const uint32_t box_bytes = static_cast<uint32_t>(a.box_rows) * 128u;
            const uint32_t box_at = static_cast<uint32_t>(half) * kBlockBytes + static_cast<uint32_t>(box) * box_bytes;
            // this lane's box of tile t: its page (looked at only when it is used), -2: none, or -3: seen by no row
            auto lookup = [&](const Segment<true>& g, int t) {
                const int j = g.place(t) * kTile + box * a.box_rows;
                if (static_cast<int>(lane) >= boxes || j >= g.kv) return -2;
                if (g.skipped(a, j, j + a.box_rows)) return -3;
                return max(-1, a.block_table[static_cast<long long>(g.b) * a.max_pages + (j >> page_bits)]);
            };
            Walker<true> walk(a);
            Segment<true> g{};
            while (ok) {
                int n[2];
                if (keys) {
                    const bool more = walk.next(g);
                    for (int x = 0; x < 2; ++x) {
                        const int first = g.rt * a.unit_tokens + x * a.tile_tokens;
                        n[x] = more && first < g.n && (pass == 0 || pass == x + 1) ? g.t1 - g.t0 : 0;
                        // tiles behind what the row tile's last row sees are for the other alone; one is always there
                        if (n[x] > 0 && a.causal)
                            while (n[x] > 1 && g.place(g.t0 + n[x] - 1) * kTile >= g.kv - g.n + min(g.n, first + a.tile_tokens)) --n[x];
                    }
                    if (more && n[0] + n[1] == 0) continue;
                    ok = all(wait(s.item_empty[count % wide::kAhead], count / wide::kAhead + 1, wide::kWaitLoad));
                    if (!ok) break;
                    if (lane == 0) {
                        Item& it = s.item[count % wide::kAhead];
                        it.g = g;
                        it.n[0] = n[0];
                        it.n[1] = n[1];
                        mbar_arrive(&s.item_full[count % wide::kAhead]);
                    }
                    __syncwarp();
                } else {
                    ok = all(wait(s.item_full[count % wide::kAhead], count / wide::kAhead, wide::kWaitLoad));
                    if (!ok) break;
                    const Item& it = s.item[count % wide::kAhead];
                    g = it.g;
                    n[0] = it.n[0];
                    n[1] = it.n[1];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.item_empty[count % wide::kAhead]);
                }
                ++count;
                const int t1 = g.t0 + max(n[0], n[1]);
                if (t1 == g.t0) break;                        // the end of the pass
                int page = lookup(g, g.t0);
                for (int x = 0; keys && ok && x < 2; ++x) {
                    if (n[x] == 0) continue;
                    ok = all(wait(s.q_empty[x], qt[x] + 1, wide::kWaitLoad));
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&s.q_full[x], static_cast<uint32_t>(a.tile_tokens * a.group) * 128u * kHalves);
                        for (int y = 0; y < kHalves; ++y)
                            tma_load_3d(s.q[x] + y * kBlockBytes, &tmQ, y * 64, g.h * a.group,
                                        g.b * a.N + g.rt * a.unit_tokens + x * a.tile_tokens, &s.q_full[x], keep);
                    }
                    __syncwarp();
                    ++qt[x];
                }
                for (int t = g.t0; ok && t < t1; ++t, ++kt) {
                    const int next = t + 1 < t1 ? lookup(g, t + 1) : -2;
                    const int slot = kt % kSlots;
                    ok = all(wait(empty[slot], kt / kSlots + 1, wide::kWaitLoad));
                    if (!ok) break;
                    const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, page != -2)) * box_bytes;
                    if (lane == 0) mbar_arrive_expect_tx(&full[slot], bytes);
                    __syncwarp();
                    if (page != -2) {
                        const int y = (g.place(t) * kTile + box * a.box_rows) & (a.page - 1);
                        int z = page * a.Hkv + g.h;
                        if (page == -3) {
                            z = a.num_pages * a.Hkv;              // outside the map: reads zeros
                        } else if (page < 0 || page >= a.num_pages) {
                            flag_input_index(ws);
                            z = g.h;
                        }
                        tma_load_3d(ring + slot * kTileBytes + box_at, map, half * 64, y, z, &full[slot], keep);
                    }
                    page = next;
                }
            }
            if (keys) grid_dependency_launch();
            if (!ok) {
                // give copies in flight time to land before the block exits
                const long long t0 = global_ns();
                while (global_ns() - t0 < a.timeout_ns) {
                }
            }
        } else if (warp >= kWarpMma) {
            // ---------------- products of row tile w: the whole warp waits, one lane issues ----------------
            // The tensor cores run one tile's products in the order of issue, so S may be written as soon as the
            // product that read P (in S) has been issued.  The tiles take turns with the end of a product and the
            // next scores: then one tile's products run while the other is in its softmax.  The waits of a turn are
            // done before it, since one takes about as long as the tensor cores' queue lasts.
            const int w = static_cast<int>(warp - kWarpMma);
            constexpr uint32_t kIdescS = attn_idesc<T, false>(kTile, kTile);
            constexpr uint32_t kIdescO = attn_idesc<T, true>(kTile, D);
            constexpr uint32_t kStep = kTileBytes >> 4;           // a tile, in descriptor units
            const uint64_t q_desc = sw128_kmajor_desc(smem_u32(s.q[w]));
            const uint64_t k_desc = sw128_kmajor_desc(smem_u32(s.k[0]));
            const uint64_t v_desc = sw128_token_rows_desc(smem_u32(s.v[0]), kBlockBytes);
            const uint32_t tS = tmem + wide::kColS + w * 128u, tP = tmem + wide::kColP + w * 128u, tO = tmem + wide::kColO + w * 128u;
            auto take_turn = [&] {
                const bool mine = w == 0 ? turn == 0 || wait(s.turn[0], turn - 1, wide::kWaitMma) : wait(s.turn[1], turn, wide::kWaitMma);
                ++turn;
                return all(mine);
            };
            while (ok) {
                ok = all(wait(s.item_full[count % wide::kAhead], count / wide::kAhead, wide::kWaitMma));
                if (!ok) break;
                const Item& it = s.item[count % wide::kAhead];
                const int n = __shfl_sync(0xFFFFFFFFu, it.n[w], 0), other = __shfl_sync(0xFFFFFFFFu, it.n[1 - w], 0);
                // tokens that the request holds from the last of these tiles on
                const int held = __shfl_sync(0xFFFFFFFFu, it.g.kv - it.g.place(it.g.t0 + max(it.n[0], it.n[1]) - 1) * kTile, 0);
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.item_empty[count % wide::kAhead]);
                ++count;
                const int most = max(n, other);
                if (most == 0) break;
                // turn t: the end of the product of key tile t - 1 and the scores of key tile t
                for (int t = 0; t <= most; ++t) {
                    const uint64_t v = v_desc + static_cast<uint32_t>((kt + t - 1) % kSlots) * kStep;
                    const uint64_t k = k_desc + static_cast<uint32_t>((kt + t) % kSlots) * kStep;
                    // what is usually there comes first, the weights last
                    if (t < most) ok = all(wait(s.k_full[(kt + t) % kSlots], (kt + t) / kSlots, wide::kWaitMma));
                    if (ok && t == 0 && n > 0) ok = all(wait(s.q_full[w], used, wide::kWaitMma));
                    if (!ok) break;
                    if (t > 0) {
                        const int slot = (kt + t - 1) % kSlots;
                        ok = all(wait(s.v_full[slot], (kt + t - 1) / kSlots, wide::kWaitMma));
                        if (!ok) break;
                        if (t <= n) {
                            if (t == most && held < kTile) {      // behind the request's end nothing may count
                                const int pieces = (kTile - held) * 8;    // of 16 bytes, per block
                                for (int y = 0; y < kHalves; ++y)
                                    for (int x = static_cast<int>(lane); x < pieces; x += 32)
                                        *reinterpret_cast<uint4*>(s.v[slot] + y * kBlockBytes + held * 128 + x * 16) =
                                            make_uint4(0u, 0u, 0u, 0u);
                                fence_proxy_async_smem();
                                __syncwarp();
                            }
                            ok = all(wait(s.p_first[w], i, wide::kWaitMma) && (t > 1 || used == 0 || wait(s.o_empty[w], used - 1, wide::kWaitMma)));
                            if (!ok) break;
                            tc_fence_after();
                            const uint32_t onto = t == 1 && pass == 0 ? 0u : 1u;   // later, O starts from what is there
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
                    if (ok && t > 0 && t <= n) ok = all(wait(s.p_last[w], i++, wide::kWaitMma));
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
            while (!mbar_try_wait(&s.drain, pass & 1) && global_ns() - t0 < a.timeout_ns) {
            }
            __syncwarp();
        } else {
            // ---------------- softmax and results of row tile w ----------------
            const int w = static_cast<int>(warp >> 3);
            const int part = static_cast<int>(warp >> 2) & 1;  // 64 of the key tile's tokens, half of the output's columns
            const uint32_t quad = warp & 3u;
            const uint32_t bar_tile = kBarTile + static_cast<uint32_t>(w), bar_rows = kBarRows + 4u * static_cast<uint32_t>(w) + quad;
            const uint32_t lanes = (quad * 32u) << 16;
            const uint32_t tS = tmem + lanes + wide::kColS + w * 128u + part * 64u, tP = tmem + lanes + wide::kColP + w * 128u + part * 32u;
            const uint32_t tO = tmem + lanes + wide::kColO + w * 128u + part * (D / 2u);
            const int row = static_cast<int>(quad * 32u + lane);
            const int row_tok = row / a.group;
            const bool row_used = row < a.tile_tokens * a.group;
            const float sl2 = a.scale * kLog2e;
            const bool falling = sl2 < 0.0f;                          // the largest score is the smallest product
            const float none = falling ? INFINITY : -INFINITY;
            // A masked score is infinite and gets no weight by that, for which the slope must not be 0: the smallest step above
            // it (no product of finite values then reaches 2^-20) stands for a scale of 0.
            const float steep = sl2 == 0.0f ? 0x1p-149f : sl2;
            auto rows_of_pass = [&](auto later) {
            constexpr bool redo = decltype(later)::value;
            while (true) {
                ok = named_bar_and(bar_tile, wide::kRowThreads, ok && wait(s.item_full[count % wide::kAhead], count / wide::kAhead, wide::kWaitSoftmax));
                if (!ok) break;
                const Item& it = s.item[count % wide::kAhead];
                const int n = it.n[w];
                if (n == 0) {
                    const int other = it.n[1 - w];
                    kt += other;
                    mbar_arrive(&s.item_empty[count++ % wide::kAhead]);
                    if (other == 0) break;
                    continue;
                }
                const Segment<true>& g = it.g;
                const int first = g.rt * a.unit_tokens + w * a.tile_tokens;   // the tile's first window token
                const int tok = first + row_tok;
                const bool valid = row_used && tok < g.n;
                // tokens that every row of the tile sees: [from, to), and those below `sinks` as far as `to`
                const int base = g.kv - g.n, last = min(g.n, first + a.tile_tokens) - 1;
                const int to = a.parents ? base : a.causal ? base + first + 1 : g.kv;
                const int from = a.window > 0 ? base + (a.parents ? g.n - 1 : last) - a.window + 1 : 0;
                const int sinks = a.window > 0 ? a.sinks : 0;
                float m2 = -INFINITY, l = 0.0f;
                for (int t = 0; t < n; ++t, ++i) {
                    const int j = g.place(g.t0 + t) * kTile;
                    const bool masked = j + kTile > to || (j < from && j + kTile > sinks);
                    uint2 sees = make_uint2(0xFFFFFFFFu, 0xFFFFFFFFu);
                    if (masked) sees = row_bits(s.args, g, tok, valid, j + part * 64);
                    bool go = wait(s.s_full[w], i, wide::kWaitSoftmax);
                    if (redo) go = named_bar_and(bar_tile, wide::kRowThreads, go);  // these meet in barriers below
                    go = all(go);
                    // 64 scores in registers
                    uint32_t r[2][32];
                    tc_fence_after();
                    tmem_ld32(tS, r[0]);
                    tmem_ld32(tS + 32, r[1]);
                    tmem_wait_ld32(r[0]);
                    tmem_wait_ld32(r[1]);
                    if (masked) {                             // an infinite score has no weight
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            if (!(((c < 32 ? sees.x : sees.y) >> (c & 31)) & 1u)) r[c >> 5][c & 31] = __float_as_uint(none);
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
                        if (t > 0) go = go && all(wait(s.pv_done[w], i - 1, wide::kWaitSoftmax));
                        ok = named_bar_and(bar_rows, 64, go);
                        if (!ok && !redo) break;                          // else at the vote below
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
                    const float2 slope = make_float2(steep, steep), shift = make_float2(-ref, -ref);
                    // 32 weights, to P: one straight piece of code, for which the compiler finds an order that keeps the
                    // exponential's unit (4 cycles a warp) at work.
                    auto weigh = [&](int x) {
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            uint32_t p[8];
#pragma unroll
                            for (int c = 16 * z; c < 16 * z + 16; c += 2) {
                                const float2 y = __ffma2_rn(make_float2(__uint_as_float(r[x][c]), __uint_as_float(r[x][c + 1])), slope, shift);
                                const float2 e = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                                sum[(c >> 1) & 1] = __fadd2_rn(sum[(c >> 1) & 1], e);
                                p[(c >> 1) & 7] = pack2(e.x, e.y, T{});
                            }
                            tmem_st8(tP + x * 16 + z * 8, p);
                        }
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
                        bool there = ok && wait(s.v_full[slot], (kt + t) / kSlots, wide::kWaitSoftmax);
                        // O is about to be changed here: the products before must be complete
                        if (there && t > 0) there = wait(s.pv_done[w], i - 1, wide::kWaitSoftmax);
                        there = all(there);
                        if (there && t == 0) {
                            uint32_t zero[16];
#pragma unroll
                            for (int c = 0; c < 16; ++c) zero[c] = 0u;
                            for (uint32_t c = 0; c < D / 2; c += 16) tmem_st16(tO + c, zero);
                            tmem_wait_st();
                        }
                        tc_fence_before();
                        ok = named_bar_and(bar_tile, wide::kRowThreads, there);     // P and O of both halves are in place
                        if (!ok) break;
                        tc_fence_after();
                        if (part == 0) {
                            // the row's mask over the whole tile: this thread has its first half
                            SeenBits<128> whole;
                            whole.all();
                            if (masked) {
                                const uint2 other = row_bits(s.args, g, tok, valid, j + 64);
                                whole.word[0] = sees.x;
                                whole.word[1] = sees.y;
                                whole.word[2] = other.x;
                                whole.word[3] = other.y;
                            }
                            move_infinities<T>(s.v[slot], kBlockBytes, kHalves, row, g.kv - j, [=](int x) { return whole.at(x); }, tP, tO,
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

                // ---------------- the tile's rows ----------------
                // The sum goes where this thread has read the other's maximum (the two sums are added, either way round):
                // this thread's own maximum may not have been read yet.
                s.half[w][1 - part][row] = l;
                ok = named_bar_and(bar_tile, wide::kRowThreads, ok);      // the warps meet again: give up together
                if (!ok) break;
                const int done = tile_results<T, D>(s.args, s, g, w, m2, i - 1);
                ok = done >= 0;
                if (!ok) continue;                                        // to the vote above
                if (!redo && done > 0) s.again = 1u;
                __syncwarp();
                mbar_arrive(&s.item_empty[count++ % wide::kAhead]);
            }
            };
            if (pass == 0) rows_of_pass(std::false_type{});
            else rows_of_pass(std::true_type{});
        }
        if (!ok) s.failed = 1u;
        __syncthreads();
        const bool stop = pass == 2 || s.again == 0u || s.failed != 0u;
        __syncthreads();                       // everyone has read them before the next pass may write them
        if (stop) break;
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, wide::kTmemCols);
    }
}

template <typename T, int D>
dspark_status launch_wide(PagedArgs& a, int grid, cudaStream_t stream) {
    constexpr size_t kSmem = sizeof(wide::Smem<D>);
    static_assert(kSmem <= 227 * 1024, "shared memory of one SM");
    a.unit_tokens = std::min(a.N, 2 * a.tile_tokens);
    PagedMaps m;
    if (!make_maps<T, D>(a, m)) return DSPARK_ERR_CUDA;
    const dspark_status st = launch_plan<true>(a, grid, stream);
    if (st != DSPARK_OK) return st;
    cudaError_t err = cudaFuncSetAttribute(wide_attention_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    if (err == cudaSuccess)
        err = launch_dependent(wide_attention_kernel<T, D>, dim3(grid), dim3(wide::kThreads), kSmem, stream, m.q, m.k, m.v, a);
    if (err != cudaSuccess) return cuda_error(err, "launch(wide_attention)");
    return launch_join<T, D, true>(a, grid, stream);
}

}  // namespace
}  // namespace dspark
