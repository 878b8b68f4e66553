// Attention of a window of new tokens per request over a paged key-value cache.
//
// A unit is one (request, key head, tile of window rows): the G query heads that share the key
// head, for as many window tokens as fit, are the up to 128 rows of one tensor-core tile, so each
// cached key and value is read from memory once for all of them.  A unit's work is its request's
// cache in tiles of 128 tokens; all units' tiles, laid end to end with a few more
// steps ahead of each unit (what starting and ending it costs), are cut into equal runs, one per CTA
// (persistent, one per SM), wherever the cuts fall.  A run's piece of a unit ("segment")
// that is not the whole unit leaves its unnormalised sums in the workspace, and a second kernel
// joins them in the order of the CTAs.  The order of every sum is fixed by the sizes alone.
//
//   warp 0      walks the run's segments, opens them to the other warps, loads (TMA) the query tile of
//               each and, page by page, the key tiles
//   warp 1      loads the value tiles
//   warp 2      issues S = Q K^T on tcgen05 (M = 128 rows, fp32 scores in tensor memory, two tiles)
//   warp 3      issues O += P V (fp32 sums in tensor memory)
//   warps 4-7   softmax: a thread per tensor-memory lane, running maximum and sum in fp32,
//               weights rounded to the cache's type into tensor memory (P, two tiles)
//   warps 8-11  (with several copies of the rows, see below) read O at a segment's end, add the
//               copies and write them while the next segment runs; with one copy the softmax
//               warps write O themselves
// The two products have a warp each because issuing one (8 instructions and their commits) takes
// about as long as a tile's loads at the memory's rate.
//
// With few rows the 128 lanes hold the rows several times over ("parts"): 4 copies of up to 32
// rows, or 2 of up to 64.  Copy k exponentiates only the k-th part of each tile's tokens and its
// P is zero elsewhere, so the copies are independent partial sums, added in the epilogue.
//
// The running maximum is raised only when a tile exceeds it by 2^8 (O, in tensor memory, is then
// rescaled): weights up to 2^8 lose nothing in a floating type, and the rescaling leaves the
// common path.  In fp16 the exponentials' reference is 2^7 below it (kHeadroom).
//
// A row must not see what lies outside its limit, but 0 * infinity is not 0.  Values past the
// request's end are zeroed in shared memory before the product (by the warp that issues it, while
// the softmax is still at work).  Where a row's result is not finite,
// the CTA goes through its run a second time with the infinities and NaN taken out of every value
// tile and added to the rows that see them; nothing else changes in that pass, so rows that do not
// see them come out bit for bit as without them.
//
// Bound by the cache's bytes where they are many: 5 requests over 70000 to 131071 tokens, 8 key heads of
// 128 (1.83 GB), take 268 us, the copy's 6.8 TB/s; 64 windows of 17 tokens over 100 to 8000 (629 MB)
// 118 us, 5.3 TB/s, where a tile's softmax over 68 rows (two copies do not fit) is nearly as long as
// its loads.  200 blocks of 8 tokens over 9 to 2000 (85 MB, D = 64) take 31 us: a unit of three tiles
// is bound by its way through the products and the softmax.  One token over 4097 takes 14.5 us, most of
// it the three kernels' starts and the chain from the plan to the join.
#include "attention_common.cuh"
#include "host_common.h"

#include <algorithm>

namespace dspark {
namespace {

constexpr int kTile = 128;                 // cached tokens per tile, and MMA rows
constexpr int kRowThreads = 128;           // softmax threads; result threads
constexpr int kAhead = 8;                  // segments between the loads and the results
constexpr int kMaxCtas = 160;
constexpr float kRaise = 8.0f;             // log2 units
constexpr uint32_t kColS = 0, kColP = 256, kColO = 384, kTmemCols = 512;
constexpr uint32_t kWaitLoad = 0x801, kWaitMma = 0x802, kWaitSoftmax = 0x803, kWaitEpilogue = 0x804;

struct PlanEntry {
    int b, kv, n;                          // the request that CTA c's run begins in, and its lengths
    int joined;                            // partial results to join: the unit cut by this run's beginning, if
    int rt, h;                             // this is the unit's first cut (else 0), its row tile and key head
    int pad[2];
    long long off, left;                   // steps into the request's units, and steps of the run
    long long pad2[2];
};

struct Plan {
    WsHeader header;
    int ctas;                              // CTAs with a run
    int pad[63];
    PlanEntry entry[kMaxCtas];
};
static_assert(sizeof(PlanEntry) == 64 && sizeof(Plan) % 256 == 0, "aligned entries, aligned partial results behind them");

struct PagedArgs {
    const void *q, *k_cache, *v_cache;
    const int32_t *block_table, *kv_len, *lengths;
    int max_pages, causal, B, N, Hq, Hkv, group, num_pages, page;
    int box_rows;                          // tokens of one TMA box: min(page, 128)
    int tile_tokens;                       // window tokens per row tile
    int rows_cap;                          // rows of one partial result
    float scale;
    void* out;
    float* lse;
    Plan* plan;
    float *part_ml, *part_o;
    long long timeout_ns;
};

// Cached tokens and window tokens of request b (none where the caller's value is out of range).
__device__ __forceinline__ bool request(const PagedArgs& a, int b, int& kv, int& n) {
    kv = a.kv_len[b];
    n = a.lengths ? a.lengths[b] : a.N;
    const bool ok = kv >= 0 && kv <= static_cast<long long>(a.max_pages) * a.page && n >= 0 && n <= a.N;
    if (!ok || kv == 0 || n == 0) kv = n = 0;
    return ok;
}

__device__ __forceinline__ int tiles_of(int kv) { return (kv + kTile - 1) / kTile; }
__device__ __forceinline__ int row_tiles_of(const PagedArgs& a, int n) { return (n + a.tile_tokens - 1) / a.tile_tokens; }

// Steps of a unit: kUnitSteps to start and end it, then its tiles.
constexpr int kUnitSteps = 3;
__device__ __forceinline__ int steps_of(int tiles) { return tiles + kUnitSteps; }
__device__ __forceinline__ long long request_steps(const PagedArgs& a, int kv, int n) {
    return n == 0 ? 0 : static_cast<long long>(row_tiles_of(a, n)) * a.Hkv * steps_of(tiles_of(kv));
}

// First step of CTA c's run, and the CTA whose run holds step w.
__device__ __forceinline__ long long run_start(long long total, int ctas, int c) {
    return ctas == 0 ? 0 : quotient(c * total, ctas);
}
__device__ __forceinline__ int run_of(long long total, int ctas, long long w) {
    return static_cast<int>(quotient((w + 1) * ctas - 1, total));
}

// One segment: tiles [t0, t1) of unit (b, rt, h), whose request has `tiles` tiles.
struct Segment {
    int b, rt, h, kv, n, tiles, t0, t1;
};

// The segments of this CTA's run.  The lengths of the request after the current one are loaded ahead.
struct Walker {
    const PagedArgs& a;
    int b, kv, n, next_kv, next_n;
    long long off, left;
    __device__ explicit Walker(const PagedArgs& args) : a(args) {
        const PlanEntry& e = a.plan->entry[blockIdx.x];
        const int4 head = *reinterpret_cast<const int4*>(&e);
        const longlong2 run = *reinterpret_cast<const longlong2*>(&e.off);
        b = head.x;
        kv = head.y;
        n = head.z;
        off = run.x;
        left = run.y;
        next_kv = next_n = 0;
        if (left > 0 && b + 1 < a.B) request(a, b + 1, next_kv, next_n);
    }
    __device__ bool next(Segment& s) {
        while (left > 0 && b < a.B) {
            const long long work = request_steps(a, kv, n);
            if (off >= work) {
                off -= work;
                ++b;
                kv = next_kv;
                n = next_n;
                if (b + 1 < a.B) request(a, b + 1, next_kv, next_n);
                continue;
            }
            s.tiles = tiles_of(kv);
            const int steps = steps_of(s.tiles);
            const int unit = static_cast<int>(quotient(off, steps));
            const int from = static_cast<int>(off - static_cast<long long>(unit) * steps);
            const int take = static_cast<int>(min(static_cast<long long>(steps - from), left));
            off += take;
            left -= take;
            s.t0 = max(0, from - kUnitSteps);
            s.t1 = from + take - kUnitSteps;
            if (s.t1 <= s.t0) continue;                    // the run ends before the unit's first tile
            s.b = b;
            s.kv = kv;
            s.n = n;
            s.rt = unit / a.Hkv;
            s.h = unit - s.rt * a.Hkv;
            return true;
        }
        return false;
    }
};

// ---------------------------------------------------------------------------
// Plan: one block.  Clears the status word, checks the lengths, and finds where each CTA's equal
// share of the tiles begins.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(PagedArgs a, int grid) {
    __shared__ long long s_warp[kPlanThreads / 32];
    __shared__ long long s_total, s_end[kPlanThreads];
    Plan* p = a.plan;
    const int tid = threadIdx.x;
    grid_dependency_launch();                              // the attention kernel sets itself up meanwhile
    if (tid < 64) reinterpret_cast<uint32_t*>(&p->header)[tid] = 0u;
    __syncthreads();

    auto work_of = [&](int b) -> long long {
        int kv, n;
        if (b >= a.B) return 0;
        if (!request(a, b, kv, n)) flag_input_index(&p->header);
        return request_steps(a, kv, n);
    };
    // inclusive scan of one value per thread; s_total receives the block's sum
    auto scan = [&](long long x) {
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(0xFFFFFFFFu, x, d);
            if (lane_id() >= static_cast<uint32_t>(d)) x += y;
        }
        __syncthreads();
        if (lane_id() == 31) s_warp[warp_id()] = x;
        __syncthreads();
        if (warp_id() == 0) {
            long long w = s_warp[lane_id()];
            for (int d = 1; d < 32; d <<= 1) {
                const long long y = __shfl_up_sync(0xFFFFFFFFu, w, d);
                if (lane_id() >= static_cast<uint32_t>(d)) w += y;
            }
            s_warp[lane_id()] = w;
            if (lane_id() == 31) s_total = w;
        }
        __syncthreads();
        return x + (warp_id() > 0 ? s_warp[warp_id() - 1] : 0);
    };

    long long total = 0, first = 0;                        // first: this thread's end among the first requests
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
        const long long end = scan(work_of(b0 + tid));
        if (b0 == 0) first = end;
        total += s_total;
    }
    const int ctas = static_cast<int>(min(static_cast<long long>(grid), total));
    if (tid == 0) p->ctas = ctas;
    // thread c looks for the request that its CTA's run begins in, among 1024 requests at a time
    const long long at = tid < ctas ? run_start(total, ctas, tid) : -1;
    if (tid >= ctas && tid < grid) p->entry[tid].left = 0;
    long long before = 0;
    for (int b0 = 0; b0 < a.B && ctas > 0; b0 += kPlanThreads) {
        s_end[tid] = a.B <= kPlanThreads ? first : before + scan(work_of(b0 + tid));
        __syncthreads();
        const long long end = before + s_total;
        if (at >= before && at < end) {
            int lo = 0, hi = min(kPlanThreads, a.B - b0) - 1;      // the first request that ends behind `at`
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                if (s_end[mid] > at) hi = mid; else lo = mid + 1;
            }
            PlanEntry e{};
            e.b = b0 + lo;
            request(a, e.b, e.kv, e.n);
            e.off = at - (lo > 0 ? s_end[lo - 1] : before);
            e.left = run_start(total, ctas, tid + 1) - at;
            const int steps = steps_of(tiles_of(e.kv));
            const int unit = static_cast<int>(quotient(e.off, steps));
            const int from = static_cast<int>(e.off - static_cast<long long>(unit) * steps);
            const long long w0 = at - from;                // the unit's first step
            e.rt = unit / a.Hkv;
            e.h = unit - e.rt * a.Hkv;
            // a cut between two of the unit's tiles, and none before it: CTAs tid - 1 .. the unit's last
            if (from > kUnitSteps && w0 + kUnitSteps >= run_start(total, ctas, tid - 1))
                e.joined = run_of(total, ctas, w0 + steps - 1) - tid + 2;
            p->entry[tid] = e;
        }
        before = end;
    }
}

template <int D, int kParts>
struct PagedCfg {
    static constexpr int kThreads = kParts == 1 ? 256 : 384;
    static constexpr int kHalves = D / 64;                        // 128-byte column blocks
    static constexpr uint32_t kBlockBytes = kTile * 128;          // one block of a tile
    static constexpr uint32_t kTileBytes = kHalves * kBlockBytes;
    static constexpr int kSlots = D == 64 ? 5 : 2;                // key tiles, and value tiles, in flight
};

template <int D, int kParts>
struct PagedSmem {
    using Cfg = PagedCfg<D, kParts>;
    alignas(1024) uint8_t k[Cfg::kSlots][Cfg::kTileBytes];
    alignas(1024) uint8_t v[Cfg::kSlots][Cfg::kTileBytes];
    alignas(1024) uint8_t q[2][Cfg::kTileBytes];
    alignas(1024) float4 stage[kTile * 8];         // 32 columns of all lanes
    float2 ml[kParts == 1 ? 1 : kAhead][kTile];    // maximum and sum of each lane, by segment
    Segment seg[kAhead];
    float row[D];
    uint32_t masks[4];
    uint32_t again, failed;                // a second pass is needed / a wait gave up
    uint64_t k_full[Cfg::kSlots], k_empty[Cfg::kSlots], v_full[Cfg::kSlots], v_empty[Cfg::kSlots];
    uint64_t seg_full[kAhead], seg_empty[kAhead];
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], s_free[2], p_ready[2], stat_full[kAhead];
    uint64_t pv_done[2];                   // by the tile's parity: O += P V of that tile is complete
    uint64_t o_empty, drain[2];
    uint32_t tmem_base;
};

template <typename T, int D, int kParts>
__global__ void __launch_bounds__(PagedCfg<D, kParts>::kThreads, 1)
paged_attention_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PagedArgs a) {
    using Cfg = PagedCfg<D, kParts>;
    constexpr int kSlots = Cfg::kSlots, kHalves = Cfg::kHalves;
    constexpr int kCols = kTile / kParts;                // tokens of a tile that a thread exponentiates
    constexpr int kRows = kTile / kParts;                // rows of a unit
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    using Smem = PagedSmem<D, kParts>;
    Smem& s = *reinterpret_cast<Smem*>(smem_raw);
    const uint32_t warp = warp_id(), lane = lane_id();
    WsHeader* ws = &a.plan->header;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&s.k_full[i], 1);
            mbar_init(&s.k_empty[i], 1);
            mbar_init(&s.v_full[i], 1);
            mbar_init(&s.v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.q_full[i], 1);
            mbar_init(&s.q_empty[i], 1);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.s_free[i], kRowThreads);
            mbar_init(&s.p_ready[i], kRowThreads);
            mbar_init(&s.pv_done[i], 1);
            mbar_init(&s.drain[i], 1);
        }
        for (int i = 0; i < kAhead; ++i) {
            mbar_init(&s.seg_full[i], 1);
            mbar_init(&s.seg_empty[i], kRowThreads);
            mbar_init(&s.stat_full[i], kRowThreads);
        }
        mbar_init(&s.o_empty, kRowThreads);
        s.again = s.failed = 0u;
        fence_mbarrier_init();
        prefetch_tensormap(&tmQ);
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (warp == 2) {
        tmem_alloc(&s.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem_base;
    grid_dependency_wait();

    // State that the roles carry from the first pass to the second, each for itself: tiles and segments
    // so far (a pass ends with a segment without tiles, which tells the other roles), and query tiles
    // (one per segment with tiles).
    int i = 0, seg = 0, qs = 0;
    bool ok = true;
    auto all = [&](bool x) { return __all_sync(0xFFFFFFFFu, x); };
    auto wait = [&](uint64_t& bar, int use, uint32_t where) {            // use: how often it completed before
        return mbar_wait_short(&bar, static_cast<uint32_t>(use) & 1u, ws, a.timeout_ns, where);
    };
    for (int pass = 0;; ++pass) {
        if (warp < 2) {
            // ---------------- loads ----------------
            const bool keys = warp == 0;
            const CUtensorMap* map = keys ? &tmK : &tmV;
            uint8_t* ring = keys ? s.k[0] : s.v[0];
            uint64_t* full = keys ? s.k_full : s.v_full;
            uint64_t* empty = keys ? s.k_empty : s.v_empty;
            const uint64_t once = l2_policy_evict_first(), keep = l2_policy_evict_last();
            const int page_bits = __ffs(a.page) - 1;
            const int boxes = kTile / a.box_rows * kHalves;
            const int box = static_cast<int>(lane) / kHalves, half = static_cast<int>(lane) % kHalves;
            const uint32_t box_bytes = static_cast<uint32_t>(a.box_rows) * 128u;
            const uint32_t box_at = static_cast<uint32_t>(half) * Cfg::kBlockBytes + static_cast<uint32_t>(box) * box_bytes;
            // this lane's box of tile t: its page (looked at only when it is used), or -2: none
            auto lookup = [&](const Segment& g, int t) {
                const int j = t * kTile + box * a.box_rows;
                if (static_cast<int>(lane) >= boxes || j >= g.kv) return -2;
                return max(-1, a.block_table[static_cast<long long>(g.b) * a.max_pages + (j >> page_bits)]);
            };
            Walker walk(a);
            Segment g{};
            bool more = keys && walk.next(g);
            while (ok) {
                if (keys) {
                    // open the segment (or the end) to the other roles, and load its query
                    bool ready = wait(s.seg_empty[seg % kAhead], seg / kAhead + 1, kWaitLoad);
                    if (more) ready = ready && wait(s.q_empty[qs & 1], (qs >> 1) + 1, kWaitLoad);
                    ok = all(ready);
                    if (!ok) break;
                    if (!more) g.t0 = g.t1 = 0;
                    if (lane == 0) {
                        s.seg[seg % kAhead] = g;
                        mbar_arrive(&s.seg_full[seg % kAhead]);
                        if (more) {
                            const uint32_t rows_bytes = static_cast<uint32_t>(a.tile_tokens * a.group) * 128u;
                            mbar_arrive_expect_tx(&s.q_full[qs & 1], rows_bytes * kHalves * kParts);
                            for (int x = 0; x < kParts * kHalves; ++x)
                                tma_load_3d(s.q[qs & 1] + (x % kHalves) * Cfg::kBlockBytes + (x / kHalves) * kRows * 128, &tmQ,
                                            (x % kHalves) * 64, g.h * a.group, g.b * a.N + g.rt * a.tile_tokens,
                                            &s.q_full[qs & 1], keep);
                        }
                    }
                    __syncwarp();
                    if (more) ++qs;
                } else {
                    ok = all(wait(s.seg_full[seg % kAhead], seg / kAhead, kWaitLoad));
                    if (!ok) break;
                    g = s.seg[seg % kAhead];
                }
                ++seg;
                if (g.t0 == g.t1) break;
                int page = lookup(g, g.t0);
                for (int t = g.t0; t < g.t1; ++t) {
                    const int next = t + 1 < g.t1 ? lookup(g, t + 1) : -2;
                    const int slot = i % kSlots;
                    ok = all(wait(empty[slot], i / kSlots + 1, kWaitLoad));
                    if (!ok) break;
                    const uint32_t n = __popc(__ballot_sync(0xFFFFFFFFu, page != -2));
                    if (lane == 0) mbar_arrive_expect_tx(&full[slot], n * box_bytes);
                    __syncwarp();
                    if (page != -2) {
                        if (page < 0 || page >= a.num_pages) {
                            flag_input_index(ws);
                            page = 0;
                        }
                        const int y = (t * kTile + box * a.box_rows) & (a.page - 1);
                        tma_load_3d(ring + slot * Cfg::kTileBytes + box_at, map, half * 64, y, page * a.Hkv + g.h, &full[slot],
                                    once);
                    }
                    page = next;
                    ++i;
                }
                if (keys) more = walk.next(g);
            }
            if (keys) grid_dependency_launch();
            if (!ok && lane == 0) {
                // give copies in flight time to land before the block exits
                for (int x = std::max(0, i - kSlots); x < i; ++x) {
                    const long long t0 = global_ns();
                    while (!mbar_try_wait(&full[x % kSlots], (x / kSlots) & 1) && global_ns() - t0 < a.timeout_ns) {
                    }
                }
                for (int x = std::max(0, qs - 2); x < qs; ++x) {
                    const long long t0 = global_ns();
                    while (!mbar_try_wait(&s.q_full[x & 1], (x >> 1) & 1) && global_ns() - t0 < a.timeout_ns) {
                    }
                }
            }
        } else if (warp < 4) {
            // ---------------- products: the whole warp waits, one lane issues ----------------
            const bool scores = warp == 2;
            constexpr uint32_t kIdescS = attn_idesc<T, false>(kTile, kTile);
            constexpr uint32_t kIdescO = attn_idesc<T, true>(kTile, D);
            constexpr uint32_t kStep = Cfg::kTileBytes >> 4;          // a tile, in descriptor units
            const uint64_t q_desc = sw128_kmajor_desc(smem_u32(s.q[0]));
            const uint64_t k_desc = sw128_kmajor_desc(smem_u32(s.k[0]));
            const uint64_t v_desc = sw128_token_rows_desc(smem_u32(s.v[0]), Cfg::kBlockBytes);
            while (ok) {
                ok = all(wait(s.seg_full[seg % kAhead], seg / kAhead, kWaitMma));
                if (!ok) break;
                const Segment& g = s.seg[seg % kAhead];
                const int n = __shfl_sync(0xFFFFFFFFu, g.t1 - g.t0, 0);
                const int held = __shfl_sync(0xFFFFFFFFu, g.kv - (g.t1 - 1) * kTile, 0);      // of the last tile
                if (n > 0 && scores) ok = all(wait(s.q_full[qs & 1], qs >> 1, kWaitMma));
                for (int x = 0; ok && x < n; ++x, ++i) {
                    const int slot = i % kSlots;
                    const bool last = x + 1 == n;
                    if (scores) {
                        ok = all(wait(s.k_full[slot], i / kSlots, kWaitMma) &&
                                 (i < 2 || wait(s.s_free[i & 1], (i >> 1) - 1, kWaitMma)));
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t q = q_desc + static_cast<uint32_t>(qs & 1) * kStep;
                        const uint64_t k = k_desc + static_cast<uint32_t>(slot) * kStep;
                        const uint32_t to = tmem + kColS + static_cast<uint32_t>(i & 1) * kTile;
                        if (elect_one()) {
#pragma unroll
                            for (int d = 0; d < D / 16; ++d) {
                                const uint64_t off = (static_cast<uint32_t>(d / 4) * Cfg::kBlockBytes + (d % 4) * 32) >> 4;
                                mma_issue<false>(to, q + off, k + off, kIdescS, d != 0 ? 1u : 0u);
                            }
                            mma_commit(&s.s_full[i & 1]);
                            mma_commit(&s.k_empty[slot]);
                            if (last) mma_commit(&s.q_empty[qs & 1]);
                        }
                    } else {
                        ok = all(wait(s.v_full[slot], i / kSlots, kWaitMma));
                        if (!ok) break;
                        if (last && held < kTile) {           // behind the request's end nothing may count
                            const int pieces = (kTile - held) * 8;        // of 16 bytes, per block
                            for (int h = 0; h < kHalves; ++h)
                                for (int y = static_cast<int>(lane); y < pieces; y += 32)
                                    *reinterpret_cast<uint4*>(s.v[slot] + h * Cfg::kBlockBytes + held * 128 + y * 16) =
                                        make_uint4(0u, 0u, 0u, 0u);
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                        ok = all(wait(s.p_ready[i & 1], i >> 1, kWaitMma) &&
                                 (x > 0 || seg == 0 || wait(s.o_empty, seg - 1, kWaitMma)));
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t v = v_desc + static_cast<uint32_t>(slot) * kStep;
                        const uint32_t p = tmem + kColP + static_cast<uint32_t>(i & 1) * 64u;
                        // in the second pass O starts from what the softmax warps put there
                        const uint32_t onto = x == 0 && pass == 0 ? 0u : 1u;
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < kTile / 16; ++k)
                                mma_issue_ta(tmem + kColO, p + k * 8, v + k * 128, kIdescO, k == 0 ? onto : 1u);
                            mma_commit(&s.pv_done[i & 1]);
                            mma_commit(&s.v_empty[slot]);
                        }
                    }
                    __syncwarp();
                }
                if (!ok) break;
                ++seg;
                if (n == 0) break;
                ++qs;
            }
            uint64_t* drain = &s.drain[scores ? 0 : 1];
            if (elect_one()) mma_commit(drain);
            __syncwarp();
            const long long t0 = global_ns();
            while (!mbar_try_wait(drain, pass & 1) && global_ns() - t0 < a.timeout_ns) {
            }
            __syncwarp();
        } else if (warp < 8) {
            // ---------------- softmax: warps 4..7 ----------------
            const uint32_t quad = warp & 3u;
            const uint32_t tlane = tmem + ((quad * 32u) << 16);
            const int line = static_cast<int>(quad * 32u + lane);         // tensor-memory lane
            const int part = line / kRows, row = line % kRows;
            const uint32_t col0 = static_cast<uint32_t>(part) * kCols;    // of a tile's tokens
            const int row_tok = row / a.group;
            const bool row_used = row < a.tile_tokens * a.group;
            const float sl2 = a.scale * kLog2e;
            const bool falling = sl2 < 0.0f;                              // the largest score is the smallest product
            if (kParts > 1 && pass == 0) {
                uint32_t zero[32];
#pragma unroll
                for (int x = 0; x < 32; ++x) zero[x] = 0u;
                for (uint32_t c = 0; c < 128; c += 32) tmem_st32(tlane + kColP + c, zero);
                tmem_wait_st();
            }
            while (ok) {
                bool go = wait(s.seg_full[seg % kAhead], seg / kAhead, kWaitSoftmax);
                // in the second pass the warps meet in barriers, so they give up together
                if (pass != 0) go = named_bar_and(2, kRowThreads, go);
                if (!__all_sync(0xFFFFFFFFu, go)) { ok = false; break; }
                const Segment g = s.seg[seg % kAhead];
                if (g.t0 == g.t1) {
                    if (kParts > 1) {
                        mbar_arrive(&s.stat_full[seg % kAhead]);
                    } else {
                        mbar_arrive(&s.o_empty);
                        mbar_arrive(&s.seg_empty[seg % kAhead]);
                    }
                    ++seg;
                    break;
                }
                const int tok = g.rt * a.tile_tokens + row_tok;           // window token of this row
                const bool valid = row_used && tok < g.n;
                const int limit = valid && a.causal ? max(0, g.kv - g.n + tok + 1) : g.kv;
                float m2 = -INFINITY, l = 0.0f;
                for (int t = g.t0; t < g.t1; ++t, ++i) {
                    bool ready = wait(s.s_full[i & 1], i >> 1, kWaitSoftmax);
                    if (pass != 0) ready = named_bar_and(2, kRowThreads, ready);
                    if (!__all_sync(0xFFFFFFFFu, ready)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t scol = tlane + kColS + static_cast<uint32_t>(i & 1) * kTile + col0;
                    const int seen = limit - t * kTile - static_cast<int>(col0);   // of this thread's columns
                    const bool masked = __any_sync(0xFFFFFFFFu, seen < kCols);
                    const float none = falling ? INFINITY : -INFINITY;
                    uint32_t r[kCols];
#pragma unroll
                    for (int c = 0; c < kCols; c += 32) tmem_ld32(scol + c, r + c);
                    tmem_wait_ld();
                    tc_fence_before();
                    mbar_arrive(&s.s_free[i & 1]);
                    if (masked) {
#pragma unroll
                        for (int c = 0; c < kCols; ++c)
                            if (c >= seen) r[c] = __float_as_uint(none);
                    }
                    float hi[4], lo[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) hi[c] = lo[c] = __uint_as_float(r[c]);
                    if (!falling) {
#pragma unroll
                        for (int c = 4; c < kCols; c += 8)
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                hi[x] = c + 4 < kCols ? fmaxf(fmaxf(hi[x], __uint_as_float(r[c + x])), __uint_as_float(r[(c + 4 + x) % kCols]))
                                                      : fmaxf(hi[x], __uint_as_float(r[c + x]));
                    } else {
#pragma unroll
                        for (int c = 4; c < kCols; ++c) lo[c & 3] = fminf(lo[c & 3], __uint_as_float(r[c]));
                    }
                    const float most = falling ? fminf(fminf(lo[0], lo[1]), fminf(lo[2], lo[3]))
                                               : fmaxf(fmaxf(hi[0], hi[1]), fmaxf(hi[2], hi[3]));
                    // NaN scores leave no maximum behind
                    const float mt = most == none ? -INFINITY : most * sl2 - HalfType<T>::kHeadroom;
                    if (t == g.t0) {
                        m2 = mt;
                    } else {
                        const bool raise = valid && mt > m2 + kRaise;
                        if (__any_sync(0xFFFFFFFFu, raise)) {
                            const bool done =
                                wait(s.pv_done[(i - 1) & 1], (i - 1) >> 1, kWaitSoftmax);
                            if (!__all_sync(0xFFFFFFFFu, done)) {
                                ok = false;
                                if (pass == 0) break;                     // else at the vote below
                            }
                            tc_fence_after();
                            const float f = raise ? exp2_approx(m2 - mt) : 1.0f;
                            if (raise) {
                                l *= f;
                                m2 = mt;
                            }
                            for (uint32_t c = 0; c < D; c += 32) {
                                uint32_t o[32];
                                tmem_ld32(tlane + kColO + c, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                                tmem_st32(tlane + kColO + c, o);
                            }
                            tmem_wait_st();
                        }
                    }
                    const float ref = m2 == -INFINITY ? 0.0f : m2;
                    const uint32_t pcol = tlane + kColP + static_cast<uint32_t>(i & 1) * 64u + col0 / 2;
#pragma unroll
                    for (int c = 0; c < kCols; ++c)
                        r[c] = __float_as_uint(exp2_approx(fmaf(__uint_as_float(r[c]), sl2, -ref)));
                    if (masked) {
#pragma unroll
                        for (int c = 0; c < kCols; ++c)
                            if (c >= seen) r[c] = 0u;
                    }
                    if (i >= 2) {                             // the product that read this P before
                        const bool done = wait(s.pv_done[i & 1], (i >> 1) - 1, kWaitSoftmax);
                        if (!__all_sync(0xFFFFFFFFu, done)) {
                            ok = false;
                            if (pass == 0) break;             // else at the vote below
                        }
                        tc_fence_after();
                    }
#pragma unroll
                    for (int c = 0; c < kCols; c += 32) {
                        uint32_t p[16];
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            p[x] = pack2(__uint_as_float(r[c + 2 * x]), __uint_as_float(r[c + 2 * x + 1]), T{});
                        tmem_st16(pcol + c / 2, p);
                    }
                    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int c = 0; c < kCols; ++c) sum[c & 3] += __uint_as_float(r[c]);
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    tmem_wait_st();
                    if (pass != 0) {
                        uint8_t* tile = s.v[i % kSlots];
                        bool there = ok && wait(s.v_full[i % kSlots], i / kSlots, kWaitSoftmax);
                        // O is about to be changed here: the products before must be complete, and before a
                        // segment's first the last reads of O
                        if (there && t != g.t0) there = wait(s.pv_done[(i - 1) & 1], (i - 1) >> 1, kWaitSoftmax);
                        else if (there && seg > 0) there = wait(s.o_empty, seg - 1, kWaitSoftmax);
                        ok = named_bar_and(2, kRowThreads, there);
                        if (!ok) break;
                        tc_fence_after();
                        if (t == g.t0) {
                            uint32_t zero[32];
#pragma unroll
                            for (int c = 0; c < 32; ++c) zero[c] = 0u;
                            for (uint32_t c = 0; c < D; c += 32) tmem_st32(tlane + kColO + c, zero);
                            tmem_wait_st();
                        }
                        const int upto = min(seen, kCols) + static_cast<int>(col0);
                        move_infinities<T>(tile, Cfg::kBlockBytes, kHalves, line, g.kv - t * kTile, static_cast<int>(col0),
                                           upto, tlane + kColP + static_cast<uint32_t>(i & 1) * 64u, tlane + kColO, s.row,
                                           s.masks, 2);
                        fence_proxy_async_smem();
                    }
                    tc_fence_before();
                    mbar_arrive(&s.p_ready[i & 1]);
                }
                if constexpr (kParts > 1) {
                    if (!ok) break;
                    s.ml[seg % kAhead][line] = make_float2(m2, l);
                    mbar_arrive(&s.stat_full[seg % kAhead]);
                } else {
                    if (ok) ok = __all_sync(0xFFFFFFFFu, wait(s.pv_done[(i - 1) & 1], (i - 1) >> 1, kWaitSoftmax));
                    if (pass != 0) ok = named_bar_and(2, kRowThreads, ok);
                    if (!ok) break;
                    tc_fence_after();
                    const bool whole = g.t0 == 0 && g.t1 == g.tiles;
                    const int head = g.h * a.group + row - row_tok * a.group;
                    const long long out_row = (static_cast<long long>(g.b) * a.N + tok) * a.Hq + head;
                    const long long part_base = static_cast<long long>(2 * blockIdx.x + (g.t0 == 0 ? 1 : 0)) * a.rows_cap;
                    const long long row0 = (static_cast<long long>(g.b) * a.N + g.rt * a.tile_tokens) * a.Hq + g.h * a.group;
                    const int rows = min(a.tile_tokens, g.n - g.rt * a.tile_tokens) * a.group;
                    const float f = whole ? (l != 0.0f ? 1.0f / l : 0.0f) : 1.0f;
                    float check[4] = {l * 0.0f, 0.0f, 0.0f, 0.0f};          // 0, or NaN
                    // 32 columns at a time through shared memory, so that four lanes write a row's piece together
                    float4* stage = s.stage + quad * 256;
                    const int piece = static_cast<int>(lane) & 3;         // eight columns
                    long long to[4];                                      // this lane's four rows (-1: none)
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int rr = static_cast<int>(quad) * 32 + y * 8 + (static_cast<int>(lane) >> 2);
                        const int rt = rr / a.group;
                        to[y] = rr >= rows ? -1
                                : whole    ? (row0 + static_cast<long long>(rt) * a.Hq + (rr - rt * a.group)) * D + piece * 8
                                           : (part_base + rr) * D + piece * 8;
                    }
#pragma unroll 2
                    for (int c = 0; c < D; c += 32) {
                        float o[32];
                        tmem_ld32(tlane + kColO + c, reinterpret_cast<uint32_t*>(o));
                        tmem_wait_ld();
                        __syncwarp();                                     // the columns before have been read
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) check[e] = fmaf(o[4 * x + e], 0.0f, check[e]);
                            stage[lane * 8 + (x ^ (lane & 7))] =
                                make_float4(o[4 * x] * f, o[4 * x + 1] * f, o[4 * x + 2] * f, o[4 * x + 3] * f);
                        }
                        __syncwarp();
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            if (to[y] < 0) continue;
                            const int from = y * 8 + (static_cast<int>(lane) >> 2);
                            const float4 p = stage[from * 8 + ((2 * piece) ^ (from & 7))];
                            const float4 q = stage[from * 8 + ((2 * piece + 1) ^ (from & 7))];
                            if (whole) {
                                const float v[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
                                *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + to[y] + c) = pack8(v, T{});
                            } else {
                                float4* dst = reinterpret_cast<float4*>(a.part_o + to[y] + c);
                                dst[0] = p;
                                dst[1] = q;
                            }
                        }
                    }
                    tc_fence_before();
                    mbar_arrive(&s.o_empty);
                    mbar_arrive(&s.seg_empty[seg % kAhead]);
                    if (valid && !whole) reinterpret_cast<float2*>(a.part_ml)[part_base + row] = make_float2(m2, l);
                    else if (valid && a.lse) a.lse[out_row] = lse_of(m2, l);
                    if (pass == 0 && valid && check[0] + check[1] + check[2] + check[3] != 0.0f) s.again = 1u;
                    __syncwarp();
                }
                ++seg;
            }
        } else if constexpr (kParts > 1) {
            // ---------------- results: warps 8..11 ----------------
            const uint32_t quad = warp & 3u;
            const uint32_t tlane = tmem + ((quad * 32u) << 16);
            const int line = static_cast<int>(quad * 32u + lane);
            const int part = line / kRows, row = line % kRows;
            const int row_tok = row / a.group, row_head = row % a.group;
            const bool row_used = row < a.tile_tokens * a.group;
            while (true) {
                ok = wait(s.seg_full[seg % kAhead], seg / kAhead, kWaitEpilogue);
                Segment g{};
                if (ok) {
                    g = s.seg[seg % kAhead];
                    ok = wait(s.stat_full[seg % kAhead], seg / kAhead, kWaitEpilogue);
                }
                const int last = i + (g.t1 - g.t0) - 1;
                if (ok && g.t1 > g.t0) ok = wait(s.pv_done[last & 1], last >> 1, kWaitEpilogue);
                ok = named_bar_and(1, kRowThreads, ok);                   // these warps meet below: give up together
                if (!ok) break;
                if (g.t0 == g.t1) {
                    mbar_arrive(&s.o_empty);
                    mbar_arrive(&s.seg_empty[seg % kAhead]);
                    ++seg;
                    break;
                }
                i = last + 1;
                tc_fence_after();
                const int tok = g.rt * a.tile_tokens + row_tok, head = g.h * a.group + row_head;
                const bool valid = row_used && tok < g.n;
                const float2* ml = s.ml[seg % kAhead];
                const float m2 = ml[line].x;
                const bool whole = g.t0 == 0 && g.t1 == g.tiles;
                const long long part_base = static_cast<long long>(2 * blockIdx.x + (g.t0 == 0 ? 1 : 0)) * a.rows_cap;
                const int rows = min(a.tile_tokens, g.n - g.rt * a.tile_tokens) * a.group;
                float top = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int k = 0; k < kParts; ++k) top = fmaxf(top, ml[k * kRows + row].x);
#pragma unroll
                for (int k = 0; k < kParts; ++k) {
                    const float2 x = ml[k * kRows + row];
                    sum += x.x == -INFINITY ? x.y : x.y * exp2_approx(x.x - top);           // x.y: 0, or NaN
                }
                const float f = (m2 == -INFINITY ? 1.0f : exp2_approx(m2 - top)) *          // this copy's factor
                                (whole ? (sum != 0.0f ? 1.0f / sum : 0.0f) : 1.0f);
                float check[4] = {ml[line].y * 0.0f, 0.0f, 0.0f, 0.0f};   // 0, or NaN
                // The copies of each row meet in shared memory, as many columns at a time as it holds of the
                // rows in use.  Lines are laid out 32 columns after 32 columns, copy by copy.
                const int lines = kParts * rows;
                const int chunks = min(D / 32, kTile / lines);            // of 32 columns, per round
                const int at_line = part * rows + row;
                const long long row0 = (static_cast<long long>(g.b) * a.N + g.rt * a.tile_tokens) * a.Hq + g.h * a.group;
#pragma unroll 1
                for (int c0 = 0; c0 < D / 32; c0 += chunks) {
                    const int c1 = min(D / 32, c0 + chunks);
#pragma unroll 1
                    for (int c = c0; c < c1; ++c) {
                        float o[32];
                        tmem_ld32(tlane + kColO + c * 32, reinterpret_cast<uint32_t*>(o));
                        tmem_wait_ld();
                        const int to = (c - c0) * lines + at_line;
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) check[e] = fmaf(o[4 * x + e], 0.0f, check[e]);
                            if (valid)
                                s.stage[to * 8 + (x ^ (to & 7))] =
                                    make_float4(o[4 * x] * f, o[4 * x + 1] * f, o[4 * x + 2] * f, o[4 * x + 3] * f);
                        }
                    }
                    if (c1 == D / 32) {
                        tc_fence_before();
                        mbar_arrive(&s.o_empty);
                    }
                    named_bar_sync(1, kRowThreads);
                    // eight columns of one row per thread and step, four threads to a row's 32
                    const int items = (c1 - c0) * rows * 4;
#pragma unroll 1
                    for (int item = line; item < items; item += kRowThreads) {
                        const int piece = item & 3, cr = item >> 2, c = cr / rows, rr = cr - c * rows;
                        float v[8] = {};
#pragma unroll
                        for (int k = 0; k < kParts; ++k) {
                            const int from = c * lines + k * rows + rr;
                            const float4 p = s.stage[from * 8 + ((2 * piece) ^ (from & 7))];
                            const float4 q = s.stage[from * 8 + ((2 * piece + 1) ^ (from & 7))];
                            v[0] += p.x; v[1] += p.y; v[2] += p.z; v[3] += p.w;
                            v[4] += q.x; v[5] += q.y; v[6] += q.z; v[7] += q.w;
                        }
                        const int col = (c0 + c) * 32 + piece * 8;
                        if (whole) {
                            const int rt = rr / a.group;
                            const long long to = row0 + static_cast<long long>(rt) * a.Hq + (rr - rt * a.group);
                            *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + to * D + col) = pack8(v, T{});
                        } else {
                            float4* dst = reinterpret_cast<float4*>(a.part_o + (part_base + rr) * D + col);
                            dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                            dst[1] = make_float4(v[4], v[5], v[6], v[7]);
                        }
                    }
                    named_bar_sync(1, kRowThreads);                       // all have read before the next round's
                }
                if (part == 0 && valid) {
                    if (!whole) reinterpret_cast<float2*>(a.part_ml)[part_base + row] = make_float2(top, sum);
                    else if (a.lse) a.lse[(static_cast<long long>(g.b) * a.N + tok) * a.Hq + head] = lse_of(top, sum);
                }
                if (pass == 0 && valid && check[0] + check[1] + check[2] + check[3] != 0.0f) s.again = 1u;
                mbar_arrive(&s.seg_empty[seg % kAhead]);
                ++seg;
            }
        }
        if (!ok) s.failed = 1u;
        __syncthreads();
        const bool stop = pass == 1 || s.again == 0u || s.failed != 0u;
        __syncthreads();                       // everyone has read them before the next pass may write them
        if (stop) break;
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------------------
// Join: block (c, y) handles four rows of the unit that CTA c's run begins inside of, where c is the
// first such CTA of the unit; a thread adds one column of a row over the unit's partial results in
// order.  All blocks together also clear the rows that see nothing because their request or window
// token does not exist.  The kernel is short on purpose: its instructions come from memory each time
// (sixteen partial rows held by each warp of a row made it slower: 5.5 us against 4.5 for 19 of them).
// ---------------------------------------------------------------------------
constexpr int kJoinRows = 4;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinRows * D) paged_join_kernel(const __grid_constant__ PagedArgs a) {
    __shared__ float s_f[kJoinRows][kMaxCtas], s_inv[kJoinRows];      // factor of each partial result, 1 / sum
    const int r = static_cast<int>(threadIdx.x) / D, col = static_cast<int>(threadIdx.x) % D;
    grid_dependency_wait();

    const int c = static_cast<int>(blockIdx.x) + 1;
    const PlanEntry& at = a.plan->entry[c < kMaxCtas ? c : 0];
    const int row = static_cast<int>(blockIdx.y) * kJoinRows + r;
    const int n = at.n, rt = at.rt, h = at.h, b = at.b;
    const int count = c < a.plan->ctas ? at.joined : 0;
    const bool active = count > 0 && row < min(a.tile_tokens, n - rt * a.tile_tokens) * a.group;
    // the row's k-th partial result: CTA c - 1 opened the unit, the others went on with it
    const long long first = static_cast<long long>(2 * (c - 1) + 1) * a.rows_cap + row;
    const long long step = 2ll * a.rows_cap;
    const int tok = rt * a.tile_tokens + row / a.group, head = h * a.group + row % a.group;
    const long long to = (static_cast<long long>(b) * a.N + tok) * a.Hq + head;
    // the first values are under way while the factors are found
    constexpr int kFirst = 8;
    const float* src = a.part_o + first * D + col;
    const long long ahead = step * D, shift = static_cast<long long>(a.rows_cap) * D;
    float v[kFirst];
    if (active) {
#pragma unroll
        for (int k = 0; k < kFirst; ++k) v[k] = k < count ? src[k * ahead - (k > 0 ? shift : 0)] : 0.0f;
    }
    if (active && col < 32) {
        constexpr int kMost = kMaxCtas / 32;
        float2 x[kMost];
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int y = 0; y < kMost; ++y) {
            const int k = col + 32 * y;
            x[y] = k < count ? reinterpret_cast<const float2*>(a.part_ml)[first + k * step - (k > 0 ? a.rows_cap : 0)]
                             : make_float2(-INFINITY, 0.0f);
        }
#pragma unroll
        for (int y = 0; y < kMost; ++y) top = fmaxf(top, x[y].x);
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
#pragma unroll
        for (int y = 0; y < kMost; ++y) {
            const bool none = x[y].x == -INFINITY;            // its sum is then 0, or NaN
            const float f = none ? x[y].y : exp2_approx(x[y].x - top);
            sum += none ? x[y].y : x[y].y * f;
            s_f[r][col + 32 * y] = f;
        }
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        if (col == 0) {
            s_inv[r] = sum != 0.0f ? 1.0f / sum : 0.0f;
            if (a.lse) a.lse[to] = lse_of(top, sum);
        }
    }
    __syncthreads();
    if (active) {
        float o = 0.0f;
#pragma unroll
        for (int k = 0; k < kFirst; ++k) o = fmaf(k < count ? s_f[r][k] : 0.0f, v[k], o);
#pragma unroll 8
        for (int k = kFirst; k < count; ++k) o = fmaf(s_f[r][k], src[k * ahead - shift], o);
        static_cast<T*>(a.out)[to * D + col] = round_to<T>(o * s_inv[r]);
    }

    // rows without a request or window token, a warp each
    const int lane = static_cast<int>(lane_id());
    const long long warps = static_cast<long long>(gridDim.x) * gridDim.y * (blockDim.x / 32);
    for (long long w = (static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * (blockDim.x / 32) + warp_id();
         w < static_cast<long long>(a.B) * a.N; w += warps) {
        const int rb = static_cast<int>(quotient(w, a.N)), i = static_cast<int>(w - static_cast<long long>(rb) * a.N);
        int kv, m;
        request(a, rb, kv, m);
        if (i < m) continue;
        uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + w * a.Hq * D);
        for (int x = lane; x < a.Hq * (D / 8); x += 32) dst[x] = make_uint4(0u, 0u, 0u, 0u);
        if (a.lse)
            for (int x = lane; x < a.Hq; x += 32) a.lse[w * a.Hq + x] = -INFINITY;
    }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
int rows_cap_of(int N, int heads) { return static_cast<int>(std::min<long long>(kTile, static_cast<long long>(N) * heads)); }

template <typename T, int D, int kParts>
cudaError_t launch_parts(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PagedArgs& a, int grid,
                         cudaStream_t stream) {
    constexpr size_t kSmem = sizeof(PagedSmem<D, kParts>);
    static_assert(kSmem <= 227 * 1024, "shared memory of one SM");
    const cudaError_t e = cudaFuncSetAttribute(paged_attention_kernel<T, D, kParts>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    if (e != cudaSuccess) return e;
    return launch_dependent(paged_attention_kernel<T, D, kParts>, dim3(grid), dim3(PagedCfg<D, kParts>::kThreads), kSmem, stream, q, k, v, a);
}

template <typename T, int D>
dspark_status launch_typed(PagedArgs a, int grid, cudaStream_t stream) {
    const uint64_t e = sizeof(T);
    CUtensorMap q, k, v;
    const uint64_t qd[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(a.Hq), static_cast<uint64_t>(a.B) * a.N};
    const uint64_t qs[2] = {D * e, static_cast<uint64_t>(a.Hq) * D * e};
    const uint32_t qb[3] = {64, static_cast<uint32_t>(a.group), static_cast<uint32_t>(a.tile_tokens)};
    const uint64_t kd[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(a.page),
                            static_cast<uint64_t>(a.num_pages) * a.Hkv};
    const uint64_t ks[2] = {D * e, static_cast<uint64_t>(a.page) * D * e};
    const uint32_t kb[3] = {64, static_cast<uint32_t>(a.box_rows), 1};
    if (!make_tensor_map(&q, HalfType<T>::kMapType, 3, a.q, qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tensor_map(&k, HalfType<T>::kMapType, 3, a.k_cache, kd, ks, kb, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tensor_map(&v, HalfType<T>::kMapType, 3, a.v_cache, kd, ks, kb, CU_TENSOR_MAP_SWIZZLE_128B))
        return DSPARK_ERR_CUDA;
    paged_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a, grid);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return cuda_error(err, "launch(paged_attention plan)");
    const int rows = a.tile_tokens * a.group;
    err = rows <= 32   ? launch_parts<T, D, 4>(q, k, v, a, grid, stream)
          : rows <= 64 ? launch_parts<T, D, 2>(q, k, v, a, grid, stream)
                       : launch_parts<T, D, 1>(q, k, v, a, grid, stream);
    if (err != cudaSuccess) return cuda_error(err, "launch(paged_attention)");
    err = launch_dependent(paged_join_kernel<T, D>, dim3(grid, (rows + kJoinRows - 1) / kJoinRows), dim3(kJoinRows * D),
                           0, stream, a);
    if (err != cudaSuccess) return cuda_error(err, "launch(paged_attention join)");
    return DSPARK_OK;
}

}  // namespace

size_t paged_attention_workspace_bytes(int B, int N, int Hq, int D) {
    if (B < 1 || N < 1 || Hq < 1 || D < 1) return 0;
    return sizeof(Plan) + 2ull * kMaxCtas * rows_cap_of(N, Hq) * (2ull + D) * sizeof(float);
}

dspark_status launch_paged_attention(const void* q, const void* k_cache, const void* v_cache, dspark_dtype dtype,
                                     const int32_t* block_table, int max_pages, const int32_t* kv_len,
                                     const int32_t* lengths, float scale, int causal, int B, int N, int Hq, int Hkv,
                                     int D, int num_pages, int page, void* out, float* lse, void* ws,
                                     cudaStream_t stream, const DeviceInfo& dev) {
    if (static_cast<long long>(num_pages) * Hkv >= (1ll << 31) || static_cast<long long>(B) * N >= (1ll << 31)) {
        set_error("paged_attention: num_pages * Hkv and B * N must be below 2^31");
        return DSPARK_ERR_UNSUPPORTED;
    }
    const int group = Hq / Hkv;
    PagedArgs a{};
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_table = block_table;
    a.kv_len = kv_len;
    a.lengths = lengths;
    a.max_pages = max_pages;
    a.causal = causal;
    a.B = B;
    a.N = N;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.group = group;
    a.num_pages = num_pages;
    a.page = page;
    a.box_rows = std::min(page, kTile);
    a.tile_tokens = std::min(N, kTile / group);
    a.rows_cap = rows_cap_of(N, Hq);
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    a.plan = static_cast<Plan*>(ws);
    a.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + sizeof(Plan));
    a.part_o = a.part_ml + 2ull * kMaxCtas * a.rows_cap * 2;
    a.timeout_ns = kDefaultTimeoutNs;
    const int grid = std::min(dev.sm_count, kMaxCtas);
    if (dtype == DSPARK_BF16)
        return D == 64 ? launch_typed<__nv_bfloat16, 64>(a, grid, stream) : launch_typed<__nv_bfloat16, 128>(a, grid, stream);
    return D == 64 ? launch_typed<__half, 64>(a, grid, stream) : launch_typed<__half, 128>(a, grid, stream);
}

}  // namespace dspark
