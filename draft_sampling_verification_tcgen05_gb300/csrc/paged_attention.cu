// Attention of a window of new tokens per request over a paged key-value cache.
//
// A unit is one (request, key head, tile of window rows): the G query heads that share the key
// head, for as many window tokens as fit, are the up to 128 rows of one tensor-core tile, so each
// cached key and value is read from memory once for all of them.  A unit's work is its request's
// cache in tiles of 128 tokens; all units' tiles, laid end to end, are cut into equal runs, one
// per CTA (persistent, one per SM), wherever the cuts fall.  A run's piece of a unit ("segment")
// that is not the whole unit leaves its unnormalised sums in the workspace, and a second kernel
// joins them in the order of the CTAs.  The order of every sum is fixed by the sizes alone.
//
//   warp 0      looks up the pages and issues the TMA loads of query, key and value tiles
//   warp 1      issues S = Q K^T and O += P V on tcgen05 (M = 128 rows, fp32 in tensor memory)
//   warps 2-5   softmax: a thread per tensor-memory lane, running maximum and sum in fp32,
//               weights rounded to the cache's type into tensor memory (P)
//
// With few rows the 128 lanes hold the rows several times over ("parts"): 4 copies of up to 32
// rows, or 2 of up to 64.  Copy k exponentiates only the k-th part of each tile's tokens and its
// P is zero elsewhere, so the copies are independent partial sums, added in the epilogue.
//
// The running maximum is raised only when a tile exceeds it by 2^8 (O, in tensor memory, is then
// rescaled): weights up to 2^8 lose nothing in a floating type, and the rescaling leaves the
// common path.
//
// A row must not see what lies outside its limit, but 0 * infinity is not 0.  Values past the
// request's end are zeroed in shared memory before the product.  Where a row's result is not finite,
// the CTA goes through its run a second time with the infinities and NaN taken out of every value
// tile and added to the rows that see them; nothing else changes in that pass, so rows that do not
// see them come out bit for bit as without them.
#include "attention_common.cuh"
#include "host_common.h"

#include <algorithm>

namespace dspark {
namespace {

constexpr int kTile = 128;                 // cached tokens per tile, and MMA rows
constexpr int kThreads = 192;
constexpr int kSoftmaxThreads = 128;
constexpr int kMaxCtas = 160;
constexpr float kRaise = 8.0f;             // log2 units
constexpr uint32_t kColS = 0, kColP = 256, kColO = 384, kTmemCols = 512;
constexpr uint32_t kWaitLoad = 0x801, kWaitMma = 0x802, kWaitSoftmax = 0x803;

struct PlanEntry {                         // where a CTA's run begins
    int b, pad;
    long long off;                         // tiles into request b's units
};

struct Plan {
    WsHeader header;
    long long total;                       // tiles of all units
    int ctas;                              // CTAs with a run
    int pad[61];
    PlanEntry entry[kMaxCtas];
};
static_assert(sizeof(Plan) % 256 == 0, "the partial results behind the plan stay aligned");

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

__device__ __forceinline__ long long run_start(const Plan* p, int c) {
    return p->ctas == 0 ? 0 : static_cast<long long>(c) * p->total / p->ctas;
}

// One segment: tiles [t0, t1) of unit (b, rt, h), whose request has `tiles` tiles.
struct Segment {
    int b, rt, h, kv, n, tiles, t0, t1;
};

struct Walker {
    const PagedArgs& a;
    int b;
    long long off, left;
    __device__ explicit Walker(const PagedArgs& args) : a(args) {
        const Plan* p = a.plan;
        const int c = blockIdx.x;
        const bool has = c < p->ctas;
        b = has ? p->entry[c].b : 0;
        off = has ? p->entry[c].off : 0;
        left = has ? run_start(p, c + 1) - run_start(p, c) : 0;
    }
    __device__ bool next(Segment& s) {
        while (left > 0 && b < a.B) {
            request(a, b, s.kv, s.n);
            s.tiles = tiles_of(s.kv);
            const long long work = static_cast<long long>(row_tiles_of(a, s.n)) * a.Hkv * s.tiles;
            if (off >= work) {
                off -= work;
                ++b;
                continue;
            }
            const int unit = static_cast<int>(off / s.tiles);
            s.b = b;
            s.rt = unit / a.Hkv;
            s.h = unit % a.Hkv;
            s.t0 = static_cast<int>(off % s.tiles);
            const long long take = min(static_cast<long long>(s.tiles - s.t0), left);
            s.t1 = s.t0 + static_cast<int>(take);
            off += take;
            left -= take;
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
    __shared__ long long s_total;
    Plan* p = a.plan;
    const int tid = threadIdx.x;
    if (tid < 64) reinterpret_cast<uint32_t*>(&p->header)[tid] = 0u;
    __syncthreads();

    auto work_of = [&](int b) -> long long {
        int kv, n;
        if (b >= a.B) return 0;
        if (!request(a, b, kv, n)) flag_input_index(&p->header);
        return static_cast<long long>(row_tiles_of(a, n)) * a.Hkv * tiles_of(kv);
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

    long long total = 0;
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
        scan(work_of(b0 + tid));
        total += s_total;
    }
    const int ctas = static_cast<int>(min(static_cast<long long>(grid), total));
    if (tid == 0) {
        p->total = total;
        p->ctas = ctas;
    }
    long long before = 0;
    for (int b0 = 0; b0 < a.B && ctas > 0; b0 += kPlanThreads) {
        const long long mine = work_of(b0 + tid);
        const long long end = before + scan(mine), begin = end - mine;
        before += s_total;
        if (mine > 0) {
            // every c with begin <= floor(c * total / ctas) < end
            long long c = (begin * ctas + total - 1) / total;
            while (c > 0 && (c - 1) * total / ctas >= begin) --c;
            for (; c < ctas; ++c) {
                const long long at = c * total / ctas;
                if (at >= end) break;
                if (at >= begin) p->entry[c] = PlanEntry{b0 + tid, 0, at - begin};
            }
        }
    }
}

__device__ __forceinline__ float lse_of(float m2, float l) {
    return l == 0.0f ? -INFINITY : ((m2 == -INFINITY ? 0.0f : m2) + log2f(l)) * kLn2;
}

template <int D>
struct PagedCfg {
    static constexpr int kHalves = D / 64;                        // 128-byte column blocks
    static constexpr uint32_t kBlockBytes = kTile * 128;          // one block of a tile
    static constexpr uint32_t kTileBytes = kHalves * kBlockBytes;
    static constexpr int kSlots = D == 128 ? 5 : 12;              // key or value tiles in flight
};

template <int D>
struct PagedSmem {
    using Cfg = PagedCfg<D>;
    alignas(1024) uint8_t ring[Cfg::kSlots][Cfg::kTileBytes];
    alignas(1024) uint8_t q[2][Cfg::kTileBytes];
    float2 ml[kTile];
    float row[D];
    uint32_t masks[4];
    uint32_t again, failed;                // a second pass is needed / a wait gave up
    uint64_t full[Cfg::kSlots], empty[Cfg::kSlots];
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], p_ready[2];
    uint64_t pv_done[2];                   // by the tile's parity: O += P V of that tile is complete
    uint64_t o_empty, drain;
    uint32_t tmem_base;
};

template <typename T, int D, int kParts>
__global__ void __launch_bounds__(kThreads, 1)
paged_attention_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PagedArgs a) {
    using Cfg = PagedCfg<D>;
    constexpr int kSlots = Cfg::kSlots, kHalves = Cfg::kHalves;
    constexpr int kCols = kTile / kParts;                // tokens of a tile that a thread exponentiates
    constexpr int kRows = kTile / kParts;                // rows of a unit
    extern __shared__ uint8_t smem_raw[];
    PagedSmem<D>& s = *reinterpret_cast<PagedSmem<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                       ~static_cast<uintptr_t>(1023));
    const uint32_t warp = warp_id(), lane = lane_id();
    WsHeader* ws = &a.plan->header;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.q_full[i], 1);
            mbar_init(&s.q_empty[i], kSoftmaxThreads);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_ready[i], kSoftmaxThreads);
            mbar_init(&s.pv_done[i], 1);
        }
        mbar_init(&s.o_empty, kSoftmaxThreads);
        s.again = s.failed = 0u;
        mbar_init(&s.drain, 1);
        fence_mbarrier_init();
        prefetch_tensormap(&tmQ);
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (warp == 1) {
        tmem_alloc(&s.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem_base;
    grid_dependency_wait();

    // state that the roles carry from the first pass to the second
    int slot = 0, i = 0, seg = 0, issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int pass = 0;; ++pass) {
    Walker walk(a);
    if (warp == 0) {
        // ---------------- loads: K0, K1, V0, K2, V1, ... in the order of the products ----------------
        const uint64_t once = l2_policy_evict_first(), keep = l2_policy_evict_last();
        const int boxes = kTile / a.box_rows * kHalves;
        const int box = static_cast<int>(lane) / kHalves, half = static_cast<int>(lane) % kHalves;
        const uint32_t box_bytes = static_cast<uint32_t>(a.box_rows) * 128u;
        const uint32_t box_at = static_cast<uint32_t>(half) * Cfg::kBlockBytes + static_cast<uint32_t>(box) * box_bytes;
        struct Load { int z, y; bool on; };
        auto lookup = [&](const Segment& g, int t) {
            Load x{0, 0, false};
            const int j = t * kTile + box * a.box_rows;
            if (static_cast<int>(lane) < boxes && j < g.kv) {
                int pg = a.block_table[static_cast<long long>(g.b) * a.max_pages + j / a.page];
                if (pg < 0 || pg >= a.num_pages) {
                    flag_input_index(ws);
                    pg = 0;
                }
                x = Load{pg * a.Hkv + g.h, j % a.page, true};
            }
            return x;
        };
        auto issue = [&](const CUtensorMap* map, const Load& x) {
            const bool ready = mbar_wait(&s.empty[slot], phase ^ 1u, ws, a.timeout_ns, kWaitLoad);
            if (!__all_sync(0xFFFFFFFFu, ready)) {
                ok = false;
                return;
            }
            const uint32_t n = __popc(__ballot_sync(0xFFFFFFFFu, x.on));
            if (lane == 0) mbar_arrive_expect_tx(&s.full[slot], n * box_bytes);
            __syncwarp();
            if (x.on) tma_load_3d(s.ring[slot] + box_at, map, half * 64, x.y, x.z, &s.full[slot], once);
            ++issued;
            if (++slot == kSlots) { slot = 0; phase ^= 1u; }
        };
        Segment g;
        Load prev{0, 0, false};
        bool have = false;
        for (; ok && walk.next(g); ++seg) {
            Load cur = lookup(g, g.t0);
            const int qb = seg & 1;
            const bool ready = mbar_wait(&s.q_empty[qb], ((seg >> 1) & 1) ^ 1u, ws, a.timeout_ns, kWaitLoad);
            if (!__all_sync(0xFFFFFFFFu, ready)) { ok = false; break; }
            if (lane == 0) {
                const uint32_t rows_bytes = static_cast<uint32_t>(a.tile_tokens * a.group) * 128u;
                mbar_arrive_expect_tx(&s.q_full[qb], rows_bytes * kHalves * kParts);
                for (int k = 0; k < kParts; ++k)
                    for (int x = 0; x < kHalves; ++x)
                        tma_load_3d(s.q[qb] + x * Cfg::kBlockBytes + k * kRows * 128, &tmQ, x * 64, g.h * a.group,
                                    g.b * a.N + g.rt * a.tile_tokens, &s.q_full[qb], keep);
            }
            __syncwarp();
            for (int t = g.t0; ok && t < g.t1; ++t) {
                const Load next = t + 1 < g.t1 ? lookup(g, t + 1) : Load{0, 0, false};
                issue(&tmK, cur);
                if (ok && have) issue(&tmV, prev);
                prev = cur;
                cur = next;
                have = true;
            }
        }
        if (ok && have) issue(&tmV, prev);
        grid_dependency_launch();
        if (!ok && lane == 0) {
            // give copies in flight time to land before the block exits
            for (int x = std::max(0, issued - kSlots); x < issued; ++x) {
                const long long t0 = global_ns();
                while (!mbar_try_wait(&s.full[x % kSlots], (x / kSlots) & 1) && global_ns() - t0 < a.timeout_ns) {
                }
            }
            for (int x = std::max(0, seg - 1); x <= seg; ++x) {
                const long long t0 = global_ns();
                while (!mbar_try_wait(&s.q_full[x & 1], (x >> 1) & 1) && global_ns() - t0 < a.timeout_ns) {
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ---------------- products ----------------
            constexpr uint32_t kIdescS = attn_idesc<T, false>(kTile, kTile);
            constexpr uint32_t kIdescO = attn_idesc<T, true>(kTile, D);
            int first_seg = 0;
            bool have = false, first = false;
            auto advance = [&] {
                if (++slot == kSlots) { slot = 0; phase ^= 1u; }
            };
            // O (+)= P V of tile i - 1; `first`: it opens segment `first_seg` (in the second pass O starts from
            // what the softmax warps put there)
            auto values = [&] {
                const int j = i - 1;
                ok = mbar_wait(&s.p_ready[j & 1], (j >> 1) & 1, ws, a.timeout_ns, kWaitMma) &&
                     (!first || first_seg == 0 ||
                      mbar_wait(&s.o_empty, (first_seg - 1) & 1, ws, a.timeout_ns, kWaitMma)) &&
                     mbar_wait(&s.full[slot], phase, ws, a.timeout_ns, kWaitMma);
                if (!ok) return;
                tc_fence_after();
                const uint32_t v = smem_u32(s.ring[slot]), p = tmem + kColP + static_cast<uint32_t>(j & 1) * 64u;
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    mma_issue_ta(tmem + kColO, p + k * 8, sw128_token_rows_desc(v + k * 2048, Cfg::kBlockBytes),
                                 kIdescO, (first && k == 0 && pass == 0) ? 0u : 1u);
                mma_commit(&s.empty[slot]);
                mma_commit(&s.pv_done[j & 1]);
                advance();
            };
            Segment g;
            for (; ok && walk.next(g); ++seg) {
                ok = mbar_wait(&s.q_full[seg & 1], (seg >> 1) & 1, ws, a.timeout_ns, kWaitMma);
                for (int t = g.t0; ok && t < g.t1; ++t) {
                    ok = mbar_wait(&s.full[slot], phase, ws, a.timeout_ns, kWaitMma);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t q = smem_u32(s.q[seg & 1]), k = smem_u32(s.ring[slot]);
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        const uint32_t at = static_cast<uint32_t>(x / 4) * Cfg::kBlockBytes + (x % 4) * 32;
                        mma_issue<false>(tmem + kColS + static_cast<uint32_t>(i & 1) * kTile, sw128_kmajor_desc(q + at),
                                         sw128_kmajor_desc(k + at), kIdescS, x != 0 ? 1u : 0u);
                    }
                    mma_commit(&s.empty[slot]);
                    mma_commit(&s.s_full[i & 1]);
                    advance();
                    if (have) values();
                    first = t == g.t0;
                    first_seg = seg;
                    have = true;
                    ++i;
                }
            }
            if (ok && have) values();
            mma_commit(&s.drain);
            const long long t0 = global_ns();
            while (!mbar_try_wait(&s.drain, pass & 1) && global_ns() - t0 < a.timeout_ns) {
            }
        }
    } else {
        // ---------------- softmax: warps 2..5 ----------------
        const uint32_t quad = warp & 3u;
        const uint32_t tlane = tmem + ((quad * 32u) << 16);
        const int line = static_cast<int>(quad * 32u + lane);         // tensor-memory lane
        const int part = line / kRows, row = line % kRows;
        const uint32_t col0 = static_cast<uint32_t>(part) * kCols;    // of a tile's tokens
        const float sl2 = a.scale * kLog2e;
        const bool falling = sl2 < 0.0f;                              // the largest score is the smallest product
        const int total = static_cast<int>(std::min<long long>(walk.left, 0x3FFFFFFF));
        if (kParts > 1 && pass == 0) {
            uint32_t zero[32];
#pragma unroll
            for (int x = 0; x < 32; ++x) zero[x] = 0u;
            for (uint32_t c = 0; c < 128; c += 32) tmem_st32(tlane + kColP + c, zero);
            tmem_wait_st();
        }
        Segment g;
        for (; ok && walk.next(g); ++seg) {
            const int tok = g.rt * a.tile_tokens + row / a.group;     // window token of this row
            const int head = g.h * a.group + row % a.group;
            const bool valid = row < a.tile_tokens * a.group && tok < g.n;
            const int limit = valid ? (a.causal ? max(0, g.kv - g.n + tok + 1) : g.kv) : g.kv;
            float m2 = -INFINITY, l = 0.0f;
            for (int t = g.t0; t < g.t1; ++t, ++i) {
                const bool ready = mbar_wait(&s.s_full[i & 1], (i >> 1) & 1, ws, a.timeout_ns, kWaitSoftmax);
                if (!__all_sync(0xFFFFFFFFu, ready)) { ok = false; break; }
                tc_fence_after();
                uint32_t r[kCols];
#pragma unroll
                for (int c = 0; c < kCols; c += 32)
                    tmem_ld32(tlane + kColS + static_cast<uint32_t>(i & 1) * kTile + col0 + c, r + c);
                tmem_wait_ld();
                const int seen = limit - t * kTile - static_cast<int>(col0);   // of this thread's columns
                const bool masked = __any_sync(0xFFFFFFFFu, seen < kCols);
                if (masked) {
                    const float none = falling ? INFINITY : -INFINITY;
#pragma unroll
                    for (int c = 0; c < kCols; ++c)
                        if (c >= seen) r[c] = __float_as_uint(none);
                }
                float hi = -INFINITY, lo = INFINITY;
                if (!falling) {
#pragma unroll
                    for (int c = 0; c < kCols; ++c) hi = fmaxf(hi, __uint_as_float(r[c]));
                } else {
#pragma unroll
                    for (int c = 0; c < kCols; ++c) lo = fminf(lo, __uint_as_float(r[c]));
                }
                const float mt = falling ? (lo == INFINITY ? -INFINITY : lo * sl2)
                                         : (hi == -INFINITY ? -INFINITY : hi * sl2);
                if (t == g.t0) {
                    m2 = mt;
                } else {
                    const bool raise = valid && mt > m2 + kRaise;
                    if (__any_sync(0xFFFFFFFFu, raise)) {
                        const bool done = mbar_wait(&s.pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1, ws, a.timeout_ns, kWaitSoftmax);
                        if (!__all_sync(0xFFFFFFFFu, done)) { ok = false; break; }
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
#pragma unroll
                for (int c = 0; c < kCols; ++c)
                    r[c] = __float_as_uint(exp2_approx(fmaf(__uint_as_float(r[c]), sl2, -ref)));
                if (masked) {
#pragma unroll
                    for (int c = 0; c < kCols; ++c)
                        if (c >= seen) r[c] = 0u;
                }
                float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < kCols; ++c) sum[c & 3] += __uint_as_float(r[c]);
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                const uint32_t pcol = tlane + kColP + static_cast<uint32_t>(i & 1) * 64u + col0 / 2;
#pragma unroll
                for (int c = 0; c < kCols; c += 32) {
                    uint32_t p[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x)
                        p[x] = pack2(__uint_as_float(r[c + 2 * x]), __uint_as_float(r[c + 2 * x + 1]), T{});
                    tmem_st16(pcol + c / 2, p);
                }
                tmem_wait_st();
                const int held = g.kv - t * kTile;
                if (held < kTile || pass != 0) {
                    const int x = i - pass * total;                   // V's place in the load order
                    const int at = 2 * total * pass + (x == total - 1 ? 2 * total - 1 : 2 * x + 2);
                    const int vs = at % kSlots;
                    bool landed = mbar_wait(&s.full[vs], (at / kSlots) & 1, ws, a.timeout_ns, kWaitSoftmax);
                    if (pass != 0 && t != g.t0)
                        landed = mbar_wait(&s.pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1, ws, a.timeout_ns, kWaitSoftmax) &&
                                 landed;
                    if (pass != 0) landed = named_bar_and(2, kSoftmaxThreads, landed);
                    if (!__all_sync(0xFFFFFFFFu, landed)) { ok = false; break; }
                    tc_fence_after();
                    if (line >= held) {                               // behind the request's end nothing may count
#pragma unroll
                        for (int h = 0; h < kHalves; ++h) {
                            uint4* p = reinterpret_cast<uint4*>(s.ring[vs] + h * Cfg::kBlockBytes + line * 128);
#pragma unroll
                            for (int y = 0; y < 8; ++y) p[y] = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    if (pass != 0) {
                        if (t == g.t0) {
                            uint32_t zero[32];
#pragma unroll
                            for (int c = 0; c < 32; ++c) zero[c] = 0u;
                            for (uint32_t c = 0; c < D; c += 32) tmem_st32(tlane + kColO + c, zero);
                            tmem_wait_st();
                        }
                        const int upto = min(seen, kCols) + static_cast<int>(col0);
                        move_infinities<T>(s.ring[vs], Cfg::kBlockBytes, kHalves, line, held, static_cast<int>(col0), upto,
                                           tlane + kColS + static_cast<uint32_t>(i & 1) * kTile, tlane + kColO, sl2, ref,
                                           s.row, s.masks, 2);
                    }
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                mbar_arrive(&s.p_ready[i & 1]);
            }
            // ---------------- the segment's result ----------------
            if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&s.pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1, ws, a.timeout_ns, kWaitSoftmax));
            // the warps that add up their copies below give up together
            if constexpr (kParts > 1) ok = named_bar_and(1, kSoftmaxThreads, ok);
            if (!ok) break;
            tc_fence_after();
            uint32_t o[D];
#pragma unroll
            for (int c = 0; c < D; c += 32) tmem_ld32(tlane + kColO + c, o + c);
            tmem_wait_ld();
            tc_fence_before();
            mbar_arrive(&s.o_empty);

            const bool whole = g.t0 == 0 && g.t1 == g.tiles;
            const long long out_row = (static_cast<long long>(g.b) * a.N + tok) * a.Hq + head;
            const long long part_row = static_cast<long long>(2 * blockIdx.x + (g.t0 == 0 ? 1 : 0)) * a.rows_cap + row;
            float check = l * 0.0f;
#pragma unroll
            for (int c = 0; c < D; ++c) check = fmaf(__uint_as_float(o[c]), 0.0f, check);
            if (pass == 0 && valid && check != 0.0f) s.again = 1u;
            if constexpr (kParts == 1) {
                const float f = whole ? (l != 0.0f ? 1.0f / l : 0.0f) : 1.0f;
                if (valid) {
                    if (whole) {
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + out_row * D);
#pragma unroll
                        for (int c = 0; c < D; c += 8) {
                            float x[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(o[c + e]) * f;
                            dst[c / 8] = pack8(x, T{});
                        }
                        if (a.lse) a.lse[out_row] = lse_of(m2, l);
                    } else {
                        uint4* dst = reinterpret_cast<uint4*>(a.part_o + part_row * D);
#pragma unroll
                        for (int c = 0; c < D; c += 4) dst[c / 4] = make_uint4(o[c], o[c + 1], o[c + 2], o[c + 3]);
                        reinterpret_cast<float2*>(a.part_ml)[part_row] = make_float2(m2, l);
                    }
                }
                mbar_arrive(&s.q_empty[seg & 1]);
            } else {
                // add the copies of each row, half of the columns at a time through the query's buffer
                s.ml[line] = make_float2(m2, l);
                named_bar_sync(1, kSoftmaxThreads);
                float top = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int k = 0; k < kParts; ++k) top = fmaxf(top, s.ml[k * kRows + row].x);
#pragma unroll
                for (int k = 0; k < kParts; ++k) {
                    const float2 x = s.ml[k * kRows + row];
                    if (x.x != -INFINITY) sum = fmaf(x.y, exp2_approx(x.x - top), sum);
                    else sum += x.y;                                  // 0, or NaN
                }
                const float f = (m2 == -INFINITY ? 1.0f : exp2_approx(m2 - top)) *
                                (whole ? (sum != 0.0f ? 1.0f / sum : 0.0f) : 1.0f);
                if (part == 0 && valid) {
                    if (!whole) reinterpret_cast<float2*>(a.part_ml)[part_row] = make_float2(top, sum);
                    else if (a.lse) a.lse[out_row] = lse_of(top, sum);
                }
                constexpr int kChunk = D / 2, kQuads = kChunk / 4;    // columns and 16-byte pieces per round
                float4* stage = reinterpret_cast<float4*>(s.q[seg & 1]);
                const int rows = min(a.tile_tokens, g.n - g.rt * a.tile_tokens) * a.group;
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int x = 0; x < kQuads; ++x) {
                        float v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = __uint_as_float(half == 0 ? o[4 * x + e] : o[kChunk + 4 * x + e]) * f;
                        stage[line * kQuads + (x ^ (line & 7))] = make_float4(v[0], v[1], v[2], v[3]);
                    }
                    named_bar_sync(1, kSoftmaxThreads);
                    for (int at = line; at < rows * (kQuads / 2); at += kSoftmaxThreads) {
                        const int rr = at / (kQuads / 2), piece = at % (kQuads / 2);     // eight columns
                        float v[8] = {};
#pragma unroll
                        for (int k = 0; k < kParts; ++k) {
                            const int from = k * kRows + rr;
                            const float4 x = stage[from * kQuads + ((2 * piece) ^ (from & 7))];
                            const float4 y = stage[from * kQuads + ((2 * piece + 1) ^ (from & 7))];
                            v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
                            v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
                        }
                        const int col = half * kChunk + piece * 8;
                        if (whole) {
                            const long long to = (static_cast<long long>(g.b) * a.N + g.rt * a.tile_tokens +
                                                  rr / a.group) * a.Hq + g.h * a.group + rr % a.group;
                            *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + to * D + col) = pack8(v, T{});
                        } else {
                            float4* dst = reinterpret_cast<float4*>(a.part_o + (part_row - row + rr) * D + col);
                            dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                            dst[1] = make_float4(v[4], v[5], v[6], v[7]);
                        }
                    }
                    named_bar_sync(1, kSoftmaxThreads);
                }
                fence_proxy_async_smem();
                mbar_arrive(&s.q_empty[seg & 1]);
            }
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
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------------------
// Join: block (c, y) handles four rows of the unit that CTA c's run begins inside of, where c is the
// first such CTA of the unit; one warp per row adds the unit's partial results in order.  All warps
// together also clear the rows that see nothing because their request or window token does not exist.
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ void __launch_bounds__(128) paged_join_kernel(const __grid_constant__ PagedArgs a) {
    constexpr int kPer = D / 32;
    const int lane = static_cast<int>(lane_id());
    grid_dependency_wait();

    const long long warps = static_cast<long long>(gridDim.x) * gridDim.y * 4;
    for (long long w = (static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * 4 + warp_id();
         w < static_cast<long long>(a.B) * a.N; w += warps) {
        const int b = static_cast<int>(w / a.N), i = static_cast<int>(w % a.N);
        int kv, n;
        request(a, b, kv, n);
        if (i < n) continue;
        uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + w * a.Hq * D);
        for (int x = lane; x < a.Hq * (D / 8); x += 32) dst[x] = make_uint4(0u, 0u, 0u, 0u);
        if (a.lse)
            for (int x = lane; x < a.Hq; x += 32) a.lse[w * a.Hq + x] = -INFINITY;
    }

    const Plan* p = a.plan;
    const int c = static_cast<int>(blockIdx.x) + 1;
    if (c >= p->ctas) return;
    const PlanEntry at = p->entry[c];
    int kv, n;
    request(a, at.b, kv, n);
    const int tiles = tiles_of(kv);
    const int t0 = static_cast<int>(at.off % tiles), unit = static_cast<int>(at.off / tiles);
    const long long w0 = run_start(p, c) - t0, w1 = w0 + tiles;
    if (t0 == 0 || w0 < run_start(p, c - 1)) return;          // no unit is cut here, or an earlier CTA joins it
    int last = c;
    while (last + 1 < p->ctas && run_start(p, last + 1) < w1) ++last;
    const int count = last - c + 2;                           // CTAs c - 1 .. last

    const int row = static_cast<int>(blockIdx.y) * 4 + static_cast<int>(warp_id());
    const int rt = unit / a.Hkv, h = unit % a.Hkv;
    const int rows = min(a.tile_tokens, n - rt * a.tile_tokens) * a.group;
    if (row >= rows) return;
    auto slot = [&](int k) {                                  // k-th contributor's partial row
        const int cta = c - 1 + k;
        return static_cast<long long>(2 * cta + (k == 0 ? 1 : 0)) * a.rows_cap + row;
    };
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
    float top = -INFINITY;
    for (int k = lane; k < count; k += 32) top = fmaxf(top, ml[slot(k)].x);
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    float sum = 0.0f, o[kPer] = {};
    for (int k0 = 0; k0 < count; k0 += 32) {
        float f = 0.0f;
        if (k0 + lane < count) {
            const float2 x = ml[slot(k0 + lane)];
            f = x.x == -INFINITY ? (x.y == x.y ? 0.0f : x.y) : exp2_approx(x.x - top);
            sum += x.x == -INFINITY ? x.y : x.y * f;
        }
        const int m = min(32, count - k0);
#pragma unroll 8
        for (int k = 0; k < m; ++k) {
            const float w = __shfl_sync(0xFFFFFFFFu, f, k);
            const float* src = a.part_o + slot(k0 + k) * D + lane * kPer;
            if constexpr (kPer == 4) {
                const float4 v = *reinterpret_cast<const float4*>(src);
                o[0] = fmaf(v.x, w, o[0]); o[1] = fmaf(v.y, w, o[1]);
                o[2] = fmaf(v.z, w, o[2]); o[3] = fmaf(v.w, w, o[3]);
            } else {
                const float2 v = *reinterpret_cast<const float2*>(src);
                o[0] = fmaf(v.x, w, o[0]); o[1] = fmaf(v.y, w, o[1]);
            }
        }
    }
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
    const int tok = rt * a.tile_tokens + row / a.group, head = h * a.group + row % a.group;
    const long long to = (static_cast<long long>(at.b) * a.N + tok) * a.Hq + head;
    T* out = static_cast<T*>(a.out) + to * D + lane * kPer;
#pragma unroll
    for (int e = 0; e < kPer; e += 2)
        *reinterpret_cast<uint32_t*>(out + e) = pack2(o[e] * inv, o[e + 1] * inv, T{});
    if (a.lse && lane == 0) a.lse[to] = lse_of(top, sum);
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
int rows_cap_of(int N, int heads) { return static_cast<int>(std::min<long long>(kTile, static_cast<long long>(N) * heads)); }

template <typename K, typename... Args>
cudaError_t launch_dependent(K kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, int D, int kParts>
cudaError_t launch_parts(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PagedArgs& a, int grid,
                         cudaStream_t stream) {
    constexpr size_t kSmem = sizeof(PagedSmem<D>) + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory of one SM");
    const cudaError_t e = cudaFuncSetAttribute(paged_attention_kernel<T, D, kParts>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    if (e != cudaSuccess) return e;
    return launch_dependent(paged_attention_kernel<T, D, kParts>, dim3(grid), dim3(kThreads), kSmem, stream, q, k, v, a);
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
    err = launch_dependent(paged_join_kernel<T, D>, dim3(grid, (rows + 3) / 4), dim3(128), 0, stream, a);
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
