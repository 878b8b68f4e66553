// Verification of a drafted tree: from the root on, the target's token behind the current node is found, and the
// child that holds it is the next node; where no child does, that token is the last.
//
// Only the rows on the way are read.  Which row comes next is known when the one before is done, so a request is a
// chain of row passes, and the requests are independent: a cluster of 1 to 16 blocks takes a request, every warp a
// part of each row, which comes to shared memory by asynchronous copies kHeld groups ahead.
//
// A row is one pass: for the largest entry, the first of equal ones, and at a temperature for fp32 sums of weights
// 2^((x - ref) / T log2 e) besides, with ref the largest of the row's first pieces.  The warp whose part holds the drawn
// share of the sum looks for the entry.  Where the sums' error could reach past the entry's ends (its bound stands at
// `eps`), and where NaN, +infinity or an overflow is in the way, a second pass decides by the exact masses, integers
// whose sum depends on no order; so the token is the exact one either way.  The blocks meet once per pass and once for
// the token: each stores a pair into all blocks of the cluster.  While they do, the row behind the largest
// entry, which is the next one most of the time, comes to the L2 cache.
//
// Bound by that chain: a row of 151936 fp32 entries in 16 blocks takes 2.3 us greedily and 4.5 us drawn, of which the
// memory's rate would explain 0.1; one greedy tree of 25 nodes 13.5 us in all.  64 drawn trees of up to 64 nodes, 230
// rows (140 MB), take 66 us, 2.1 TB/s, as long as the deepest path needs with 8 blocks.  (Exact masses in every
// row: 104 us; with the row read again by the second pass and barriers of the cluster: 234.)
#include "half_common.cuh"
#include "mass_common.cuh"
#include "tree_common.cuh"

#include <algorithm>

namespace dspark {
namespace {

constexpr int kThreads = 256;
constexpr int kWarpBits = 3, kWarps = 1 << kWarpBits;
static_assert(kThreads == 32 * kWarps, "warps of a block");
constexpr int kBlocks = 4;                 // per SM
constexpr int kClusterMost = 16;
constexpr int kGroup = 4;                  // rounds of 32 pieces that are loaded and looked at together
constexpr int kHeld = 3;                   // groups in shared memory: under way, or the last ones

struct VerifyArgs {
    TreeArgs tree;
    const void* target;
    const float *temperature, *u;          // null: temperature 0
    int cluster_bits;                      // 2^cluster_bits blocks take a request
};

constexpr int kTurns = 4;
struct alignas(16) Pair { u64 key, sum; };

struct Shared {
    uint4 held[kHeld][kGroup][kThreads];
    Pair pair[kTurns][kClusterMost];       // what the cluster's blocks tell each other, kTurns exchanges in turn
    Pair warp_pair[kTurns][kWarps];
    int parent[kTreeMost], token[kTreeMost];
    int path[kTreeMost], out[kTreeMost];
    uint64_t bar[kTurns];
};
constexpr uint32_t kWaitPeer = 0xB01;
// A test build makes a wait run out: limits of 2 ms, and block DSPARK_LATE_RANK of a cluster 20 ms late at its
// exchange DSPARK_LATE_AT (expressions in the names of the kernel).
#ifdef DSPARK_LATE_AT
constexpr long long kPeerLimitNs = 2000000;
#else
constexpr long long kPeerLimitNs = kDefaultTimeoutNs;
#endif
constexpr long long kUnderWayNs = 100000;  // far more than a store into another block's shared memory takes

__device__ __forceinline__ void copy_async(void* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(kLeft) : "memory"); }

// The largest of three; NaN where one is NaN.
__device__ __forceinline__ float max3_nan(float x, float y, float z) {
    float m;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(x), "f"(y), "f"(z));
    return m;
}

// One row: V entries from `row` on, taken as 16-byte pieces of memory.  The first and the last piece may reach
// beyond the row: their other entries count as -infinity and are not read.
template <typename T>
struct Row {
    static constexpr int kPer = 16 / sizeof(T);
    const T* row;
    int V, shift;                          // entries of the first piece ahead of the row
    __device__ __forceinline__ Row(const T* p, int v) : row(p), V(v) {
        shift = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
    }
    __device__ __forceinline__ int pieces() const { return (shift + V + kPer - 1) / kPer; }
    __device__ __forceinline__ int id(int piece) const { return piece * kPer - shift; }
    __device__ __forceinline__ int first_whole() const { return shift > 0 ? 1 : 0; }             // the pieces that lie
    __device__ __forceinline__ int behind_whole() const { return (shift + V) / kPer; }           // within the row
    __device__ __noinline__ uint4 edge(int piece) const {
        const int v = id(piece);
        T x[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) x[e] = v + e >= 0 && v + e < V ? row[v + e] : static_cast<T>(-INFINITY);
        uint4 w;
        memcpy(&w, x, 16);
        return w;
    }
    static __device__ __forceinline__ uint4 nothing() {    // entries of -infinity
        const uint32_t w = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;
        return make_uint4(w, w, w, w);
    }
    static __device__ __forceinline__ void unpack(const uint4& w, float* x) {
        if constexpr (sizeof(T) == 4) {
            x[0] = __uint_as_float(w.x);
            x[1] = __uint_as_float(w.y);
            x[2] = __uint_as_float(w.z);
            x[3] = __uint_as_float(w.w);
        } else {
            unpack8(w, x, T{});
        }
    }
};

template <typename T, bool kCluster>
__global__ void __launch_bounds__(kThreads, kBlocks) verify_tree_kernel(const __grid_constant__ VerifyArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Shared& s = *reinterpret_cast<Shared*>(smem_raw);
    constexpr int kPer = Row<T>::kPer;
    const TreeArgs& t = a.tree;
    const int tid = threadIdx.x, warp = static_cast<int>(warp_id()), lane = static_cast<int>(lane_id());
    const int C = kCluster ? 1 << a.cluster_bits : 1, warp_bits = (kCluster ? a.cluster_bits : 0) + kWarpBits;
    const int rank = kCluster ? static_cast<int>(cluster_rank()) : 0;
    const int b = static_cast<int>(blockIdx.x) >> (kCluster ? a.cluster_bits : 0);
    const int self = rank * kWarps + warp;                 // among the cluster's warps, in the order of the row
    uint32_t flags = 0;

    const int nodes = tree_nodes(t, b);
    const int n = max(nodes, 0);
    if (nodes < 0) flags |= DSPARK_STATUS_INPUT_RANGE;
    bool bad = false;
    for (int i = tid; i < n; i += kThreads) tree_node(t, b, i, s.parent[i], s.token[i], bad);
    for (int i = tid; i < t.N; i += kThreads) s.path[i] = s.out[i] = -1;
    if (bad) flags |= DSPARK_STATUS_INPUT_RANGE;
    float T_b = a.temperature ? a.temperature[b] : 0.0f;
    if (!(T_b >= 0.0f) || T_b == INFINITY) {
        flags |= DSPARK_STATUS_NUMERIC;
        T_b = 0.0f;
    }
    const bool greedy = T_b == 0.0f;
    const float inv = greedy ? 0.0f : fminf(1.0f / T_b, 3.402823466e38f);

    // What the blocks tell each other travels as asynchronous stores into every block, which complete on an mbarrier
    // there.  Of any three turns at least one is an exchange of all blocks, which a block answers when all its warps
    // have come to it, so what the turn after those overwrites has been read.
    int turn = 0;
    auto told = [&](uint32_t bytes) {                      // false where the wait gave up, in all warps of the block alike
        bool ok = true;
        if constexpr (kCluster) {
            uint64_t* bar = &s.bar[turn % kTurns];
            if (tid == 0) mbar_arrive_expect_tx(bar, bytes);
            ok = __syncthreads_and(mbar_wait_short(bar, static_cast<uint32_t>(turn / kTurns) & 1u, t.ws, kPeerLimitNs, kWaitPeer)) != 0;
        } else {
            __syncthreads();
        }
        ++turn;
        return ok;
    };
    auto late = [&] {
#ifdef DSPARK_LATE_AT
        if (kCluster && turn == DSPARK_LATE_AT && rank == DSPARK_LATE_RANK) {
            const long long t0 = global_ns();
            while (global_ns() - t0 < 20000000) {
            }
        }
#endif
    };
    // A pair of every block: the largest of the warps' `key`s and the sum of their `sum`s (added by `add`).  Lane r then has those of block r, 0 where there is none.
    auto exchange = [&](u64 key, u64 sum, auto add, Pair& all) {
        late();
        const int now = turn % kTurns;
        if (lane == 0) s.warp_pair[now][warp] = Pair{key, sum};
        __syncthreads();
        if (warp == 0) {
            Pair mine = s.warp_pair[now][lane % kWarps];   // every kWarps lanes come to the same
            mine.key = warp_max_u64(mine.key);
#pragma unroll
            for (int d = kWarps / 2; d > 0; d >>= 1) mine.sum = add(mine.sum, __shfl_xor_sync(0xFFFFFFFFu, mine.sum, d));
            if (kCluster && lane < C)
                send2(remote(&s.pair[now][rank], static_cast<uint32_t>(lane)), mine.key, mine.sum,
                      remote(&s.bar[now], static_cast<uint32_t>(lane)));
            if (!kCluster && lane == 0) s.pair[now][0] = mine;
        }
        const bool ok = told(static_cast<uint32_t>(C) * 16u);
        all = lane < C ? s.pair[now][lane] : Pair{0, 0};
        return ok;
    };
    // A value that only one warp of the cluster has (`here`).
    auto hear = [&](bool here, u64 mine, u64& value) {
        late();
        const int now = turn % kTurns;
        if (kCluster && here && lane < C)
            send(remote(&s.pair[now][0].key, static_cast<uint32_t>(lane)), mine, remote(&s.bar[now], static_cast<uint32_t>(lane)));
        if (!kCluster && here && lane == 0) s.pair[now][0].key = mine;
        const bool ok = told(8u);
        value = s.pair[now][0].key;
        return ok;
    };
    // The first child of `node` that holds token y (kTreeMost: none).
    auto child_of = [&](int node, int y) {
        uint32_t child = kTreeMost;
        for (int i = lane; i < n; i += 32)
            if (i > 0 && s.parent[i] == node && s.token[i] == y) child = min(child, static_cast<uint32_t>(i));
        return static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, child));
    };
    if (kCluster && tid == 0) {
        for (int i = 0; i < kTurns; ++i) mbar_init(&s.bar[i], 1);
        fence_mbarrier_init();
    }
    __syncthreads();
    if constexpr (kCluster) {                              // no block stores into one that has not begun
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    grid_dependency_wait();                                // the status word has been cleared

    int node = 0, accepted = 0;
    bool ok = true;
    for (int k = 0; k < n; ++k) {
        auto row_of = [&](int i) { return Row<T>(static_cast<const T*>(a.target) + (static_cast<long long>(b) * t.N + i) * t.V, t.V); };
        const Row<T> row = row_of(node);
        // this warp's pieces, in rounds of 32 and groups of rounds
        auto first_piece = [&](const Row<T>& r, int w) { return static_cast<int>((static_cast<long long>(r.pieces()) * w) >> warp_bits); };
        const int lo = first_piece(row, self), hi = first_piece(row, self + 1);
        const int rounds = (hi - lo + 31) / 32, groups = (rounds + kGroup - 1) / kGroup;
        auto piece_of = [&](int x) { return lo + 32 * x + lane; };
        const uint4 nothing = Row<T>::nothing();           // behind the last piece
        const int whole0 = row.first_whole(), whole1 = row.behind_whole();
        auto start = [&](int g) {                          // a group's loads; an empty one behind the last keeps the count
            if (g < groups) {
#pragma unroll
                for (int x = 0; x < kGroup; ++x) {
                    const int j = piece_of(g * kGroup + x);
                    uint4* to = &s.held[g % kHeld][x][tid];
                    if (j >= whole0 && j < min(hi, whole1)) copy_async(to, row.row + row.id(j));
                    else *to = j < hi ? row.edge(j) : nothing;
                }
            }
            copy_commit();
        };
        // a round again, after the pass: from shared memory, or from the L2 cache
        auto piece = [&](int x) {
            const int j = piece_of(x);
            if (x / kGroup >= groups - kHeld) return s.held[x / kGroup % kHeld][x % kGroup][tid];
            if (j >= whole0 && j < min(hi, whole1)) return __ldg(reinterpret_cast<const uint4*>(row.row + row.id(j)));
            return j < hi ? row.edge(j) : nothing;
        };
        const float drawn = greedy ? 0.0f : a.u[static_cast<long long>(b) * t.N + node];
#pragma unroll
        for (int g = 0; g < kHeld; ++g) start(g);

        // ---- one pass: the largest entry, the first of equal ones; without greed sums of weights for a first answer ----
        // These weights are relative to `ref`, the largest of the row's first pieces, which all warps look at.
        float ref = 0.0f;
        if (!greedy) {
            float v[kPer], top = -INFINITY;
            Row<T>::unpack(lane >= whole0 && lane < whole1 ? __ldg(reinterpret_cast<const uint4*>(row.row + row.id(lane)))
                           : lane < row.pieces()           ? row.edge(lane)
                                                           : nothing,
                           v);
#pragma unroll
            for (int e = 0; e < kPer; ++e) top = fmaxf(top, v[e]);
            top = float_from_order_bits(__reduce_max_sync(0xFFFFFFFFu, float_order_bits(top)));
            if (top > -INFINITY && top < INFINITY) ref = top;
        }
        const float2 slope2 = make_float2(inv * kLog2e, inv * kLog2e), shift2 = make_float2(-ref * slope2.x, -ref * slope2.x);
        auto quick = [&](const float* v, int e) {          // 2^((v - ref) / T * log2 e), two at once
            const float2 z = __ffma2_rn(make_float2(v[e], v[e + 1]), slope2, shift2);
            return make_float2(exp2_approx(z.x), exp2_approx(z.y));
        };
        const int per = (groups + 31) / 32;                // lane l keeps the sums of `per` groups together, the l-th such
        float2 sum2[2] = {};
        float group_sum = 0.0f;
        float best = -INFINITY, odd_value = -INFINITY;     // odd_value: NaN where one is met
        int best_piece = lo;
        uint4 best_raw = nothing;
        auto look = [&](const uint4& raw, int j) {
            float v[kPer];
            Row<T>::unpack(raw, v);
            float top = max3_nan(v[0], v[1], v[2]);
            if constexpr (kPer == 4) {
                top = max3_nan(top, v[3], v[3]);
            } else {
                top = max3_nan(top, v[3], v[4]);
                top = max3_nan(top, v[5], v[6]);
                top = max3_nan(top, v[7], v[7]);
            }
            odd_value = max3_nan(odd_value, top, top);
            if (top > best) {
                best = top;
                best_piece = j;
                best_raw = raw;
            }
            if (!greedy) {
#pragma unroll
                for (int e = 0; e < kPer; e += 2) sum2[(e >> 1) & 1] = __fadd2_rn(sum2[(e >> 1) & 1], quick(v, e));
            }
        };
        auto lane_sum = [&]() {                            // of the group that has been looked at
            const float sum = (sum2[0].x + sum2[0].y) + (sum2[1].x + sum2[1].y);
            sum2[0] = sum2[1] = make_float2(0.0f, 0.0f);
            return sum;
        };
        for (int g0 = 0; g0 < groups; g0 += kHeld) {
            float sum[kHeld];
#pragma unroll
            for (int g = 0; g < kHeld; ++g) {
                sum[g] = 0.0f;
                if (g0 + g >= groups) continue;
                copy_wait<kHeld - 1>();
#pragma unroll
                for (int x = 0; x < kGroup; ++x) look(s.held[g][x][tid], piece_of((g0 + g) * kGroup + x));
                sum[g] = lane_sum();
                start(g0 + g + kHeld);
            }
            if (greedy) continue;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1)
#pragma unroll
                for (int g = 0; g < kHeld; ++g) sum[g] += __shfl_xor_sync(0xFFFFFFFFu, sum[g], d);
#pragma unroll
            for (int g = 0; g < kHeld; ++g)
                if (lane == (per == 1 ? g0 + g : (g0 + g) / per)) group_sum += sum[g];
        }
        float warp_sum = group_sum;
        if (!greedy)
            for (int d = 16; d > 0; d >>= 1) warp_sum += __shfl_xor_sync(0xFFFFFFFFu, warp_sum, d);
        bool clean = __all_sync(0xFFFFFFFFu, odd_value < INFINITY);           // no NaN, no +infinity
        if (!clean) {                                      // once more without them
            best = -INFINITY;
            for (int x = 0; x < rounds; ++x) {
                float v[kPer];
                const uint4 raw = piece(x);
                Row<T>::unpack(raw, v);
                float top = -INFINITY;
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if (v[e] < INFINITY) top = fmaxf(top, v[e]);
                if (top > best) {
                    best = top;
                    best_piece = piece_of(x);
                    best_raw = raw;
                }
            }
        }
        u64 key = 0;                                       // 0: nothing finite
        if (best > -INFINITY) {
            float v[kPer];
            Row<T>::unpack(best_raw, v);
#pragma unroll
            for (int e = kPer - 1; e >= 0; --e)
                if (v[e] == best) key = argmax_key(best, static_cast<uint32_t>(row.id(best_piece) + e));
        }
        key = warp_max_u64(key);
        auto add_floats = [](u64 x, u64 y) {
            return static_cast<u64>(__float_as_uint(__uint_as_float(static_cast<uint32_t>(x)) + __uint_as_float(static_cast<uint32_t>(y))));
        };
        Pair all;
        // a block that met NaN or +infinity says so by a sum of NaN; a sum that is not a number by itself (a slope that
        // overflows) counts as infinite
        ok = exchange(key, __float_as_uint(!clean ? NAN : warp_sum == warp_sum ? warp_sum : INFINITY), add_floats, all);
        if (!ok) break;
        const float block_sum = __uint_as_float(static_cast<uint32_t>(all.sum));
        clean = __all_sync(0xFFFFFFFFu, block_sum == block_sum);
        key = warp_max_u64(all.key);
        if (!clean || key == 0) flags |= DSPARK_STATUS_NUMERIC;
        int y = key != 0 ? static_cast<int>(key_index(key)) : 0;
        int child = child_of(node, y);

        if (!greedy && key != 0) {
            if (child < n) {                               // the likeliest next row is under way to the L2 cache meanwhile
                const Row<T> next = row_of(child);
                const int to = min(first_piece(next, self + 1), next.behind_whole());
                for (int j = max(first_piece(next, self), next.first_whole()) + 8 * lane; j < to; j += 8 * 32)
                    prefetch_l2(next.row + next.id(j));
            }
            const float m = float_from_order_bits(static_cast<uint32_t>(key >> 32));
            float u = drawn;
            if (!(u >= 0.0f && u < 1.0f)) {
                flags |= DSPARK_STATUS_INPUT_RANGE;
                u = u >= 1.0f ? 0x1.fffffep-1f : 0.0f;
            }
            const uint32_t share = static_cast<uint32_t>(u * 0x1p24f);        // exact: a power of two, then the floor
            // Which of the first `count` lanes' values q, end to end, holds `rest`; leaves in `rest` what is behind its beginning
            // (-1: none).  The lanes behind them hold 0, but fp32 sums of theirs are added in another order and may be larger than
            // the last value's: their votes do not count.
            auto locate = [&](auto q, int count, auto& rest) {
                auto in = q;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const auto o = __shfl_up_sync(0xFFFFFFFFu, in, d);
                    if (lane >= d) in += o;
                }
                const int at = __ffs(__ballot_sync(0xFFFFFFFFu, in > rest) & (0xFFFFFFFFu >> (32 - count))) - 1;
                if (at > 0) rest -= __shfl_sync(0xFFFFFFFFu, in, at - 1);
                return at;
            };
            // Whether this warp holds `rest`, given the blocks' values and the warps' of this block; exactly one does (where
            // a rounding leaves it behind all, the last).
            auto owns = [&](auto of_blocks, auto of_warps, auto& rest) {
                const int r = locate(of_blocks, C, rest);
                if ((r < 0 ? C - 1 : r) != rank) return false;
                const int w = locate(of_warps, kWarps, rest);
                return (w < 0 ? kWarps - 1 : w) == warp;
            };

            // ---- the first answer: from the fp32 sums, where their error cannot reach the entry's ends ----
            // With r_v the real weight: the exact mass differs from 2^40 r_v by the roundings of (x - m) * inv, 2^-23 of
            // up to 28 (what is smaller has no mass), expf's 2 ulp and the floor; the quick weight by those of the
            // slope, 1.5 * 2^-24 of up to 41 in log2 units, of the multiply-add, 2^-24 of its result, and ex2's 2 ulp
            // (a common factor counts for nothing); the sums by 2^-24 a step.  `slack` is more than all that.
            const float far = (m - ref) * slope2.x;
            const float reach = far >= 0.0f ? fmaxf(41.0f, far) : 41.0f - far;
            const float eps = 7e-6f + 5e-8f * reach + 6e-8f * static_cast<float>(rounds * (kPer / 4) + 64) + 2e-12f * static_cast<float>(t.V);
            float total = block_sum;
            for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
            u64 found = 0;                                 // the entry's id + 1
            if (clean && total > 0x1p-60f && total < 0x1p100f) {
                const int last = (turn - 1) % kTurns;
                float rest = total * u;
                const bool here = owns(block_sum, lane < kWarps ? __uint_as_float(static_cast<uint32_t>(s.warp_pair[last][lane].sum)) : 0.0f, rest);
                if (here) {
                    const float slack = eps * total;
                    const int l = locate(group_sum, 32, rest);                // a lane without groups has no rounds either
                    for (int x0 = l * per * kGroup; l >= 0 && x0 < min((l + 1) * per * kGroup, rounds); x0 += kGroup) {
                        float part[kGroup];
#pragma unroll
                        for (int x = 0; x < kGroup; ++x) {
                            float v[kPer];
                            Row<T>::unpack(x0 + x < rounds ? piece(x0 + x) : nothing, v);
                            float2 w = quick(v, 0);
#pragma unroll
                            for (int e = 2; e < kPer; e += 2) w = __fadd2_rn(w, quick(v, e));
                            part[x] = w.x + w.y;
                        }
#pragma unroll
                        for (int d = 1; d < 32; d <<= 1)                      // inclusive sums over the lanes, round by round
#pragma unroll
                            for (int x = 0; x < kGroup; ++x) {
                                const float o = __shfl_up_sync(0xFFFFFFFFu, part[x], d);
                                if (lane >= d) part[x] += o;
                            }
                        int at = -1;
                        uint32_t over = 0;
#pragma unroll
                        for (int x = 0; x < kGroup; ++x) {
                            if (at >= 0) continue;
                            over = __ballot_sync(0xFFFFFFFFu, part[x] > rest);
                            if (over != 0) {
                                at = x;
                                if (over & 1u) continue;
                                rest -= __shfl_sync(0xFFFFFFFFu, part[x], __ffs(over) - 2);
                            } else {
                                rest -= __shfl_sync(0xFFFFFFFFu, part[x], 31);
                            }
                        }
                        if (at < 0) continue;              // in a later round
                        float v[kPer], from = 0.0f;
                        Row<T>::unpack(piece(x0 + at), v);
#pragma unroll
                        for (int e = 0; e < kPer; e += 2) {
                            const float2 w = quick(v, e);
                            if (rest >= from + slack && rest + slack < from + w.x) found = static_cast<u64>(row.id(piece_of(x0 + at)) + e) + 1;
                            from += w.x;
                            if (rest >= from + slack && rest + slack < from + w.y) found = static_cast<u64>(row.id(piece_of(x0 + at)) + e) + 2;
                            from += w.y;
                        }
                        found = __shfl_sync(0xFFFFFFFFu, found, __ffs(over) - 1);
                        break;
                    }
                }
                ok = hear(here, found, found);
                if (!ok) break;
            }

            if (found == 0) {
                // ---- exact masses ----
                const float2 shift = make_float2(-m, -m), slope = make_float2(inv, inv);
                auto weights = [&](const uint4& raw, float* w) {   // the roundings of (x - m) * inv, two at once
                    Row<T>::unpack(raw, w);
#pragma unroll
                    for (int e = 0; e < kPer; ++e) w[e] = w[e] < INFINITY ? w[e] : -INFINITY;
#pragma unroll
                    for (int e = 0; e < kPer; e += 2) {
                        const float2 z = __fmul2_rn(__fadd2_rn(make_float2(w[e], w[e + 1]), shift), slope);
                        w[e] = expf(z.x);
                        w[e + 1] = expf(z.y);
                    }
                };
                u64 kept = 0;
                for (int g = 0; g < groups; ++g) {
                    uint4 raw[kGroup];
#pragma unroll
                    for (int x = 0; x < kGroup; ++x) raw[x] = piece(g * kGroup + x);
                    MassSum sum;
#pragma unroll
                    for (int x = 0; x < kGroup; ++x) {
                        float w[kPer];
                        weights(raw[x], w);
#pragma unroll
                        for (int e = 0; e < kPer; e += 2) sum.add(make_float2(w[e], w[e + 1]));
                        sum.count(kPer);
                    }
                    const u64 q = sum.warp_value();
                    if (lane == (per == 1 ? g : g / per)) kept += q;
                }
                ok = exchange(0, warp_sum_u64(kept), [](u64 x, u64 y) { return x + y; }, all);
                if (!ok) break;
                const int last = (turn - 1) % kTurns;
                u64 rest = share_of(warp_sum_u64(all.sum), share);
                const bool here = owns(all.sum, lane < kWarps ? s.warp_pair[last][lane].sum : 0, rest);
                if (here) {
                    for (int x = locate(kept, 32, rest) * per * kGroup; x < rounds; ++x) {
                        float w[kPer];
                        u64 sum = 0;
                        weights(piece(x), w);
#pragma unroll
                        for (int e = 0; e < kPer; ++e) sum += mass_of(w[e]);
                        const int l = locate(sum, 32, rest);
                        if (l < 0) {
                            rest -= warp_sum_u64(sum);
                            continue;
                        }
                        u64 ahead = 0;
#pragma unroll
                        for (int e = 0; e < kPer; ++e) {
                            const u64 qe = mass_of(w[e]);
                            if (lane == l && found == 0 && ahead + qe > rest) found = static_cast<u64>(row.id(piece_of(x)) + e) + 1;
                            ahead += qe;
                        }
                        found = warp_max_u64(found);
                        break;
                    }
                }
                ok = hear(here, found, found);
                if (!ok) break;
            }
            if (static_cast<int>(found) - 1 != y) {
                y = static_cast<int>(found) - 1;
                child = child_of(node, y);
            }
        }

        if (tid == 0) {
            s.path[k] = node;
            s.out[k] = y;
        }
        if (child >= n) break;
        node = child;
        ++accepted;
    }

    if constexpr (kCluster) {                              // no block ends while another still stores into it
        if (!ok) {
            copy_wait<0>();
            const long long t0 = global_ns();
            while (global_ns() - t0 < kUnderWayNs) {
            }
        }
        __syncwarp();
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    }
    if (flags) set_status(t.ws, flags);
    if (rank == 0) {
        __syncthreads();
        for (int i = tid; i < t.N; i += kThreads) {
            t.out_tokens[static_cast<long long>(b) * t.N + i] = s.out[i];
            t.path[static_cast<long long>(b) * t.N + i] = s.path[i];
        }
        if (tid == 0) t.num_accepted[b] = accepted;
    }
}

// The walk alone, the target's tokens given: a warp per request, eight nodes to a lane.
constexpr int kWalkWarps = 4;

__global__ void __launch_bounds__(32 * kWalkWarps) walk_tree_kernel(const __grid_constant__ TreeArgs t, const int32_t* target) {
    constexpr int kMine = kTreeMost / 32;
    const int lane = static_cast<int>(lane_id());
    const int b = static_cast<int>(blockIdx.x) * kWalkWarps + static_cast<int>(warp_id());
    if (b >= t.B) return grid_dependency_wait();
    const int nodes = tree_nodes(t, b), n = max(nodes, 0);
    const long long at = static_cast<long long>(b) * t.N;
    bool bad = nodes < 0;
    int parent[kMine], token[kMine], behind[kMine], path[kMine], out[kMine];      // node 32 x + lane
#pragma unroll
    for (int x = 0; x < kMine; ++x) {
        const int i = 32 * x + lane;
        parent[x] = token[x] = behind[x] = -1;
        path[x] = out[x] = -1;
        if (i >= n) continue;
        tree_node(t, b, i, parent[x], token[x], bad);
        behind[x] = target[at + i];
    }
    int node = 0, accepted = 0;
    for (int k = 0; k < n; ++k) {
        int y = 0;
#pragma unroll
        for (int x = 0; x < kMine; ++x)
            if (node >> 5 == x) y = __shfl_sync(0xFFFFFFFFu, behind[x], node & 31);
        uint32_t child = kTreeMost;
#pragma unroll
        for (int x = kMine - 1; x >= 0; --x) {
            const int i = 32 * x + lane;
            if (i > 0 && i < n && parent[x] == node && token[x] == y) child = static_cast<uint32_t>(i);
            if (k >> 5 == x && (k & 31) == lane) {
                path[x] = node;
                out[x] = y;
            }
        }
        child = __reduce_min_sync(0xFFFFFFFFu, child);
        if (child >= static_cast<uint32_t>(n)) break;
        node = static_cast<int>(child);
        ++accepted;
    }
#pragma unroll
    for (int x = 0; x < kMine; ++x) {
        const int i = 32 * x + lane;
        if (i >= t.N) continue;
        t.out_tokens[at + i] = out[x];
        t.path[at + i] = path[x];
    }
    if (lane == 0) t.num_accepted[b] = accepted;
    grid_dependency_wait();                                // the status word has been cleared
    if (bad) flag_input_index(t.ws);
}

template <typename T>
dspark_status launch_typed(const VerifyArgs& a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.tree.B) << a.cluster_bits);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 1u << a.cluster_bits;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = a.cluster_bits > 0 ? 2 : 1;
    const auto kernel = a.cluster_bits > 0 ? verify_tree_kernel<T, true> : verify_tree_kernel<T, false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(Shared)));
    if (e == cudaSuccess && a.cluster_bits > 3) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e != cudaSuccess) return cuda_error(e, "launch(verify_tree)");
    return DSPARK_OK;
}

}  // namespace

dspark_status launch_verify_tree(const void* target, dspark_dtype dtype, const float* temperature, const float* u,
                                 const int32_t* parents, const int32_t* draft_tokens, const int32_t* lengths, int B, int N,
                                 int V, int32_t* out_tokens, int32_t* num_accepted, int32_t* path, void* ws,
                                 cudaStream_t stream, const DeviceInfo& dev) {
    VerifyArgs a{};
    a.tree = TreeArgs{parents, draft_tokens, lengths, B, N, V, V - 1, out_tokens, num_accepted, path, static_cast<WsHeader*>(ws)};
    a.target = target;
    a.temperature = temperature;
    a.u = u;
    // As many blocks per request as the SMs hold at once, while a block's part of a row stays worth an exchange.  64 requests
    // of 151936 entries: 8 blocks each 66 us; 16, which then wait for room, 70; 4 take 82.  One request with one row to draw from:
    // of 4000 entries 5.8 us in one block, 6.7 in two; of 8000, where two are taken, 6.5 and 7.3; of 32000 9.4, 8.7 in two,
    // 7.5 in four, 7.2 in eight (which are taken), 7.1 in 16.
    while ((2 << a.cluster_bits) <= kClusterMost && static_cast<long long>(B) * (2 << a.cluster_bits) <= static_cast<long long>(kBlocks) * dev.sm_count &&
           V / (2 << a.cluster_bits) >= 8 * kThreads)
        ++a.cluster_bits;
    const dspark_status st = clear_header(ws, stream);
    if (st != DSPARK_OK) return st;
    return dtype == DSPARK_F32 ? launch_typed<float>(a, stream) : launch_typed<__nv_bfloat16>(a, stream);
}

dspark_status launch_verify_tree_tokens(const int32_t* target_tokens, const int32_t* parents, const int32_t* draft_tokens,
                                        const int32_t* lengths, int B, int N, int32_t* out_tokens, int32_t* num_accepted,
                                        int32_t* path, void* ws, cudaStream_t stream) {
    const TreeArgs t{parents, draft_tokens, lengths, B, N, 0, INT32_MAX, out_tokens, num_accepted, path, static_cast<WsHeader*>(ws)};
    const dspark_status st = clear_header(ws, stream);
    if (st != DSPARK_OK) return st;
    const cudaError_t e = launch_dependent(walk_tree_kernel, dim3((B + kWalkWarps - 1) / kWalkWarps), dim3(32 * kWalkWarps), 0,
                                           stream, t, target_tokens);
    if (e != cudaSuccess) return cuda_error(e, "launch(verify_tree_tokens)");
    return DSPARK_OK;
}

}  // namespace dspark
