// Verification of a drafted tree: from the root on, the target's token behind the current node is found, and the
// child that holds it is the next node; where no child does, that token is the last.
//
// Only the rows on the way are read.  Which row comes next is known when the one before is done, so a request is a
// chain of row passes, and the requests are independent: a cluster of 1 to 16 blocks takes a request, every warp a
// part of each row.  A row at temperature 0 is one pass for the largest entry, kept in shared memory as far as it
// fits.  Otherwise a second pass sums the entries' masses, integers, so that no sum depends on an order, and the warp
// whose part holds the drawn share looks for the entry.  The warps meet once per pass and once for the token; a
// value of each goes to all blocks of the cluster.  While a row's masses are summed, the row behind its largest entry,
// which is the next one most of the time, comes to the L2 cache.
#include "half_common.cuh"
#include "mass_common.cuh"
#include "tree_common.cuh"

#include <algorithm>

namespace dspark {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlocks = 4;                 // per SM
constexpr int kClusterMost = 16;
constexpr int kBatch = 6;                  // 16-byte pieces that a thread has under way beside those held
constexpr int kHeld = 12;                  // pieces of a row that a thread holds in shared memory

struct VerifyArgs {
    TreeArgs tree;
    const void* target;
    const float *temperature, *u;          // null: temperature 0
    int cluster;
};

struct Shared {
    uint4 held[kHeld][kThreads];
    u64 slot[2][kClusterMost * kWarps];    // what the cluster's warps tell each other, two exchanges in turn
    int parent[kTreeMost], token[kTreeMost];
    int path[kTreeMost], out[kTreeMost];
    uint64_t bar[2];
};
constexpr uint32_t kWaitPeer = 0xB01;
constexpr long long kUnderWayNs = 100000;  // far more than a store into another block's shared memory takes

__device__ __forceinline__ void copy_async(void* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

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
    __device__ __forceinline__ bool whole(int piece) const { return id(piece) >= 0 && id(piece) + kPer <= V; }
    __device__ __forceinline__ uint4 load(int piece) const {
        const int v = id(piece);
        if (v >= 0 && v + kPer <= V) return __ldg(reinterpret_cast<const uint4*>(row + v));
        uint4 w;
        T* x = reinterpret_cast<T*>(&w);
#pragma unroll
        for (int e = 0; e < kPer; ++e) x[e] = v + e >= 0 && v + e < V ? row[v + e] : static_cast<T>(-INFINITY);
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
    const int C = kCluster ? a.cluster : 1;
    const int rank = kCluster ? static_cast<int>(cluster_rank()) : 0;
    const int b = static_cast<int>(blockIdx.x) / C;
    const int warps = C * kWarps, self = rank * kWarps + warp;               // of the cluster, in the order of the row
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

    // A value of every warp of the cluster for all of them; lane l then has those of warps 4 l .. 4 l + 3 (0 where
    // there is none).  The values travel as asynchronous stores that complete on an mbarrier of the receiving block.
    // What the next exchange but one overwrites has been read: all have answered the next one by then.  False where
    // the wait gave up.
    int turn = 0;                                          // exchanges so far
    auto exchange = [&](u64 mine, u64 (&all)[4]) {
        const int odd = turn & 1;
        bool ok = true;
        if constexpr (kCluster) {
            if (tid == 0) mbar_arrive_expect_tx(&s.bar[odd], static_cast<uint32_t>(warps) * 8u);
            if (lane < C)
                send(remote(&s.slot[odd][self], static_cast<uint32_t>(lane)), mine, remote(&s.bar[odd], static_cast<uint32_t>(lane)));
            ok = mbar_wait_short(&s.bar[odd], static_cast<uint32_t>(turn >> 1) & 1u, t.ws, kDefaultTimeoutNs, kWaitPeer);
            ok = __all_sync(0xFFFFFFFFu, ok);
        } else {
            if (lane == 0) s.slot[odd][self] = mine;
            __syncthreads();
        }
        ++turn;
#pragma unroll
        for (int x = 0; x < 4; ++x) all[x] = 4 * lane + x < warps ? s.slot[odd][4 * lane + x] : 0;
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
        mbar_init(&s.bar[0], 1);
        mbar_init(&s.bar[1], 1);
        fence_mbarrier_init();
    }
    __syncthreads();
    if constexpr (kCluster) {                              // no block stores into one that has not begun
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    grid_dependency_wait();                                // the status word has been cleared

    // A key's low word tells the entry by a number from 2^31 on; without that bit the warp met NaN or +infinity.
    constexpr u64 kClean = 1ull << 31;
    int node = 0, accepted = 0;
    bool ok = true;
    for (int k = 0; k < n; ++k) {
        auto row_of = [&](int i) { return Row<T>(static_cast<const T*>(a.target) + (static_cast<long long>(b) * t.N + i) * t.V, t.V); };
        const Row<T> row = row_of(node);
        // this warp's pieces, in rounds of 32; the first kHeld rounds stay in shared memory
        auto first_piece = [&](const Row<T>& r, int w) { return static_cast<int>(static_cast<long long>(r.pieces()) * w / warps); };
        const int lo = first_piece(row, self), hi = first_piece(row, self + 1);
        const int rounds = (hi - lo + 31) / 32;
        const int held = min(rounds, kHeld);
        auto piece_of = [&](int x) { return lo + 32 * x + lane; };
        const uint4 nothing = Row<T>::nothing();           // where the last round has no piece for a lane

        // ---- the largest entry, the first of equal ones ----
#pragma unroll 4
        for (int x = 0; x < held; ++x) {
            const int j = piece_of(x);
            if (j < hi && row.whole(j)) copy_async(&s.held[x][tid], row.row + row.id(j));
            else s.held[x][tid] = j < hi ? row.load(j) : nothing;
        }
        float best = -INFINITY;
        int best_piece = -1;
        bool clean = true;                                 // no NaN, no +infinity
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
            if (!(top < INFINITY)) {
                clean = false;
                top = -INFINITY;
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if (v[e] < INFINITY) top = fmaxf(top, v[e]);
            }
            if (top > best) {
                best = top;
                best_piece = j;
            }
        };
        for (int x0 = kHeld; x0 < rounds; x0 += kBatch) {
            uint4 raw[kBatch];
#pragma unroll
            for (int x = 0; x < kBatch; ++x) raw[x] = piece_of(x0 + x) < hi ? row.load(piece_of(x0 + x)) : nothing;
#pragma unroll
            for (int x = 0; x < kBatch; ++x) look(raw[x], piece_of(x0 + x));
        }
        // the pieces held come before the others
        const float later = best;
        const int later_piece = best_piece;
        best = -INFINITY;
        best_piece = -1;
        copy_wait();
#pragma unroll 4
        for (int x = 0; x < held; ++x) look(s.held[x][tid], piece_of(x));
        if (later > best) {
            best = later;
            best_piece = later_piece;
        }
        u64 key = 0;                                       // 0: nothing finite
        if (best_piece >= 0) {
            const int x = (best_piece - lo) / 32;
            float v[kPer];
            Row<T>::unpack(x < kHeld ? s.held[x][tid] : row.load(best_piece), v);
#pragma unroll
            for (int e = kPer - 1; e >= 0; --e)
                if (v[e] == best) key = argmax_key(best, static_cast<uint32_t>(row.id(best_piece) + e));
        }
        key = warp_max_u64(key) | kClean;
        if (!__all_sync(0xFFFFFFFFu, clean)) key &= ~kClean;
        u64 all[4];
        ok = exchange(key, all);
        if (!ok) break;
        clean = true;
        key = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (4 * lane + x < warps && !(all[x] & kClean)) clean = false;
            key = max(key, all[x] | kClean);
        }
        clean = __all_sync(0xFFFFFFFFu, clean);
        key = warp_max_u64(key);
        if (key >> 32 == 0) key = 0;
        if (!clean) flags |= DSPARK_STATUS_NUMERIC;
        int y = key != 0 ? static_cast<int>(key_index(key)) : 0;
        if (key == 0) flags |= DSPARK_STATUS_NUMERIC;
        int child = child_of(node, y);

        if (!greedy && key != 0) {
            if (child < n) {                               // the likeliest next row is under way to the L2 cache meanwhile
                const Row<T> next = row_of(child);
                const int to = first_piece(next, self + 1);
                for (int j = first_piece(next, self) + 8 * lane; j < to; j += 8 * 32)
                    if (next.whole(j)) prefetch_l2(next.row + next.id(j));
            }
            // ---- masses: lane g keeps the sum of the warp's g-th group of rounds ----
            const float m = float_from_order_bits(static_cast<uint32_t>(key >> 32));
            const float2 shift = make_float2(-m, -m), slope = make_float2(inv, inv);
            auto weights = [&](const uint4& raw, float* w, bool filter) {  // the roundings of (x - m) * inv, two at once
                Row<T>::unpack(raw, w);
                if (filter)
#pragma unroll
                    for (int e = 0; e < kPer; ++e) w[e] = w[e] < INFINITY ? w[e] : -INFINITY;
#pragma unroll
                for (int e = 0; e < kPer; e += 2) {
                    const float2 z = __fmul2_rn(__fadd2_rn(make_float2(w[e], w[e + 1]), shift), slope);
                    w[e] = expf(z.x);
                    w[e + 1] = expf(z.y);
                }
            };
            // A round's masses: fewer than 2^27 in each half, so the halves' sums over a group of up to 16 stay within 32 bits.
            auto add_round = [&](MassSum& sum, const uint4& raw, bool filter) {
                float w[kPer];
                weights(raw, w, filter);
#pragma unroll
                for (int e = 0; e < kPer; e += 2) sum.add(make_float2(w[e], w[e + 1]));
                sum.count(kPer);
            };
            auto piece = [&](int x) { return piece_of(x) < hi ? row.load(piece_of(x)) : nothing; };
            const int per = (rounds + 31) / 32;            // rounds of a group
            u64 kept = 0;
            auto sum_groups = [&](bool filter) {
                if (per == 1) {
#pragma unroll 4
                    for (int x = 0; x < held; ++x) {
                        MassSum sum;
                        add_round(sum, s.held[x][tid], filter);
                        const u64 q = sum.warp_value();
                        if (lane == x) kept = q;
                    }
                }
                for (int g = per == 1 ? held : 0; g * per < rounds; ) {
                    // kBatch rounds' loads ahead: as many groups, or part of one
                    uint4 raw[kBatch];
                    if (per == 1) {
#pragma unroll
                        for (int x = 0; x < kBatch; ++x) raw[x] = g + x < rounds ? piece(g + x) : nothing;
#pragma unroll
                        for (int x = 0; x < kBatch; ++x) {
                            MassSum sum;
                            add_round(sum, raw[x], filter);
                            const u64 q = sum.warp_value();
                            if (lane == g + x) kept = q;
                        }
                        g += kBatch;
                    } else {
                        u64 q = 0;
                        for (int x0 = g * per; x0 < min((g + 1) * per, rounds); x0 += kBatch) {
                            const int end = min((g + 1) * per, rounds);
#pragma unroll
                            for (int x = 0; x < kBatch; ++x)
                                raw[x] = x0 + x >= end ? nothing : x0 + x < kHeld ? s.held[x0 + x][tid] : piece(x0 + x);
                            MassSum sum;
#pragma unroll
                            for (int x = 0; x < kBatch; ++x) add_round(sum, raw[x], filter);
                            q += sum.warp_value();
                        }
                        if (lane == g) kept = q;
                        ++g;
                    }
                }
            };
            if (clean) sum_groups(false);
            else sum_groups(true);
            u64 q[4];
            ok = exchange(warp_sum_u64(kept), q);
            if (!ok) break;
            const u64 mine = (q[0] + q[1]) + (q[2] + q[3]);
            u64 before = mine;                             // inclusive, then ahead of this lane's warps
            for (int d = 1; d < 32; d <<= 1) {
                const u64 o = __shfl_up_sync(0xFFFFFFFFu, before, d);
                if (lane >= d) before += o;
            }
            const u64 total = __shfl_sync(0xFFFFFFFFu, before, 31);
            before -= mine;
            float u = a.u[static_cast<long long>(b) * t.N + node];
            if (!(u >= 0.0f && u < 1.0f)) {
                flags |= DSPARK_STATUS_INPUT_RANGE;
                u = u >= 1.0f ? 0x1.fffffep-1f : 0.0f;
            }
            const u64 want = share_of(total, static_cast<uint32_t>(u * 0x1p24f));  // exact: a power of two, then the floor
            // the warp whose part holds the share, and the mass ahead of it there
            int owner = -1;
            u64 rest = 0;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                if (before <= want && want < before + q[x]) {
                    owner = 4 * lane + x;
                    rest = want - before;
                }
                before += q[x];
            }
            const int at = __ffs(__ballot_sync(0xFFFFFFFFu, owner >= 0)) - 1;      // some lane: want < total
            owner = __shfl_sync(0xFFFFFFFFu, owner, at);
            rest = __shfl_sync(0xFFFFFFFFu, rest, at);
            u64 found = 0;                                 // the entry's id + 1, in the one warp that finds it
            if (owner == self) {
                u64 incl = kept;
                for (int d = 1; d < 32; d <<= 1) {
                    const u64 o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
                    if (lane >= d) incl += o;
                }
                const int g = __ffs(__ballot_sync(0xFFFFFFFFu, incl > rest)) - 1;
                rest -= __shfl_sync(0xFFFFFFFFu, incl - kept, g);
                for (int x = g * per; x < rounds; ++x) {
                    float w[kPer];
                    u64 sum = 0;
                    weights(x < kHeld ? s.held[x][tid] : piece(x), w, !clean);
#pragma unroll
                    for (int e = 0; e < kPer; ++e) sum += mass_of(w[e]);
                    u64 in = sum;
                    for (int d = 1; d < 32; d <<= 1) {
                        const u64 o = __shfl_up_sync(0xFFFFFFFFu, in, d);
                        if (lane >= d) in += o;
                    }
                    const uint32_t over = __ballot_sync(0xFFFFFFFFu, in > rest);
                    if (over == 0) {
                        rest -= __shfl_sync(0xFFFFFFFFu, in, 31);
                        continue;
                    }
                    if (lane == __ffs(over) - 1) {
                        u64 ahead = in - sum;
#pragma unroll
                        for (int e = 0; e < kPer; ++e) {
                            const u64 qe = mass_of(w[e]);
                            if (found == 0 && ahead + qe > rest) found = static_cast<u64>(row.id(piece_of(x)) + e) + 1;
                            ahead += qe;
                        }
                    }
                    found = __shfl_sync(0xFFFFFFFFu, found, __ffs(over) - 1);
                    break;
                }
            }
            ok = exchange(found, all);
            if (!ok) break;
            y = static_cast<int>(warp_max_u64(max(max(all[0], all[1]), max(all[2], all[3])))) - 1;
            child = child_of(node, y);
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
            copy_wait();
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
    cfg.gridDim = dim3(static_cast<unsigned>(a.tree.B) * static_cast<unsigned>(a.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = static_cast<unsigned>(a.cluster);
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = a.cluster > 1 ? 2 : 1;
    const auto kernel = a.cluster > 1 ? verify_tree_kernel<T, true> : verify_tree_kernel<T, false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(Shared)));
    if (e == cudaSuccess && a.cluster > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
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
    a.tree = TreeArgs{parents, draft_tokens, lengths, B, N, V, out_tokens, num_accepted, path, static_cast<WsHeader*>(ws)};
    a.target = target;
    a.temperature = temperature;
    a.u = u;
    // As many blocks per request as the SMs hold, while a block's part of a row stays worth an exchange.
    a.cluster = 1;
    while (a.cluster < kClusterMost && 2ll * a.cluster * B <= static_cast<long long>(kBlocks) * dev.sm_count &&
           V / (2 * a.cluster) >= 4 * kThreads)
        a.cluster *= 2;
    const dspark_status st = clear_header(ws, stream);
    if (st != DSPARK_OK) return st;
    return dtype == DSPARK_F32 ? launch_typed<float>(a, stream) : launch_typed<__nv_bfloat16>(a, stream);
}

dspark_status launch_verify_tree_tokens(const int32_t* target_tokens, const int32_t* parents, const int32_t* draft_tokens,
                                        const int32_t* lengths, int B, int N, int32_t* out_tokens, int32_t* num_accepted,
                                        int32_t* path, void* ws, cudaStream_t stream) {
    const TreeArgs t{parents, draft_tokens, lengths, B, N, INT32_MAX, out_tokens, num_accepted, path, static_cast<WsHeader*>(ws)};
    const dspark_status st = clear_header(ws, stream);
    if (st != DSPARK_OK) return st;
    const cudaError_t e = launch_dependent(walk_tree_kernel, dim3((B + kWalkWarps - 1) / kWalkWarps), dim3(32 * kWalkWarps), 0,
                                           stream, t, target_tokens);
    if (e != cudaSuccess) return cuda_error(e, "launch(verify_tree_tokens)");
    return DSPARK_OK;
}

}  // namespace dspark
