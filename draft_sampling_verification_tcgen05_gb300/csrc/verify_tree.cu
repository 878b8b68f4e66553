// Verification of a drafted tree: from the root on, the target's token behind the current node is found, and the
// child that holds it is the next node; where no child does, that token is the last.
//
// Only the rows on the way are read.  Which row comes next is known when the one before is done, so a request is a
// chain of row passes, and the requests are independent: a cluster of 1 to 16 blocks takes a request, every block a
// part of each row.  A row at temperature 0 is one pass for the largest entry.  Otherwise a second pass (from the L2
// cache, as a rule) sums the entries' masses, integers, so that no sum depends on an order, and the warp whose part
// holds the drawn share looks for the entry in one of its 32 pieces of that part.
#include "half_common.cuh"
#include "mass_common.cuh"
#include "tree_common.cuh"

#include <algorithm>

namespace dspark {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kClusterMost = 16;
constexpr int kBatch = 8;                  // 16-byte pieces that a thread has under way

struct VerifyArgs {
    TreeArgs tree;
    const void* target;
    const float *temperature, *u;          // null: temperature 0
    int cluster;
};

struct Shared {
    u64 slot[2][kClusterMost];             // what the blocks tell each other, two exchanges in turn
    u64 warp_value[kWarps];
    int parent[kTreeMost], token[kTreeMost];
    int path[kTreeMost], out[kTreeMost];
    u64 found;
    int next;
};

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
    __device__ __forceinline__ uint4 load(int piece) const {
        const int v = id(piece);
        if (v >= 0 && v + kPer <= V) return __ldg(reinterpret_cast<const uint4*>(row + v));
        uint4 w;
        T* x = reinterpret_cast<T*>(&w);
#pragma unroll
        for (int e = 0; e < kPer; ++e) x[e] = v + e >= 0 && v + e < V ? row[v + e] : static_cast<T>(-INFINITY);
        return w;
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
__global__ void __launch_bounds__(kThreads, 2) verify_tree_kernel(const __grid_constant__ VerifyArgs a) {
    __shared__ Shared s;
    constexpr int kPer = Row<T>::kPer;
    const TreeArgs& t = a.tree;
    const int tid = threadIdx.x, warp = static_cast<int>(warp_id()), lane = static_cast<int>(lane_id());
    const int C = kCluster ? a.cluster : 1;
    const int rank = kCluster ? static_cast<int>(cluster_rank()) : 0;
    const int b = static_cast<int>(blockIdx.x) / C;
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

    // Values of all blocks, in the order of the blocks; `odd` alternates from exchange to exchange.
    int odd = 0;
    auto exchange = [&](u64 mine) {                        // mine: in thread 0 .. C - 1 of the block
        if constexpr (kCluster) {
            odd ^= 1;
            if (tid < C) {
                const uint32_t to = remote(&s.slot[odd][rank], static_cast<uint32_t>(tid));
                asm volatile("st.shared::cluster.u64 [%0], %1;" :: "r"(to), "l"(mine) : "memory");
            }
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        } else {
            if (tid == 0) s.slot[0][0] = mine;
            __syncthreads();
        }
    };
    __syncthreads();
    if constexpr (kCluster) {                              // no block stores into one that has not begun
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    }

    int node = 0, accepted = 0;
    for (int k = 0; k < n; ++k) {
        const Row<T> row(static_cast<const T*>(a.target) + (static_cast<long long>(b) * t.N + node) * t.V, t.V);
        // this warp's pieces
        const long long pieces = row.pieces(), part = static_cast<long long>(rank) * kWarps + warp, parts = static_cast<long long>(C) * kWarps;
        const int lo = static_cast<int>(pieces * part / parts), hi = static_cast<int>(pieces * (part + 1) / parts);

        // ---- the largest entry, the first of equal ones ----
        float best = -INFINITY;
        int best_piece = -1;
        bool odd_value = false;                            // NaN or +infinity
        for (int j0 = lo; j0 < hi; j0 += 32 * kBatch) {
            uint4 raw[kBatch];
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
                const int j = j0 + 32 * x + lane;
                if (j < hi) raw[x] = row.load(j);
            }
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
                const int j = j0 + 32 * x + lane;
                if (j >= hi) continue;
                float v[kPer];
                Row<T>::unpack(raw[x], v);
                float top = -INFINITY;
#pragma unroll
                for (int e = 0; e < kPer; ++e) {
                    const bool fine = v[e] < INFINITY;
                    odd_value = odd_value || !fine;
                    if (fine && v[e] > top) top = v[e];
                }
                if (top > best) {
                    best = top;
                    best_piece = j;
                }
            }
        }
        u64 key = 0;                                       // 0: nothing finite
        if (best_piece >= 0) {
            float v[kPer];
            Row<T>::unpack(row.load(best_piece), v);
#pragma unroll
            for (int e = kPer - 1; e >= 0; --e)
                if (v[e] == best) key = argmax_key(best, static_cast<uint32_t>(row.id(best_piece) + e));
        }
        if (odd_value) flags |= DSPARK_STATUS_NUMERIC;
        key = warp_max_u64(key);
        __syncthreads();                                   // all have read the row's values before
        if (lane == 0) s.warp_value[warp] = key;
        __syncthreads();
        if (warp == 0) key = warp_max_u64(lane < kWarps ? s.warp_value[lane] : 0);
        exchange(key);
        key = 0;
        for (int r = 0; r < C; ++r) key = max(key, s.slot[odd][r]);
        int y = key != 0 ? static_cast<int>(key_index(key)) : 0;
        if (key == 0) flags |= DSPARK_STATUS_NUMERIC;

        if (!greedy && key != 0) {
            // ---- masses: lane l keeps the sum of the l-th of the 32 pieces that the warp's part is cut into ----
            const float m = float_from_order_bits(static_cast<uint32_t>(key >> 32));
            auto mass_in = [&](const uint4& w) {
                float v[kPer];
                Row<T>::unpack(w, v);
                u64 q = 0;
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if (v[e] < INFINITY) q += mass_of(expf(__fmul_rn(__fsub_rn(v[e], m), inv)));
                return q;
            };
            const int per = max(1, (hi - lo + 32 * 32 - 1) / (32 * 32));           // rounds of 32 pieces
            u64 kept = 0;
            for (int x = 0; x < 32; ++x) {
                u64 q = 0;
                for (int y0 = 0; y0 < per; ++y0) {
                    const int j = lo + (x * per + y0) * 32 + lane;
                    if (j < hi) q += mass_in(row.load(j));
                }
                q = warp_sum_u64(q);
                if (lane == x) kept = q;
            }
            const u64 mine = warp_sum_u64(kept);
            __syncthreads();
            if (lane == 0) s.warp_value[warp] = mine;
            __syncthreads();
            u64 block = 0;
            for (int w = 0; w < kWarps; ++w) block += s.warp_value[w];
            exchange(block);
            u64 total = 0, before = 0;
            for (int r = 0; r < C; ++r) {
                if (r < rank) before += s.slot[odd][r];
                total += s.slot[odd][r];
            }
            for (int w = 0; w < warp; ++w) before += s.warp_value[w];
            float u = a.u[static_cast<long long>(b) * t.N + node];
            if (!(u >= 0.0f && u < 1.0f)) {
                flags |= DSPARK_STATUS_INPUT_RANGE;
                u = u >= 1.0f ? 0x1.fffffep-1f : 0.0f;
            }
            const u64 want = share_of(total, static_cast<uint32_t>(u * 0x1p24f));  // exact: a power of two, then the floor
            u64 found = 0;                                 // the entry's id + 1, in the one warp that finds it
            if (before <= want && want < before + mine) {
                u64 incl = kept;
                for (int d = 1; d < 32; d <<= 1) {
                    const u64 o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
                    if (lane >= d) incl += o;
                }
                u64 rest = want - before;                  // mass ahead of the entry in this warp's part
                const int x = __ffs(__ballot_sync(0xFFFFFFFFu, incl > rest)) - 1;
                rest -= __shfl_sync(0xFFFFFFFFu, incl - kept, x);
                for (int y0 = 0; y0 < per; ++y0) {
                    const int j = lo + (x * per + y0) * 32 + lane;
                    uint4 w{};
                    u64 q = 0;
                    if (j < hi) {
                        w = row.load(j);
                        q = mass_in(w);
                    }
                    u64 in = q;
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
                        float v[kPer];
                        Row<T>::unpack(w, v);
                        u64 ahead = in - q;
#pragma unroll
                        for (int e = 0; e < kPer; ++e) {
                            const u64 qe = v[e] < INFINITY ? mass_of(expf(__fmul_rn(__fsub_rn(v[e], m), inv))) : 0;
                            if (found == 0 && ahead + qe > rest) found = static_cast<u64>(row.id(j) + e) + 1;
                            ahead += qe;
                        }
                        s.found = found;
                    }
                    break;
                }
                __syncwarp();
            }
            // the block that holds the entry tells the others; exactly one does
            u64 block_before = 0;
            for (int r = 0; r < rank; ++r) block_before += s.slot[odd][r];
            __syncthreads();
            exchange(block_before <= want && want < block_before + block ? s.found : 0);
            u64 id = 0;
            for (int r = 0; r < C; ++r) id = max(id, s.slot[odd][r]);
            y = static_cast<int>(id) - 1;
        }

        // ---- the first child that holds the token ----
        int child = kTreeMost;
        if (warp == 0) {
            for (int i = lane; i < n; i += 32)
                if (s.parent[i] == node && s.token[i] == y && i > 0) child = min(child, i);
            child = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, static_cast<uint32_t>(child)));
            if (lane == 0) {
                s.next = child;
                s.path[k] = node;
                s.out[k] = y;
            }
        }
        __syncthreads();
        child = s.next;
        if (child >= n) break;
        node = child;
        ++accepted;
    }

    if constexpr (kCluster) {                              // no block ends while another still stores into it
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    }
    grid_dependency_wait();                                // the status word has been cleared
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
    cudaError_t e = cudaSuccess;
    if (a.cluster > 8) e = cudaFuncSetAttribute(verify_tree_kernel<T, true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess)
        e = a.cluster > 1 ? cudaLaunchKernelEx(&cfg, verify_tree_kernel<T, true>, a) : cudaLaunchKernelEx(&cfg, verify_tree_kernel<T, false>, a);
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
    // As many blocks per request as the SMs hold, two on each, while a block's part of a row stays worth a launch.
    a.cluster = 1;
    while (a.cluster < kClusterMost && 2ll * a.cluster * B <= 2ll * dev.sm_count && V / (2 * a.cluster) >= 2 * kThreads) a.cluster *= 2;
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
