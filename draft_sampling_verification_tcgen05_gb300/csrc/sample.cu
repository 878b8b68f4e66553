// Sampling with temperature, top-k, min-p and top-p from given uniforms.
//
// The kept set is a prefix of the entries ordered by (logit, largest first; id, smallest first), so it
// is described by its last entry, the cut, and every sum is of integers (a weight's mass is
// floor(w * 2^40)), so the cut, the total and the token depend on no order of summation.
//
// With as many rows as SMs a row is a block's, which passes over it in memory (the rows under way
// fit the L2 cache, so later passes find them there), and the blocks take row after row from a queue,
// the longest first; with fewer rows a cluster of 2 to 16 blocks
// shares a row, each with a copy of its part in shared memory.  Sums, counts and lists then travel as
// asynchronous stores into the receiving block's shared memory that complete on an mbarrier there (a
// cluster's barrier waits for all earlier stores: 2000 cycles and more each time, an exchange takes a
// third of that).  A warp passes over a run of neighbouring entries, so sums by id come with any pass.
// What a row needs, and no more, is done:
//   1. the largest entry, and the largest of each thread; a greedy row is settled by that
//   2. with a small top-k: a histogram of the largest logits of groups of entries (at least 2 k groups)
//      gives a bound that at least k entries reach; those entries, usually a few more than k, go to a
//      list from the threads' parts whose largest entry reaches it, and one block settles min-p, top-p and the token on it: a histogram of counts and masses
//      over 1024 parts of the range, then over the part that holds the cut, until that is one entry
//   3. else the total mass of the entries that min-p leaves; entries of mass at most (Q - need) / count
//      cannot be needed for top-p
//   4. the cut is closed in on among the others: a histogram of counts over 2048 parts of their range,
//      bounds of each part's mass from its edges, the parts that can hold the cut are the next range,
//      and the mass above it is summed exactly; once the range's entries fit the list, they are settled
//      there; a range that bounds do not make smaller (two logits, many times each, where the wanted mass is
//      reached between them) is halved by an exact sum; a range of one repeated logit is settled by id
//   5. the token, where the list did not give it: kept masses of the runs, then the run that holds the
//      drawn mass again.  Probabilities: zeros and the list's entries, or a pass over the row
// A row that needs 3 and 4 is bound by its instructions (an exponential and an exact mass per entry and
// pass), the others by memory.  576 rows of 151936 with their distributions (700 MB), every third row without
// top-k, take 303 us, 2.3 TB/s: about 123 us for such a row on its SM, 41 us for one with a list, 24 us for a
// greedy one.  Rows in their order 443 us, the longest first 366 us, from a queue 332 us, lean passes where neither
// top-k nor min-p is set 314 us (with the sum above the cut and its list in passes of their own 326 us), packed
// arithmetic 307 us, a list from the parts that reach it 303 us; two blocks of half the threads per SM 446 us (the
// rows under way no longer fit the L2 cache).  One row takes 11 us, a chain of exchanges.
#include "attention_common.cuh"
#include "device_common.cuh"
#include "half_common.cuh"
#include "host_common.h"

#include <algorithm>

namespace dspark {
namespace {

constexpr int kMaxCluster = 16;
constexpr int kPlanThreads = 1024;
constexpr int kList = 2048;                // entries of the list
constexpr int kBins = 2048;
// What depends on the threads of a block.
template <int kThreads>
struct Block {
    static constexpr int kWarps = kThreads / 32;
    static constexpr int kPerThread = kBins / kThreads;
    static constexpr int kParts = kThreads;                       // of the list's range, a thread each
    static constexpr int kHist = 3 * kParts > kBins ? 3 * kParts : kBins;
};
constexpr int kFew = 256;                  // entries that are settled by comparing each with all
constexpr int kBatch = 4;                  // 16-byte pieces that a thread has under way
constexpr uint32_t kWaitPeer = 0xA01;
// A test build makes a wait run out: limits of 2 ms, and block DSPARK_LATE_RANK of a cluster 20 ms late at its
// exchange DSPARK_LATE_AT (expressions in the names of sample_row).
#ifdef DSPARK_LATE_AT
constexpr long long kPeerLimitNs = 2000000;
#else
constexpr long long kPeerLimitNs = kDefaultTimeoutNs;
#endif
constexpr long long kUnderWayNs = 100000;  // far more than a store into another block's shared memory takes

struct Plan {
    WsHeader header;
    unsigned int next;                     // of the queue
    int pad[63];
};

struct SampleArgs {
    const void* logits;
    const float* temperature;
    const int32_t* top_k;
    const float *top_p, *min_p, *u;
    int R, V;
    int cluster, slice;                    // blocks of a row, entries of a block
    int resident;                          // a block's part is held in shared memory
    int queue;                             // blocks take row after row
    int32_t* tokens;
    float* probs;
    WsHeader* ws;
    Plan* plan;
    int32_t* order;                        // with a queue: the rows as they are taken
};

using u64 = unsigned long long;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Address of the same shared variable in block `rank` of the cluster.
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
// Asynchronous stores and an addition there, counted in bytes on an mbarrier of the same block.
__device__ __forceinline__ void send(uint32_t at, u64 v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];"
                 :: "r"(at), "l"(v), "r"(bar) : "memory");
}
__device__ __forceinline__ void send32(uint32_t at, uint32_t v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];"
                 :: "r"(at), "r"(v), "r"(bar) : "memory");
}
__device__ __forceinline__ void send_add(uint32_t at, uint32_t v, uint32_t bar) {
    asm volatile("red.async.relaxed.cluster.shared::cluster.mbarrier::complete_tx::bytes.add.u32 [%0], %1, [%2];"
                 :: "r"(at), "r"(v), "r"(bar) : "memory");
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// floor(total * frac / 2^24), total < 2^62, frac <= 2^24.
__device__ __forceinline__ u64 share_of(u64 total, uint32_t frac) {
    return (total >> 24) * frac + (((total & 0xFFFFFFull) * frac) >> 24);
}

// floor(w * 2^40) in two halves of 20 bits, w <= 1.  Scalings by 2^20 are exact; adding 2^23 rounded toward
// zero leaves the floor of a value below 2^23 in the low bits (a conversion instruction runs at an
// eighth of an addition's rate).  The halves come with 2^23's bits, kHalfBias, on top.
constexpr uint32_t kHalfBias = 0x4B000000u;
__device__ __forceinline__ void mass_halves_biased(float w, uint32_t& hi, uint32_t& lo) {
    const float s = __fmul_rn(w, 0x1p20f), t = __fadd_rz(s, 0x1p23f);
    hi = __float_as_uint(t);
    lo = __float_as_uint(__fadd_rz(__fmul_rn(__fsub_rn(s, __fsub_rn(t, 0x1p23f)), 0x1p20f), 0x1p23f));
}
__device__ __forceinline__ void mass_halves(float w, uint32_t& hi, uint32_t& lo) {
    mass_halves_biased(w, hi, lo);
    hi -= kHalfBias;
    lo -= kHalfBias;
}
__device__ __forceinline__ u64 mass_of(float w) {
    uint32_t hi, lo;
    mass_halves(w, hi, lo);
    return (static_cast<u64>(hi) << 20) + lo;
}
// A sum of masses, of fewer than 4096 entries, which are counted apart (by the piece where all are added).
struct MassSum {
    uint32_t hi = 0, lo = 0, n = 0;
    __device__ __forceinline__ void add(float w) {
        uint32_t h, l;
        mass_halves_biased(w, h, l);
        hi += h;
        lo += l;
    }
    // Two masses at once, by packed instructions (the same roundings).
    __device__ __forceinline__ void add(float2 w) {
        const float2 scale = make_float2(0x1p20f, 0x1p20f), one = make_float2(0x1p23f, 0x1p23f);
        const float2 s = __fmul2_rn(w, scale), t = __fadd2_rz(s, one);
        const float2 rest = __fadd2_rn(s, __fadd2_rn(one, make_float2(-t.x, -t.y)));
        const float2 u = __fadd2_rz(__fmul2_rn(rest, scale), one);
        hi += __float_as_uint(t.x) + __float_as_uint(t.y);
        lo += __float_as_uint(u.x) + __float_as_uint(u.y);
    }
    __device__ __forceinline__ void count(uint32_t k) { n += k; }             // entries that were added
    __device__ __forceinline__ u64 value() const {
        return (static_cast<u64>(hi - n * kHalfBias) << 20) + (lo - n * kHalfBias);
    }
};
// floor(y) for 0 <= y < 2^23, likewise.
__device__ __forceinline__ int floor_of(float y) {
    return static_cast<int>(__float_as_uint(__fadd_rz(y, 0x1p23f)) - kHalfBias);
}

template <int kThreads>
struct alignas(16) Shared {
    static constexpr int kWarps = Block<kThreads>::kWarps, kHist = Block<kThreads>::kHist;
    u64 red[2][kMaxCluster][4];            // values exchanged by the blocks, two exchanges in turn
    union {
        u64 list[kList];                   // argmax keys: of this block, then in the first block of all
        struct {                           // while there is no list:
            uint32_t share[kBins];         // all blocks' counts of the bins that this block adds up
            uint32_t bins[kBins];          // in the first block: all blocks' counts
        };
    };
    uint32_t hist[kHist];                  // counts (kBins), or on the list counts and masses' halves of kParts parts
    u64 segment[kMaxCluster * kWarps];     // of the first block: mass or count of each warp's run
    u64 warp_sum[4][kWarps];
    u64 out[4];                            // what the first block tells the others
    u64 run[kWarps];                       // mass of the list's entries in each run of this block
    u64 found;                             // the entry that locate() was asked for
    uint32_t list_count, next;
    u64 bar_red[2], bar_out, bar_hist, bar_list, bar_segment, bar_found, bar_share, bar_bins;
};

struct Reduced { u64 a, b, c, d; };

// ---------------------------------------------------------------------------
// Plan: one block.  Clears the status word and the queue and, where the blocks take their rows from a
// queue, orders the rows by what they take, the longest first.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads) sample_plan_kernel(const __grid_constant__ SampleArgs p) {
    constexpr int kKinds = 5;
    __shared__ int s_at[kKinds];
    const int tid = threadIdx.x;
    grid_dependency_launch();                                                 // the other kernel's blocks get ready
    if (tid < static_cast<int>(sizeof(Plan) / 4)) reinterpret_cast<uint32_t*>(p.plan)[tid] = 0u;
    if (!p.queue) return;
    auto kind = [&](int r) {                                // closed in on; all summed; on a long list; a short one; greedy
        const int k = p.top_k[r];
        if (!(p.temperature[r] > 0.0f) || k == 1) return 4;
        if (k > 0 && k <= kList / 2) return k > kFew ? 2 : 3;
        return p.top_p[r] < 1.0f ? 0 : 1;
    };
    if (tid < kKinds) s_at[tid] = 0;
    __syncthreads();
    for (int r = tid; r < p.R; r += kPlanThreads)
        for (int x = kind(r) + 1; x < kKinds; ++x) atomicAdd(&s_at[x], 1);    // rows ahead of the later kinds
    __syncthreads();
    for (int r = tid; r < p.R; r += kPlanThreads) p.order[atomicAdd(&s_at[kind(r)], 1)] = r;
}

// One row.  False, in all threads of the block, where a wait for the other blocks gave up: nothing is sent
// or written any more then.
template <typename T, int kThreads>
__device__ __forceinline__ bool sample_row(const SampleArgs& p, Shared<kThreads>& s, T* const held, const long long r) {
    constexpr int kWarps = Block<kThreads>::kWarps, kPerThread = Block<kThreads>::kPerThread, kParts = Block<kThreads>::kParts;
    const int tid = threadIdx.x, V = p.V;
    const uint32_t warp = warp_id(), lane = lane_id();
    const int C = p.cluster;
    const uint32_t rank = C > 1 ? cluster_rank() : 0u;
    const T* const global = static_cast<const T*>(p.logits) + r * V;
    const int v0 = min(V, static_cast<int>(rank) * p.slice), v1 = min(V, v0 + p.slice), n = v1 - v0;

    for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0u;
    if (tid == 0) s.list_count = 0u;
    if (C > 1) {
        if (tid == 0) {
            for (u64* b = s.bar_red; b <= &s.bar_bins; ++b) mbar_init(reinterpret_cast<uint64_t*>(b), 1);
            fence_mbarrier_init();
        }
        __syncthreads();
        // the others may write here from now on; waited for ahead of the first exchange
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    // Waits for `bytes` that other blocks send to `bar` here; `uses` counts its phases.  All of the block's threads
    // come out with the same `ok`: whoever finds it false leaves sample_row.
    bool ok = true;
    auto receive = [&](u64& bar, int& uses, uint32_t bytes) {
        uint64_t* b = reinterpret_cast<uint64_t*>(&bar);
        if (tid == 0) mbar_arrive_expect_tx(b, bytes);
        const bool there = mbar_wait(b, static_cast<uint32_t>(uses++) & 1u, p.ws, kPeerLimitNs, kWaitPeer);
        ok = __syncthreads_and(there) != 0;
    };
    int used_red[2] = {0, 0}, used_out = 0, used_hist = 0, used_list = 0, used_segment = 0, used_found = 0, used_share = 0,
        used_bins = 0;

    // ---- parameters, each read as the nearest valid value ----
    uint32_t flags = 0;
    float temp = p.temperature[r], top_p = p.top_p[r], min_p = p.min_p[r], u = p.u[r];
    int k = p.top_k[r];
    if (!(temp >= 0.0f) || isinf(temp)) { temp = 0.0f; flags |= DSPARK_STATUS_NUMERIC; }
    if (!(top_p >= 0.0f && top_p <= 1.0f)) { top_p = top_p < 0.0f ? 0.0f : 1.0f; flags |= DSPARK_STATUS_INPUT_RANGE; }
    if (!(min_p >= 0.0f && min_p <= 1.0f)) { min_p = min_p > 1.0f ? 1.0f : 0.0f; flags |= DSPARK_STATUS_INPUT_RANGE; }
    if (!(u >= 0.0f && u < 1.0f)) { u = u >= 1.0f ? 0x1.fffffep-1f : 0.0f; flags |= DSPARK_STATUS_INPUT_RANGE; }
    if (k <= 0 || k > V) k = V;
    if (temp == 0.0f) k = 1;
    const float inv = temp == 0.0f ? 1.0f : fminf(__fdiv_rn(1.0f, temp), 3.402823466e+38f);
    const uint32_t P = static_cast<uint32_t>(top_p * 0x1p24f), U = static_cast<uint32_t>(u * 0x1p24f);

    // Ordered bits of an entry; 0 for one that takes no part (NaN, infinities).
    auto bits = [](float x) { return x < INFINITY && x > -INFINITY ? float_order_bits(x) : 0u; };
    auto key_of = [](float x, int v) { return argmax_key(x, static_cast<uint32_t>(v)); };
    auto key_logit = [](u64 key) { return float_from_order_bits(static_cast<uint32_t>(key >> 32)); };

    // ---- exchanges ----
    int turn = 0;
#ifdef DSPARK_LATE_AT
    int exchanges = 0;
#endif
    // Every block's four values, added up (a, b) or by maximum (c, d); the arguments count in thread 0 only.
    // Afterwards s.red[turn ^ 1][i] holds block i's.
    auto exchange = [&](u64 a, u64 b, u64 c, u64 d) {
#ifdef DSPARK_LATE_AT
        if (C > 1 && exchanges++ == DSPARK_LATE_AT && rank == DSPARK_LATE_RANK) {
            const long long t0 = global_ns();
            while (global_ns() - t0 < 20000000) {
            }
        }
#endif
        if (tid == 0) {
            u64* mine = s.red[turn][rank];
            mine[0] = a; mine[1] = b; mine[2] = c; mine[3] = d;
        }
        __syncthreads();
        if (C > 1) {
            const uint32_t to = static_cast<uint32_t>(tid >> 2);
            if (tid < C * 4 && to != rank)
                send(remote(&s.red[turn][rank][tid & 3], to), s.red[turn][rank][tid & 3], remote(&s.bar_red[turn], to));
            receive(s.bar_red[turn], used_red[turn], static_cast<uint32_t>(C - 1) * 32u);
        }
        Reduced x{0, 0, 0, 0};
        if (!ok) return x;
        for (int i = 0; i < C; ++i) {
            const u64* y = s.red[turn][i];
            x.a += y[0];
            x.b += y[1];
            x.c = max(x.c, y[2]);
            x.d = max(x.d, y[3]);
        }
        turn ^= 1;
        return x;
    };
    // Sums (a, b) and maxima (c, d) over the block's threads, in its first warp.
    auto block = [&](u64& a, u64& b, u64& c, u64& d) {
        a = warp_sum_u64(a);
        b = warp_sum_u64(b);
        c = warp_max_u64(c);
        d = warp_max_u64(d);
        __syncthreads();
        if (lane == 0) {
            s.warp_sum[0][warp] = a;
            s.warp_sum[1][warp] = b;
            s.warp_sum[2][warp] = c;
            s.warp_sum[3][warp] = d;
        }
        __syncthreads();
        if (warp == 0) {
            const bool in = lane < kWarps;
            a = warp_sum_u64(in ? s.warp_sum[0][lane] : 0);
            b = warp_sum_u64(in ? s.warp_sum[1][lane] : 0);
            c = warp_max_u64(in ? s.warp_sum[2][lane] : 0);
            d = warp_max_u64(in ? s.warp_sum[3][lane] : 0);
        }
    };
    static_assert(kWarps <= 32, "a warp adds up the warps");
    auto reduce = [&](u64 a, u64 b, u64 c, u64 d) {
        block(a, b, c, d);
        return exchange(a, b, c, d);
    };
    // Inclusive sums over the block's threads, on top of a0 and b0.
    auto scan = [&](u64& a, u64& b, u64 a0, u64 b0) {
        for (int d = 1; d < 32; d <<= 1) {
            const u64 y = __shfl_up_sync(0xFFFFFFFFu, a, d), z = __shfl_up_sync(0xFFFFFFFFu, b, d);
            if (lane >= static_cast<uint32_t>(d)) {
                a += y;
                b += z;
            }
        }
        if (lane == 31) {
            s.warp_sum[0][warp] = a;
            s.warp_sum[1][warp] = b;
        }
        __syncthreads();
        // the warps' sums ahead of this one
        u64 y = lane < warp ? s.warp_sum[0][lane] : 0, z = lane < warp ? s.warp_sum[1][lane] : 0;
        a += a0 + warp_sum_u64(y);
        b += b0 + warp_sum_u64(z);
    };
    // What the first block has put into s.out, in every block.
    auto hear = [&] {
        if (rank == 0) {
            __syncthreads();
            const uint32_t to = static_cast<uint32_t>(tid >> 2);
            if (tid < C * 4 && to != 0) send(remote(&s.out[tid & 3], to), s.out[tid & 3], remote(&s.bar_out, to));
        } else {
            receive(s.bar_out, used_out, 32u);
        }
    };

    // ---- the row, in 16-byte pieces: entry e of piece i is place0 + i * kPiece + e ----
    // The first and last piece may reach into the rows beside this one; in shared memory they stay pieces.
    constexpr int kPiece = 16 / sizeof(T);
    const int pad = static_cast<int>((reinterpret_cast<uintptr_t>(global + v0) & 15u) / sizeof(T));
    const int pieces = n > 0 ? (pad + n + kPiece - 1) / kPiece : 0, place0 = v0 - pad;
    const uint4* const row16 = reinterpret_cast<const uint4*>(global + place0);
    const int per_run = (pieces + kWarps - 1) / kWarps;
    const int run0 = min(pieces, static_cast<int>(warp) * per_run), run1 = min(pieces, run0 + per_run);   // this warp's
    auto whole = [&](int i) { return place0 + i * kPiece >= v0 && place0 + (i + 1) * kPiece <= v1; };
    auto fetch = [&](int i, bool from_memory) {                               // piece i; 0 outside the row
        if (!from_memory) return reinterpret_cast<const uint4*>(held)[i];
        if (whole(i)) return __ldg(row16 + i);
        T y[kPiece];
        for (int e = 0; e < kPiece; ++e) {
            const int v = place0 + i * kPiece + e;
            y[e] = v >= v0 && v < v1 ? global[v] : T(0.0f);
        }
        return *reinterpret_cast<const uint4*>(y);
    };
    auto unpack = [&](const uint4& w, int i, float (&x)[kPiece]) {            // as fp32; NaN outside the row
        T y[kPiece];
        *reinterpret_cast<uint4*>(y) = w;
#pragma unroll
        for (int e = 0; e < kPiece; ++e) x[e] = to_float(y[e]);
        if (!whole(i)) {
#pragma unroll
            for (int e = 0; e < kPiece; ++e) {
                const int v = place0 + i * kPiece + e;
                if (v < v0 || v >= v1) x[e] = NAN;
            }
        }
    };
    // Calls f(piece, its entries) for this warp's run, by whole warps; entries outside the row, and pieces past
    // the run's end, come as NaN.
    const int whole0 = pad > 0 ? 1 : 0, whole1 = min(run1, (pad + n) / kPiece);   // pieces wholly inside, of this run
    auto pass = [&](bool from_memory, auto f) {
        int i0 = run0;
        for (; i0 < run1; ) {
            const bool full = i0 >= whole0 && i0 + 32 * kBatch <= whole1;
            if (full) {
                uint4 w[kBatch];
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    const int i = i0 + j * 32 + static_cast<int>(lane);
                    w[j] = from_memory ? __ldg(row16 + i) : reinterpret_cast<const uint4*>(held)[i];
                }
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    T y[kPiece];
                    *reinterpret_cast<uint4*>(y) = w[j];
                    float x[kPiece];
#pragma unroll
                    for (int e = 0; e < kPiece; ++e) x[e] = to_float(y[e]);
                    f(i0 + j * 32 + static_cast<int>(lane), x, w[j], j);
                }
                i0 += 32 * kBatch;
            } else {
                const int i = i0 + static_cast<int>(lane);
                const uint4 w = i < run1 ? fetch(i, from_memory) : make_uint4(0u, 0u, 0u, 0u);
                float x[kPiece];
                unpack(w, i, x);
                if (i >= run1) {
#pragma unroll
                    for (int e = 0; e < kPiece; ++e) x[e] = NAN;
                }
                f(i, x, w, 0);
                i0 += 32;
            }
        }
    };
    const bool streamed = p.resident == 0;

    // ---- 1. the largest entries ----
    float tops[kBatch];                                                       // of this thread's pieces, in turn
    int at[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
        tops[j] = -INFINITY;
        at[j] = 0;
    }
    uint32_t odd = 0;
    pass(true, [&](int i, float (&x)[kPiece], const uint4& w, int j) {
        if (!streamed && i < run1) reinterpret_cast<uint4*>(held)[i] = w;
        float top = x[0], sum = x[0];
#pragma unroll
        for (int e = 1; e < kPiece; ++e) {
            top = fmaxf(top, x[e]);
            sum += x[e];
        }
        if (top == INFINITY || !(sum == sum)) {                               // rare: something that is skipped
            top = -INFINITY;
#pragma unroll
            for (int e = 0; e < kPiece; ++e) {
                const int v = place0 + i * kPiece + e;
                if (!(x[e] < INFINITY)) odd |= i < run1 && v >= v0 && v < v1 ? 1u : 0u;    // not what lies outside
                else top = fmaxf(top, x[e]);
            }
        }
        if (top > tops[j]) {
            tops[j] = top;
            at[j] = i;
        }
    });
    __syncwarp();
    // this thread's largest entry: the first of them within the first piece that has it
    u64 best = 0;
    {
        float top = tops[0];
        int i = at[0];
#pragma unroll
        for (int j = 1; j < kBatch; ++j)
            if (tops[j] > top || (tops[j] == top && at[j] < i)) {
                top = tops[j];
                i = at[j];
            }
        if (top > -INFINITY) {
            float x[kPiece];
            unpack(fetch(i, streamed), i, x);
#pragma unroll
            for (int e = kPiece - 1; e >= 0; --e)
                if (x[e] == top) best = key_of(top, place0 + i * kPiece + e);
        }
    }
    if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    // For a small top-k: groups of entries, at least 2 k of them if there can be, and their largest: 1 to 32
    // threads' entries, or a thread's every kBatch-th piece.
    int span = 32;
    while (span > 1 && (C * kThreads) / span < 2 * k) span >>= 2;             // 32, 8, 2, 0: single threads
    span = max(span, 1);
    const bool fine = C * kThreads < 2 * k;
    uint32_t group = static_cast<uint32_t>(best >> 32);
    for (int d = 1; d < span; d <<= 1) group = max(group, __shfl_xor_sync(0xFFFFFFFFu, group, d));
    uint32_t leads = group != 0 && (lane & (span - 1)) == 0 ? 1u : 0u, least_group = group;
    if (fine) {
        leads = 0;
        least_group = 0xFFFFFFFFu;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const uint32_t b = bits(tops[j]);
            if (b == 0) continue;
            ++leads;
            least_group = min(least_group, b);
        }
        if (leads == 0) least_group = 0;
    }
    // c: the largest entry; d: the smallest of the groups' largest, as its complement
    const Reduced x = reduce(odd, leads, best, least_group != 0 ? 0xFFFFFFFFu - least_group : 0u);
    if (!ok) return false;
    if (x.a != 0) flags |= DSPARK_STATUS_NUMERIC;
    const bool clean = x.a == 0;                                              // no NaN, no infinity but -infinity
    const uint32_t top_bits = static_cast<uint32_t>(x.c >> 32);
    if (top_bits == 0) flags |= DSPARK_STATUS_NUMERIC;
    if (rank == 0 && tid == 0 && flags) set_status(p.ws, flags);
    const float m = float_from_order_bits(top_bits);
    const int groups = static_cast<int>(x.b);                                 // groups with an entry
    const float bottom = float_from_order_bits(0xFFFFFFFFu - static_cast<uint32_t>(x.d));

    auto weight = [&](float l) { return expf(__fmul_rn(__fsub_rn(l, m), inv)); };
    auto weights = [&](float l, float k) {
        const float2 y = __fmul2_rn(__fadd2_rn(make_float2(l, k), make_float2(-m, -m)), make_float2(inv, inv));
        return make_float2(expf(y.x), expf(y.y));
    };

    u64 cut = 0, total = 0;                                                   // the kept set: key >= cut; its mass
    u64 limit = 0;                                                            // likewise after top-k, while top-p is sought
    int token = -1;                                                           // once it is known
    bool in_list = false;                                                     // the blocks' lists hold the kept set
    // Calls f(logit, id, whether it takes part so far) for the entries of at least `least`, where few are: by
    // whole warps, a warp being there as long as one of its entries is.
    auto each = [&](float least, auto f) {
        pass(streamed, [&](int i, const float (&x)[kPiece], const uint4&, int) {
            float top = x[0];
#pragma unroll
            for (int e = 1; e < kPiece; ++e) top = fmaxf(top, x[e]);
            if (!__any_sync(0xFFFFFFFFu, top >= least)) return;
#pragma unroll
            for (int e = 0; e < kPiece; ++e) {
                bool in = x[e] >= least && x[e] < INFINITY;
                if (!__any_sync(0xFFFFFFFFu, in)) continue;
                const int v = place0 + i * kPiece + e;
                if (limit != 0) in = in && key_of(x[e], v) >= limit;
                f(x[e], v, in);
            }
        });
    };
    // The same, by threads, where many are: only for those that take part.
    auto every = [&](float least, auto f) {
        pass(streamed, [&](int i, const float (&x)[kPiece], const uint4&, int) {
#pragma unroll
            for (int e = 0; e < kPiece; ++e) {
                if (!(x[e] >= least && x[e] < INFINITY)) continue;
                const int v = place0 + i * kPiece + e;
                if (limit != 0 && key_of(x[e], v) < limit) continue;
                f(x[e], v);
            }
        });
    };
    // Entries for which `yes` go to this block's list, as long as they fit.
    auto append = [&](bool yes, float l, int v) {
        const uint32_t vote = __ballot_sync(0xFFFFFFFFu, yes);
        if (vote == 0) return;
        uint32_t at = 0;
        if (lane == 0) at = atomicAdd(&s.list_count, __popc(vote));
        at = __shfl_sync(0xFFFFFFFFu, at, 0) + __popc(vote & ((1u << lane) - 1u));
        if (yes && at < kList) s.list[at] = key_of(l, v);
    };
    // The blocks' lists, one behind the other, in the first block, unless they are more than kList together;
    // tells their number.  Every block's own entries stay the first s.list_count of its list.
    auto gather = [&] {
        __syncthreads();
        const uint32_t mine = s.list_count;
        const Reduced all = exchange(mine, 0, 0, 0);
        if (!ok) return 0;
        if (all.a <= kList && C > 1) {
            if (rank != 0) {
                uint32_t before = 0;
                for (int i = 0; i < static_cast<int>(rank); ++i) before += static_cast<uint32_t>(s.red[turn ^ 1][i][0]);
                for (uint32_t i = tid; i < mine; i += kThreads)
                    send(remote(&s.list[before + i], 0), s.list[i], remote(&s.bar_list, 0));
            } else {
                receive(s.bar_list, used_list, 8u * static_cast<uint32_t>(all.a - mine));
                if (!ok) return 0;
            }
        }
        __syncthreads();
        if (tid == 0) s.list_count = all.a <= kList ? mine : 0u;
        __syncthreads();
        return static_cast<int>(min(all.a, static_cast<u64>(kList) + 1));
    };

    // First block: settles the cut on the list of `count` entries, behind `above` entries of mass `over`: at
    // most kk entries in all, and of those as many as reach the mass `need` (~0: top-p's share of them).
    // Leaves {cut, mass, token + 1 if nothing is above the list, else 0} in s.out.
    auto settle = [&](int count, u64 above, u64 over, u64 kk, u64 need) {
        if (count <= kFew) {
            // a thread per entry: its rank and the mass before it, by comparison with all entries
            u64* const masses = reinterpret_cast<u64*>(s.hist);
            u64 key = 0, mass = 0;
            if (tid < count) {
                key = s.list[tid];
                const float w = weight(key_logit(key));
                mass = w < min_p ? ~0ull : mass_of(w);                        // ~0: it takes no part
                masses[tid] = mass;
            }
            const bool part = tid < count && mass != ~0ull;
            __syncthreads();
            u64 rank_of = above, before = over;
            if (part)
                for (int i = 0; i < count; ++i) {
                    const u64 other = s.list[i], q = masses[i];
                    if (other > key && q != ~0ull) {
                        ++rank_of;
                        before += q;
                    }
                }
            const bool counted = part && rank_of < kk;
            u64 sum = counted ? mass : 0, none = 0, zero = 0, nil = 0;
            block(sum, none, zero, nil);
            if (tid == 0) s.out[0] = over + sum;
            __syncthreads();
            const u64 upto_k = s.out[0];
            if (need == ~0ull) need = max(1ull, share_of(upto_k, P));
            const bool keep = counted && (before < need || rank_of == 0);
            const int number = __syncthreads_count(keep);
            if (keep && rank_of + 1 == above + static_cast<u64>(number)) {    // the last of them
                s.out[0] = key;
                s.out[1] = before + mass;
            }
            if (tid < count) masses[tid] = keep ? mass : 0;
            if (tid == 0) s.out[2] = 0;
            __syncthreads();
            if (above == 0 && keep) {
                // by id: the one in which the drawn mass falls
                const u64 t = share_of(s.out[1], U);
                const uint32_t id = key_index(key);
                u64 ahead = 0;
                for (int i = 0; i < count; ++i)
                    if (key_index(s.list[i]) < id) ahead += masses[i];
                if (ahead <= t && t < ahead + mass) s.out[2] = static_cast<u64>(id) + 1;
            }
            __syncthreads();
            return;
        }
        // this thread's entries that take part, and their masses' halves
        constexpr int kPer = kList / kThreads;
        u64 key[kPer];
        uint32_t qh[kPer], ql[kPer];
        u64 sum = 0, number = 0, low = 0, high = 0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int i = e * kThreads + tid;
            key[e] = i < count ? s.list[i] : 0;
            qh[e] = ql[e] = 0;
            if (key[e] == 0) continue;
            const float w = weight(key_logit(key[e]));
            if (w < min_p) {
                key[e] = 0;
                continue;
            }
            mass_halves(w, qh[e], ql[e]);
            sum += (static_cast<u64>(qh[e]) << 20) + ql[e];
            ++number;
            low = max(low, ~key[e]);
            high = max(high, key[e]);
        }
        block(sum, number, low, high);
        if (tid == 0) {
            s.out[0] = sum;
            s.out[1] = number;
            s.out[2] = ~low;
            s.out[3] = high;
        }
        __syncthreads();
        sum = s.out[0];
        number = s.out[1];
        const u64 bottom_key = s.out[2], top_key = s.out[3];
        // Of the entries with keys in [lo, hi], the largest key first, behind c_before entries of mass m_before:
        // the first with which the count reaches want_count, or the mass want_mass (the other is ~0); it is
        // there.  Returns its key, and the mass up to it.
        auto descend = [&](const u64 (&key)[kPer], u64 lo, u64 hi, u64 c_before, u64 m_before, u64 want_count, u64 want_mass,
                           u64& upto) {
            for (int level = 0; level < 8; ++level) {                         // 10 bits each time
                int shift = 0;
                while (((hi - lo) >> shift) >= kParts) ++shift;
                __syncthreads();
#pragma unroll
                for (int y = 0; y < 3; ++y) s.hist[y * kParts + tid] = 0u;
                __syncthreads();
#pragma unroll
                for (int e = 0; e < kPer; ++e) {
                    if (key[e] < lo || key[e] > hi) continue;
                    const int part = static_cast<int>((hi - key[e]) >> shift);
                    atomicAdd(&s.hist[part], 1u);
                    atomicAdd(&s.hist[kParts + part], qh[e]);
                    atomicAdd(&s.hist[2 * kParts + part], ql[e]);
                }
                __syncthreads();
                const u64 c = s.hist[tid], q = (static_cast<u64>(s.hist[kParts + tid]) << 20) + s.hist[2 * kParts + tid];
                u64 ci = c, qi = q;
                scan(ci, qi, c_before, m_before);
                const bool crosses = want_count != ~0ull ? ci - c < want_count && ci >= want_count
                                                         : qi - q < want_mass && qi >= want_mass;
                if (crosses) {
                    s.out[0] = static_cast<u64>(tid);
                    s.out[1] = c;
                    s.out[2] = ci - c;
                    s.out[3] = qi - q;
                }
                __syncthreads();
                const u64 part = s.out[0], in_part = s.out[1];
                c_before = s.out[2];
                m_before = s.out[3];
                const u64 first = hi - (part << shift), length = (1ull << shift) - 1;
                lo = first - lo > length ? first - length : lo;
                hi = first;
                if (in_part == 1) break;
            }
            // the one entry left
            __syncthreads();
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (key[e] >= lo && key[e] <= hi) {
                    s.out[0] = key[e];
                    s.out[1] = m_before + (static_cast<u64>(qh[e]) << 20) + ql[e];
                }
            __syncthreads();
            upto = s.out[1];
            return s.out[0];
        };
        u64 last = bottom_key, upto = over + sum;
        if (above + number > kk) last = descend(key, bottom_key, top_key, above, over, kk, ~0ull, upto);
        if (need == ~0ull) need = max(1ull, share_of(upto, P));
        if (need < upto) last = descend(key, last, top_key, above, over, ~0ull, need, upto);
        u64 drawn = 0;
        if (above == 0) {
            // by id: the first with which the mass exceeds the drawn share
            u64 id_key[kPer];
#pragma unroll
            for (int e = 0; e < kPer; ++e) id_key[e] = key[e] >= last ? (key[e] & 0xFFFFFFFFull) + 1 : 0;
            u64 unused;
            const u64 found = descend(id_key, 1, 1ull << 32, 0, 0, ~0ull, share_of(upto, U) + 1, unused);
            drawn = static_cast<u64>(key_index(found - 1)) + 1;
        }
        __syncthreads();
        if (tid == 0) {
            s.out[0] = last;
            s.out[1] = upto;
            s.out[2] = drawn;
        }
        __syncthreads();
    };
    auto settled_on_list = [&] {
        hear();
        cut = s.out[0];
        total = s.out[1];
        token = static_cast<int>(s.out[2]) - 1;
        in_list = token >= 0;
    };

    bool settled = top_bits == 0 || k == 1;                                   // nothing to keep, or one entry
    if (settled) {
        cut = top_bits == 0 ? ~0ull : x.c;
        total = top_bits == 0 ? 0 : 1ull << 40;
        token = top_bits == 0 ? 0 : static_cast<int>(key_index(x.c));
        in_list = true;
        if (top_bits != 0 && token >= v0 && token < v1 && tid == 0) {
            s.list[0] = cut;
            s.list_count = 1u;
        }
        __syncthreads();
    }

    // ---- 2. a small top-k ----
    // A range that can be parted evenly (not of one value, and finite).
    auto even = [&](float lowest) { return m - lowest > 1e-30f && m - lowest < 1e38f; };
    if (!settled && k <= groups && k <= kList / 2 && even(bottom)) {
        const float scale = (kBins - 1) / (m - bottom);
        auto enter = [&](uint32_t b) {
            const int bin = min(kBins - 1, static_cast<int>((m - float_from_order_bits(b)) * scale));
            if (rank != 0) send_add(remote(&s.hist[bin], 0), 1u, remote(&s.bar_hist, 0));
            else atomicAdd(&s.hist[bin], 1u);
        };
        if (!fine) {
            if (leads != 0) enter(group);
        } else {
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (bits(tops[j]) != 0) enter(bits(tops[j]));
        }
        if (rank == 0) {
            if (C > 1) receive(s.bar_hist, used_hist, 4u * static_cast<uint32_t>(x.b - s.red[turn ^ 1][0][1]));
            if (!ok) return false;
            __syncthreads();
            // the first bin up to which there are k
            u64 c[kPerThread], sum = 0, none = 0;
#pragma unroll
            for (int e = 0; e < kPerThread; ++e) sum += c[e] = s.hist[tid * kPerThread + e];
            u64 incl = sum;
            scan(incl, none, 0, 0);
            u64 before = incl - sum;
#pragma unroll
            for (int e = 0; e < kPerThread; ++e) {
                if (before < static_cast<u64>(k) && before + c[e] >= static_cast<u64>(k))
                    s.out[0] = static_cast<u64>(tid * kPerThread + e);
                before += c[e];
            }
        }
        hear();
        if (!ok) return false;
        const float reach = static_cast<float>(s.out[0] + 1);
        // a logit that no entry of those parts is below
        const float least = m - reach / scale * (1.0f + 1e-5f) - fabsf(m) * 2.5e-7f;
        auto list = [&](float l, int v, bool in) { append(in && (m - l) * scale < reach, l, v); };
        // Few of the parts whose largest entries are known reach it, and only those are looked at again: the
        // j-th pieces of a lane, in all the full batches of this warp's run.
        uint8_t* const hot = reinterpret_cast<uint8_t*>(s.segment) + warp * (32 * kBatch);
        int parts = 0;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const uint32_t vote = __ballot_sync(0xFFFFFFFFu, tops[j] >= least);
            if (tops[j] >= least) hot[parts + __popc(vote & ((1u << lane) - 1u))] = static_cast<uint8_t>(j * 32 + lane);
            parts += __popc(vote);
        }
        __syncwarp();
        const int full0 = run0 < whole0 ? min(run1, run0 + 32) : run0;         // as pass() goes
        const int batches = max(0, (whole1 - full0) / (32 * kBatch)), full1 = full0 + 32 * kBatch * batches;
        if (4 * parts * batches > run1 - run0) {
            each(least, list);
        } else {
            auto look = [&](bool there, int i, const uint4& w) {
                float x[kPiece];
                unpack(w, i, x);
#pragma unroll
                for (int e = 0; e < kPiece; ++e) {
                    const bool in = there && x[e] >= least && x[e] < INFINITY;
                    if (__any_sync(0xFFFFFFFFu, in)) list(x[e], place0 + i * kPiece + e, in);
                }
            };
            for (int end = 0; end < 2; ++end) {                               // what is in no full batch
                const int to = end == 0 ? full0 : run1;
                for (int i0 = end == 0 ? run0 : full1; i0 < to; i0 += 32) {
                    const int i = i0 + static_cast<int>(lane);
                    look(i < to, i, i < to ? fetch(i, streamed) : make_uint4(0u, 0u, 0u, 0u));
                }
            }
            const int work = parts * batches;
            for (int t0 = 0; t0 < work; t0 += 64) {
                uint4 w[2];
                int at_piece[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int t = t0 + 32 * y + static_cast<int>(lane);
                    const int part = t / batches, id = t < work ? hot[part] : 0;
                    at_piece[y] = t < work ? full0 + (t - part * batches) * (32 * kBatch) + id : run0;
                    w[y] = t < work ? fetch(at_piece[y], streamed) : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int y = 0; y < 2; ++y) look(t0 + 32 * y + static_cast<int>(lane) < work, at_piece[y], w[y]);
            }
        }
        const int count = gather();
        if (!ok) return false;
        if (count <= kList) {
            if (rank == 0) settle(count, 0, 0, static_cast<u64>(k), ~0ull);
            settled_on_list();
            if (!ok) return false;
            settled = true;
        }
    }

    // With every run's sum in the first block's s.segment: the first id at which the sum of value(logit, id)
    // over all ids up to it exceeds t, known to one warp of the cluster, which calls found(id) in all lanes.
    auto locate = [&](u64 t, auto value, auto found) {
        if (rank == 0) {
            if (C > 1) receive(s.bar_segment, used_segment, static_cast<uint32_t>(C - 1) * kWarps * 8u);
            if (!ok) return;
            __syncthreads();
        }
        if (rank == 0 && warp == 0) {
            u64 before = 0;
            for (int i0 = 0; i0 < C * kWarps; i0 += 32) {
                const u64 mass = i0 + static_cast<int>(lane) < C * kWarps ? s.segment[i0 + lane] : 0;
                u64 incl = mass;
                for (int d = 1; d < 32; d <<= 1) {
                    const u64 y = __shfl_up_sync(0xFFFFFFFFu, incl, d);
                    if (lane >= static_cast<uint32_t>(d)) incl += y;
                }
                incl += before;
                if (incl > t && incl - mass <= t) {
                    s.out[0] = static_cast<u64>(i0) + lane;
                    s.out[1] = t - (incl - mass);
                }
                before = __shfl_sync(0xFFFFFFFFu, incl, 31);
            }
        }
        hear();
        if (!ok) return;
        if (s.out[0] == rank * kWarps + warp) {
            // a lane sums neighbouring pieces of the run; then the lanes share the pieces of the one it is in
            u64 left = s.out[1];
            const int per_lane = ((run1 - run0 + 31) / 32) | 1;               // odd: the lanes meet no bank twice
            int a0 = min(run1, run0 + static_cast<int>(lane) * per_lane), a1 = min(run1, a0 + per_lane);
            auto add = [&](int i) {
                float y[kPiece];
                unpack(fetch(i, streamed), i, y);
                u64 sum = 0;
#pragma unroll
                for (int e = 0; e < kPiece; ++e) sum += value(y[e], place0 + i * kPiece + e);
                return sum;
            };
            auto pick = [&](u64 own, int& at) {                               // the lane whose sum passes `left`
                u64 incl = own;
                for (int d = 1; d < 32; d <<= 1) {
                    const u64 y = __shfl_up_sync(0xFFFFFFFFu, incl, d);
                    if (lane >= static_cast<uint32_t>(d)) incl += y;
                }
                const uint32_t vote = __ballot_sync(0xFFFFFFFFu, incl > left);
                at = vote != 0 ? __ffs(static_cast<int>(vote)) - 1 : 31;
                const u64 y = __shfl_sync(0xFFFFFFFFu, vote != 0 ? incl - own : incl, at);
                left -= y;
                return vote != 0;
            };
            u64 sum = 0;
            for (int i = a0; i < a1; ++i) sum += add(i);
            int at;
            if (pick(sum, at)) {
                a0 = __shfl_sync(0xFFFFFFFFu, a0, at);
                a1 = __shfl_sync(0xFFFFFFFFu, a1, at);
                for (int i = a0; i < a1; i += 32) {
                    const int mine = i + static_cast<int>(lane);
                    if (!pick(mine < a1 ? add(mine) : 0, at)) continue;
                    float y[kPiece];
                    unpack(fetch(i + at, streamed), i + at, y);
                    int v = place0 + (i + at) * kPiece;
#pragma unroll
                    for (int e = 0; e < kPiece; ++e) {
                        const u64 q = value(y[e], v);
                        if (q > left) break;
                        left -= q;
                        ++v;
                    }
                    found(v);
                    break;
                }
            }
        }
    };
    auto report_run = [&](u64 sum) {                                          // lane 0's: this run's sum
        if (lane != 0) return;
        if (rank != 0) send(remote(&s.segment[rank * kWarps + warp], 0), sum, remote(&s.bar_segment, 0));
        else s.segment[warp] = sum;
    };
    auto set_token = [&](int v) {
        if (lane == 0) p.tokens[r] = v;
    };

    // ---- 3. and 4. ----
    bool runs_known = false;                                                  // the runs' kept masses are reported
    if (!settled) {
        // Closes in on the cut: the first entry of the order with which the count reaches `want_count`, or the
        // mass `want_mass` (the other is ~0).  `lowest`: no entry below this logit can be the cut.
        // Where the cut comes from a list, `run_mass` receives the mass that this warp's run has above the list.
        u64 run_mass = 0;
        auto close_in = [&](u64 want_count, u64 want_mass, float lowest) {
            u64 above = 0, over = 0;                                          // count and mass above the range
            run_mass = 0;
            runs_known = false;
            bool linear = even(lowest);                                       // parts of equal width, or of equal bits
            uint32_t hi = top_bits, lo = float_order_bits(lowest);
            for (int i = tid; i < kBins; i += kThreads) s.share[i] = 0u;
            exchange(0, 0, 0, 0);                                             // all blocks' shares are clear
            if (!ok) return;
            // A level leaves a range of less than half, or the next one halves it: the range is one logit, at the
            // latest, after twice the 32 bits.
            constexpr int kLevels = 72;
            bool halve = false;
            for (int level = 0; level < kLevels; ++level) {
                const float scale = linear ? kBins / (m - lowest) : 0.0f;
                int shift = 0;
                while (((hi - lo) >> shift) >= kBins) ++shift;
                const float from = float_from_order_bits(lo);
                // an entry's part, or kBins
                auto part_of = [&](float l, bool in) {
                    const uint32_t b = float_order_bits(l);
                    if (!in || b > hi || (min_p != 0.0f && weight(l) < min_p)) return kBins;
                    return linear ? min(kBins - 1, floor_of((m - l) * scale)) : static_cast<int>((hi - b) >> shift);
                };
                __syncthreads();
                if (tid == 0) s.list_count = 0u;
                for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0u;
                __syncthreads();
                const bool plain = linear && limit == 0 && min_p == 0.0f && clean;    // no more than the range to look at
                // The first and last part that can hold the cut, and whether the entries in them fit the list; to halve
                // the range, all the parts behind its middle.
                int first = (static_cast<int>((hi - lo) >> shift) + 1) / 2, last = kBins - 1;
                bool fits = false;
                if (!halve) {
                    if (plain) {
                        pass(streamed, [&](int, const float (&x)[kPiece], const uint4&, int) {
#pragma unroll
                            for (int e = 0; e < kPiece; ++e) {
                                const int part = min(kBins - 1, floor_of((m - x[e]) * scale));
                                if (x[e] >= from) atomicAdd(&s.hist[part], 1u);
                            }
                        });
                    } else {
                        every(from, [&](float l, int) {
                            const int part = part_of(l, true);
                            if (part < kBins) atomicAdd(&s.hist[part], 1u);
                        });
                    }
                    __syncthreads();
                    if (C > 1) {
                        // each block adds up its share of the bins over all blocks, for the first one
                        const int share = kBins / C, bin0 = static_cast<int>(rank) * share;
                        for (int i = tid; i < kBins; i += kThreads) {
                            const uint32_t to = static_cast<uint32_t>(i / share);
                            if (to != rank) send_add(remote(&s.share[i], to), s.hist[i], remote(&s.bar_share, to));
                            else atomicAdd(&s.share[i], s.hist[i]);
                        }
                        receive(s.bar_share, used_share, static_cast<uint32_t>((C - 1) * share) * 4u);
                        if (!ok) return;
                        __syncthreads();
                        for (int i = bin0 + tid; i < bin0 + share; i += kThreads) {
                            if (rank != 0) send32(remote(&s.bins[i], 0), s.share[i], remote(&s.bar_bins, 0));
                            else s.bins[i] = s.share[i];
                            s.share[i] = 0u;                                  // the next level comes after an exchange
                        }
                        if (rank == 0) receive(s.bar_bins, used_bins, static_cast<uint32_t>(kBins - share) * 4u);
                        if (!ok) return;
                    } else {
                        for (int i = tid; i < kBins; i += kThreads) s.bins[i] = s.hist[i];
                    }
                    __syncthreads();
                    if (rank == 0) {
                        // bounds of each part's mass from its edges, with room for the rounding of edges and expf
                        u64 c[kPerThread], least[kPerThread], most[kPerThread], in_least = 0, in_most = 0;
#pragma unroll
                        for (int e = 0; e < kPerThread; ++e) {
                            const int i = tid * kPerThread + e;
                            c[e] = s.bins[i];
                            least[e] = most[e] = c[e];
                            if (want_count == ~0ull) {
                                float hi_edge, lo_edge;
                                if (linear) {
                                    const float rounding = fabsf(m) * 2.5e-7f;
                                    hi_edge = m - (i / scale) * (1.0f - 1e-5f) + rounding;
                                    lo_edge = i == kBins - 1 ? lowest : m - ((i + 1) / scale) * (1.0f + 1e-5f) - rounding;
                                } else {
                                    const uint32_t first = hi - min(hi - lo, static_cast<uint32_t>(i) << shift);
                                    const uint32_t last = hi - min(hi - lo, (static_cast<uint32_t>(i + 1) << shift) - 1u);
                                    hi_edge = float_from_order_bits(first);
                                    lo_edge = float_from_order_bits(last);
                                }
                                most[e] = c[e] * (mass_of(fminf(1.0f, weight(hi_edge) * (1.0f + 1e-4f))) + 1);
                                least[e] = c[e] * mass_of(fminf(1.0f, fmaxf(0.0f, weight(lo_edge) * (1.0f - 1e-4f))));
                            }
                            in_least += least[e];
                            in_most += most[e];
                        }
                        u64 least_before = in_least, most_before = in_most;
                        if (tid == 0) s.out[0] = s.out[1] = kBins - 1;        // first and last part that can hold the cut
                        scan(least_before, most_before, 0, 0);
                        least_before -= in_least;
                        most_before -= in_most;
                        const u64 want = want_count != ~0ull ? want_count - above : want_mass - over;
#pragma unroll
                        for (int e = 0; e < kPerThread; ++e) {
                            const u64 i = static_cast<u64>(tid * kPerThread + e);
                            if (most_before < want && most_before + most[e] >= want) s.out[0] = i;
                            if (least_before < want && least_before + least[e] >= want) s.out[1] = i;
                            least_before += least[e];
                            most_before += most[e];
                        }
                        __syncthreads();
                        // the entries in those parts
                        u64 inside = 0, none = 0, zero = 0, nil = 0;
#pragma unroll
                        for (int e = 0; e < kPerThread; ++e) {
                            const u64 i = static_cast<u64>(tid * kPerThread + e);
                            if (i >= s.out[0] && i <= s.out[1]) inside += c[e];
                        }
                        block(inside, none, zero, nil);
                        if (tid == 0) s.out[2] = inside;
                    }
                    hear();
                    if (!ok) return;
                    first = static_cast<int>(s.out[0]);
                    last = static_cast<int>(s.out[1]);
                    fits = s.out[2] <= kList;
                }
                __syncthreads();                                              // the bins' place may become the list's
                // above those parts: summed; in them: listed if they fit, else bounded
                u64 more = 0, high = 0, low = 0;
                MassSum mass;
                auto inside = [&](float l, int v) {
                    if (fits) {
                        s.list[atomicAdd(&s.list_count, 1u)] = key_of(l, v);
                    } else {
                        high = max(high, static_cast<u64>(float_order_bits(l)));
                        low = max(low, static_cast<u64>(0xFFFFFFFFu - float_order_bits(l)));
                    }
                };
                if (plain) {
                    // The parts do not rise with the logit: bounds found once are compared with, instead of parts.
                    auto largest = [&](int part) {                            // ordered bits, of a logit of this part or a later one
                        uint32_t below = lo, above = top_bits + 1u;           // lo is in the last part, or beyond all
                        while (above - below > 1u) {
                            const uint32_t mid = below + (above - below) / 2u;
                            const float l = float_from_order_bits(mid);
                            if (min(kBins - 1, floor_of((m - l) * scale)) >= part) below = mid;
                            else above = mid;
                        }
                        return below;
                    };
                    const float ceiling = first > 0 ? float_from_order_bits(largest(first)) : INFINITY;   // above it: summed
                    const float ground = last < kBins - 1 ? float_from_order_bits(largest(last + 1) + 1u) : from;
                    uint32_t entries_above = 0;
                    pass(streamed, [&](int i, const float (&x)[kPiece], const uint4&, int) {
#pragma unroll
                        for (int e = 0; e < kPiece; e += 2) {
                            const bool in0 = x[e] > ceiling, in1 = x[e + 1] > ceiling;
                            const float2 w = weights(x[e], x[e + 1]);
                            mass.add(make_float2(in0 ? w.x : 0.0f, in1 ? w.y : 0.0f));
                            entries_above += (in0 ? 1u : 0u) + (in1 ? 1u : 0u);
                            if (x[e] >= ground && !in0) inside(x[e], place0 + i * kPiece + e);
                            if (x[e + 1] >= ground && !in1) inside(x[e + 1], place0 + i * kPiece + e + 1);
                        }
                        mass.count(kPiece);
                    });
                    more = entries_above;
                } else {
                    every(from, [&](float l, int v) {
                        const int part = part_of(l, true);
                        if (part < first) {
                            mass.add(weight(l));
                            mass.count(1);
                            ++more;
                        } else if (part <= last) {
                            inside(l, v);
                        }
                    });
                }
                const u64 own = mass.value();
                const Reduced y = reduce(own, more, high, low);
                if (!ok) return;
                if (halve && (want_count != ~0ull ? above + y.b >= want_count : over + y.a >= want_mass)) {
                    lo = hi - (static_cast<uint32_t>(first) << shift) + 1u;   // it is in the upper half
                    halve = false;
                    continue;
                }
                run_mass += warp_sum_u64(own);
                over += y.a;
                above += y.b;
                if (fits) {
                    const int count = gather();
                    if (!ok) return;
                    if (rank == 0) settle(count, above, over, want_count, want_mass);
                    settled_on_list();
                    if (!ok) return;
                    if (token < 0) {
                        // the runs' sums: the list's kept entries join those above it
                        __syncthreads();
                        if (tid < kWarps) s.run[tid] = 0;
                        __syncthreads();
                        for (uint32_t i = tid; i < s.list_count; i += kThreads) {
                            const u64 key = s.list[i];
                            if (key < cut) continue;
                            const int place = (static_cast<int>(key_index(key)) - place0) / kPiece;
                            atomicAdd(&s.run[place / per_run], mass_of(weight(key_logit(key))));
                        }
                        __syncthreads();
                        run_mass += s.run[warp];
                        runs_known = true;
                    }
                    return;
                }
                linear = false;
                const uint32_t width = hi - lo;
                hi = static_cast<uint32_t>(y.c);
                lo = 0xFFFFFFFFu - static_cast<uint32_t>(y.d);
                // Bounds cannot part large groups of equal logits where the wanted mass is reached between them.
                halve = hi - lo > width / 2u;
                if (hi == lo) {
                    // one logit, repeated: so many of them by id
                    const u64 q = mass_of(weight(float_from_order_bits(hi)));
                    const u64 take = want_count != ~0ull ? want_count - above
                                     : q == 0          ? 1
                                                       : max(1ull, (want_mass - over + q - 1) / q);
                    auto tie = [&](float l, int v) -> u64 { return bits(l) == hi && key_of(l, v) >= limit ? 1 : 0; };
                    u64 ties = 0;
                    pass(streamed, [&](int i, const float (&y)[kPiece], const uint4&, int) {
#pragma unroll
                        for (int e = 0; e < kPiece; ++e) ties += tie(y[e], place0 + i * kPiece + e);
                    });
                    report_run(warp_sum_u64(ties));
                    locate(take - 1, tie, [&](int v) {
                        const u64 key = key_of(float_from_order_bits(hi), v);
                        if (C == 1) s.found = key;
                        else if (lane < static_cast<uint32_t>(C))
                            send(remote(&s.found, lane), key, remote(&s.bar_found, lane));
                    });
                    if (!ok) return;
                    if (C > 1) receive(s.bar_found, used_found, 8u);
                    else __syncthreads();
                    if (!ok) return;
                    cut = s.found;
                    total = over + take * q;
                    return;
                }
            }
            if (rank == 0 && tid == 0) set_status(p.ws, DSPARK_STATUS_INTERNAL);   // not reached: see kLevels
        };

        // The mass, first of all entries alike where neither min-p nor top-k nor something odd is in the way (what lies
        // outside the row weighs nothing); the smallest entry is then only asked for if the mass needs it.
        MassSum mass;
        float lowest = -INFINITY;
        u64 entries = static_cast<u64>(V);
        bool alike = clean && min_p == 0.0f && k == V;
        if (alike) {
            pass(streamed, [&](int, const float (&x)[kPiece], const uint4&, int) {
#pragma unroll
                for (int e = 0; e < kPiece; e += 2) mass.add(weights(fmaxf(x[e], -INFINITY), fmaxf(x[e + 1], -INFINITY)));
                mass.count(kPiece);
            });
            const u64 own = mass.value();
            total = reduce(own, 0, 0, 0).a;
            if (!ok) return false;
            run_mass = warp_sum_u64(own);
            const u64 need = max(1ull, share_of(total, P));
            alike = need >= total || (total - need) / entries > 0;
        }
        if (!alike) {
            // what min-p leaves
            mass = MassSum();
            uint32_t count = 0;
            float smallest = INFINITY;
            pass(streamed, [&](int, const float (&x)[kPiece], const uint4&, int) {
#pragma unroll
                for (int e = 0; e < kPiece; ++e) {
                    const bool finite = fabsf(x[e]) < INFINITY;
                    float w = finite ? weight(x[e]) : 0.0f;
                    const bool in = finite && w >= min_p;
                    if (!in) w = 0.0f;
                    mass.add(w);
                    count += in ? 1u : 0u;
                    if (in) smallest = fminf(smallest, x[e]);
                }
                mass.count(kPiece);
            });
            const u64 own = mass.value();
            const Reduced all = reduce(own, count, 0, count != 0 ? 0xFFFFFFFFu - float_order_bits(smallest) : 0u);
            if (!ok) return false;
            lowest = float_from_order_bits(0xFFFFFFFFu - static_cast<uint32_t>(all.d));
            entries = all.b;
            total = all.a;
            run_mass = warp_sum_u64(own);
        }
        runs_known = true;                                                    // if everything is kept
        if (static_cast<u64>(k) < entries) {
            close_in(static_cast<u64>(k), ~0ull - 1, lowest);
            if (!ok) return false;
            limit = cut;
            entries = static_cast<u64>(k);
        }
        const u64 need = max(1ull, share_of(total, P));                       // the first entry (mass 2^40) is kept anyway
        if (need < total) {
            // Entries of mass at most z weigh no more than total - need together: the cut is not among them.
            const u64 z = (total - need) / entries;
            float least = lowest;
            if (z > 0) least = fmaxf(lowest, m + (logf(__ull2float_rn(z) * 0x1p-40f) * (1.0f + 1e-5f) - 1e-5f) / inv);
            token = -1;                                                       // what top-k's list said is not the last word
            in_list = false;
            close_in(~0ull, need, least);
            if (!ok) return false;
        }
        if (token < 0 && runs_known) report_run(run_mass);
    }

    // ---- 5. the token, and the probabilities ----
    if (p.queue && tid == 0) s.next = gridDim.x + atomicAdd(&p.plan->next, 1u);   // the next row: no earlier, for the order
    const float cut_logit = cut == 0 ? -INFINITY : key_logit(cut);
    auto kept = [&](float l, int v) {                                         // weight of a kept entry, else 0
        if (!(l >= cut_logit) || bits(l) == 0 || key_of(l, v) < cut) return 0.0f;
        const float w = weight(l);
        return w < min_p ? 0.0f : w;
    };
    if (token < 0) {
        if (!runs_known) {
            MassSum mass;
            pass(streamed, [&](int i, const float (&y)[kPiece], const uint4&, int) {
#pragma unroll
                for (int e = 0; e < kPiece; ++e)
                    if (y[e] >= cut_logit) {
                        mass.add(kept(y[e], place0 + i * kPiece + e));
                        mass.count(1);
                    }
            });
            report_run(warp_sum_u64(mass.value()));
        }
        locate(share_of(total, U), [&](float l, int v) { return mass_of(kept(l, v)); }, set_token);
        if (!ok) return false;
    } else if (rank == 0 && warp == 0) {
        set_token(token);
    }
    if (p.probs == nullptr) return true;
    const float norm = 0x1p40f / __ull2float_rn(total);
    float* const probs = p.probs + r * V;
    auto share = [&](float w) { return w >= 0x1p-40f ? w * norm : 0.0f; };    // 0 where the mass is
    if (in_list) {
        // zeros, then this block's part of the list
        const int head = min(n, static_cast<int>((16u - (reinterpret_cast<uintptr_t>(probs + v0) & 15u)) & 15u) / 4);
        const int quads = (n - head) / 4;
        for (int i = tid; i < head; i += kThreads) probs[v0 + i] = 0.0f;
        for (int i = tid; i < quads; i += kThreads)
            __stcs(reinterpret_cast<float4*>(probs + v0 + head) + i, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
        for (int i = head + 4 * quads + tid; i < n; i += kThreads) probs[v0 + i] = 0.0f;
        __syncthreads();
        for (uint32_t i = tid; i < s.list_count; i += kThreads) {
            const u64 key = s.list[i];
            if (key >= cut) probs[key_index(key)] = share(weight(key_logit(key)));
        }
    } else {
        // 16-byte stores where the two rows are aligned alike (fp32 logits)
        pass(streamed, [&](int i, const float (&x)[kPiece], const uint4&, int) {
            if (i >= run1) return;
            float y[kPiece];
            const int v = place0 + i * kPiece;
#pragma unroll
            for (int e = 0; e < kPiece; ++e) y[e] = x[e] >= cut_logit ? share(kept(x[e], v + e)) : 0.0f;
            if (kPiece == 4 && whole(i)) {
                __stcs(reinterpret_cast<float4*>(probs + v), *reinterpret_cast<const float4*>(y));
            } else {
#pragma unroll
                for (int e = 0; e < kPiece; ++e)
                    if (v + e >= v0 && v + e < v1) probs[v + e] = y[e];
            }
        });
    }
    return true;
}

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const __grid_constant__ SampleArgs p) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Shared<kThreads>& s = *reinterpret_cast<Shared<kThreads>*>(smem_raw);
    T* const held = reinterpret_cast<T*>(smem_raw + sizeof(s));
    grid_dependency_wait();
    int place = static_cast<int>(blockIdx.x) / p.cluster;
    bool ok;
    while (true) {
        ok = sample_row(p, s, held, p.queue ? p.order[place] : place);
        if (!p.queue) break;
        __syncthreads();
        place = static_cast<int>(s.next);
        __syncthreads();
        if (place >= p.R) break;
    }
    if (!ok) {
        // No block may end while another can still send to it.  One that has received everything has nothing under
        // way to it; one that gave up stays until all others have ended or come here (the barrier counts threads
        // that have ended as arrived), and until what they sent before has had time to arrive.
        asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
        asm volatile("barrier.cluster.wait;" ::: "memory");
        const long long t0 = global_ns();
        while (global_ns() - t0 < kUnderWayNs) {
        }
    }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
template <typename T, int kThreads>
cudaError_t launch_blocks(SampleArgs p, cudaStream_t stream, const DeviceInfo& dev) {
    using S = Shared<kThreads>;
    p.resident = sizeof(S) + static_cast<size_t>(p.slice) * sizeof(T) + 32 <= dev.smem_optin ? 1 : 0;
    const size_t smem = sizeof(S) + (p.resident ? static_cast<size_t>(p.slice) * sizeof(T) + 32 : 0);
    auto kernel = sample_kernel<T, kThreads>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.queue ? static_cast<unsigned>(dev.sm_count) : static_cast<unsigned>(p.R) * static_cast<unsigned>(p.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(p.cluster);
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    sample_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T>
cudaError_t launch_typed(SampleArgs p, cudaStream_t stream, const DeviceInfo& dev) {
    // Blocks per row: doubled until every SM has one, while a block keeps kMinSlice entries.  That may end at up to
    // twice the SMs, which costs a second round of blocks and still wins with long rows: 39 rows of 151936 take 72 us
    // on 4 blocks each and 107 us on 2, 77 rows 109 us on 2 and 166 us on 1 (86 us on 4), 120 rows 123 and 169 us.
    // Where it does not: 72 rows of 32000 on 4 blocks 49 us, on 2 39 us; 150 rows of 151936 on 2 114 us, on 1 107 us.
    constexpr int kMinSlice = 4096;
    auto slice_of = [&](int blocks) { return ((p.V + blocks - 1) / blocks + 7) / 8 * 8; };
    int c = 1;
    while (c < kMaxCluster && static_cast<long long>(p.R) * c < dev.sm_count && slice_of(2 * c) >= kMinSlice) c *= 2;
    p.cluster = c;
    p.queue = c == 1 && p.R > dev.sm_count ? 1 : 0;
    p.slice = slice_of(c);
    // Half the threads meet sooner at their barriers; with long parts the passes count, which want them all.
    // 512 against 1024 threads: parts of 9496 entries 11 and 15 us (one row), of 16000 38 and 42 us (76 rows), of
    // 35000 58 and 61 us (100 rows), of 37984 76 and 72 us (38 rows), of 75968 133 and 109 us (76 rows).
    constexpr int kShortSlice = 32768;
    return p.slice <= kShortSlice ? launch_blocks<T, 512>(p, stream, dev) : launch_blocks<T, 1024>(p, stream, dev);
}

}  // namespace

size_t sample_workspace_bytes(int R) { return R < 1 ? 0 : sizeof(Plan) + static_cast<size_t>(R) * sizeof(int32_t); }

dspark_status launch_sample(const void* logits, dspark_dtype dtype, const float* temperature, const int32_t* top_k,
                            const float* top_p, const float* min_p, const float* u, int R, int V, int32_t* tokens,
                            float* probs, void* ws, cudaStream_t stream, const DeviceInfo& dev) {
    if (static_cast<long long>(R) * kMaxCluster >= (1ll << 31)) {
        set_error("sample: too many rows (R=%d)", R);
        return DSPARK_ERR_UNSUPPORTED;
    }
    SampleArgs p{logits, temperature, top_k, top_p, min_p, u, R, V, 1, 0, 0, 0, tokens, probs, static_cast<WsHeader*>(ws),
                 static_cast<Plan*>(ws), reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + sizeof(Plan))};
    const cudaError_t e = dtype == DSPARK_F32 ? launch_typed<float>(p, stream, dev)
                                              : launch_typed<__nv_bfloat16>(p, stream, dev);
    if (e != cudaSuccess) return cuda_error(e, "launch(sample)");
    return DSPARK_OK;
}

}  // namespace dspark
