// Sampling with temperature, top-k, min-p and top-p from given uniforms.
//
// The kept set is a prefix of the entries ordered by (logit, largest first; id, smallest first), so it
// is described by its last entry, the cut, and every sum is of integers (a weight's mass is
// floor(w * 2^40)), so the cut, the total and the token depend on no order of summation.
//
// A cluster of 1 to 16 blocks holds one row in shared memory, read once from memory; the passes below
// run on that copy, partial sums and counts travel through distributed shared memory.  What a row
// needs, and no more, is done:
//   1. load the row, its largest logit m, and each thread's largest (their smallest bounds a range)
//   2. with top-k (k up to the number of threads): a histogram of the threads' largest logits gives a
//      bound that at least k entries reach; those entries, usually a few more than k, go to a list
//      that one block sorts, and min-p and top-p are settled on the list
//   3. else the total mass of the entries that min-p leaves; entries of mass at most (Q - need) / count
//      cannot be needed for top-p, and if the others fit, they go to the list in the same way
//   4. else (a wide nucleus, a very large k) the cut is closed in on: a histogram of counts over 2048
//      parts of the range, bounds of each part's mass from its edges, the parts that can hold the cut
//      are the next range, and the mass above it is summed exactly; once the range's entries fit the
//      list, it is sorted; a range of one repeated logit is settled by id
//   5. one pass sums the kept masses of contiguous runs and writes the probabilities; the run that
//      holds the drawn mass is gone through again for the token
#include "device_common.cuh"
#include "half_common.cuh"
#include "host_common.h"

#include <algorithm>

namespace dspark {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kList = 2048;                // entries of the list
constexpr int kBins = 2048;
constexpr int kPerThread = kBins / kThreads;

struct SampleArgs {
    const void* logits;
    const float* temperature;
    const int32_t* top_k;
    const float *top_p, *min_p, *u;
    int R, V;
    int cluster, slice;                    // blocks of a row, entries of a block (a multiple of 8)
    int resident;                          // the slice is held in shared memory
    int32_t* tokens;
    float* probs;
    WsHeader* ws;
};

using u64 = unsigned long long;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Address of the same shared variable in block `rank` of the cluster, and accesses through it.
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void remote_store(uint32_t at, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" :: "r"(at), "l"(v) : "memory");
}
__device__ __forceinline__ void remote_add(uint32_t at, uint32_t v) {
    asm volatile("red.shared::cluster.add.u32 [%0], %1;" :: "r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t remote_take(uint32_t at, uint32_t v) {
    uint32_t old;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(at), "r"(v) : "memory");
    return old;
}
__device__ __forceinline__ uint32_t remote_load(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// floor(total * frac / 2^24), total < 2^62, frac <= 2^24.
__device__ __forceinline__ u64 share_of(u64 total, uint32_t frac) {
    return (total >> 24) * frac + (((total & 0xFFFFFFull) * frac) >> 24);
}

// floor(w * 2^40) in two halves of at most 20 bits (w <= 1): both scalings by 2^20 are exact, and
// 32-bit conversions and additions are cheaper than 64-bit ones.
__device__ __forceinline__ void mass_halves(float w, uint32_t& hi, uint32_t& lo) {
    const float s = __fmul_rn(w, 0x1p20f);
    hi = static_cast<uint32_t>(s);
    lo = static_cast<uint32_t>(__fmul_rn(__fsub_rn(s, static_cast<float>(hi)), 0x1p20f));
}
__device__ __forceinline__ u64 mass_of(float w) {
    uint32_t hi, lo;
    mass_halves(w, hi, lo);
    return (static_cast<u64>(hi) << 20) + lo;
}

struct alignas(16) Shared {
    u64 red[2][kMaxCluster][4];            // values exchanged by the blocks, two exchanges in turn
    u64 list[kList];                       // of the first block: argmax keys
    uint32_t hist[kBins];                  // counts, all blocks' in the first one
    uint32_t list_count, pad;
    u64 found;                             // the entry that locate() was asked for
    u64 segment[kMaxCluster * kWarps];     // of the first block: mass or count of each warp's run
    u64 warp_sum[4][kWarps];
    u64 out[4];                            // what the first block tells the others
};

struct Reduced { u64 a, b, c, d; };

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ SampleArgs p) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Shared& s = *reinterpret_cast<Shared*>(smem_raw);
    T* const held = reinterpret_cast<T*>(smem_raw + sizeof(Shared));
    const int tid = threadIdx.x, V = p.V;
    const uint32_t warp = warp_id(), lane = lane_id();
    const int C = p.cluster;
    const uint32_t rank = C > 1 ? cluster_rank() : 0u;
    const long long r = blockIdx.x / C;
    const T* const global = static_cast<const T*>(p.logits) + r * V;
    const int v0 = min(V, static_cast<int>(rank) * p.slice), v1 = min(V, v0 + p.slice), n = v1 - v0;
    auto sync = [&] { if (C > 1) cluster_sync(); else __syncthreads(); };

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

    // ---- exchanges ----
    int turn = 0;
    // Every block's four values, added up (a, b) or by maximum (c, d); the arguments count in thread 0 only.
    auto exchange = [&](u64 a, u64 b, u64 c, u64 d) {
        Reduced x{a, b, c, d};
        if (tid == 0) {
            u64* mine = s.red[turn][rank];
            mine[0] = a; mine[1] = b; mine[2] = c; mine[3] = d;
        }
        if (C > 1) {
            __syncthreads();
            if (tid < C * 4 && static_cast<uint32_t>(tid >> 2) != rank)
                remote_store(remote(&s.red[turn][rank][tid & 3], static_cast<uint32_t>(tid >> 2)), s.red[turn][rank][tid & 3]);
        }
        sync();
        x = Reduced{0, 0, 0, 0};
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
    // Sums (a, b) and maxima (c, d) over the block's threads, in thread 0, then exchanged.
    auto reduce = [&](u64 a, u64 b, u64 c, u64 d) {
        a = warp_sum_u64(a);
        b = warp_sum_u64(b);
        c = warp_max_u64(c);
        d = warp_max_u64(d);
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
        return exchange(a, b, c, d);
    };
    // What the first block has put into s.out, in every block.
    auto hear = [&] {
        __syncthreads();
        if (C > 1 && rank == 0 && tid < C * 4 && (tid >> 2) != 0)
            remote_store(remote(&s.out[tid & 3], static_cast<uint32_t>(tid >> 2)), s.out[tid & 3]);
        sync();
    };

    // ---- 1. the row ----
    // Entry v is held at v - v0 + pad, so that 16-byte pieces of the row stay pieces in shared memory.
    constexpr int kPiece = 16 / sizeof(T);
    const int pad = p.resident ? static_cast<int>((reinterpret_cast<uintptr_t>(global + v0) & 15u) / sizeof(T)) : 0;
    const T* const row = p.resident ? held + pad - v0 : global;              // row[v], v in [v0, v1)
    uint32_t top = 0, odd = 0;
    auto look = [&](float x) {
        if (!(x < INFINITY)) odd = 1;                                         // NaN and +infinity; not -infinity
        top = max(top, bits(x));
    };
    if (p.resident) {
        const int pieces = (pad + n + kPiece - 1) / kPiece;
        const T* const base = global + v0 - pad;
#pragma unroll 4
        for (int i = tid; i < pieces; i += kThreads) {
            T x[kPiece];
            const int first = i * kPiece - pad;                               // of the piece, in the slice
            if (first >= 0 && first + kPiece <= n) {
                *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(base + i * kPiece);
#pragma unroll
                for (int e = 0; e < kPiece; ++e) look(to_float(x[e]));
                *reinterpret_cast<uint4*>(held + i * kPiece) = *reinterpret_cast<const uint4*>(x);
            } else {
                for (int e = 0; e < kPiece; ++e) {
                    if (first + e < 0 || first + e >= n) continue;
                    const T y = base[i * kPiece + e];
                    look(to_float(y));
                    held[i * kPiece + e] = y;
                }
            }
        }
    } else {
        for (int v = v0 + tid; v < v1; v += kThreads) look(to_float(row[v]));
    }
    const uint32_t mine = top;                                                // this thread's largest
    if (tid == 0) s.list_count = 0u;
    for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0u;
    // c: the largest; d: the smallest of the threads' largest, as its complement
    Reduced x = reduce(odd, mine != 0 ? 1 : 0, mine, mine != 0 ? 0xFFFFFFFFu - mine : 0u);
    if (x.a != 0) flags |= DSPARK_STATUS_NUMERIC;
    const uint32_t top_bits = static_cast<uint32_t>(x.c);
    if (top_bits == 0) flags |= DSPARK_STATUS_NUMERIC;
    if (rank == 0 && tid == 0 && flags) set_status(p.ws, flags);
    const float m = float_from_order_bits(top_bits);
    const int groups = static_cast<int>(x.b);                                 // threads with an entry
    const float bottom = float_from_order_bits(0xFFFFFFFFu - static_cast<uint32_t>(x.d));

    auto weight = [&](float l) { return expf(__fmul_rn(__fsub_rn(l, m), inv)); };

    u64 cut = 0, total = 0;                                                   // the kept set: argmax_key >= cut; its mass
    u64 limit = 0;                                                            // likewise after top-k, while top-p is sought
    // Entries that min-p and `limit` leave.  Calls f(bits, id, logit).
    auto each = [&](auto f) {
        for (int v = v0 + tid; v < v1; v += kThreads) {
            const float l = to_float(row[v]);
            const uint32_t b = bits(l);
            if (b != 0 && argmax_key(l, static_cast<uint32_t>(v)) >= limit) f(b, v, l);
        }
    };
    // Entries for which in(bits, id, logit) holds go to the list; returns how many there are (the list
    // holds them if they are no more than kList).
    auto append = [&](bool yes, float l, int v) {                             // warp-converged
        const uint32_t vote = __ballot_sync(0xFFFFFFFFu, yes);
        if (vote == 0) return;
        uint32_t at = 0;
        const uint32_t count_at = C > 1 ? remote(&s.list_count, 0) : 0;
        if (lane == 0) at = C > 1 ? remote_take(count_at, __popc(vote)) : atomicAdd(&s.list_count, __popc(vote));
        at = __shfl_sync(0xFFFFFFFFu, at, 0) + __popc(vote & ((1u << lane) - 1u));
        if (yes && at < kList) {
            const u64 key = argmax_key(l, static_cast<uint32_t>(v));
            if (C > 1) remote_store(remote(&s.list[at], 0), key);
            else s.list[at] = key;
        }
    };
    auto each_converged = [&](auto f) {                                       // f is called by whole warps: in, id, logit
        const int end = v0 + (n + 31) / 32 * 32;
        for (int v = v0 + tid; v < end; v += kThreads) {
            const float l = v < v1 ? to_float(row[v]) : -INFINITY;
            f(bits(l) != 0 && argmax_key(l, static_cast<uint32_t>(v)) >= limit, v, l);
        }
    };

    // Bitonic sort of list[0 .. size), size a power of two, the largest first, by the calling block.
    auto sort = [&](int size) {
        for (int span = 2; span <= size; span <<= 1)
            for (int step = span >> 1; step > 0; step >>= 1) {
                __syncthreads();
                for (int i = tid; i < size / 2; i += kThreads) {
                    const int a = 2 * i - (i & (step - 1)), b = a + step;
                    const u64 ka = s.list[a], kb = s.list[b];
                    if (((a & span) == 0) == (ka < kb)) {
                        s.list[a] = kb;
                        s.list[b] = ka;
                    }
                }
            }
        __syncthreads();
    };
    auto key_logit = [&](u64 key) { return float_from_order_bits(static_cast<uint32_t>(key >> 32)); };

    // First block: settles the cut on the list of `count` entries, behind `above` entries of mass `over`: at
    // most kk entries in all, and of those as many as reach the mass `need` (~0: top-p's share of them).
    // Leaves {cut, mass} in s.out.
    auto settle = [&](int count, u64 above, u64 over, u64 kk, u64 need) {
        int size = 2;
        while (size < count) size <<= 1;
        for (int i = count + tid; i < size; i += kThreads) s.list[i] = 0;
        sort(size);
        // per thread kPerThread neighbours: masses, their prefix
        constexpr int kPer = kList / kThreads;
        u64 q[kPer], sum = 0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int i = tid * kPer + e;
            q[e] = 0;
            if (i < count && above + static_cast<u64>(i) < kk) {
                const float w = weight(key_logit(s.list[i]));
                if (w >= min_p) q[e] = mass_of(w) + (1ull << 62);             // bit 62: it takes part
            }
        }
        // the entries that take part are a prefix of the list: their masses' sum
#pragma unroll
        for (int e = 0; e < kPer; ++e) sum += q[e] & ~(1ull << 62);
        u64 incl = sum;
        for (int d = 1; d < 32; d <<= 1) {
            const u64 y = __shfl_up_sync(0xFFFFFFFFu, incl, d);
            if (lane >= static_cast<uint32_t>(d)) incl += y;
        }
        if (lane == 31) s.warp_sum[0][warp] = incl;
        __syncthreads();
        u64 before = over + incl - sum, all = over;
        for (uint32_t w = 0; w < kWarps; ++w) {
            if (w < warp) before += s.warp_sum[0][w];
            all += s.warp_sum[0][w];
        }
        if (need == ~0ull) need = share_of(all, P);
        // kept: what takes part while the mass before it is short of what is needed (the first of all is kept
        // anyway); the last of them is the cut
        uint32_t last = 0;                                                    // its place + 1
        u64 upto = 0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int i = tid * kPer + e;
            const bool keep = (q[e] >> 62) != 0 && (before < need || (above == 0 && i == 0));
            before += q[e] & ~(1ull << 62);
            if (keep) {
                last = static_cast<uint32_t>(i) + 1u;
                upto = before;
            }
        }
        const uint32_t best = __reduce_max_sync(0xFFFFFFFFu, last);
        if (best != 0 ? last == best : lane == 0) {
            s.warp_sum[2][warp] = best;
            s.warp_sum[3][warp] = upto;
        }
        __syncthreads();
        if (tid == 0) {
            uint32_t w = 0;
            for (uint32_t y = 1; y < kWarps; ++y)
                if (s.warp_sum[2][y] != 0) w = y;
            s.out[0] = s.list[max(1ull, s.warp_sum[2][w]) - 1];
            s.out[1] = s.warp_sum[3][w];
        }
        __syncthreads();
    };

    bool settled = top_bits == 0;                                             // nothing to keep: cut 0, total 0
    if (settled) cut = ~0ull;

    // ---- 2. a small top-k ----
    // A range that can be parted evenly (not of one value, and finite).
    auto even = [&](float lowest) { return m - lowest > 1e-30f && m - lowest < 1e38f; };
    if (!settled && k <= groups && k <= kList / 2 && even(bottom)) {
        const float scale = (kBins - 1) / (m - bottom);
        if (mine != 0) {
            const int bin = min(kBins - 1, static_cast<int>((m - float_from_order_bits(mine)) * scale));
            if (C > 1) remote_add(remote(&s.hist[bin], 0), 1u);
            else atomicAdd(&s.hist[bin], 1u);
        }
        sync();
        if (rank == 0) {
            // the first bin up to which there are k
            uint32_t c[kPerThread], sum = 0;
#pragma unroll
            for (int e = 0; e < kPerThread; ++e) sum += c[e] = s.hist[tid * kPerThread + e];
            uint32_t incl = sum;
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, incl, d);
                if (lane >= static_cast<uint32_t>(d)) incl += y;
            }
            if (lane == 31) s.warp_sum[0][warp] = incl;
            __syncthreads();
            uint32_t before = incl - sum;
            for (uint32_t w = 0; w < warp; ++w) before += static_cast<uint32_t>(s.warp_sum[0][w]);
            for (int e = 0; e < kPerThread; ++e) {
                if (before < static_cast<uint32_t>(k) && before + c[e] >= static_cast<uint32_t>(k))
                    s.out[0] = static_cast<u64>(tid * kPerThread + e);
                before += c[e];
            }
        }
        hear();
        const float reach = static_cast<float>(s.out[0] + 1);
        each_converged([&](bool in, int v, float l) { append(in && (m - l) * scale < reach, l, v); });
        sync();
        const uint32_t count = C > 1 ? remote_load(remote(&s.list_count, 0)) : s.list_count;
        if (count <= kList) {
            if (rank == 0) settle(static_cast<int>(count), 0, 0, static_cast<u64>(k), ~0ull);
            hear();
            cut = s.out[0];
            total = s.out[1];
            settled = true;
        } else {
            sync();                                                           // all have read the count
            if (tid == 0) s.list_count = 0u;
        }
    }

    // This warp's run of neighbouring entries.
    const int per_run = ((n + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int run0 = min(v1, v0 + static_cast<int>(warp) * per_run), run1 = min(v1, run0 + per_run);
    // With every run's sum in the first block's s.segment: the first id at which the sum of value(logit, id)
    // over all ids up to it exceeds t, known to one warp of the cluster, which calls found(id) in all lanes.
    auto locate = [&](u64 t, auto value, auto found) {
        sync();
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
        if (s.out[0] == rank * kWarps + warp) {
            u64 left = s.out[1];
            for (int b = run0; b < run1; b += 32) {
                const int v = b + static_cast<int>(lane);
                u64 incl = v < run1 ? value(to_float(row[v]), v) : 0;
                for (int d = 1; d < 32; d <<= 1) {
                    const u64 y = __shfl_up_sync(0xFFFFFFFFu, incl, d);
                    if (lane >= static_cast<uint32_t>(d)) incl += y;
                }
                const uint32_t vote = __ballot_sync(0xFFFFFFFFu, incl > left);
                if (vote != 0) {
                    found(b + __ffs(static_cast<int>(vote)) - 1);
                    break;
                }
                left -= __shfl_sync(0xFFFFFFFFu, incl, 31);
            }
        }
    };
    auto report_run = [&](u64 sum) {                                          // lane 0's: this run's sum
        if (lane != 0) return;
        if (C > 1) remote_store(remote(&s.segment[rank * kWarps + warp], 0), sum);
        else s.segment[warp] = sum;
    };

    // ---- 3. and 4. ----
    if (!settled) {
        // Closes in on the cut: the first entry of the order with which the count reaches `want_count`, or the
        // mass `want_mass` (the other is ~0).  `lowest`: no entry below this logit can be the cut.
        auto close_in = [&](u64 want_count, u64 want_mass, float lowest) {
            u64 above = 0, over = 0;                                          // count and mass above the range
            bool linear = even(lowest);                                       // parts of equal width, or of equal bits
            uint32_t hi = top_bits, lo = float_order_bits(lowest);
            while (true) {
                const float scale = linear ? kBins / (m - lowest) : 0.0f;
                int shift = 0;
                while (((hi - lo) >> shift) >= kBins) ++shift;
                auto bin_of = [&](uint32_t b, float l) {
                    return linear ? min(kBins - 1, static_cast<int>((m - l) * scale)) : static_cast<int>((hi - b) >> shift);
                };
                sync();
                if (tid == 0) s.list_count = 0u;
                for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0u;
                __syncthreads();
                each([&](uint32_t b, int, float l) {
                    if (b >= lo && b <= hi && weight(l) >= min_p) atomicAdd(&s.hist[bin_of(b, l)], 1u);
                });
                sync();
                if (rank != 0)
                    for (int i = tid; i < kBins; i += kThreads)
                        if (s.hist[i] != 0) remote_add(remote(&s.hist[i], 0), s.hist[i]);
                sync();
                if (rank == 0) {
                    // bounds of each part's mass from its edges, with room for the rounding of edges and expf
                    uint32_t c[kPerThread];
                    u64 least[kPerThread], most[kPerThread], sum_least = 0, sum_most = 0;
#pragma unroll
                    for (int e = 0; e < kPerThread; ++e) {
                        const int i = tid * kPerThread + e;
                        c[e] = s.hist[i];
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
                            least[e] = c[e] * mass_of(fmaxf(0.0f, weight(lo_edge) * (1.0f - 1e-4f)));
                        }
                        sum_least += least[e];
                        sum_most += most[e];
                    }
                    u64 in_least = sum_least, in_most = sum_most;
                    for (int d = 1; d < 32; d <<= 1) {
                        const u64 y = __shfl_up_sync(0xFFFFFFFFu, in_least, d), z = __shfl_up_sync(0xFFFFFFFFu, in_most, d);
                        if (lane >= static_cast<uint32_t>(d)) {
                            in_least += y;
                            in_most += z;
                        }
                    }
                    if (lane == 31) {
                        s.warp_sum[0][warp] = in_least;
                        s.warp_sum[1][warp] = in_most;
                    }
                    if (tid == 0) {
                        s.out[0] = s.out[1] = kBins - 1;                      // first and last part that can hold the cut
                    }
                    __syncthreads();
                    u64 least_before = in_least - sum_least, most_before = in_most - sum_most;
                    for (uint32_t w = 0; w < warp; ++w) {
                        least_before += s.warp_sum[0][w];
                        most_before += s.warp_sum[1][w];
                    }
                    const u64 want = want_count != ~0ull ? want_count - above : want_mass - over;
#pragma unroll
                    for (int e = 0; e < kPerThread; ++e) {
                        const u64 i = static_cast<u64>(tid * kPerThread + e);
                        if (most_before < want && most_before + most[e] >= want) s.out[0] = i;
                        if (least_before < want && least_before + least[e] >= want) s.out[1] = i;
                        least_before += least[e];
                        most_before += most[e];
                    }
                }
                hear();
                const int first = static_cast<int>(s.out[0]), last = static_cast<int>(s.out[1]);
                // above those parts: summed; in them: counted, bounded and, if they fit, listed
                u64 more = 0, high = 0, low = 0;
                uint32_t mass_hi = 0, mass_lo = 0, inside = 0;
                each_converged([&](bool in, int v, float l) {
                    const uint32_t b = bits(l);
                    in = in && b >= lo && b <= hi;
                    float w = 0.0f;
                    int bin = kBins;
                    if (in) {
                        bin = bin_of(b, l);
                        w = weight(l);
                        in = w >= min_p;
                    }
                    if (in && bin < first) {
                        uint32_t qh, ql;
                        mass_halves(w, qh, ql);
                        mass_hi += qh;
                        mass_lo += ql;
                        ++more;
                    }
                    const bool here = in && bin >= first && bin <= last;
                    if (here) {
                        ++inside;
                        high = max(high, static_cast<u64>(b));
                        low = max(low, static_cast<u64>(0xFFFFFFFFu - b));
                    }
                    append(here, l, v);
                });
                const Reduced y = reduce((static_cast<u64>(mass_hi) << 20) + mass_lo, more + (static_cast<u64>(inside) << 32), high, low);
                over += y.a;
                above += y.b & 0xFFFFFFFFull;
                const u64 count = y.b >> 32;
                if (count <= kList) {
                    if (rank == 0) settle(static_cast<int>(count), above, over, want_count, want_mass);
                    hear();
                    cut = s.out[0];
                    total = s.out[1];
                    return;
                }
                linear = false;
                hi = static_cast<uint32_t>(y.c);
                lo = 0xFFFFFFFFu - static_cast<uint32_t>(y.d);
                if (hi == lo) {
                    // one logit, repeated: so many of them by id
                    const u64 q = mass_of(weight(float_from_order_bits(hi)));
                    const u64 take = want_count != ~0ull ? want_count - above
                                     : q == 0          ? 1
                                                       : max(1ull, (want_mass - over + q - 1) / q);
                    u64 ties = 0;
                    for (int v = run0 + static_cast<int>(lane); v < run1; v += 32) {
                        const float l = to_float(row[v]);
                        if (bits(l) == hi && argmax_key(l, static_cast<uint32_t>(v)) >= limit) ++ties;
                    }
                    report_run(warp_sum_u64(ties));
                    locate(take - 1,
                           [&](float l, int v) -> u64 {
                               return bits(l) == hi && argmax_key(l, static_cast<uint32_t>(v)) >= limit ? 1 : 0;
                           },
                           [&](int v) {
                               if (lane < static_cast<uint32_t>(C)) {
                                   const u64 key = argmax_key(float_from_order_bits(hi), static_cast<uint32_t>(v));
                                   if (C > 1) remote_store(remote(&s.found, lane), key);
                                   else s.found = key;
                               }
                           });
                    sync();
                    cut = s.found;
                    total = over + take * q;
                    return;
                }
            }
        };

        // what min-p leaves
        uint32_t mass_hi = 0, mass_lo = 0, count = 0, low = 0;
        each([&](uint32_t b, int, float l) {
            const float w = weight(l);
            if (w < min_p) return;
            uint32_t qh, ql;
            mass_halves(w, qh, ql);
            mass_hi += qh;
            mass_lo += ql;
            ++count;
            low = max(low, 0xFFFFFFFFu - b);
        });
        const Reduced all = reduce((static_cast<u64>(mass_hi) << 20) + mass_lo, count, 0, low);
        const float lowest = float_from_order_bits(0xFFFFFFFFu - static_cast<uint32_t>(all.d));
        u64 entries = all.b;
        total = all.a;
        if (static_cast<u64>(k) < entries) {
            close_in(static_cast<u64>(k), ~0ull - 1, lowest);
            limit = cut;
            entries = static_cast<u64>(k);
        }
        const u64 need = max(1ull, share_of(total, P));       // the first entry (mass 2^40) is kept anyway
        if (need < total) {
            // Entries of mass at most z weigh no more than total - need together: the cut is not among them.
            const u64 z = (total - need) / entries;
            float least = lowest;
            if (z > 0) least = fmaxf(lowest, m + (logf(__ull2float_rn(z) * 0x1p-40f) * (1.0f + 1e-5f) - 1e-5f) / inv);
            sync();
            if (tid == 0) s.list_count = 0u;
            sync();
            each_converged([&](bool in, int v, float l) { append(in && l >= least && weight(l) >= min_p, l, v); });
            sync();
            const uint32_t listed = C > 1 ? remote_load(remote(&s.list_count, 0)) : s.list_count;
            if (listed <= kList) {
                if (rank == 0) settle(static_cast<int>(listed), 0, 0, ~0ull, need);
                hear();
                cut = s.out[0];
                total = s.out[1];
            } else {
                close_in(~0ull, need, least);
            }
        }
    }

    // ---- 5. the kept entries' runs, and the probabilities ----
    const float cut_logit = cut == 0 ? -INFINITY : float_from_order_bits(static_cast<uint32_t>(cut >> 32));
    auto kept = [&](float l, int v) {                                         // weight of a kept entry, else 0
        if (!(l >= cut_logit) || bits(l) == 0 || argmax_key(l, static_cast<uint32_t>(v)) < cut) return 0.0f;
        const float w = weight(l);
        return w < min_p ? 0.0f : w;
    };
    const bool some = top_bits != 0;
    if (some || p.probs != nullptr) {
        const float norm = __fmul_rn(__ull2float_rn(total), 0x1p-40f);
        float* const probs = p.probs != nullptr ? p.probs + r * V : nullptr;
        uint32_t mass_hi = 0, mass_lo = 0;
#pragma unroll 4
        for (int v = run0 + static_cast<int>(lane); v < run1; v += 32) {
            const float w = some ? kept(to_float(row[v]), v) : 0.0f;
            float y = 0.0f;
            if (w > 0.0f) {
                uint32_t qh, ql;
                mass_halves(w, qh, ql);
                mass_hi += qh;
                mass_lo += ql;
                if (probs != nullptr && (qh | ql) != 0) y = __fdiv_rn(w, norm);
            }
            if (probs != nullptr) probs[v] = y;
        }
        if (some) report_run(warp_sum_u64((static_cast<u64>(mass_hi) << 20) + mass_lo));
    }
    if (some) {
        locate(share_of(total, U), [&](float l, int v) { return mass_of(kept(l, v)); },
               [&](int v) {
                   if (lane == 0) p.tokens[r] = v;
               });
        sync();                                                               // shared memory lives as long as it is read
    } else if (rank == 0 && tid == 0) {
        p.tokens[r] = 0;
    }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
template <typename T>
cudaError_t launch_typed(SampleArgs p, cudaStream_t stream, const DeviceInfo& dev) {
    const size_t room = dev.smem_optin - sizeof(Shared) - 64;
    // Blocks per row: enough that two blocks' copies fit an SM; with few rows, more, as long as a block keeps
    // kMinSlice entries, so that all SMs share the row's passes.
    constexpr int kMinSlice = 4096;
    constexpr size_t kCopy = 80 * 1024;
    int c = 1;
    auto slice_of = [&](int blocks) { return ((p.V + blocks - 1) / blocks + 7) / 8 * 8; };
    while (c < kMaxCluster && slice_of(c) * sizeof(T) > kCopy) c *= 2;
    while (c < kMaxCluster && static_cast<long long>(p.R) * c < 2ll * dev.sm_count && slice_of(2 * c) >= kMinSlice) c *= 2;
    p.cluster = c;
    p.slice = slice_of(c);
    p.resident = static_cast<size_t>(p.slice) * sizeof(T) <= room ? 1 : 0;
    const size_t smem = sizeof(Shared) + (p.resident ? static_cast<size_t>(p.slice) * sizeof(T) + 32 : 0);
    cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.R) * static_cast<unsigned>(c));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(c);
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sample_kernel<T>, p);
}

}  // namespace

dspark_status launch_sample(const void* logits, dspark_dtype dtype, const float* temperature, const int32_t* top_k,
                            const float* top_p, const float* min_p, const float* u, int R, int V, int32_t* tokens,
                            float* probs, void* ws, cudaStream_t stream, const DeviceInfo& dev) {
    if (static_cast<long long>(R) * kMaxCluster >= (1ll << 31)) {
        set_error("sample: too many rows (R=%d)", R);
        return DSPARK_ERR_UNSUPPORTED;
    }
    dspark_status st = clear_workspace(ws, sizeof(WsHeader), stream);
    if (st != DSPARK_OK) return st;
    SampleArgs p{logits, temperature, top_k, top_p, min_p, u, R, V, 1, 0, 0, tokens, probs, static_cast<WsHeader*>(ws)};
    const cudaError_t e = dtype == DSPARK_F32 ? launch_typed<float>(p, stream, dev)
                                              : launch_typed<__nv_bfloat16>(p, stream, dev);
    if (e != cudaSuccess) return cuda_error(e, "launch(sample)");
    return DSPARK_OK;
}

}  // namespace dspark
