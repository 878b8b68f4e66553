// Moves within a paged key-value cache: the accepted path of a drafted tree behind the tokens before it
// (dspark_kv_compact), and whole pages for sequences that part (dspark_kv_copy_pages).
//
// Compaction is in place: token base + path[i] goes to base + i, and path[i] >= i.  A thread owns sixteen bytes of
// every token (one layer, cache and head, and the place within the head), so no other thread writes what it reads,
// and takes the tokens in ascending order, kBatch loads ahead of their stores.  A store of batch x goes to a place
// below every token of the later batches, so nothing is overwritten before it has been read.
// Bound by its chain of loads (lengths, path, table, then one batch): 3.9 us for a path of one request in one layer,
// 8.5 us for 64 requests in 24 layers' caches (24 MB), 2.9 TB/s.
//
// Page copies are bound by the memory: 500 pages of 32 KB in both caches of 24 layers (1.57 GB read and written) take
// 228 us, 6.9 TB/s, with eight 16-byte loads of a thread under way.
#include "attention_common.cuh"
#include "device_common.cuh"
#include "host_common.h"
#include "tree_common.cuh"

#include <algorithm>

namespace dspark {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 8;                  // tokens, or 16-byte pieces of a page, that a thread has under way

struct CompactArgs {
    uint4 *k, *v;                          // layer l is l * layer pieces of 16 bytes further
    const int32_t *block_table, *kv_len, *lengths, *path, *num_accepted;
    int32_t* kv_out;
    long long layer;
    int layers, max_pages, B, N, Hkv, row, num_pages, page;     // row: pieces of a token's head
    WsHeader* ws;
};

// Block (x, b): kThreads of request b's columns.
__global__ void __launch_bounds__(kThreads) kv_compact_kernel(const __grid_constant__ CompactArgs a) {
    __shared__ long long s_src[kTreeMost], s_dst[kTreeMost];    // of head 0, in pieces; -1: not moved
    const int tid = threadIdx.x;
    for (int b = static_cast<int>(blockIdx.y); b < a.B; b += static_cast<int>(gridDim.y)) {
        const int kv = a.kv_len[b], n = a.lengths ? a.lengths[b] : a.N, accepted = a.num_accepted[b];
        bool ok = n >= 0 && n <= a.N && kv >= n && kv <= static_cast<long long>(a.max_pages) * a.page && accepted >= 0 &&
                  accepted <= max(n - 1, 0);
        const int kept = ok && n > 0 ? accepted + 1 : 0, base = kv - n;
        if (tid < kept) {
            const int32_t* path = a.path + static_cast<long long>(b) * a.N;
            const int at = path[tid], before = tid > 0 ? path[tid - 1] : -1;
            ok = at > before && at < n;
            s_src[tid] = s_dst[tid] = -1;
            if (ok && at > tid) {                          // at >= tid, as the path ascends
                auto place = [&](int j) {
                    const int in_table = j / a.page, p = a.block_table[static_cast<long long>(b) * a.max_pages + in_table];
                    return p < 0 || p >= a.num_pages ? -1ll
                                                     : (static_cast<long long>(p) * a.Hkv * a.page + (j - in_table * a.page)) * a.row;
                };
                const long long src = place(base + at), dst = place(base + tid);
                if (src < 0 || dst < 0) {
                    grid_dependency_wait();
                    flag_input_index(a.ws);
                } else {
                    s_src[tid] = src;
                    s_dst[tid] = dst;
                }
            }
        }
        ok = __syncthreads_and(ok) != 0;
        if (blockIdx.x == 0 && tid == 0) {
            a.kv_out[b] = !ok || n == 0 ? kv : base + kept;
            if (!ok) {
                grid_dependency_wait();                    // the status word has been cleared
                flag_input_index(a.ws);
            }
        }
        if (ok) {
            const int columns = a.layers * 2 * a.Hkv * a.row;
            const int c = static_cast<int>(blockIdx.x) * kThreads + tid;
            const int piece = c % a.row, head = c / a.row % a.Hkv, rest = c / a.row / a.Hkv;
            uint4* cache = (rest & 1 ? a.v : a.k) + static_cast<long long>(rest >> 1) * a.layer +
                           static_cast<long long>(head) * a.page * a.row + piece;
            for (int i0 = 0; i0 < kept && c < columns; i0 += kBatch) {
                uint4 x[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (i0 + i < kept && s_src[i0 + i] >= 0) x[i] = cache[s_src[i0 + i]];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (i0 + i < kept && s_src[i0 + i] >= 0) cache[s_dst[i0 + i]] = x[i];
            }
        }
        __syncthreads();                                   // the places are written again for the next request
    }
    grid_dependency_wait();
}

struct CopyArgs {
    uint4 *k, *v;
    const int32_t *src, *dst, *used;
    long long layer;                       // pieces of 16 bytes between layers
    int layers, M, Hkv, row, num_pages, page;
    WsHeader* ws;
};

// Item (pair, layer, cache) per block, in turn.
__global__ void __launch_bounds__(kThreads) kv_copy_kernel(const __grid_constant__ CopyArgs a) {
    const int tid = threadIdx.x;
    auto good = [&](int m) {
        const int from = a.src[m], to = a.dst[m], used = a.used ? a.used[m] : a.page;
        return from >= 0 && from < a.num_pages && to >= 0 && to < a.num_pages && used >= 0 && used <= a.page;
    };
    if (blockIdx.x == 0) {
        // the status word is this block's alone, so nothing has to clear it before
        bool bad = false;
        for (int m = tid; m < a.M; m += kThreads) bad |= !good(m);
        bad = __syncthreads_or(bad) != 0;
        if (tid < static_cast<int>(sizeof(WsHeader) / 4)) reinterpret_cast<uint32_t*>(a.ws)[tid] = 0u;
        __syncthreads();
        if (tid == 0 && bad) flag_input_index(a.ws);
    }
    const int pieces = a.Hkv * a.page * a.row, head = a.page * a.row;
    const long long items = static_cast<long long>(a.M) * a.layers * 2;
    for (long long item = blockIdx.x; item < items; item += gridDim.x) {
        const int m = static_cast<int>(item / (2 * a.layers)), rest = static_cast<int>(item - static_cast<long long>(m) * 2 * a.layers);
        if (!good(m) || a.src[m] == a.dst[m]) continue;
        uint4* cache = (rest & 1 ? a.v : a.k) + static_cast<long long>(rest >> 1) * a.layer;
        const uint4* from = cache + static_cast<long long>(a.src[m]) * pieces;
        uint4* to = cache + static_cast<long long>(a.dst[m]) * pieces;
        const int filled = (a.used ? a.used[m] : a.page) * a.row;              // pieces of a head
        const bool whole = filled == head;
        for (int p0 = 0; p0 < pieces; p0 += kThreads * kBatch) {
            uint4 x[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int p = p0 + i * kThreads + tid;
                if (p < pieces && (whole || p % head < filled)) x[i] = from[p];
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int p = p0 + i * kThreads + tid;
                if (p < pieces && (whole || p % head < filled)) to[p] = x[i];
            }
        }
    }
}

}  // namespace

dspark_status launch_kv_compact(void* k_cache, void* v_cache, long long layer_stride, int layers, const int32_t* block_table,
                                int max_pages, const int32_t* kv_len, const int32_t* lengths, const int32_t* path,
                                const int32_t* num_accepted, int B, int N, int Hkv, int D, int num_pages, int page,
                                int32_t* kv_len_out, void* ws, cudaStream_t stream) {
    const int row = D / 8;
    const CompactArgs a{static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache), block_table, kv_len, lengths, path, num_accepted,
                        kv_len_out, layer_stride / 8, layers, max_pages, B, N, Hkv, row, num_pages, page, static_cast<WsHeader*>(ws)};
    const dspark_status st = clear_header(ws, stream);
    if (st != DSPARK_OK) return st;
    const int columns = layers * 2 * Hkv * row;
    const cudaError_t e = launch_dependent(kv_compact_kernel, dim3((columns + kThreads - 1) / kThreads, std::min(B, 65535)),
                                           dim3(kThreads), 0, stream, a);
    if (e != cudaSuccess) return cuda_error(e, "launch(kv_compact)");
    return DSPARK_OK;
}

dspark_status launch_kv_copy_pages(void* k_cache, void* v_cache, long long layer_stride, int layers, const int32_t* src,
                                   const int32_t* dst, const int32_t* used, int M, int Hkv, int D, int num_pages, int page,
                                   void* ws, cudaStream_t stream) {
    const CopyArgs a{static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache), src, dst, used, layer_stride / 8, layers, M, Hkv,
                     D / 8, num_pages, page, static_cast<WsHeader*>(ws)};
    const long long items = static_cast<long long>(M) * layers * 2;
    kv_copy_kernel<<<static_cast<unsigned>(std::min(items, 1ll << 30)), kThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_error(e, "launch(kv_copy_pages)");
    return DSPARK_OK;
}

}  // namespace dspark
