// Attention of a window of new tokens per request over a paged key-value cache.
//
// One warp per (request, window row, query head): the row's query in registers, the cached keys
// one after another, a running maximum and sum (the softmax in one pass), all in fp32.
#include "device_common.cuh"
#include "half_common.cuh"
#include "host_common.h"

namespace dspark {
namespace {

struct PagedArgs {
    const void *q, *k_cache, *v_cache;
    const int32_t *block_table, *kv_len, *lengths;
    int max_pages, causal, B, N, Hq, Hkv, num_pages, page;
    float scale;
    void* out;
    float* lse;
    WsHeader* ws;
};

template <typename T, int D>
__global__ void __launch_bounds__(128) paged_attention_kernel(PagedArgs a) {
    constexpr int kPer = D / 32;                      // values of a row per lane (2 or 4)
    const long long row = static_cast<long long>(blockIdx.x) * 4 + warp_id();
    if (row >= static_cast<long long>(a.B) * a.N * a.Hq) return;
    const int h = static_cast<int>(row % a.Hq);
    const int i = static_cast<int>(row / a.Hq % a.N), b = static_cast<int>(row / a.Hq / a.N);
    const int lane = lane_id();
    int kv = a.kv_len[b], n = a.lengths ? a.lengths[b] : a.N;
    if (kv < 0 || kv > static_cast<long long>(a.max_pages) * a.page || n < 0 || n > a.N) {
        if (lane == 0) flag_input_index(a.ws);
        kv = n = 0;
    }
    const int limit = i >= n ? 0 : a.causal ? kv - n + i + 1 : kv;
    const int hk = h / (a.Hq / a.Hkv);

    float q[kPer], o[kPer] = {};
    auto load = [&](const void* base, long long at, float* x) {
        const T* p = static_cast<const T*>(base) + at + lane * kPer;
#pragma unroll
        for (int e = 0; e < kPer; e += 2) {
            const float2 v = unpack2(*reinterpret_cast<const uint32_t*>(p + e), T{});
            x[e] = v.x;
            x[e + 1] = v.y;
        }
    };
    load(a.q, row * D, q);
    float m = -INFINITY, l = 0.0f;
    bool bad = false;
    for (int j = 0; j < limit; ++j) {
        int pg = a.block_table[static_cast<long long>(b) * a.max_pages + j / a.page];
        if (pg < 0 || pg >= a.num_pages) {
            bad = true;
            pg = 0;
        }
        const long long at = ((static_cast<long long>(pg) * a.Hkv + hk) * a.page + j % a.page) * D;
        float k[kPer], v[kPer];
        load(a.k_cache, at, k);
        load(a.v_cache, at, v);
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) s = fmaf(q[e], k[e], s);
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        s *= a.scale;
        const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.0f : mn;
        const float c = expf((m == -INFINITY ? ref : m) - ref), w = expf(s - ref);
        l = l * c + w;
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] = o[e] * c + w * v[e];
        m = mn;
    }
    if (bad && lane == 0) flag_input_index(a.ws);
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    T* out = static_cast<T*>(a.out) + row * D + lane * kPer;
#pragma unroll
    for (int e = 0; e < kPer; e += 2)
        *reinterpret_cast<uint32_t*>(out + e) = pack2(o[e] * inv, o[e + 1] * inv, T{});
    if (a.lse && lane == 0) a.lse[row] = l != 0.0f ? (m == -INFINITY ? 0.0f : m) + logf(l) : -INFINITY;
}

}  // namespace

size_t paged_attention_workspace_bytes(int B, int N, int Hq, int D) {
    return B < 1 || N < 1 || Hq < 1 || D < 1 ? 0 : sizeof(WsHeader);
}

dspark_status launch_paged_attention(const void* q, const void* k_cache, const void* v_cache, dspark_dtype dtype,
                                     const int32_t* block_table, int max_pages, const int32_t* kv_len,
                                     const int32_t* lengths, float scale, int causal, int B, int N, int Hq, int Hkv,
                                     int D, int num_pages, int page, void* out, float* lse, void* ws,
                                     cudaStream_t stream, const DeviceInfo&) {
    dspark_status st = clear_workspace(ws, sizeof(WsHeader), stream);
    if (st != DSPARK_OK) return st;
    PagedArgs a{q, k_cache, v_cache, block_table, kv_len, lengths, max_pages, causal, B, N, Hq, Hkv, num_pages, page,
                scale, out, lse, static_cast<WsHeader*>(ws)};
    const long long blocks = (static_cast<long long>(B) * N * Hq + 3) / 4;
    if (blocks >= (1ll << 31)) {
        set_error("paged_attention: too many rows (B=%d N=%d Hq=%d)", B, N, Hq);
        return DSPARK_ERR_UNSUPPORTED;
    }
    const unsigned grid = static_cast<unsigned>(blocks);
    if (dtype == DSPARK_BF16) {
        if (D == 64) paged_attention_kernel<__nv_bfloat16, 64><<<grid, 128, 0, stream>>>(a);
        else paged_attention_kernel<__nv_bfloat16, 128><<<grid, 128, 0, stream>>>(a);
    } else {
        if (D == 64) paged_attention_kernel<__half, 64><<<grid, 128, 0, stream>>>(a);
        else paged_attention_kernel<__half, 128><<<grid, 128, 0, stream>>>(a);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_error(e, "launch(paged_attention)");
    return DSPARK_OK;
}

}  // namespace dspark
