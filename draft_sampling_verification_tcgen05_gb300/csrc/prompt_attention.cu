// Attention within packed prompts of different lengths.
//
// One warp per (token, query head): the row's query in registers, its sequence's keys one after
// another, a running maximum and sum (the softmax in one pass), all in fp32.
#include "device_common.cuh"
#include "half_common.cuh"
#include "host_common.h"

namespace dspark {
namespace {

struct PromptArgs {
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    const int32_t* cu_seqlens;
    int causal, B, T, Hq, Hkv;
    float scale;
    void* out;
    float* lse;
    WsHeader* ws;
};

template <typename T, int D>
__global__ void __launch_bounds__(128) prompt_attention_kernel(PromptArgs a) {
    constexpr int kPer = D / 32;                      // values of a row per lane (2 or 4)
    const long long row = static_cast<long long>(blockIdx.x) * 4 + warp_id();
    if (row >= static_cast<long long>(a.T) * a.Hq) return;
    const int h = static_cast<int>(row % a.Hq), t = static_cast<int>(row / a.Hq);
    const int lane = lane_id(), hk = h / (a.Hq / a.Hkv);
    // the token's sequence, from the bounds as their running maximum clipped to [0, T]
    int begin = 0, end = 0, lo = 0;
    bool bad = false;
    for (int b = 0; b <= a.B; ++b) {
        const int c = a.cu_seqlens[b], hi = max(lo, min(max(c, 0), a.T));
        bad = bad || c != hi;
        if (b > 0 && lo <= t && t < hi) {
            begin = lo;
            end = a.causal ? t + 1 : hi;
        }
        lo = hi;
    }
    if (bad && lane == 0) flag_input_index(a.ws);

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
    load(a.q, t * a.q_stride + static_cast<long long>(h) * D, q);
    float m = -INFINITY, l = 0.0f;
    for (int j = begin; j < end; ++j) {
        float k[kPer], v[kPer];
        load(a.k, j * a.k_stride + static_cast<long long>(hk) * D, k);
        load(a.v, j * a.v_stride + static_cast<long long>(hk) * D, v);
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
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    T* out = static_cast<T*>(a.out) + row * D + lane * kPer;
#pragma unroll
    for (int e = 0; e < kPer; e += 2)
        *reinterpret_cast<uint32_t*>(out + e) = pack2(o[e] * inv, o[e + 1] * inv, T{});
    if (a.lse && lane == 0) a.lse[row] = l != 0.0f ? (m == -INFINITY ? 0.0f : m) + logf(l) : -INFINITY;
}

}  // namespace

dspark_status launch_prompt_attention(const void* q, const void* k, const void* v, dspark_dtype dtype,
                                      long long q_stride, long long k_stride, long long v_stride,
                                      const int32_t* cu_seqlens, float scale, int causal, int B, int T, int Hq,
                                      int Hkv, int D, void* out, float* lse, void* ws, cudaStream_t stream,
                                      const DeviceInfo&) {
    dspark_status st = clear_workspace(ws, sizeof(WsHeader), stream);
    if (st != DSPARK_OK) return st;
    PromptArgs a{q, k, v, q_stride, k_stride, v_stride, cu_seqlens, causal, B, T, Hq, Hkv, scale, out, lse,
                 static_cast<WsHeader*>(ws)};
    const long long blocks = (static_cast<long long>(T) * Hq + 3) / 4;
    if (blocks >= (1ll << 31)) {
        set_error("prompt_attention: too many rows (T=%d Hq=%d)", T, Hq);
        return DSPARK_ERR_UNSUPPORTED;
    }
    const unsigned grid = static_cast<unsigned>(blocks);
    if (dtype == DSPARK_BF16) {
        if (D == 64) prompt_attention_kernel<__nv_bfloat16, 64><<<grid, 128, 0, stream>>>(a);
        else prompt_attention_kernel<__nv_bfloat16, 128><<<grid, 128, 0, stream>>>(a);
    } else {
        if (D == 64) prompt_attention_kernel<__half, 64><<<grid, 128, 0, stream>>>(a);
        else prompt_attention_kernel<__half, 128><<<grid, 128, 0, stream>>>(a);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_error(e, "launch(prompt_attention)");
    return DSPARK_OK;
}

}  // namespace dspark
