// Appending new tokens to a paged key-value cache, with the position rotation on the way.
//
// Each head row of a token is read once, normalised and rotated in fp32 registers, rounded once
// and written once: queries to their output, keys and values to the cache slot of the token.
//
// A row of D values is held by D / 16 adjacent lanes, sixteen values (two 16-byte chunks) each.
// The chunks of a lane are chosen so that a rotation's two halves meet in the lane: with halves
// rot/2 apart, lane j of the rotated part holds chunks j and j + rot/16; with interleaved pairs,
// chunks 2j and 2j + 1.  The norm's mean is a shuffle sum over the row's lanes.
#include "device_common.cuh"
#include "half_common.cuh"
#include "host_common.h"

#include <algorithm>

namespace dspark {
namespace {

struct AppendArgs {
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    const int32_t *positions, *slots;
    const float* cos_sin;
    const float *q_norm, *k_norm;
    float eps;
    int max_positions, rot;
    int T, Hq, Hkv, D;
    void *q_out, *k_cache, *v_cache;
    int num_pages, page;
    WsHeader* ws;
};

constexpr int kThreads = 256;

// One head row per group of `lanes` (a power of two >= D / 16) lanes.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(AppendArgs a, int lanes) {
    const int rows = a.Hq + 2 * a.Hkv;
    const long long item = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) / lanes;
    const int j = threadIdx.x & (lanes - 1);
    const bool in_range = item < static_cast<long long>(a.T) * rows;
    const int t = in_range ? static_cast<int>(item / rows) : 0;
    const int row = in_range ? static_cast<int>(item % rows) : 0;
    const bool active = in_range && j < a.D / 16;

    const int pos = a.positions[t], slot = a.slots[t];
    const bool pos_ok = pos >= 0 && pos < a.max_positions;
    const bool slot_ok = slot >= -1 && static_cast<long long>(slot) < static_cast<long long>(a.num_pages) * a.page;
    if (in_range && row == 0 && j == 0 && !(pos_ok && slot_ok)) flag_input_index(a.ws);

    const T* src;
    T* dst = nullptr;
    const float* weight = nullptr;
    bool rotated = true;
    if (row < a.Hq) {
        src = static_cast<const T*>(a.q) + t * a.q_stride + static_cast<long long>(row) * a.D;
        dst = static_cast<T*>(a.q_out) + (static_cast<long long>(t) * a.Hq + row) * a.D;
        weight = a.q_norm;
    } else {
        const bool key = row < a.Hq + a.Hkv;
        const int h = row - a.Hq - (key ? 0 : a.Hkv);
        src = (key ? static_cast<const T*>(a.k) + t * a.k_stride : static_cast<const T*>(a.v) + t * a.v_stride) +
              static_cast<long long>(h) * a.D;
        if (slot_ok && slot >= 0 && pos_ok)
            dst = static_cast<T*>(key ? a.k_cache : a.v_cache) +
                  ((static_cast<long long>(slot / a.page) * a.Hkv + h) * a.page + slot % a.page) * a.D;
        weight = key ? a.k_norm : nullptr;
        rotated = key;
    }

    // the lane's two chunks of eight values
    const int half = a.rot / 16;
    int c0 = 2 * j, c1 = 2 * j + 1;
    if (!kInterleaved && j < half) {
        c0 = j;
        c1 = j + half;
    }
    float x[16];
    if (active) {
        unpack8(*reinterpret_cast<const uint4*>(src + 8 * c0), x, T{});
        unpack8(*reinterpret_cast<const uint4*>(src + 8 * c1), x + 8, T{});
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 0.0f;
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
    for (int d = lanes >> 1; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
    if (!active || dst == nullptr) return;

    if (weight != nullptr) {
        const float r = rsqrtf(ss / static_cast<float>(a.D) + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] *= r * weight[8 * c0 + i];
            x[8 + i] *= r * weight[8 * c1 + i];
        }
    }
    if (rotated && j < half) {
        if (pos_ok) {
            const float* cs = a.cos_sin + static_cast<long long>(pos) * a.rot;
            float c[8], s[8];
            load8(cs + 8 * j, c);
            load8(cs + a.rot / 2 + 8 * j, s);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float& u = kInterleaved ? x[2 * i] : x[i];
                float& w = kInterleaved ? x[2 * i + 1] : x[8 + i];
                const float p = u, q = w;
                u = p * c[i] - q * s[i];
                w = q * c[i] + p * s[i];
            }
        }
    }
    if (!pos_ok) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 0.0f;
    }
    *reinterpret_cast<uint4*>(dst + 8 * c0) = pack8(x, T{});
    *reinterpret_cast<uint4*>(dst + 8 * c1) = pack8(x + 8, T{});
}

}  // namespace

dspark_status launch_kv_append(const void* q, const void* k, const void* v, dspark_dtype dtype, long long q_stride,
                               long long k_stride, long long v_stride, const int32_t* positions, const int32_t* slots,
                               const float* cos_sin, int max_positions, int rot, int interleaved, const float* q_norm,
                               const float* k_norm, float eps, int T, int Hq, int Hkv, int D, void* q_out,
                               void* k_cache, void* v_cache, int num_pages, int page, void* ws, cudaStream_t stream,
                               const DeviceInfo&) {
    dspark_status st = clear_workspace(ws, sizeof(WsHeader), stream);
    if (st != DSPARK_OK) return st;
    AppendArgs a{q, k, v, q_stride, k_stride, v_stride, positions, slots, cos_sin, q_norm, k_norm, eps,
                 max_positions, rot, T, Hq, Hkv, D, q_out, k_cache, v_cache, num_pages, page,
                 static_cast<WsHeader*>(ws)};
    int lanes = 1;
    while (lanes < D / 16) lanes *= 2;
    const long long threads = static_cast<long long>(T) * (Hq + 2 * Hkv) * lanes;
    const long long blocks = (threads + kThreads - 1) / kThreads;
    if (blocks >= (1ll << 31)) {
        set_error("kv_append: too many rows (T=%d Hq=%d Hkv=%d)", T, Hq, Hkv);
        return DSPARK_ERR_UNSUPPORTED;
    }
    const unsigned grid = static_cast<unsigned>(blocks);
    if (dtype == DSPARK_BF16) {
        if (interleaved) kv_append_kernel<__nv_bfloat16, true><<<grid, kThreads, 0, stream>>>(a, lanes);
        else kv_append_kernel<__nv_bfloat16, false><<<grid, kThreads, 0, stream>>>(a, lanes);
    } else {
        if (interleaved) kv_append_kernel<__half, true><<<grid, kThreads, 0, stream>>>(a, lanes);
        else kv_append_kernel<__half, false><<<grid, kThreads, 0, stream>>>(a, lanes);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_error(e, "launch(kv_append)");
    return DSPARK_OK;
}

}  // namespace dspark
