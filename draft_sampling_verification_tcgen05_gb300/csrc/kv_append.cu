// Appending new tokens to a paged key-value cache, with the position rotation on the way.
//
// Each head row of a token is read once, normalised and rotated in fp32 registers, rounded once
// and written once: queries to their output, keys and values to the cache slot of the token.
//
// A row of D values is held by D / 16 adjacent lanes, sixteen values (two 16-byte chunks) each.
// The chunks of a lane are chosen so that a rotation's two halves meet in the lane: with halves
// rot/2 apart, lane j of the rotated part holds chunks j and j + rot/16; with interleaved pairs,
// chunks 2j and 2j + 1.  The norm's mean is a shuffle sum over the row's lanes.
//
// It is bound by memory.  A lane takes kRows rows of one token: their loads are under way together,
// and the token's angles, twice a row's bytes, are read once for all of them.  8191 tokens of 32 + 2 * 8
// heads of 128 in fp16 (201 MB) take 37.5 us, 5.4 TB/s of the 6.8 that a copy reaches; two rows a lane
// 40 us, one row 49 us.  What counts beside the rows is how many loads the registers leave room for: four
// rows in six blocks of 128 threads (80 registers) 37.5 us, in two of 256 (109 registers) 45 us, in four of
// 256 (64 registers) 51 us.
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

constexpr int kThreads = 128;
constexpr int kRowsMost = 4;
constexpr int kFew = 2048;                                 // threads per SM

// Bounds of the tokens' positions and slots; a token outside them gets zeros and no slot.
__device__ __forceinline__ bool position_ok(const AppendArgs& a, int pos) { return pos >= 0 && pos < a.max_positions; }
__device__ __forceinline__ bool slot_ok(const AppendArgs& a, int slot) { return slot >= -1 && slot < a.num_pages * a.page; }

// kRows head rows of a token per group of 2^lane_bits (>= D / 16) lanes: rows g, g + groups, ...
template <typename T, bool kInterleaved, int kRows>
__global__ void __launch_bounds__(kThreads, 6) kv_append_kernel(const __grid_constant__ AppendArgs a, int lane_bits, uint32_t groups) {
    if (blockIdx.x == 0) {
        // the status word is this block's alone, so nothing has to clear it before
        bool bad = false;
        for (int t = threadIdx.x; t < a.T; t += kThreads) bad |= !position_ok(a, a.positions[t]) || !slot_ok(a, a.slots[t]);
        bad = __syncthreads_or(bad) != 0;
        if (threadIdx.x < sizeof(WsHeader) / 4) reinterpret_cast<uint32_t*>(a.ws)[threadIdx.x] = 0u;
        __syncthreads();
        if (threadIdx.x == 0 && bad) flag_input_index(a.ws);
    }
    const int rows = a.Hq + 2 * a.Hkv;
    const int lanes = 1 << lane_bits;
    const uint32_t item = (blockIdx.x * static_cast<uint32_t>(kThreads / 32) << (5 - lane_bits)) + (threadIdx.x >> lane_bits);
    const int j = static_cast<int>(threadIdx.x) & (lanes - 1);
    const uint32_t token = item / groups;
    const int g = static_cast<int>(item - token * groups);
    const bool in_range = token < static_cast<uint32_t>(a.T);
    const long long t = in_range ? token : 0;
    const bool active = in_range && j < a.D / 16;

    // the lane's two chunks of eight values
    const int half = a.rot / 16;
    int c0 = 2 * j, c1 = 2 * j + 1;
    if (!kInterleaved && j < half) {
        c0 = j;
        c1 = j + half;
    }
    uint4 raw[kRows][2];
#pragma unroll
    for (int y = 0; y < kRows; ++y) {
        const int row = g + y * static_cast<int>(groups);
        raw[y][0] = raw[y][1] = make_uint4(0u, 0u, 0u, 0u);
        if (!active || row >= rows) continue;
        const T* src = row < a.Hq           ? static_cast<const T*>(a.q) + t * a.q_stride + static_cast<long long>(row) * a.D
                       : row < a.Hq + a.Hkv ? static_cast<const T*>(a.k) + t * a.k_stride + static_cast<long long>(row - a.Hq) * a.D
                                            : static_cast<const T*>(a.v) + t * a.v_stride +
                                                  static_cast<long long>(row - a.Hq - a.Hkv) * a.D;
        raw[y][0] = *reinterpret_cast<const uint4*>(src + 8 * c0);
        raw[y][1] = *reinterpret_cast<const uint4*>(src + 8 * c1);
    }
    const int pos = a.positions[t], slot = a.slots[t];
    const bool pos_ok = position_ok(a, pos);
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = 1.0f;
        s[i] = 0.0f;
    }
    const bool turns = active && pos_ok && j < half;
    if (turns) {
        const float* cs = a.cos_sin + static_cast<long long>(pos) * a.rot;
        load8(cs + 8 * j, c);
        load8(cs + a.rot / 2 + 8 * j, s);
    }
    T *keys = nullptr, *values = nullptr;                  // of key head 0
    if (pos_ok && slot >= 0 && slot_ok(a, slot)) {
        const int in_page = slot / a.page;
        const long long at = (static_cast<long long>(in_page) * a.Hkv * a.page + (slot - in_page * a.page)) * a.D;
        keys = static_cast<T*>(a.k_cache) + at;
        values = static_cast<T*>(a.v_cache) + at;
    }

#pragma unroll
    for (int y = 0; y < kRows; ++y) {
        const int row = g + y * static_cast<int>(groups);
        const bool query = row < a.Hq, value = row >= a.Hq + a.Hkv;
        T* dst = nullptr;
        if (active && row < rows) {
            if (query) dst = static_cast<T*>(a.q_out) + (t * a.Hq + row) * a.D;
            else if (!value && keys) dst = keys + static_cast<long long>(row - a.Hq) * a.page * a.D;
            else if (value && values) dst = values + static_cast<long long>(row - a.Hq - a.Hkv) * a.page * a.D;
        }
        float x[16];
        unpack8(raw[y][0], x, T{});
        unpack8(raw[y][1], x + 8, T{});
        const float* weight = query ? a.q_norm : value ? nullptr : a.k_norm;
        if (a.q_norm || a.k_norm) {                        // the same for all lanes: they meet in the sum
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
            for (int d = lanes >> 1; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
            if (weight != nullptr && active) {
                const float r = rsqrtf(ss / static_cast<float>(a.D) + a.eps);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[i] *= r * weight[8 * c0 + i];
                    x[8 + i] *= r * weight[8 * c1 + i];
                }
            }
        }
        if (dst == nullptr) continue;
        if (!value && turns) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float& u = kInterleaved ? x[2 * i] : x[i];
                float& w = kInterleaved ? x[2 * i + 1] : x[8 + i];
                const float p = u, q = w;
                u = p * c[i] - q * s[i];
                w = q * c[i] + p * s[i];
            }
        }
        if (!pos_ok) {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = 0.0f;
        }
        *reinterpret_cast<uint4*>(dst + 8 * c0) = pack8(x, T{});
        *reinterpret_cast<uint4*>(dst + 8 * c1) = pack8(x + 8, T{});
    }
}

template <typename T, bool kInterleaved>
void launch_rows(const AppendArgs& a, int lane_bits, int rows, unsigned grid, uint32_t groups, cudaStream_t stream) {
    if (rows == 1) kv_append_kernel<T, kInterleaved, 1><<<grid, kThreads, 0, stream>>>(a, lane_bits, groups);
    else kv_append_kernel<T, kInterleaved, kRowsMost><<<grid, kThreads, 0, stream>>>(a, lane_bits, groups);
}

}  // namespace

dspark_status launch_kv_append(const void* q, const void* k, const void* v, dspark_dtype dtype, long long q_stride,
                               long long k_stride, long long v_stride, const int32_t* positions, const int32_t* slots,
                               const float* cos_sin, int max_positions, int rot, int interleaved, const float* q_norm,
                               const float* k_norm, float eps, int T, int Hq, int Hkv, int D, void* q_out,
                               void* k_cache, void* v_cache, int num_pages, int page, void* ws, cudaStream_t stream,
                               const DeviceInfo& dev) {
    AppendArgs a{q, k, v, q_stride, k_stride, v_stride, positions, slots, cos_sin, q_norm, k_norm, eps,
                 max_positions, rot, T, Hq, Hkv, D, q_out, k_cache, v_cache, num_pages, page,
                 static_cast<WsHeader*>(ws)};
    int lane_bits = 0;
    while ((1 << lane_bits) < D / 16) ++lane_bits;
    // One row per lane while that leaves the SMs room for more: the calls are then short, and latency counts.
    // With 48 heads of 128 the bound is at 800 tokens, one row against four there 5.9 and 6.0 us; 64 tokens 2.8
    // and 4.6 us, 2400 tokens 13.9 and 11.9 us.
    const int all = Hq + 2 * Hkv;
    const long long threads = (static_cast<long long>(T) * all) << lane_bits;
    const int rows = threads <= static_cast<long long>(dev.sm_count) * kFew ? 1 : kRowsMost;
    const uint32_t groups = static_cast<uint32_t>((all + rows - 1) / rows);
    const long long items = static_cast<long long>(T) * groups;
    if (items >= (1ll << 31)) {
        set_error("kv_append: too many rows (T=%d Hq=%d Hkv=%d)", T, Hq, Hkv);
        return DSPARK_ERR_UNSUPPORTED;
    }
    const unsigned grid = static_cast<unsigned>(((items << lane_bits) + kThreads - 1) / kThreads);
    if (dtype == DSPARK_BF16) {
        if (interleaved) launch_rows<__nv_bfloat16, true>(a, lane_bits, rows, grid, groups, stream);
        else launch_rows<__nv_bfloat16, false>(a, lane_bits, rows, grid, groups, stream);
    } else {
        if (interleaved) launch_rows<__half, true>(a, lane_bits, rows, grid, groups, stream);
        else launch_rows<__half, false>(a, lane_bits, rows, grid, groups, stream);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_error(e, "launch(kv_append)");
    return DSPARK_OK;
}

}  // namespace dspark
