// Sampling with temperature, top-k, min-p and top-p from given uniforms.
//
// The kept set is a prefix of the entries ordered by (logit, largest first; id, smallest first).
// Its last entry is found in two steps of exact integer arithmetic: the 32 ordered bits of the
// last entry's logit, one bit at a time (is the count, or the mass, of the entries above still
// short of what is wanted?), then its id among the entries that share that logit.
// One block per row; every step reads the row again.
#include "device_common.cuh"
#include "half_common.cuh"
#include "host_common.h"

namespace dspark {
namespace {

constexpr int kThreads = 1024;

struct SampleArgs {
    const void* logits;
    const float* temperature;
    const int32_t* top_k;
    const float *top_p, *min_p, *u;
    int R, V;
    int32_t* tokens;
    float* probs;
    WsHeader* ws;
};

__device__ __forceinline__ float load_logit(const float* p, int v) { return p[v]; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p, int v) { return __bfloat162float(p[v]); }

// floor(total * frac / 2^24), total < 2^62, frac <= 2^24.
__device__ __forceinline__ unsigned long long share(unsigned long long total, uint32_t frac) {
    return (total >> 24) * frac + (((total & 0xFFFFFFull) * frac) >> 24);
}

__device__ unsigned long long block_sum(unsigned long long x, unsigned long long* s) {
    x = warp_sum_u64(x);
    __syncthreads();
    if (lane_id() == 0) s[warp_id()] = x;
    __syncthreads();
    unsigned long long r = 0;
    for (int w = 0; w < kThreads / 32; ++w) r += s[w];
    return r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(SampleArgs a) {
    __shared__ unsigned long long s_sum[kThreads / 32];
    __shared__ int s_token;
    const int r = blockIdx.x, tid = threadIdx.x, V = a.V;
    const T* x = static_cast<const T*>(a.logits) + static_cast<long long>(r) * V;

    // parameters, each read as the nearest valid value
    uint32_t flags = 0;
    float temp = a.temperature[r], top_p = a.top_p[r], min_p = a.min_p[r], u = a.u[r];
    int k = a.top_k[r];
    if (!(temp >= 0.0f) || isinf(temp)) { temp = 0.0f; flags |= DSPARK_STATUS_NUMERIC; }
    if (!(top_p >= 0.0f && top_p <= 1.0f)) { top_p = top_p < 0.0f ? 0.0f : 1.0f; flags |= DSPARK_STATUS_INPUT_RANGE; }
    if (!(min_p >= 0.0f && min_p <= 1.0f)) { min_p = min_p > 1.0f ? 1.0f : 0.0f; flags |= DSPARK_STATUS_INPUT_RANGE; }
    if (!(u >= 0.0f && u < 1.0f)) { u = u >= 1.0f ? 0x1.fffffep-1f : 0.0f; flags |= DSPARK_STATUS_INPUT_RANGE; }
    if (k <= 0 || k > V) k = V;
    if (temp == 0.0f) k = 1;
    const float inv = temp == 0.0f ? 1.0f : fminf(__fdiv_rn(1.0f, temp), 3.402823466e+38f);

    // an entry's ordered bits (0: skipped), and its weight
    auto bits = [&](float v) { return v < INFINITY && v > -INFINITY ? float_order_bits(v) : 0u; };
    uint32_t top = 0, odd = 0;
    for (int v = tid; v < V; v += kThreads) {
        const float l = load_logit(x, v);
        if (!(l < INFINITY)) odd = 1;
        top = max(top, bits(l));
    }
    if (__syncthreads_or(odd)) flags |= DSPARK_STATUS_NUMERIC;
    {
        __shared__ uint32_t s_top;
        if (tid == 0) { s_top = 0; s_token = 0; }
        __syncthreads();
        atomicMax(&s_top, top);
        __syncthreads();
        top = s_top;
    }
    if (top == 0) flags |= DSPARK_STATUS_NUMERIC;
    const float m = float_from_order_bits(top);
    auto weight = [&](float l) { return expf(__fmul_rn(__fsub_rn(l, m), inv)); };
    auto mass = [&](float w) { return static_cast<unsigned long long>(__fmul_rn(w, 0x1p40f)); };

    // The entries with ordered bits >= key, of those with exactly `key` the ones with id < id_end:
    // count and mass.
    auto above = [&](uint32_t key, int id_end, unsigned long long& count, unsigned long long& sum) {
        unsigned long long c = 0, s = 0;
        for (int v = tid; v < V; v += kThreads) {
            const float l = load_logit(x, v);
            const uint32_t b = bits(l);
            if (b == 0 || b < key || (b == key && v >= id_end)) continue;
            const float w = weight(l);
            if (w < min_p) continue;
            c += 1;
            s += mass(w);
        }
        count = block_sum(c, s_sum);
        sum = block_sum(s, s_sum);
    };
    // The largest (key, id) prefix end at which `enough(count, mass)` first holds; all entries if never.
    auto cut = [&](auto enough, uint32_t& key, int& id_end, unsigned long long& sum) {
        unsigned long long c, s;
        key = 1;
        id_end = V;
        above(1, V, c, s);
        sum = s;
        if (!enough(c, s)) return;
        uint32_t lo = 1, hi = top;                    // the largest key with enough at or above it
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo + 1) / 2;
            above(mid, V, c, s);
            if (enough(c, s)) lo = mid; else hi = mid - 1;
        }
        key = lo;
        int a0 = 1, b0 = V;                           // the smallest id_end with enough
        while (a0 < b0) {
            const int mid = a0 + (b0 - a0) / 2;
            above(key, mid, c, s);
            if (enough(c, s)) b0 = mid; else a0 = mid + 1;
        }
        id_end = b0;
        above(key, id_end, c, sum);
    };
    uint32_t key;
    int id_end;
    unsigned long long Q, Q2;
    cut([&](unsigned long long c, unsigned long long) { return c >= static_cast<unsigned long long>(k); }, key, id_end, Q);
    const unsigned long long need = share(Q, static_cast<uint32_t>(top_p * 0x1p24f));
    uint32_t key2;
    int id_end2;
    cut([&](unsigned long long c, unsigned long long s) { return s >= need && c >= 1; }, key2, id_end2, Q2);
    if (key2 > key || (key2 == key && id_end2 < id_end)) { key = key2; id_end = id_end2; }
    else Q2 = Q;

    // the draw: the first id whose inclusive prefix mass exceeds t
    const unsigned long long t = share(Q2, static_cast<uint32_t>(u * 0x1p24f));
    auto kept = [&](float l, int v) {
        const uint32_t b = bits(l);
        if (b == 0 || b < key || (b == key && v >= id_end)) return 0.0f;
        const float w = weight(l);
        return w < min_p ? 0.0f : w;
    };
    int lo = 0, hi = V - 1;
    while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        unsigned long long s = 0;
        for (int v = tid; v <= mid; v += kThreads) s += mass(kept(load_logit(x, v), v));
        s = block_sum(s, s_sum);
        if (s > t) hi = mid; else lo = mid + 1;
    }
    if (tid == 0) {
        a.tokens[r] = top == 0 ? 0 : lo;
        if (flags) set_status(a.ws, flags);
    }
    if (a.probs != nullptr) {
        const float total = __fmul_rn(__ull2float_rn(Q2), 0x1p-40f);
        for (int v = tid; v < V; v += kThreads) {
            const float w = top == 0 ? 0.0f : kept(load_logit(x, v), v);
            a.probs[static_cast<long long>(r) * V + v] = mass(w) > 0 ? __fdiv_rn(w, total) : 0.0f;
        }
    }
}

}  // namespace

dspark_status launch_sample(const void* logits, dspark_dtype dtype, const float* temperature, const int32_t* top_k,
                            const float* top_p, const float* min_p, const float* u, int R, int V, int32_t* tokens,
                            float* probs, void* ws, cudaStream_t stream, const DeviceInfo&) {
    dspark_status st = clear_workspace(ws, sizeof(WsHeader), stream);
    if (st != DSPARK_OK) return st;
    SampleArgs a{logits, temperature, top_k, top_p, min_p, u, R, V, tokens, probs, static_cast<WsHeader*>(ws)};
    if (dtype == DSPARK_F32) sample_kernel<float><<<R, kThreads, 0, stream>>>(a);
    else sample_kernel<__nv_bfloat16><<<R, kThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_error(e, "launch(sample)");
    return DSPARK_OK;
}

}  // namespace dspark
