// Integer masses of weights, shares of them, and what the blocks of a cluster need to exchange them.
#pragma once

#include "device_common.cuh"

namespace dspark {

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
// Asynchronous store there, counted in bytes on an mbarrier of the same block.
__device__ __forceinline__ void send(uint32_t at, u64 v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];"
                 :: "r"(at), "l"(v), "r"(bar) : "memory");
}
// Likewise of two values that lie together, 16-byte aligned.
__device__ __forceinline__ void send2(uint32_t at, u64 v, u64 w, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [%0], {%1, %2}, [%3];"
                 :: "r"(at), "l"(v), "l"(w), "r"(bar) : "memory");
}

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
    // The warp's sum, of fewer than 128 entries in each lane (its halves then stay within 32 bits).
    __device__ __forceinline__ u64 warp_value() const {
        return (static_cast<u64>(__reduce_add_sync(0xFFFFFFFFu, hi - n * kHalfBias)) << 20) +
               __reduce_add_sync(0xFFFFFFFFu, lo - n * kHalfBias);
    }
    __device__ __forceinline__ u64 value() const {
        return (static_cast<u64>(hi - n * kHalfBias) << 20) + (lo - n * kHalfBias);
    }
};
}  // namespace dspark
