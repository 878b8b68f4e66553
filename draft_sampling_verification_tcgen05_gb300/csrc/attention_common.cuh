// Building blocks shared by the attention kernels: operand descriptors of the two products,
// tensor-memory transfers, the exponential, and launches that overlap their predecessor's end.
#pragma once

#include "device_common.cuh"
#include "half_common.cuh"

namespace dspark {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// kHeadroom: how far below a tile's maximum, in log2 units, the softmax puts its reference.  The weights of the
// product with the values have the values' type, since kind::f16 takes no other.  bf16 has fp32's exponents, so
// their size does not matter.  fp16 rounds what is below 2^-14 to a fixed step of 2^-24, and the sum of the weights,
// in fp32, does not: many small weights beside a large one would be lost from the product alone.  With the largest
// weight at 2^7 (2^15 before the reference follows) that step is 2^-31 of it.
template <typename T> struct HalfType;
template <> struct HalfType<__nv_bfloat16> {
    static constexpr uint32_t kMmaFormat = 1;
    static constexpr float kHeadroom = 0.0f;
    static constexpr CUtensorMapDataType kMapType = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
};
template <> struct HalfType<__half> {
    static constexpr uint32_t kMmaFormat = 0;
    static constexpr float kHeadroom = 7.0f;
    static constexpr CUtensorMapDataType kMapType = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
};

// kind::f16 instruction descriptor, fp32 accumulation, M x N tile, A K-major; B K-major (keys) or, with
// kTokenRows, stored token by token with the output's columns contiguous (values).
template <typename T, bool kTokenRows>
__host__ __device__ constexpr uint32_t attn_idesc(int M, int N) {
    return (1u << 4) | (HalfType<T>::kMmaFormat << 7) | (HalfType<T>::kMmaFormat << 10) |
           (kTokenRows ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Descriptor of a value tile in shared memory: 64-column blocks `block_bytes` apart, each with one
// 128-byte swizzled row per token (8 tokens: 1024 bytes).
__device__ __forceinline__ uint64_t sw128_token_rows_desc(uint32_t smem_addr, uint32_t block_bytes) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);      // start address
    d |= static_cast<uint64_t>(block_bytes >> 4) << 16;           // leading offset: next 64 columns
    d |= static_cast<uint64_t>(1024 >> 4) << 32;                  // stride offset: next 8 tokens
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;                          // 128-byte swizzle
    return d;
}

// One lane of a converged warp.  The tensor-core warp runs its waits and address arithmetic with all
// lanes, so that operands stay in uniform registers, and lets one lane issue: issued from a branch that
// only lane 0 had entered, each instruction cost about 100 cycles of operand moves.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// 32 lanes x 32 bits, 32 consecutive columns into r[0..31].
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// Waits for the loads so far; names the 32 registers whose use has to come after it.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                   "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                   "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :: "memory");
}

// The largest of three; NaN counts only where all are.
__device__ __forceinline__ float max3(float x, float y, float z) {
    float m;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(x), "f"(y), "f"(z));
    return m;
}

// 2^x (at most 2 ulp; -infinity gives 0).
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void tmem_st1(uint32_t taddr, uint32_t r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" :: "r"(taddr), "r"(r) : "memory");
}

// Whether a packed pair holds an infinity or NaN (an exponent of all ones).
__device__ __forceinline__ bool pair_not_finite(uint32_t w, __nv_bfloat16) {
    return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

__device__ __forceinline__ bool pair_not_finite(uint32_t w, __half) {
    return (w & 0x7C00u) == 0x7C00u || (w & 0x7C000000u) == 0x7C000000u;
}

// Takes the infinities and NaN out of a value tile (128 token rows of `halves` 128-byte swizzled
// blocks) before its product, which would spread them to rows that do not see them (0 * infinity is
// NaN), and adds weight * value of each to the rows that do.  Called by 128 softmax threads together
// (named barrier `bar`): thread `line` owns token row `line` of the tile and one output row, which
// sees this tile's tokens [first, seen).  The rows' weights are at taddr_p, packed as the product
// takes them, the output row at taddr_o (complete up to the tile before); `row` and `masks` are
// scratch in shared memory.
template <typename T>
__device__ __noinline__ void move_infinities(uint8_t* tile, uint32_t block_bytes, int halves, int line, int held, int first,
                                             int seen, uint32_t taddr_p, uint32_t taddr_o, float* row, uint32_t* masks,
                                             uint32_t bar) {
    bool bad = false;
    if (line < held) {
        for (int x = 0; x < halves; ++x) {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(tile + x * block_bytes + line * 128);
            for (int y = 0; y < 32; ++y) bad = bad || pair_not_finite(p[y], T{});
        }
    }
    const uint32_t vote = __ballot_sync(0xFFFFFFFFu, bad);
    if ((line & 31) == 0) masks[line >> 5] = vote;
    named_bar_sync(bar, 128);
    for (int t = 0; t < 128; ++t) {
        if (((masks[t >> 5] >> (t & 31)) & 1u) == 0u) continue;
        if (line == t) {
            for (int x = 0; x < halves; ++x) {
                uint32_t* p = reinterpret_cast<uint32_t*>(tile + x * block_bytes + line * 128);
                for (int y = 0; y < 32; ++y) {
                    const int at = (y & 3) | ((((y >> 2) ^ line) & 7) << 2);      // the swizzle: where pair y is
                    const uint32_t w = p[at];
                    const bool odd = pair_not_finite(w, T{});
                    const float2 v = unpack2(w, T{});
                    const float lo = v.x - v.x == 0.0f ? 0.0f : v.x, hi = v.y - v.y == 0.0f ? 0.0f : v.y;
                    row[64 * x + 2 * y] = lo;
                    row[64 * x + 2 * y + 1] = hi;
                    if (odd) p[at] = (lo == 0.0f ? w & 0xFFFFu : 0u) | (hi == 0.0f ? w & 0xFFFF0000u : 0u);
                }
            }
        }
        named_bar_sync(bar, 128);
        const uint32_t pair = tmem_ld1(taddr_p + static_cast<uint32_t>(t >> 1));
        tmem_wait_ld();
        const float2 ws = unpack2(pair, T{});
        const float w = (t & 1) != 0 ? ws.y : ws.x;
        for (int d = 0; d < 64 * halves; ++d) {
            const float v = row[d];
            if (v == 0.0f) continue;
            const float o = __uint_as_float(tmem_ld1(taddr_o + static_cast<uint32_t>(d)));
            tmem_wait_ld();
            tmem_st1(taddr_o + static_cast<uint32_t>(d), __float_as_uint(t >= first && t < seen ? fmaf(w, v, o) : o));
            tmem_wait_st();
        }
        named_bar_sync(bar, 128);
    }
}

// mbar_wait with the waiting itself out of line: what is inlined where a wait is usually over is a few
// instructions.
inline __device__ __noinline__ bool mbar_wait_longer(uint64_t* bar, uint32_t parity, WsHeader* ws, long long timeout_ns, uint32_t where) {
    return mbar_wait(bar, parity, ws, timeout_ns, where);
}

__device__ __forceinline__ bool mbar_wait_short(uint64_t* bar, uint32_t parity, WsHeader* ws, long long timeout_ns, uint32_t where) {
    return mbar_try_wait(bar, parity) || mbar_wait_longer(bar, parity, ws, timeout_ns, where);
}

// Named barrier that also tells whether `ok` holds in all its threads.
__device__ __forceinline__ bool named_bar_and(uint32_t id, uint32_t nthreads, bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %3, 0;\n\t"
        "barrier.cta.red.and.pred p, %1, %2, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r) : "r"(id), "r"(nthreads), "r"(static_cast<uint32_t>(ok)) : "memory");
    return r != 0;
}

// Quotients of non-negative values: the 32-bit division where it can serve (the 64-bit one is a long
// dependent chain, and every role starts its work with one).
__device__ __forceinline__ long long quotient(long long x, long long y) {
    if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
    return x / y;
}

// Log-sum-exp from the maximum in log2 units and the sum relative to it.
__device__ __forceinline__ float lse_of(float m2, float l) {
    return l == 0.0f ? -INFINITY : ((m2 == -INFINITY ? 0.0f : m2) + log2f(l)) * kLn2;
}

// Programmatic dependent launch: wait until the preceding kernel of the stream has completed and its
// writes are visible / allow the next one to be launched (it waits by itself before it reads).
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dependency_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Launch of a kernel that starts while its predecessor ends (it calls grid_dependency_wait itself).
template <typename K, typename... Args>
cudaError_t launch_dependent(K kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace dspark
