// dspark_paged_attention: arguments and launches of the kernels of paged_attention.cuh.
#include "paged_attention.cuh"

namespace dspark {

size_t paged_attention_workspace_bytes(int B, int N, int Hq, int D) {
    if (B < 1 || N < 1 || Hq < 1 || D < 1) return 0;
    return partials_end(rows_cap_of(N, Hq), D);
}

dspark_status launch_paged_attention(const void* q, const void* k_cache, const void* v_cache, dspark_dtype dtype,
                                     const int32_t* block_table, int max_pages, const int32_t* kv_len,
                                     const int32_t* lengths, float scale, int causal, int B, int N, int Hq, int Hkv,
                                     int D, int num_pages, int page, void* out, float* lse, void* ws,
                                     cudaStream_t stream, const DeviceInfo& dev) {
    if (static_cast<long long>(num_pages) * Hkv >= (1ll << 31) || static_cast<long long>(B) * N >= (1ll << 31)) {
        set_error("paged_attention: num_pages * Hkv and B * N must be below 2^31");
        return DSPARK_ERR_UNSUPPORTED;
    }
    const PagedArgs a = paged_args(q, k_cache, v_cache, block_table, max_pages, kv_len, lengths, scale, causal, B, N, Hq, Hkv, D,
                                   num_pages, page, out, lse, ws);
    const int grid = std::min(dev.sm_count, kMaxCtas);
    if (dtype == DSPARK_BF16)
        return D == 64 ? launch_typed<__nv_bfloat16, 64, false>(a, grid, stream) : launch_typed<__nv_bfloat16, 128, false>(a, grid, stream);
    return D == 64 ? launch_typed<__half, 64, false>(a, grid, stream) : launch_typed<__half, 128, false>(a, grid, stream);
}

}  // namespace dspark
