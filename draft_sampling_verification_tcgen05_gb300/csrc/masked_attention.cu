// dspark_tree_attention and dspark_window_attention: arguments and launches of the kernels of paged_attention.cuh and
// wide_attention.cuh with masks.  Both go through one instantiation: the masks are looked at only in the tiles that a
// row does not see as a whole, a tree's last one to three and the two ends of a window, so a switch at run time costs
// nothing.
#include "wide_attention.cuh"

namespace dspark {

namespace {

int words_of(int N) { return (N + 31) / 32; }
int wide_cap_of(int N, int heads) { return static_cast<int>(std::min<long long>(2 * kTile, static_cast<long long>(N) * heads)); }

template <typename T, int D>
dspark_status launch(PagedArgs& a, int grid, cudaStream_t stream) {
    // More rows than a tile holds: two tiles against one stream of keys and values (wide_attention.cuh), except where
    // requests bring their own lengths and two tiles hold the longest.  Most of them then fill one tile, and a block that has one
    // tile has nothing to do while that is in its softmax; two blocks' worth of single tiles it is then.  The host knows neither
    // how many rows the requests use nor how long their contexts are, so this is a guess from the call's shape; where the other
    // side was the faster one (marked), it costs 3 us, 5 % and 17 %.
    // Measured, the kernels of a call, wide / one tile at a time, 8 heads of keys, four (or eight) of queries to each, bf16, in us:
    //   lengths given      16 trees of up to 64 nodes, 500 to 8000 keys   65.7 / 57.0     16 of up to 17 of 8 heads each  55.8 / 45.7
    //                      33 of up to 64, D = 64, a window of 2048       79.5 / 74.9     1 of 64, 1000 keys              22.2 / 19.3
    //                      4 of up to 64, 20000 to 60000 keys (marked)   138.4 / 146.0    64 of up to 64, 100 to 1000
    //                                                                                     keys (marked)                   64.8 / 75.6
    //                      8 of up to 200, 200 to 4000 keys               45.8 / 45.1     2 chunks of up to 4096,
    //                                                                                     a window of 1024               140.2 / 185.9
    //   every row used     16 trees of 64 nodes, 500 to 8000 keys         72.0 / 75.8     16 of 17, 8 heads each          64.4 / 72.5
    //                      4 of 64, 20000 to 60000 keys                  147.0 / 184.0    64 of 64, 100 to 1000           69.4 / 92.9
    //                      2 chunks of 4096, a window of 1024            185.9 / 256.1    1 of 64, 1000 keys (marked)     22.5 / 19.6
    if (a.N > (a.lengths ? 2 : 1) * a.tile_tokens) return launch_wide<T, D>(a, grid, stream);
    return launch_typed<T, D, true>(a, grid, stream);
}

}  // namespace

size_t tree_attention_workspace_bytes(int B, int N, int Hq, int D) {
    if (B < 1 || N < 1 || Hq < 1 || D < 1) return 0;
    return partials_end(wide_cap_of(N, Hq), D) + static_cast<size_t>(B) * N * (words_of(N) + 1) * sizeof(uint32_t);
}

size_t window_attention_workspace_bytes(int B, int N, int Hq, int D) {
    if (B < 1 || N < 1 || Hq < 1 || D < 1) return 0;
    return partials_end(wide_cap_of(N, Hq), D);
}

dspark_status launch_masked_attention(const void* q, const void* k_cache, const void* v_cache, dspark_dtype dtype,
                                      const int32_t* block_table, int max_pages, const int32_t* kv_len,
                                      const int32_t* lengths, const int32_t* parents, int window, int sinks, float scale,
                                      int causal, int B, int N, int Hq, int Hkv, int D, int num_pages, int page, void* out,
                                      float* lse, void* ws, cudaStream_t stream, const DeviceInfo& dev) {
    if (static_cast<long long>(num_pages) * Hkv >= (1ll << 31) || static_cast<long long>(B) * N >= (1ll << 31)) {
        set_error("%s_attention: num_pages * Hkv and B * N must be below 2^31", parents ? "tree" : "window");
        return DSPARK_ERR_UNSUPPORTED;
    }
    PagedArgs a = paged_args(q, k_cache, v_cache, block_table, max_pages, kv_len, lengths, scale, causal, B, N, Hq, Hkv, D,
                             num_pages, page, out, lse, ws);
    a.rows_cap = wide_cap_of(N, Hq);
    set_partials(a);
    a.parents = parents;
    a.words = words_of(N);
    a.ancestors = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + partials_end(a.rows_cap, D));
    a.window = std::min(window, 1 << 30);                  // as wide as a table can be: positions stay within 32 bits
    a.sinks = sinks;
    const int grid = std::min(dev.sm_count, kMaxCtas);
    if (dtype == DSPARK_BF16) return D == 64 ? launch<__nv_bfloat16, 64>(a, grid, stream) : launch<__nv_bfloat16, 128>(a, grid, stream);
    return D == 64 ? launch<__half, 64>(a, grid, stream) : launch<__half, 128>(a, grid, stream);
}

}  // namespace dspark
