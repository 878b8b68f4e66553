// A drafted tree of one request as the verification kernels see it, and the status word's clearing beside the
// launch that follows.
#pragma once

#include "attention_common.cuh"
#include "device_common.cuh"
#include "host_common.h"

namespace dspark {

struct TreeArgs {
    const int32_t *parents, *draft_tokens, *lengths;
    int B, N, V;                           // V: entries of a row (0: there are none)
    int last;                              // the largest token
    int32_t *out_tokens, *num_accepted, *path;
    WsHeader* ws;
};

// Nodes of request b's tree (-1: out of range).
__device__ __forceinline__ int tree_nodes(const TreeArgs& a, int b) {
    const int n = a.lengths ? a.lengths[b] : a.N;
    return n < 0 || n > a.N ? -1 : n;
}

// Parent and token of node i < n as the walk takes them: what is out of range is flagged and makes the node one
// that is never reached.
__device__ __forceinline__ void tree_node(const TreeArgs& a, int b, int i, int& parent, int& token, bool& bad) {
    const long long at = static_cast<long long>(b) * a.N + i;
    parent = a.parents[at];
    token = a.draft_tokens[at];
    if (parent < -1 || parent >= i) {
        bad = true;
        parent = -1;
    }
    if (i > 0 && (token < 0 || token > a.last)) {
        bad = true;
        parent = -1;
    }
}

static __global__ void __launch_bounds__(64) clear_header_kernel(WsHeader* ws) {
    grid_dependency_launch();
    reinterpret_cast<uint32_t*>(ws)[threadIdx.x] = 0u;
}

// Clears the status word; a kernel that is launched as its dependent waits (grid_dependency_wait) before it sets bits.
inline dspark_status clear_header(void* ws, cudaStream_t stream) {
    clear_header_kernel<<<1, sizeof(WsHeader) / 4, 0, stream>>>(static_cast<WsHeader*>(ws));
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? DSPARK_OK : cuda_error(e, "launch(clear status)");
}

}  // namespace dspark
