// ea_tree.cu - a tree of drafted tokens: its ancestor masks before the target model
// runs over it, and the walk that accepts a path after.
//
// Both are a launch and a few dependent steps on chip, one CTA a sequence; latency is all
// there is (64 trees of 128 nodes: 2.0 us and 3.0 us).
//   tree_plan_kernel    pointer doubling: after round k a node holds its ancestors up
//                       to 2^k - 1 steps away and a pointer to the one 2^k away, so
//                       a chain of 128 takes seven rounds
//   tree_accept_kernel  one warp, four nodes a lane: each step votes on which node is
//                       the first child that holds the model's token
#include <cuda_runtime.h>

#include "ea_device.cuh"
#include "ea_internal.h"

namespace ea {

static_assert(EA_MAX_TREE == 128, "a node's ancestors are four words");

// The nodes of a sequence; a count outside [0, T] is reported and counts as none.
__device__ __forceinline__ int tree_nodes(const int32_t *n_nodes, int b, int T, uint32_t *err)
{
    const int n = n_nodes ? n_nodes[b] : T;
    if (n >= 0 && n <= T)
        return n;
    if (threadIdx.x == 0)
        raise_error(err, EA_DEVERR_CHECK);
    return 0;
}

__global__ void __launch_bounds__(EA_MAX_TREE) tree_plan_kernel(const int32_t *parents, const int32_t *n_nodes,
                                                                int T, int32_t *depth, uint4 *mask, uint32_t *err)
{
    __shared__ uint4 up[EA_MAX_TREE];
    __shared__ int to[EA_MAX_TREE];
    const int b = blockIdx.x, t = threadIdx.x;
    const int n = tree_nodes(n_nodes, b, T, err);
    int p = t < n ? parents[static_cast<int64_t>(b) * T + t] : -1;
    if (p < -1 || p >= t) {
        if (t < n)
            raise_error(err, EA_DEVERR_CHECK);
        p = -1;
    }
    uint4 a = make_uint4(0u, 0u, 0u, 0u);
    const uint32_t bit = t < n ? 1u << (t & 31) : 0u;
    if (t < 32)
        a.x = bit;
    else if (t < 64)
        a.y = bit;
    else if (t < 96)
        a.z = bit;
    else
        a.w = bit;
    while (__syncthreads_or(p >= 0)) {
        up[t] = a;
        to[t] = p;
        __syncthreads();
        if (p >= 0) {
            const uint4 v = up[p];
            a = make_uint4(a.x | v.x, a.y | v.y, a.z | v.z, a.w | v.w);
            p = to[p];
        }
    }
    if (t < T) {
        const int64_t at = static_cast<int64_t>(b) * T + t;
        mask[at] = a;
        depth[at] = t < n ? __popc(a.x) + __popc(a.y) + __popc(a.z) + __popc(a.w) - 1 : 0;
    }
}

struct AcceptArgs {
    const int32_t *tokens, *parents, *targets, *n_nodes;
    int32_t *path, *n_accepted, *next_token;
    uint32_t *err;
    int T;
};

__global__ void __launch_bounds__(32) tree_accept_kernel(const AcceptArgs a)
{
    __shared__ int target[EA_MAX_TREE];
    const int b = blockIdx.x, lane = threadIdx.x;
    const int n = tree_nodes(a.n_nodes, b, a.T, a.err);
    const int64_t base = static_cast<int64_t>(b) * a.T;
    int parent[4], token[4];
    bool bad = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int t = 32 * k + lane;
        parent[k] = -1;
        token[k] = 0;
        if (t < n) {
            parent[k] = a.parents[base + t];
            token[k] = a.tokens[base + t];
            target[t] = a.targets[base + t];
            if (parent[k] < -1 || parent[k] >= t) {
                bad = true;
                parent[k] = -1;
            }
        }
    }
    if (bad)
        raise_error(a.err, EA_DEVERR_CHECK);
    __syncwarp();
    // node 0 is the last sampled token; a child comes after its parent, so the walk ends
    int count = 0, mine[4] = {-1, -1, -1, -1}, next = -1;
    for (int at = n > 0 ? 0 : -1; at >= 0;) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (count == 32 * k + lane)
                mine[k] = at;
        ++count;
        next = target[at];
        int first = -1;
#pragma unroll
        for (int k = 3; k >= 0; --k) {
            const uint32_t hit = __ballot_sync(0xffffffffu, parent[k] == at && token[k] == next);
            if (hit)
                first = 32 * k + __ffs(hit) - 1;
        }
        at = first;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (32 * k + lane < a.T)
            a.path[base + 32 * k + lane] = mine[k];
    if (lane == 0) {
        a.n_accepted[b] = count;
        a.next_token[b] = next;
    }
}

static bool tree_ws_ok(const void *ws, size_t bytes)
{
    return ws && !(reinterpret_cast<uintptr_t>(ws) & 255u) && bytes >= sizeof(ea_ws_header);
}

} // namespace ea

using namespace ea;

extern "C" ea_status ea_tree_plan(const int32_t *parents, const int32_t *n_nodes, int B, int T, int32_t *depth,
                                  int32_t *mask, void *workspace, size_t ws_bytes, void *stream)
{
    if (!parents || !depth || !mask || B < 1 || T < 1 || (reinterpret_cast<uintptr_t>(mask) & 15u))
        return EA_ERR_INVALID_ARG;
    if (T > EA_MAX_TREE)
        return EA_ERR_UNSUPPORTED;
    if (!tree_ws_ok(workspace, ws_bytes))
        return EA_ERR_WORKSPACE;
    tree_plan_kernel<<<B, EA_MAX_TREE, 0, static_cast<cudaStream_t>(stream)>>>(
        parents, n_nodes, T, depth, reinterpret_cast<uint4 *>(mask), &static_cast<ea_ws_header *>(workspace)->error);
    return cudaGetLastError() == cudaSuccess ? EA_OK : EA_ERR_CUDA;
}

extern "C" ea_status ea_tree_accept(const int32_t *tokens, const int32_t *parents, const int32_t *targets,
                                    const int32_t *n_nodes, int B, int T, int32_t *path, int32_t *n_accepted,
                                    int32_t *next_token, void *workspace, size_t ws_bytes, void *stream)
{
    if (!tokens || !parents || !targets || !path || !n_accepted || !next_token || B < 1 || T < 1)
        return EA_ERR_INVALID_ARG;
    if (T > EA_MAX_TREE)
        return EA_ERR_UNSUPPORTED;
    if (!tree_ws_ok(workspace, ws_bytes))
        return EA_ERR_WORKSPACE;
    AcceptArgs a{tokens, parents, targets, n_nodes, path, n_accepted, next_token,
                 &static_cast<ea_ws_header *>(workspace)->error, T};
    tree_accept_kernel<<<B, 32, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? EA_OK : EA_ERR_CUDA;
}
