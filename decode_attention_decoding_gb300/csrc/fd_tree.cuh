// fd_tree.cuh -- attention of a tree of drafted tokens over a KV cache (sm_103a).
//
// Request b's cache holds L positions, the last t of them the tree's nodes.
// The query rows of kv head g are r = i * G + h (node i, query head g * G + h).
// Row r sees position p when p < L - t, or when node i's mask row has the bit
// of node p - (L - t).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "fd_device.cuh"
#include "fd_sched.h"

namespace fd {

constexpr int kMaxTree = 256;        // nodes of a tree
constexpr int kMaxTreeRows = 4096;   // nodes x query heads of a kv head

struct TreeParams {
    const uint16_t *q;
    const uint8_t *k, *v;
    const uint64_t *mask;          // null: causal among the nodes
    long long mask_stride;
    const int32_t *tree_lens, *seq_lens, *block_table;
    float *o, *lse;
    unsigned int *ws_err;
    int batch, tree_len, words, hq, hkv, group, head_dim, cap;
    int page_size, max_blocks, num_pages;   // contiguous: block_table null, page_size = s_max
    float scale, v_scale;
    int q_f16;
};

// Request b's cache length and node count; a value out of range is clamped,
// and reported in *err when err is given.
struct TreeReq {
    int L, t;
};
__device__ __forceinline__ TreeReq tree_req(const TreeParams &p, int b, unsigned int *err)
{
    const int l = p.seq_lens ? p.seq_lens[b] : p.cap, n = p.tree_lens ? p.tree_lens[b] : p.tree_len;
    TreeReq r;
    r.L = min(max(l, 0), p.cap);
    r.t = min(max(n, 0), p.tree_len);
    if (err && (r.L != l || r.t != n))
        atomicOr(err, kErrLength);
    return r;
}

cudaError_t launch_tree_simple(int kv, const TreeParams &p, cudaStream_t stream);

}  // namespace fd
