// fd_tree.cuh -- attention of a tree of drafted tokens over a KV cache (sm_103a):
// parameters, and how the work is divided among CTAs.
//
// Request b's cache holds L positions, the last t of them the tree's nodes.
// The query rows of kv head g are r = i * G + h (node i, query head g * G + h).
// Row r sees position p when p < L - t, or when node i's mask row has the bit
// of node p - (L - t).
//
// A call with n query rows a kv head multiplies every K and V row by n rows:
// 4 n D operations on 4 D bytes (16-bit cache), n operations a byte.  GB300
// reads 6.8 TB/s and multiplies 1.87 PFLOP/s, 275 operations a byte: up to
// some 180 rows (the weights are taken in two parts, 1.5 times the products)
// the call is bound by reading the cache once, above by the tensor cores.
// Hence tcgen05 MMAs with the query rows as the 128 rows of the MMA (fewer
// rows waste tensor-core time that such a call has to spare), K and V through
// shared memory once per 128 or 256 rows, and the cache split among all SMs
// whatever the number of requests.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "fd_device.cuh"
#include "fd_sched.h"

namespace fd {

constexpr int kMaxTree = 256;        // nodes of a tree
constexpr int kMaxTreeRows = 4096;   // nodes x query heads of a kv head
constexpr int kTreeMaxCtas = 256;    // split CTAs (sizes the workspace)

// Cost of a segment start in tiles of the split (below).  Measured on GB300
// with 3, 4, 5, 7: 16 ragged GQA-4 requests of up to 8192 tokens 72, 69, 73, 75
// us, 64 of up to 16384 371, 370, 368, 371, one of 2048 tokens 17.4, 17.4, 18.2,
// 18.2.
constexpr int kTreeSegCost = 4;

// A scale of 0 becomes this one, so that a hidden score (-inf) keeps its
// weight of 0; scores below 1e30 are still 0.
constexpr float kTreeLeastScale = 1e-37f;

// Units of 128 positions that a tensor-core accumulator sums before it is
// flushed (fd_tree_kernel.cuh).
constexpr int kTreeFlush = 16;

// Positions of a tile: K and V tiles of at most 32 KB each.
__host__ __device__ constexpr int tree_tile(int d) { return d == 256 ? 64 : 128; }
// Groups of 128 softmax threads, each with an accumulator of D tensor-memory columns.
__host__ __device__ constexpr int tree_groups(int d) { return d == 256 ? 1 : 2; }

struct TreeParams {
    const uint16_t *q;
    const uint8_t *k, *v;          // the cache: read by loader threads, and for values that are not finite
    const uint64_t *mask;          // null: causal among the nodes
    long long mask_stride;
    const int32_t *tree_lens, *seq_lens, *block_table;
    float *o, *lse;
    float *ws_o, *ws_lse;          // partials: [2 ctas][D / 4][slot_rows][4], [2 ctas][slot_rows]
    float *ws_sums;                // flushed accumulators: [ctas][groups][D / 4][sum_rows][4]
    long long *ws_cost;            // [batch + 1]: cost position of each request, then the total
    unsigned int *ws_err;
    unsigned long long timeout_ns;
    int batch, tree_len, words, hq, hkv, group, cap;
    int page_size, max_blocks, num_pages;   // contiguous: block_table null, page_size = s_max
    int rows;                      // query rows of a segment: 128, or 256 (two row tiles)
    int slot_rows;                 // rows of a partial: min(rows, tree_len * group)
    int sum_rows;                  // rows of a group's flushed accumulator: min(128, tree_len * group)
    int box_rows;                  // positions of one TMA box
    int k_slots, v_slots;          // K and V tiles in shared memory
    int raw_slots;                 // tiles of FP8 codes, of K and of V each
    uint32_t off_k, off_v, off_raw, off_misc;
    float scale_log2, v_scale;     // scale_log2 > 0 (a negative scale's sign goes to q)
    int q_f16, negate_q, starve;
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

// The work.  Request b has segs = hkv * ceil(t G / rows) segments (kv head g,
// row group m: segment g * groups + m) of nb = ceil(L / tile) tiles each, none
// if L or t is 0.  As in fd_sched.h a segment start costs kTreeSegCost tiles
// (loading q, the epilogue): segment s of b lies at the positions
//     cost(b) + s (nb + W) + W + j,  j < nb,
// and with C positions in all, CTA c of P' = min(P, C) owns the tiles at
// positions [ceil(c C / P'), ceil((c + 1) C / P')).  The CTAs of a segment are
// consecutive and each owns some of its tiles.  A CTA that owns a whole
// segment writes its output; the others write a partial.  A CTA has at most
// two of those, the segment that it finds begun (slot 2 c) and the one that it
// leaves unfinished (slot 2 c + 1, or 2 c if it found it begun).
struct TreeSeg {
    int nb, groups, segs;
};
template <int D>
__device__ __forceinline__ TreeSeg tree_seg(const TreeParams &p, TreeReq r)
{
    TreeSeg s = {0, 0, 0};
    if (r.L > 0 && r.t > 0) {
        s.nb = (r.L - 1) / tree_tile(D) + 1;   // L may be close to 2^31
        s.groups = (r.t * p.group + p.rows - 1) / p.rows;
        s.segs = p.hkv * s.groups;
    }
    return s;
}
__device__ __forceinline__ long long tree_cost(TreeSeg s) { return (long long)s.segs * (s.nb + kTreeSegCost); }

struct TreeSplit {
    long long cost;   // C
    int ctas;         // P'
    // x / y for 0 <= x; a 64-bit division costs some 100 instructions
    __device__ __forceinline__ static long long quotient(long long x, long long y)
    {
        return x >> 32 == 0 && y >> 32 == 0 ? (long long)((uint32_t)x / (uint32_t)y) : x / y;
    }
    __device__ __forceinline__ int cta_at(long long pos) const { return (int)quotient(pos * ctas, cost); }
    __device__ __forceinline__ long long begin(int c) const { return quotient(cost * c + ctas - 1, ctas); }
};
__device__ __forceinline__ TreeSplit tree_split(long long cost, int grid)
{
    return {cost, cost < grid ? (int)cost : grid};
}

// Host side.
struct TreeLaunch {
    int grid;
    size_t smem_bytes, smem_optin;
    cudaStream_t stream;
};
// How the cache reaches shared memory: 16-bit tiles by TMA; FP8 codes by TMA,
// converted by four warps; or copied by four warps (pages under 8 tokens: a TMA
// box's rows would not reach the swizzle's 1 KB).
enum : int { kTreeTma = 0, kTreeConvert = 1, kTreeCopy = 2 };

// F16: the MMAs' type, fp16 or bf16: the query's, and fp16 for FP8 caches.
template <int D, bool F16, int KV, int LOAD>
cudaError_t launch_tree_variant(const TreeParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv,
                                const TreeLaunch &c);

#define FD_TREE_VARIANTS_D(X, D)                                                              \
    X(D, false, kKvBf16, kTreeTma) X(D, true, kKvF16, kTreeTma)                               \
    X(D, true, kKvE4m3, kTreeConvert) X(D, true, kKvE5m2, kTreeConvert)                       \
    X(D, false, kKvBf16, kTreeCopy) X(D, true, kKvF16, kTreeCopy)                             \
    X(D, true, kKvE4m3, kTreeCopy) X(D, true, kKvE5m2, kTreeCopy)
#define FD_TREE_VARIANTS(X) FD_TREE_VARIANTS_D(X, 64) FD_TREE_VARIANTS_D(X, 128) FD_TREE_VARIANTS_D(X, 256)
#define FD_EXTERN_TREE(D, F16, KV, LOAD)                                                                          \
    extern template cudaError_t launch_tree_variant<D, F16, KV, LOAD>(const TreeParams &, const CUtensorMap &,    \
                                                                       const CUtensorMap &, const TreeLaunch &);
FD_TREE_VARIANTS(FD_EXTERN_TREE)
#undef FD_EXTERN_TREE

cudaError_t launch_tree_merge(int head_dim, const TreeParams &p, int grid_ctas, cudaStream_t stream);

}  // namespace fd
