// Joins the tree kernel's partials: a row's output is
//     sum_c 2^(lse_c - M) O_c / sum_c 2^(lse_c - M),   M = max_c lse_c,
// over the CTAs c that had some of its segment, and zeros (lse -inf) for the
// rows of segments that have no tiles.  Segments that one CTA had whole are
// written already.
#include "fd_tree.cuh"

namespace fd {

constexpr int kMergeRows = 32;      // query rows of a CTA, a lane each
constexpr int kMergeWarps = 8;

// grid: (kv head x row group x 32 rows, request).  Partials are laid out
// [D / 4][row][4], so that a warp (32 rows of one 4-dim column) reads 512
// consecutive bytes; the rows are turned round in shared memory for the write.
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) tree_merge_kernel(const __grid_constant__ TreeParams p, int ctas)
{
    constexpr int kPad = D + 4;
    __shared__ __align__(16) float s_o[kMergeRows * kPad];
    __shared__ float s_lse[kMergeRows];
    constexpr int kCols = D / 4 / kMergeWarps;   // 4-dim columns of a warp
    constexpr float kNegInf = -__builtin_huge_valf();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int all_groups = (p.tree_len * p.group + p.rows - 1) / p.rows, blocks = (p.slot_rows + kMergeRows - 1) / kMergeRows;
    const int b = blockIdx.y, rb = blockIdx.x % blocks, gm = blockIdx.x / blocks;
    const int g = gm / all_groups, mg = gm - g * all_groups;
    const int first = mg * p.rows + rb * kMergeRows;            // the block's first query row of the kv head
    const int rows = min(kMergeRows, min(p.rows - rb * kMergeRows, p.tree_len * p.group - first));
    pdl_launch_dependents();
    pdl_wait_prior_grid();
    if (rows <= 0)
        return;
    const TreeSeg s = tree_seg<D>(p, tree_req(p, b, nullptr));
    float4 acc[kCols];
#pragma unroll
    for (int k = 0; k < kCols; ++k)
        acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    float lse = kNegInf;
    if (mg < s.groups) {
        const TreeSplit split = tree_split(p.ws_cost[p.batch], ctas);
        const long long pos = p.ws_cost[b] + (long long)(g * s.groups + mg) * (s.nb + kTreeSegCost) + kTreeSegCost;
        const int c0 = split.cta_at(pos), c1 = split.cta_at(pos + s.nb - 1);
        if (c0 == c1)
            return;
        if (lane < rows) {
            const int srow = rb * kMergeRows + lane;
            auto slot = [&](int c) { return 2 * c + (c == c0 ? 1 : 0); };
            float top = kNegInf;
            for (int c = c0; c <= c1; ++c)
                top = fmaxf(top, p.ws_lse[slot(c) * p.slot_rows + srow]);
            const float ref = top == kNegInf ? 0.f : top;
            float sum = 0.f;
            for (int c = c0; c <= c1; ++c) {
                const float x = p.ws_lse[slot(c) * p.slot_rows + srow];
                if (x == kNegInf)
                    continue;   // saw nothing, and wrote nothing
                const float w = exp2_approx(x - ref);
                sum += w;
                const float *src = p.ws_o + ((long long)slot(c) * (D / 4) + warp * kCols) * p.slot_rows * 4 + srow * 4;
#pragma unroll
                for (int k = 0; k < kCols; ++k) {
                    const float4 o = *reinterpret_cast<const float4 *>(src + (long long)k * p.slot_rows * 4);
                    acc[k].x = fmaf(w, o.x, acc[k].x);
                    acc[k].y = fmaf(w, o.y, acc[k].y);
                    acc[k].z = fmaf(w, o.z, acc[k].z);
                    acc[k].w = fmaf(w, o.w, acc[k].w);
                }
            }
            if (sum != 0.f) {   // true for NaN
                const float inv = 1.f / sum;
#pragma unroll
                for (int k = 0; k < kCols; ++k) {
                    acc[k].x *= inv;
                    acc[k].y *= inv;
                    acc[k].z *= inv;
                    acc[k].w *= inv;
                }
                lse = (ref + log2f(sum)) * 0.6931471805599453f;
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kCols; ++k)
        *reinterpret_cast<float4 *>(s_o + lane * kPad + (warp * kCols + k) * 4) = acc[k];
    if (warp == 0)
        s_lse[lane] = lse;
    __syncthreads();
    for (int e = threadIdx.x; e < rows * (D / 4); e += 32 * kMergeWarps) {
        const int r = e / (D / 4), c = e - r * (D / 4), i = (first + r) / p.group, h = first + r - i * p.group;
        const long long row = ((long long)b * p.tree_len + i) * p.hq + g * p.group + h;
        *reinterpret_cast<float4 *>(p.o + row * D + 4 * c) = *reinterpret_cast<const float4 *>(s_o + r * kPad + 4 * c);
        if (c == 0 && p.lse)
            p.lse[row] = s_lse[r];
    }
}

template <int D>
static cudaError_t launch_merge_d(const TreeParams &p, int ctas, cudaStream_t stream)
{
    const int groups = (p.tree_len * p.group + p.rows - 1) / p.rows, blocks = (p.slot_rows + kMergeRows - 1) / kMergeRows;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.hkv * groups * blocks), (unsigned)p.batch);
    cfg.blockDim = dim3(32 * kMergeWarps);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D>, p, ctas);
}

cudaError_t launch_tree_merge(int head_dim, const TreeParams &p, int grid_ctas, cudaStream_t stream)
{
    return head_dim == 64 ? launch_merge_d<64>(p, grid_ctas, stream)
           : head_dim == 128 ? launch_merge_d<128>(p, grid_ctas, stream) : launch_merge_d<256>(p, grid_ctas, stream);
}

}  // namespace fd
