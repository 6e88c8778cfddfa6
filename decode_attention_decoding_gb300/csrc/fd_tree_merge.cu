// Joins the tree kernel's partials: a row's output is
//     sum_c 2^(lse_c - M) O_c / sum_c 2^(lse_c - M),   M = max_c lse_c,
// over the CTAs c that had some of its segment, and zeros (lse -inf) for the
// rows of segments that have no tiles.  Segments that one CTA had whole are
// written already.
#include "fd_tree.cuh"

namespace fd {

constexpr int kMergeRows = 32;      // query rows of a CTA, a lane each
constexpr int kMergeScanBatch = 32; // requests whose positions every warp finds itself

// 4-dim columns of a warp, and partials whose loads are in flight together:
// 16 loads of 16 bytes a thread.
__host__ __device__ constexpr int merge_cols(int d) { return d == 256 ? 4 : 2; }
__host__ __device__ constexpr int merge_warps(int d) { return d / 4 / merge_cols(d); }

// grid: (kv head x row group x 32 rows, request).  Partials are laid out
// [D / 4][row][4], so that a warp (32 rows of one 4-dim column) reads 512
// consecutive bytes; the rows are turned round in shared memory for the write.
//
// A short call waits for this kernel's chain of loads, so it is kept short:
// with up to 32 requests the segment's place comes from the lengths, which are
// read before the split kernel ends (it has waited for the kernels that may
// have written them), and one round trip brings the statistics and the sums
// of several partials.
template <int D>
__global__ void __launch_bounds__(32 * merge_warps(D)) tree_merge_kernel(const __grid_constant__ TreeParams p, int ctas)
{
    constexpr int kPad = D + 4, kCols = merge_cols(D), kWarps = merge_warps(D), kTogether = 16 / kCols;
    __shared__ __align__(16) float s_o[kMergeRows * kPad];
    __shared__ float s_lse[kMergeRows];
    constexpr float kNegInf = -__builtin_huge_valf();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int all_groups = (p.tree_len * p.group + p.rows - 1) / p.rows, blocks = (p.slot_rows + kMergeRows - 1) / kMergeRows;
    const int b = blockIdx.y, rb = blockIdx.x % blocks, gm = blockIdx.x / blocks;
    const int g = gm / all_groups, mg = gm - g * all_groups;
    const int first = mg * p.rows + rb * kMergeRows;            // the block's first query row of the kv head
    const int rows = min(kMergeRows, min(p.rows - rb * kMergeRows, p.tree_len * p.group - first));
    pdl_launch_dependents();
    if (rows <= 0)
        return;
    const TreeSeg s = tree_seg<D>(p, tree_req(p, b, nullptr));
    long long cost_b = 0, cost = 0;
    if (p.batch <= kMergeScanBatch) {
        const long long mine = lane < p.batch ? tree_cost(tree_seg<D>(p, tree_req(p, lane, nullptr))) : 0;
        long long x = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off)
                x += y;
        }
        cost = __shfl_sync(0xffffffffu, x, 31);
        cost_b = __shfl_sync(0xffffffffu, x - mine, b);
    }
    pdl_wait_prior_grid();
    float4 acc[kCols];
#pragma unroll
    for (int k = 0; k < kCols; ++k)
        acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    float lse = kNegInf;
    if (mg < s.groups) {
        if (p.batch > kMergeScanBatch) {
            cost = p.ws_cost[p.batch];
            cost_b = p.ws_cost[b];
        }
        const TreeSplit split = tree_split(cost, ctas);
        const long long pos = cost_b + (long long)(g * s.groups + mg) * (s.nb + kTreeSegCost) + kTreeSegCost;
        const int c0 = split.cta_at(pos), c1 = split.cta_at(pos + s.nb - 1);
        if (c0 == c1)
            return;
        if (lane < rows) {
            const int srow = rb * kMergeRows + lane;
            float top = kNegInf, sum = 0.f;
            for (int c = c0; c <= c1; c += kTogether) {
                float x[kTogether];
                float4 o[kTogether][kCols];
#pragma unroll
                for (int n = 0; n < kTogether; ++n) {
                    // the first CTA of a segment left it, the others found it begun
                    const int slot = 2 * (c + n) + (c + n == c0 ? 1 : 0);
                    x[n] = kNegInf;
                    if (c + n <= c1) {
                        x[n] = p.ws_lse[slot * p.slot_rows + srow];
                        const float *src = p.ws_o + ((long long)slot * (D / 4) + warp * kCols) * p.slot_rows * 4 + srow * 4;
#pragma unroll
                        for (int k = 0; k < kCols; ++k)
                            o[n][k] = *reinterpret_cast<const float4 *>(src + (long long)k * p.slot_rows * 4);
                    }
                }
                float higher = top;
#pragma unroll
                for (int n = 0; n < kTogether; ++n)
                    higher = fmaxf(higher, x[n]);
                // at least fp32's least normal number: an infinite sum stays infinite however small
                // its weight is, and 10^-38 of a finite one does not matter
                auto weight = [](float y) { return y < -126.f ? 1.1754944e-38f : exp2_approx(y); };   // NaN: NaN
                const float ref = higher == kNegInf ? 0.f : higher, down = weight(top - ref);
                sum *= down;
#pragma unroll
                for (int k = 0; k < kCols; ++k)
                    acc[k] = make_float4(acc[k].x * down, acc[k].y * down, acc[k].z * down, acc[k].w * down);
                top = higher;
#pragma unroll
                for (int n = 0; n < kTogether; ++n) {
                    if (x[n] == kNegInf)
                        continue;   // no partial, or one that saw nothing and wrote nothing
                    const float w = weight(x[n] - ref);
                    sum += w;
#pragma unroll
                    for (int k = 0; k < kCols; ++k) {
                        acc[k].x = fmaf(w, o[n][k].x, acc[k].x);
                        acc[k].y = fmaf(w, o[n][k].y, acc[k].y);
                        acc[k].z = fmaf(w, o[n][k].z, acc[k].z);
                        acc[k].w = fmaf(w, o[n][k].w, acc[k].w);
                    }
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
                lse = ((top == kNegInf ? 0.f : top) + log2f(sum)) * 0.6931471805599453f;
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kCols; ++k)
        *reinterpret_cast<float4 *>(s_o + lane * kPad + (warp * kCols + k) * 4) = acc[k];
    if (warp == 0)
        s_lse[lane] = lse;
    __syncthreads();
    for (int e = threadIdx.x; e < rows * (D / 4); e += 32 * kWarps) {
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
    cfg.blockDim = dim3(32 * merge_warps(D));
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
