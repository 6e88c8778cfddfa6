// The tree attention on CUDA cores, one warp per query row: a tile of 32
// positions is staged in shared memory as fp32, a lane forms the score of one
// position, the warp updates its running maximum and sum, and each lane
// accumulates head_dim / 32 of the output's dims.
#include "fd_tree.cuh"

namespace fd {

constexpr int kSimpleRows = 8, kSimpleKeys = 32;

template <int KV, int D>
__global__ void __launch_bounds__(kSimpleRows * 32) tree_simple_kernel(const __grid_constant__ TreeParams p)
{
    extern __shared__ float s_kv[];
    constexpr int kRow = D + 1;   // a lane reads one row: an odd stride hits every bank
    float *sk = s_kv, *sv = s_kv + kSimpleKeys * kRow, *sq = sv + kSimpleKeys * kRow;
    const int b = blockIdx.z, g = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool reports = blockIdx.x == 0 && g == 0 && threadIdx.x == 0;
    const TreeReq req = tree_req(p, b, reports ? p.ws_err : nullptr);
    const int r = blockIdx.x * kSimpleRows + warp, i = r / p.group, h = r - i * p.group;
    const int base = req.L - req.t;
    const bool live = i < req.t && base + i >= 0, in_call = i < p.tree_len;
    const long long row = ((long long)b * p.tree_len + i) * p.hq + g * p.group + h;
    if (in_call)
        for (int d = lane; d < D; d += 32) {
            const uint32_t w = p.q[row * D + d];
            sq[warp * D + d] = p.q_f16 ? f16x2_to_float2(w).x : __uint_as_float(w << 16);
        }
    float m = -INFINITY, l = 0.f, acc[D / 32] = {};
    for (int t0 = 0; t0 < req.L; t0 += kSimpleKeys) {
        __syncthreads();
        for (int e = threadIdx.x; e < kSimpleKeys * D; e += kSimpleRows * 32) {
            const int j = e / D, d = e - j * D, pos = t0 + j;
            float kx = 0.f, vx = 0.f;
            if (pos < req.L) {
                long long at = (long long)b * p.page_size + pos;
                if (p.block_table) {
                    int page = p.block_table[(long long)b * p.max_blocks + pos / p.page_size];
                    if ((unsigned)page >= (unsigned)p.num_pages) {
                        atomicOr(p.ws_err, kErrPage);
                        page = 0;
                    }
                    at = (long long)page * p.page_size + pos % p.page_size;
                }
                const long long el = (at * p.hkv + g) * D + d;
                if constexpr (kv_is_fp8(KV)) {
                    kx = fp8x2_to_float2<KV>(p.k[el]).x;
                    vx = fp8x2_to_float2<KV>(p.v[el]).x;
                } else {
                    kx = x2_to_float2<KV == kKvF16>(reinterpret_cast<const uint16_t *>(p.k)[el]).x;
                    vx = x2_to_float2<KV == kKvF16>(reinterpret_cast<const uint16_t *>(p.v)[el]).x;
                }
            }
            sk[j * kRow + d] = kx;
            sv[j * kRow + d] = vx;
        }
        __syncthreads();
        if (!live)
            continue;
        const int pos = t0 + lane, node = pos - base;
        bool sees = pos < req.L;
        if (sees && node >= 0)
            sees = p.mask ? (p.mask[b * p.mask_stride + (long long)i * p.words + (node >> 6)] >> (node & 63)) & 1 : node <= i;
        float s = 0.f;
        for (int d = 0; d < D; ++d)
            s = fmaf(sq[warp * D + d], sk[lane * kRow + d], s);
        s = sees ? s * p.scale : -INFINITY;
        float mt = s;
#pragma unroll
        for (int off = 16; off; off >>= 1)
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, off));
        const float mn = fmaxf(m, mt), mu = mn == -INFINITY ? 0.f : mn;
        const float w = sees ? expf(s - mu) : 0.f, c = expf(m - mu);
        float ws = w;
#pragma unroll
        for (int off = 16; off; off >>= 1)
            ws += __shfl_xor_sync(0xffffffffu, ws, off);
        l = l * c + ws;
        m = mn;
#pragma unroll
        for (int n = 0; n < D / 32; ++n)
            acc[n] *= c;
        const unsigned seen = __ballot_sync(0xffffffffu, sees);
        for (int j = 0; j < kSimpleKeys; ++j) {
            const float wj = __shfl_sync(0xffffffffu, w, j);
            if (seen >> j & 1)   // what a row does not see must not reach it, infinities included
#pragma unroll
                for (int n = 0; n < D / 32; ++n)
                    acc[n] = fmaf(wj, sv[j * kRow + lane + 32 * n], acc[n]);
        }
    }
    if (!in_call)
        return;
    const bool any = l != 0.f;   // also when l is not a number
#pragma unroll
    for (int n = 0; n < D / 32; ++n)
        p.o[row * D + lane + 32 * n] = any ? acc[n] / l * p.v_scale : 0.f;
    if (p.lse && lane == 0)
        p.lse[row] = any ? m + logf(l) : -INFINITY;
}

template <int KV, int D>
static cudaError_t launch_simple(const TreeParams &p, cudaStream_t stream)
{
    const size_t smem = sizeof(float) * (2 * kSimpleKeys * (D + 1) + kSimpleRows * D);
    cudaError_t e = cudaFuncSetAttribute(tree_simple_kernel<KV, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess)
        return e;
    const dim3 grid((unsigned)ceil_div(p.tree_len * p.group, kSimpleRows), (unsigned)p.hkv, (unsigned)p.batch);
    tree_simple_kernel<KV, D><<<grid, kSimpleRows * 32, smem, stream>>>(p);
    return cudaGetLastError();
}

template <int KV>
static cudaError_t launch_simple_kv(const TreeParams &p, cudaStream_t s)
{
    return p.head_dim == 64 ? launch_simple<KV, 64>(p, s)
           : p.head_dim == 128 ? launch_simple<KV, 128>(p, s) : launch_simple<KV, 256>(p, s);
}

cudaError_t launch_tree_simple(int kv, const TreeParams &p, cudaStream_t s)
{
    switch (kv) {
    case kKvBf16: return launch_simple_kv<kKvBf16>(p, s);
    case kKvF16: return launch_simple_kv<kKvF16>(p, s);
    case kKvE4m3: return launch_simple_kv<kKvE4m3>(p, s);
    default: return launch_simple_kv<kKvE5m2>(p, s);
    }
}

}  // namespace fd
