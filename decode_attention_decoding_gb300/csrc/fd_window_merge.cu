// Joins the window kernel's partials: with the reference exponents m_s, the sums
// of weights l_s and of weighted V rows x_s of the CTAs s that had some of a
// segment,
//     O = v_scale sum_s 2^(m_s - M) x_s / sum_s 2^(m_s - M) l_s,   M = max_s m_s,
// and zeros (LSE -inf) for requests that see nothing.  Segments that one CTA
// had whole are written already.
#include "fd_window.cuh"

namespace fd {

constexpr int kWindowMergeThreads = 128;
constexpr int kWindowMergeTogether = 4;   // partials whose loads a thread has in flight

// grid: (kv head, request, column).  A thread owns 4 dims and every S-th partial.
template <int D>
__global__ void __launch_bounds__(kWindowMergeThreads) window_merge_kernel(const __grid_constant__ WindowParams p, int ctas, int warps,
                                                                           float shift)
{
    constexpr int kLanes = D / 4, S = kWindowMergeThreads / kLanes;
    constexpr float kNegInf = -__builtin_huge_valf(), kLeast = 1.1754944e-38f;
    __shared__ float4 s_x[S][kLanes];
    __shared__ float2 s_ml[S];
    const int head = blockIdx.x, b = blockIdx.y, col = blockIdx.z;
    const int d = threadIdx.x % kLanes, s = threadIdx.x / kLanes;
    pdl_launch_dependents();
    pdl_wait_prior_grid();
    const int heads = p.hkv / p.team, h = head / p.team, lead = head - h * p.team;
    const int *prefix = p.ws_prefix, *nonempty = prefix + p.batch + 1;
    const int nb = (prefix[b + 1] - prefix[b]) / heads;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    float top = kNegInf, sum = 0.f;
    if (nb > 0) {
        Schedule sch = {prefix, nonempty, p.batch, heads, kWindowSegCost, 0};
        const long long cost = sch.cost();
        const int teams = window_workers(cost, ctas, warps / p.team);
        sch.P = ctas * teams;
        const long long pos = sch.seg_pos(b, h), end = pos + nb;
        const int w0 = sch.cta_at(pos), w1 = sch.cta_at(end - 1);
        // the last worker went on to another segment: it left this one's end apart
        const bool apart = end + kWindowSegCost < cost && sch.cta_at(end + kWindowSegCost) == w1;
        const int wl = apart ? w1 - 1 : w1, c0 = w0 / teams, c1 = wl / teams;
        if (w0 == w1 || (!apart && c0 == c1))
            return;
        const int n = c1 - c0 + 1 + (apart ? 1 : 0);
        for (int k = s; k < n; k += S * kWindowMergeTogether) {
            float2 ml[kWindowMergeTogether];
            float4 y[kWindowMergeTogether];
            float higher = top;
#pragma unroll
            for (int e = 0; e < kWindowMergeTogether; ++e) {
                const int kk = k + e * S;
                ml[e] = make_float2(kNegInf, 0.f);
                if (kk < n) {
                    const int cta = c0 + kk;
                    const long long slot = cta > c1 ? (long long)(2 * w1) * p.team + lead
                                                    : (long long)(2 * max(w0, cta * teams) + 1) * p.team + lead;
                    ml[e] = p.ws_ml[slot * p.cols + col];
                    y[e] = *reinterpret_cast<const float4 *>(p.ws_o + (slot * p.cols + col) * D + 4 * d);
                }
                higher = fmaxf(higher, ml[e].x);
            }
            const float ref = higher == kNegInf ? 0.f : higher, down = fmaxf(exp2_approx(top - ref), kLeast);
            sum *= down;
            x = make_float4(x.x * down, x.y * down, x.z * down, x.w * down);
            top = higher;
#pragma unroll
            for (int e = 0; e < kWindowMergeTogether; ++e) {
                if (k + e * S >= n)
                    continue;
                const float f = fmaxf(exp2_approx(ml[e].x - ref), kLeast);
                sum = fmaf(f, ml[e].y, sum);
                x.x = fmaf(f, y[e].x, x.x);
                x.y = fmaf(f, y[e].y, x.y);
                x.z = fmaf(f, y[e].z, x.z);
                x.w = fmaf(f, y[e].w, x.w);
            }
        }
        s_x[s][d] = x;
        if (d == 0)
            s_ml[s] = make_float2(top, sum);
        __syncthreads();
        if (s > 0)
            return;
#pragma unroll
        for (int e = 1; e < S; ++e)
            top = fmaxf(top, s_ml[e].x);
        const float ref = top == kNegInf ? 0.f : top;
        sum = 0.f;
        x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int e = 0; e < S; ++e) {
            const float f = fmaxf(exp2_approx(s_ml[e].x - ref), kLeast);
            const float4 y = s_x[e][d];
            sum = fmaf(f, s_ml[e].y, sum);
            x.x = fmaf(f, y.x, x.x);
            x.y = fmaf(f, y.y, x.y);
            x.z = fmaf(f, y.z, x.z);
            x.w = fmaf(f, y.w, x.w);
        }
    } else if (s > 0)
        return;
    const int i = col / p.group;
    const long long row = (long long)(b * p.q_len + i) * p.hq + head * p.group + (col - i * p.group);
    const float f = sum == 0.f ? 0.f : p.v_scale / sum;
    *reinterpret_cast<float4 *>(p.o + row * D + 4 * d) = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
    if (d == 0 && p.lse)
        p.lse[row] = sum == 0.f ? kNegInf : ((top == kNegInf ? 0.f : top) - shift + log2f(sum)) * 0.6931471805599453f;
}

template <int D>
static cudaError_t launch_merge_d(const WindowParams &p, int ctas, int warps, float shift, cudaStream_t stream)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.hkv, (unsigned)p.batch, (unsigned)p.cols);
    cfg.blockDim = dim3(kWindowMergeThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, window_merge_kernel<D>, p, ctas, warps, shift);
}

cudaError_t launch_window_merge(int head_dim, const WindowParams &p, int grid_ctas, int warps, float shift, cudaStream_t stream)
{
    return head_dim == 64 ? launch_merge_d<64>(p, grid_ctas, warps, shift, stream)
           : head_dim == 128 ? launch_merge_d<128>(p, grid_ctas, warps, shift, stream) : launch_merge_d<256>(p, grid_ctas, warps, shift, stream);
}

}  // namespace fd
