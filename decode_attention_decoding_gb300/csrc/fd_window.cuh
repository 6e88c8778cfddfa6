// fd_window.cuh -- decode attention through a sliding window with sinks, over
// 16-bit, FP8 and 4-bit caches (sm_103a): parameters, and how the work is
// divided among warps.
//
// The T = q_len new tokens of a request of length L sit at positions L - T + i.
// Position t is visible to the token at position p when t <= p and
// (t < sinks or t > p - window).  What some new token sees is
//     [0, head) and [first, L),
//     first = min(L, max(sinks, L - T - window + 1)), head = min(sinks, first),
// and that is all a call reads: "row" v < head + L - first is position v if
// v < head, else v - head + first.  Without a window first = head = 0.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "fd_device.cuh"
#include "fd_sched.h"

namespace fd {

constexpr int kKvE2m1 = 4;           // 4-bit cache (after fd_device.cuh's kKv*)
constexpr int kWindowMaxCtas = 160;  // split CTAs (sizes the workspace)
constexpr int kWindowMaxWarps = 16;  // warps of a split CTA
constexpr int kWindowMaxColumns = 16;

// Cost of a segment start, in tiles (fd_sched.h): a warp loads the query and
// flushes its outputs there.  Measured on GB300 with 0, 1, 2, 4 (us): 64
// requests of up to 16384 positions in 4 bits 129.7, 126.5, 127.0, 128.5, 8 of
// 16 columns 117.8, 116.7, 116.6, 115.7; others alike.
constexpr int kWindowSegCost = 1;

constexpr int kWindowAbout = 32;   // bytes that say what a tile is

// Shape of the split kernel for head dim D, a cache of type KV and MMAs of 8 NT
// query columns.
template <int D_, int KV_, int NT_>
struct WindowCfg {
    static constexpr int D = D_, KV = KV_, NT = NT_;
    static constexpr bool kFp4 = KV == kKvE2m1, kFp8 = KV == kKvE4m3 || KV == kKvE5m2;
    static constexpr bool kF16 = KV != kKvBf16;              // type of the MMAs
    static constexpr bool kInf = KV == kKvBf16 || KV == kKvF16 || KV == kKvE5m2;   // types with infinities
    static constexpr int kParts = kF16 ? 2 : 3;              // 16-bit parts of a softmax weight
    // The reference of a column's weights is its largest score so far, of weight 2^kShift: fp16 remainders of small weights
    // keep their bits.
    static constexpr float kShift = kF16 ? 14.f : 0.f;
    static constexpr int kRow = kFp4 ? D / 2 : kFp8 ? D : 2 * D;   // bytes of a row
    static constexpr int kGran = kRow / 16;                  // 16-byte pieces of a row
    static constexpr int kScaleRow = kFp4 ? D / 16 : 0;      // bytes of a row's block scales
    // Rows of a tile, and warps of a CTA (12 and 16 leave 168 and 128 registers a thread, fewer 255).  Every warp has two
    // tiles, one on its way: some 64 KB in flight on an SM, more of it was slower wherever memory is the bound (a window
    // of 4096 over 64 GQA-4 requests, 8 warps: 166 us with one tile ahead, 186 with two).  Measured over 400 MB in 8
    // requests of 8 heads (us, 1 / 8 / 16 columns), rows x warps: 4 bits, 64 dims: 32 x 12 114 / 117 / 161, 64 x 8
    // 107 / 114 / 149, 64 x 12 98 / 105 / 147, 64 x 16 92 / 101 / 162; 128 dims: 32 x 12 88 / 99 / 144, 64 x 8 85 / 93 /
    // 134; 256 dims: 16 x 8 99 / 114 / 163, 32 x 8 85 / 102 / 151 (no room with 16 columns); FP8, 64 dims: 32 x 12
    // 73 / 78 / 95, 64 x 8 71 / 75 / 96; 128 dims: 16 x 8 86 / 91 / 106, 32 x 8 67 / 74 / 93, 64 x 4 69 / 82 / 126; 256
    // dims: 16 x 8 67 / 78 / 101, 32 x 4 69 / 85 / 123; 16 bits, 64 dims: 16 x 8 86 / 87 / 93, 32 x 8 69 / 70 / 76, 64 x 4
    // 71 / 74 / 85; 128 dims: 16 x 8 68 / 71 / 77, 32 x 4 69 / 72 / 85.  The floor is 59.  The shapes taken, since weights
    // come from differences of scores: 4 bits 94 / 102 / 149, 86 / 92 / 132, 82 / 98 / 164, FP8 69 / 73 / 101, 68 / 72 / 93,
    // 67 / 72 / 100, 16 bits 67 / 68 / 75, 66 / 68 / 74, 66 / 77 / 104 (64, 128, 256 dims).
    static constexpr int kTile = kFp4   ? (D < 256 ? 64 : NT == 1 ? 32 : 16)
                                 : kFp8 ? (D == 64 ? (NT == 1 ? 64 : 32) : D == 128 ? 32 : 16)
                                        : (D == 64 ? 32 : 16);
    static constexpr int kWarps = kFp4 && D == 64 ? (NT == 1 ? 16 : 12) : kFp8 && D == 64 && NT == 2 ? 12 : !kFp4 && !kFp8 && D == 256 ? 4 : 8;
    static constexpr int kStage = 2 * kTile * (kRow + kScaleRow);
    // Two words a lane of each k step of the query: in registers where there are some left.
    static constexpr bool kQueryShared = NT == 2;
    static constexpr int kQuery = kQueryShared ? 16 * D * NT : 0;
    static constexpr int kSums = (int)sizeof(float) * NT * 8 * (D + 2);   // bytes of a warp's sums, left in its ring at the end
    static constexpr int kStages = 2;
    static constexpr int kRing = (kStage + kWindowAbout) * kStages + kQuery;   // bytes of a warp's tiles, of what each is, and of the query
};

struct WindowParams {
    const uint16_t *q;
    const uint8_t *k, *v, *ks, *vs;    // cache rows; block scales of a 4-bit cache
    const int32_t *block_table, *seq_lens;
    float *o, *lse;
    float *ws_o;                       // partials [slots][cols][D]: sums of weight * V ...
    float2 *ws_ml;                     // ... and [slots][cols]: their reference exponent and sum of weights
    unsigned int *ws_counts;           // of a segment that several CTAs have: partials written; by its first worker, 0 between calls
    unsigned int *ws_err;
    int batch, q_len, hq, hkv, group, cols, cap;
    int page_size, max_blocks, num_pages;   // contiguous: block_table null, page_size = s_max, num_pages = batch
    int page_shift;                    // page_size = 2^page_shift, or -1
    uint32_t row_page, row_token, row_head; // cache row = page * row_page + slot * row_token + head * row_head
    int window, sinks;                 // window 0: none
    int team;                          // adjacent kv heads that a team of as many warps reads side by side
    float scale_log2, v_scale;         // scale_log2 includes k_scale; > 0 (a negative scale's sign goes to q)
    int q_f16, negate_q;
};

// What a request's new tokens see together.
struct WindowReq {
    int L, head, first, rows;   // L = rows + first - head
};
__device__ __forceinline__ WindowReq window_req(const WindowParams &p, int b, unsigned int *err)
{
    const int l = p.seq_lens ? p.seq_lens[b] : p.cap;
    WindowReq r;
    r.L = min(max(l, 0), p.cap);
    if (err && r.L != l)
        atomicOr(err, kErrLength);
    r.head = r.first = 0;
    if (p.window) {
        const long long back = (long long)r.L - p.q_len - p.window + 1;
        r.first = (int)min((long long)r.L, max((long long)p.sinks, back));
        r.head = min(p.sinks, r.first);
    }
    r.rows = r.L - r.first + r.head;
    return r;
}
__device__ __forceinline__ int window_pos(const WindowReq &r, int row) { return row < r.head ? row : row - r.head + r.first; }

// fd_sched.h's Schedule with divisions of 32 bits where they do: a short call
// waits for them (a 64-bit division costs some 100 instructions).
static __device__ __noinline__ long long window_divide(long long x, long long y) { return x / y; }
__device__ __forceinline__ long long window_quotient(long long x, long long y)
{
    return ((unsigned long long)x | (unsigned long long)y) >> 32 == 0 ? (long long)((uint32_t)x / (uint32_t)y) : window_divide(x, y);
}
struct WindowSchedule : Schedule {
    long long total;   // cost()
    int busy;          // ctas()
    __device__ __forceinline__ int cta_at(long long pos) const { return (int)window_quotient(pos * busy, total); }
    // the first tile of CTA c (as Schedule::tile_at of its first cost position)
    __device__ __forceinline__ int first_tile(int c) const
    {
        const long long x = window_quotient(total * c + busy - 1, busy);
        if (x >= total)
            return tiles();
        int lo = 0, hi = batch - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if ((long long)prefix[mid + 1] + (long long)w * hkv * nonempty[mid + 1] > x)
                hi = mid;
            else
                lo = mid + 1;
        }
        const int nb = (prefix[lo + 1] - prefix[lo]) / hkv;
        const long long q = x - ((long long)prefix[lo] + (long long)w * hkv * nonempty[lo]) - w;
        if (q <= 0)
            return prefix[lo];
        long long h = window_quotient(q, nb + w), j = q - h * (nb + w);
        if (j >= nb) {   // in the gap before head h + 1
            ++h;
            j = 0;
        }
        return prefix[lo] + (int)(h * nb + j);
    }
};

// Workers (teams of p.team warps) of a CTA of a call of this cost: no more
// than there is work for, so that a short call spreads over all SMs.
__device__ __forceinline__ int window_workers(long long cost, int grid, int most)
{
    const long long want = window_quotient(cost + grid - 1, grid);
    return want < 1 ? 1 : want < most ? (int)want : most;
}

// Short segments are not split over CTAs: joining a segment's parts (fence, count, partials through L2) takes as long as
// this many tiles of a warp.  Measured on GB300, one request of 32 heads in 4 bits: 128 positions 10.1 us split and 6.4
// whole, 512 10.5 and 7.3, 1024 10.6 and 9.6, 1536 10.8 and 11.7; 58 requests of 65 visible positions, 16 columns of 256
// dims 41 and 29.
__device__ __forceinline__ int window_join_tiles(int cols, int d) { return 2 + cols * d / 1024; }
// CTAs that a call's segments are split over: n of them for a segment take the time of tiles / n and of n partials, which
// one CTA reads; a warp's tile takes about as long as 60000 values of partials.  Measured on GB300 with 25000, 60000,
// 150000, no limit (us): 65536 positions of one kv head in 4 bits, 16 columns 31.3, 30.4, 32.9, 39.0; 16384, 8 columns
// 15.3, 14.9, 16.5, 21.4; two requests of 8 kv heads, 16 columns, 685 visible positions in E5M2 25.9, 19.0, 19.0, 19.0.
__device__ __forceinline__ int window_ctas(int grid, int segments, int tiles, int cols, int d)
{
    const float n = sqrtf((float)segments * tiles * (60000.f / (cols * d)));
    return n >= grid ? grid : max(1, (int)n);
}

// A scale of 0 becomes this one, so that a hidden score (-inf) keeps its
// weight of 0; scores below 1e30 are still 0.
constexpr float kWindowLeastScale = 1e-37f;

// Host side.
struct WindowLaunch {
    int grid;
    size_t smem_optin;
    cudaStream_t stream;
    cudaEvent_t start_event, end_event;   // recorded around the split kernel, or null
};

template <int D, int KV>
cudaError_t launch_window_variant(const WindowParams &p, const WindowLaunch &c);

#define FD_WINDOW_VARIANTS_D(X, D) X(D, kKvBf16) X(D, kKvF16) X(D, kKvE4m3) X(D, kKvE5m2) X(D, kKvE2m1)
#define FD_WINDOW_VARIANTS(X) FD_WINDOW_VARIANTS_D(X, 64) FD_WINDOW_VARIANTS_D(X, 128) FD_WINDOW_VARIANTS_D(X, 256)
#define FD_EXTERN_WINDOW(D, KV) extern template cudaError_t launch_window_variant<D, KV>(const WindowParams &, const WindowLaunch &);
FD_WINDOW_VARIANTS(FD_EXTERN_WINDOW)
#undef FD_EXTERN_WINDOW

bool record_event(cudaEvent_t ev, cudaStream_t stream);   // fd_api.cu

}  // namespace fd
