// fd_window.cu -- decode attention through a window with sinks, and over 4-bit
// caches (fd_window_decode, fd_decode4 and their paged forms): argument checks
// and launch.
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "fd.h"
#include "fd_launch.h"
#include "fd_window.cuh"

namespace fd {
namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool scale_ok(float x) { return x == 0.f || (x > 0.f && x < __builtin_huge_valf()); }

// The counts lie at the same place for every shape: each call leaves them at 0.
struct WindowWorkspace {
    size_t counts, ml, o, total;
};
WindowWorkspace window_workspace(int cols, int d)
{
    const size_t slots = 2 * (size_t)kWindowMaxCtas * kWindowMaxWarps;
    WindowWorkspace w;
    w.counts = 256;
    w.ml = align_up(w.counts + sizeof(unsigned int) * slots / 2, 256);
    w.o = align_up(w.ml + sizeof(float2) * slots * cols, 256);
    w.total = align_up(w.o + sizeof(float) * slots * cols * d, 256);
    return w;
}

int q_len_of(const fd_options *opts) { return opts && opts->q_len > 0 ? opts->q_len : 1; }

// A call, whatever its cache.
struct WindowCall {
    const void *q, *k, *v, *ks, *vs;   // ks: null unless the cache is in 4 bits
    bool fp4;
    const int32_t *block_table, *seq_lens, *seq_lens_host;
    int max_blocks, batch, hq, hkv, d, page_size, num_pages, window, sinks;
    float scale;
    float *o, *lse;
    void *ws;
    size_t ws_bytes;
    const fd_options *opts;
    cudaStream_t stream;
};

fd_status run(const WindowCall &a)
{
    const fd_options *opts = a.opts;
    if (a.batch < 0 || a.hq <= 0 || a.hkv <= 0 || a.hq % a.hkv != 0 || a.window < 0 || a.sinks < 0)
        return FD_ERR_INVALID_ARG;
    if (opts && (opts->num_ctas < 0 || opts->num_ctas > kWindowMaxCtas || opts->dtype < 0 || opts->dtype > 1 ||
                 opts->kv_dtype < FD_KV_AS_Q || opts->kv_dtype > (a.fp4 ? FD_KV_AS_Q : FD_KV_FP8_E5M2) || opts->q_len < 0 ||
                 !scale_ok(opts->k_scale) || !scale_ok(opts->v_scale)))
        return FD_ERR_INVALID_ARG;
    const long long cap = a.block_table ? (long long)a.max_blocks * a.page_size : a.page_size;
    if (a.seq_lens_host)
        for (int b = 0; b < a.batch; ++b)
            if (a.seq_lens_host[b] < 0 || a.seq_lens_host[b] > cap)
                return FD_ERR_INVALID_ARG;
    const int q_len = q_len_of(opts);
    const size_t need = fd_window_workspace_size(a.batch, a.hq, a.hkv, a.d, q_len);
    // rows have 32-bit numbers, and so have tiles (of at least 16 rows; a segment start counts as one)
    const long long rows = (long long)a.num_pages * a.page_size;
    long long span = cap;
    if (a.window && (long long)a.window + a.sinks + q_len < span)
        span = (long long)a.window + a.sinks + q_len;
    if (need == 0 || cap >= (1ll << 31) || rows >= (1ll << 32) || rows * a.hkv >= (1ll << 32) - 1 ||
        (span / 16 + 2) * a.hkv * a.batch >= (1ll << 31))
        return FD_ERR_UNSUPPORTED;
    if (a.batch == 0)
        return FD_OK;
    if (!a.q || !a.k || !a.v || (a.fp4 && (!a.ks || !a.vs)) || !a.o || !a.ws)
        return FD_ERR_INVALID_ARG;
    if (!aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.ks, 16) || !aligned(a.vs, 16) ||
        !aligned(a.o, 16) || !aligned(a.ws, 256) || !aligned(a.seq_lens, 4) || !aligned(a.block_table, 4) || !aligned(a.lse, 4))
        return FD_ERR_INVALID_ARG;
    if (a.ws_bytes < need)
        return FD_ERR_WORKSPACE_TOO_SMALL;

    DeviceInfo dev;
    const fd_status st = device_info(&dev);
    if (st != FD_OK)
        return st;
    const bool f16 = opts && opts->dtype == FD_DTYPE_F16;
    const int kv_dtype = opts ? opts->kv_dtype : FD_KV_AS_Q;
    const int kv = a.fp4 ? kKvE2m1 : kv_dtype == FD_KV_FP8_E4M3 ? kKvE4m3 : kv_dtype == FD_KV_FP8_E5M2 ? kKvE5m2 : f16 ? kKvF16 : kKvBf16;
    WindowParams p;
    std::memset(&p, 0, sizeof p);
    p.q = static_cast<const uint16_t *>(a.q);
    p.k = static_cast<const uint8_t *>(a.k);
    p.v = static_cast<const uint8_t *>(a.v);
    p.ks = static_cast<const uint8_t *>(a.ks);
    p.vs = static_cast<const uint8_t *>(a.vs);
    p.block_table = a.block_table;
    p.seq_lens = a.seq_lens;
    p.o = a.o;
    p.lse = a.lse;
    p.batch = a.batch;
    p.q_len = q_len;
    p.hq = a.hq;
    p.hkv = a.hkv;
    p.group = a.hq / a.hkv;
    p.cols = p.group * q_len;
    p.cap = (int)cap;
    p.page_size = a.page_size;
    p.page_shift = a.page_size > 0 && (a.page_size & (a.page_size - 1)) == 0 ? __builtin_ctz((unsigned)a.page_size) : -1;
    p.max_blocks = a.max_blocks;
    p.num_pages = a.num_pages;
    p.row_page = (uint32_t)a.page_size * (uint32_t)a.hkv;
    p.row_token = a.fp4 ? 1u : (uint32_t)a.hkv;
    p.row_head = a.fp4 ? (uint32_t)a.page_size : 1u;
    p.window = a.window;
    p.sinks = a.window ? a.sinks : 0;
    const bool scaled = kv >= kKvE4m3;
    const float scale = a.scale * (scaled && opts && opts->k_scale != 0.f ? opts->k_scale : 1.f);
    p.negate_q = scale < 0.f;
    p.scale_log2 = (p.negate_q ? -scale : scale) * 1.4426950408889634f;
    if (p.scale_log2 < kWindowLeastScale)
        p.scale_log2 = kWindowLeastScale;
    p.v_scale = scaled && opts && opts->v_scale != 0.f ? opts->v_scale : 1.f;
    p.q_f16 = f16;
    // Rows of a kv head are hkv rows apart unless the cache is in 4 bits: where they are short, adjacent
    // heads are read side by side.
    p.team = 1;
    if (!a.fp4) {
        const int row = a.d * (kv == kKvBf16 || kv == kKvF16 ? 2 : 1);
        if (row == 64 && a.hkv % 4 == 0)
            p.team = 4;
        else if (row <= 128 && a.hkv % 2 == 0)
            p.team = 2;
    }
    const WindowWorkspace w = window_workspace(p.cols, a.d);
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    p.ws_err = reinterpret_cast<unsigned int *>(ws);
    p.ws_counts = reinterpret_cast<unsigned int *>(ws + w.counts);
    p.ws_ml = reinterpret_cast<float2 *>(ws + w.ml);
    p.ws_o = reinterpret_cast<float *>(ws + w.o);
    WindowLaunch c;
    c.grid = opts && opts->num_ctas > 0 ? opts->num_ctas : dev.sms < kWindowMaxCtas ? dev.sms : kWindowMaxCtas;
    c.smem_optin = (size_t)dev.smem_optin;
    c.stream = a.stream;
    c.start_event = opts ? static_cast<cudaEvent_t>(opts->split_start_event) : nullptr;
    c.end_event = opts ? static_cast<cudaEvent_t>(opts->split_end_event) : nullptr;
    cudaError_t e = cudaErrorInvalidValue;
#define FD_PICK_WINDOW(D, KV)                       \
    if (a.d == D && kv == KV)                       \
        e = launch_window_variant<D, KV>(p, c);
    FD_WINDOW_VARIANTS(FD_PICK_WINDOW)
#undef FD_PICK_WINDOW
    return e == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

}  // namespace
}  // namespace fd

using namespace fd;

extern "C" {

size_t fd_window_workspace_size(int batch, int num_q_heads, int num_kv_heads, int head_dim, int q_len)
{
    if (batch < 0 || batch > kMaxBatch || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
        num_kv_heads > 65535 || q_len < 1 || (long long)(num_q_heads / num_kv_heads) * q_len > kWindowMaxColumns ||
        (head_dim != 64 && head_dim != 128 && head_dim != 256))
        return 0;
    return window_workspace(num_q_heads / num_kv_heads * q_len, head_dim).total;
}

fd_status fd_window_decode(const void *q, const void *k, const void *v, const int32_t *seq_lens_dev,
                           const int32_t *seq_lens_host, int batch, int num_q_heads, int num_kv_heads, int head_dim,
                           int s_max, int window, int sinks, float scale, float *o, float *lse, void *workspace,
                           size_t workspace_bytes, const fd_options *opts, fd_stream_t stream)
{
    if (s_max < 0 || window < 1)
        return FD_ERR_INVALID_ARG;
    const WindowCall a = {q, k, v, nullptr, nullptr, false, nullptr, seq_lens_dev, seq_lens_host, 0, batch, num_q_heads,
                          num_kv_heads, head_dim, s_max, batch, window, sinks, scale, o, lse, workspace, workspace_bytes,
                          opts, reinterpret_cast<cudaStream_t>(stream)};
    return run(a);
}

fd_status fd_window_decode_paged(const void *q, const void *k_pages, const void *v_pages, const int32_t *block_table,
                                 int max_blocks_per_seq, const int32_t *seq_lens_dev, const int32_t *seq_lens_host,
                                 int batch, int num_q_heads, int num_kv_heads, int head_dim, int page_size,
                                 int num_pages, int window, int sinks, float scale, float *o, float *lse,
                                 void *workspace, size_t workspace_bytes, const fd_options *opts, fd_stream_t stream)
{
    if (!block_table || !seq_lens_dev || max_blocks_per_seq <= 0 || page_size <= 0 || num_pages <= 0 || window < 1)
        return FD_ERR_INVALID_ARG;
    const WindowCall a = {q, k_pages, v_pages, nullptr, nullptr, false, block_table, seq_lens_dev, seq_lens_host,
                          max_blocks_per_seq, batch, num_q_heads, num_kv_heads, head_dim, page_size, num_pages, window,
                          sinks, scale, o, lse, workspace, workspace_bytes, opts, reinterpret_cast<cudaStream_t>(stream)};
    return run(a);
}

fd_status fd_decode4(const void *q, const fd_cache4 *cache, const int32_t *seq_lens_dev, const int32_t *seq_lens_host,
                     int batch, int num_q_heads, int num_kv_heads, int head_dim, int s_max, int window, int sinks,
                     float scale, float *o, float *lse, void *workspace, size_t workspace_bytes, const fd_options *opts,
                     fd_stream_t stream)
{
    if (!cache || s_max < 0)
        return FD_ERR_INVALID_ARG;
    const WindowCall a = {q, cache->k_codes, cache->v_codes, cache->k_scales, cache->v_scales, true, nullptr, seq_lens_dev,
                          seq_lens_host, 0, batch, num_q_heads, num_kv_heads, head_dim, s_max, batch, window, sinks, scale,
                          o, lse, workspace, workspace_bytes, opts, reinterpret_cast<cudaStream_t>(stream)};
    return run(a);
}

fd_status fd_decode4_paged(const void *q, const fd_cache4 *cache, const int32_t *block_table, int max_blocks_per_seq,
                           const int32_t *seq_lens_dev, const int32_t *seq_lens_host, int batch, int num_q_heads,
                           int num_kv_heads, int head_dim, int page_size, int num_pages, int window, int sinks,
                           float scale, float *o, float *lse, void *workspace, size_t workspace_bytes,
                           const fd_options *opts, fd_stream_t stream)
{
    if (!cache || !block_table || !seq_lens_dev || max_blocks_per_seq <= 0 || page_size <= 0 || num_pages <= 0)
        return FD_ERR_INVALID_ARG;
    const WindowCall a = {q, cache->k_codes, cache->v_codes, cache->k_scales, cache->v_scales, true, block_table,
                          seq_lens_dev, seq_lens_host, max_blocks_per_seq, batch, num_q_heads, num_kv_heads, head_dim,
                          page_size, num_pages, window, sinks, scale, o, lse, workspace, workspace_bytes, opts,
                          reinterpret_cast<cudaStream_t>(stream)};
    return run(a);
}

}  // extern "C"
