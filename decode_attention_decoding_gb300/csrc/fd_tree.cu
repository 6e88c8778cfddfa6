// fd_tree.cu -- attention of a tree of drafted tokens over a KV cache
// (fd_tree_decode, fd_tree_decode_paged): argument checks and launch.
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "fd.h"
#include "fd_device.cuh"
#include "fd_sched.h"
#include "fd_tree.cuh"

namespace fd {
namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool scale_ok(float x) { return x == 0.f || (x > 0.f && x < __builtin_huge_valf()); }

// The checks that need no layout.
fd_status check_tree(const void *q, const void *k, const void *v, const void *mask, long long mask_stride,
                     const void *tree_lens, const void *seq_lens, int batch, int tree_len, int hq, int hkv,
                     int head_dim, const float *o, const float *lse, const void *ws, size_t ws_bytes,
                     const fd_options *opts)
{
    if (batch < 0 || hq <= 0 || hkv <= 0 || hq % hkv != 0 || tree_len <= 0)
        return FD_ERR_INVALID_ARG;
    if (!q || !k || !v || !o || !ws)
        return FD_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(ws, 256) ||
        !aligned(mask, 8) || !aligned(tree_lens, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4))
        return FD_ERR_INVALID_ARG;
    const long long words = (tree_len + 63) / 64;
    if (mask && mask_stride != 0 && mask_stride < words * tree_len)
        return FD_ERR_INVALID_ARG;
    if (opts && (opts->num_ctas < 0 || opts->num_ctas > kMaxCtas || opts->dtype < 0 || opts->dtype > 1 ||
                 opts->kv_dtype < FD_KV_AS_Q || opts->kv_dtype > FD_KV_FP8_E5M2 || !scale_ok(opts->k_scale) ||
                 !scale_ok(opts->v_scale) || opts->q_len < 0 || opts->q_len > 1))
        return FD_ERR_INVALID_ARG;
    if (fd_tree_workspace_size(batch, tree_len, hq, hkv, head_dim) == 0)
        return FD_ERR_UNSUPPORTED;
    if (ws_bytes < fd_tree_workspace_size(batch, tree_len, hq, hkv, head_dim))
        return FD_ERR_WORKSPACE_TOO_SMALL;
    return FD_OK;
}

bool host_lens_ok(const int32_t *lens, int batch, long long cap)
{
    if (lens)
        for (int b = 0; b < batch; ++b)
            if (lens[b] < 0 || lens[b] > cap)
                return false;
    return true;
}

fd_status launch(TreeParams p, const fd_options *opts, void *workspace, fd_stream_t stream)
{
    const bool f16 = opts && opts->dtype == FD_DTYPE_F16;
    const int kv_dtype = opts ? opts->kv_dtype : FD_KV_AS_Q;
    const int kv = kv_dtype == FD_KV_FP8_E4M3 ? kKvE4m3
                   : kv_dtype == FD_KV_FP8_E5M2 ? kKvE5m2 : (f16 ? kKvF16 : kKvBf16);
    const bool fp8 = kv_is_fp8(kv);
    p.scale *= fp8 && opts->k_scale != 0.f ? opts->k_scale : 1.f;
    p.v_scale = fp8 && opts->v_scale != 0.f ? opts->v_scale : 1.f;
    p.q_f16 = f16;
    p.words = (p.tree_len + 63) / 64;
    p.group = p.hq / p.hkv;
    p.ws_err = static_cast<unsigned int *>(workspace);
    return launch_tree_simple(kv, p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

}  // namespace
}  // namespace fd

using namespace fd;

extern "C" {

size_t fd_tree_workspace_size(int batch, int tree_len, int num_q_heads, int num_kv_heads, int head_dim)
{
    if (batch < 0 || batch > kMaxBatch || tree_len < 1 || tree_len > kMaxTree || num_q_heads <= 0 ||
        num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
        (head_dim != 64 && head_dim != 128 && head_dim != 256) ||
        (long long)(num_q_heads / num_kv_heads) * tree_len > kMaxTreeRows)
        return 0;
    return 256;
}

fd_status fd_tree_decode(const void *q, const void *k, const void *v, const uint64_t *tree_mask,
                         long long mask_stride, const int32_t *tree_lens_dev, const int32_t *seq_lens_dev,
                         const int32_t *seq_lens_host, int batch, int tree_len, int num_q_heads, int num_kv_heads,
                         int head_dim, int s_max, float scale, float *o, float *lse, void *workspace,
                         size_t workspace_bytes, const fd_options *opts, fd_stream_t stream)
{
    fd_status st = check_tree(q, k, v, tree_mask, mask_stride, tree_lens_dev, seq_lens_dev, batch, tree_len,
                              num_q_heads, num_kv_heads, head_dim, o, lse, workspace, workspace_bytes, opts);
    if (st != FD_OK)
        return st;
    if (s_max < 0 || !host_lens_ok(seq_lens_host, batch, s_max))
        return FD_ERR_INVALID_ARG;
    if ((long long)batch * s_max >= (1ll << 31))
        return FD_ERR_UNSUPPORTED;
    if (batch == 0)
        return FD_OK;
    TreeParams p;
    std::memset(&p, 0, sizeof p);
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint8_t *>(k);
    p.v = static_cast<const uint8_t *>(v);
    p.mask = tree_mask;
    p.mask_stride = mask_stride;
    p.tree_lens = tree_lens_dev;
    p.seq_lens = seq_lens_dev;
    p.batch = batch;
    p.tree_len = tree_len;
    p.hq = num_q_heads;
    p.hkv = num_kv_heads;
    p.head_dim = head_dim;
    p.cap = s_max;
    p.page_size = s_max;
    p.scale = scale;
    p.o = o;
    p.lse = lse;
    return launch(p, opts, workspace, stream);
}

fd_status fd_tree_decode_paged(const void *q, const void *k_pages, const void *v_pages, const int32_t *block_table,
                               int max_blocks_per_seq, const uint64_t *tree_mask, long long mask_stride,
                               const int32_t *tree_lens_dev, const int32_t *seq_lens_dev,
                               const int32_t *seq_lens_host, int batch, int tree_len, int num_q_heads,
                               int num_kv_heads, int head_dim, int page_size, int num_pages, float scale, float *o,
                               float *lse, void *workspace, size_t workspace_bytes, const fd_options *opts,
                               fd_stream_t stream)
{
    fd_status st = check_tree(q, k_pages, v_pages, tree_mask, mask_stride, tree_lens_dev, seq_lens_dev, batch,
                              tree_len, num_q_heads, num_kv_heads, head_dim, o, lse, workspace, workspace_bytes,
                              opts);
    if (st != FD_OK)
        return st;
    const long long cap = (long long)max_blocks_per_seq * page_size;
    if (!block_table || !seq_lens_dev || !aligned(block_table, 4) || max_blocks_per_seq <= 0 || page_size <= 0 ||
        num_pages <= 0 || !host_lens_ok(seq_lens_host, batch, cap))
        return FD_ERR_INVALID_ARG;
    if (!((page_size < kTileTokens && kTileTokens % page_size == 0) || page_size % kTileTokens == 0) ||
        cap >= (1ll << 31) || (long long)num_pages * page_size >= (1ll << 31))
        return FD_ERR_UNSUPPORTED;
    if (batch == 0)
        return FD_OK;
    TreeParams p;
    std::memset(&p, 0, sizeof p);
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint8_t *>(k_pages);
    p.v = static_cast<const uint8_t *>(v_pages);
    p.mask = tree_mask;
    p.mask_stride = mask_stride;
    p.tree_lens = tree_lens_dev;
    p.seq_lens = seq_lens_dev;
    p.block_table = block_table;
    p.max_blocks = max_blocks_per_seq;
    p.num_pages = num_pages;
    p.page_size = page_size;
    p.batch = batch;
    p.tree_len = tree_len;
    p.hq = num_q_heads;
    p.hkv = num_kv_heads;
    p.head_dim = head_dim;
    p.cap = (int)cap;
    p.scale = scale;
    p.o = o;
    p.lse = lse;
    return launch(p, opts, workspace, stream);
}

}  // extern "C"
