// fd_tree.cu -- attention of a tree of drafted tokens over a KV cache
// (fd_tree_decode, fd_tree_decode_paged): argument checks and launch.
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "fd.h"
#include "fd_launch.h"
#include "fd_tree.cuh"
#include "fd_tree_kernel.cuh"

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
    if (opts && (opts->num_ctas < 0 || opts->num_ctas > kTreeMaxCtas || opts->dtype < 0 || opts->dtype > 1 ||
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

// Shared memory of the split kernel: the query rows, then rings of K and V
// tiles in what is left, then the barriers.  An odd slot goes to K, whose tiles
// are wanted a step earlier.  FP8 codes wait in rings of their own; two
// converted tiles of each are enough, the rest holds codes.
template <int D>
void plan_tree_smem(TreeParams *p, TreeLaunch *c, int load)
{
    using C = TreeCfg<D, kTreeTma>;   // the sizes used here are the same for every loader
    const size_t q = (size_t)(p->rows / 128) * C::kQBytes, misc = align_up(sizeof(TreeMisc), 16);
    size_t left = c->smem_optin - q - misc;
    p->raw_slots = 0;
    int slots = 4;
    if (load == kTreeConvert) {
        const int raw = (int)((left - 4 * C::kSlotBytes) / (2 * C::kRawBytes));
        p->raw_slots = raw < kTreeMaxRaw ? raw : kTreeMaxRaw;
        left -= 2 * (size_t)p->raw_slots * C::kRawBytes;
    }
    slots = (int)(left / C::kSlotBytes);
    slots = slots < 2 * kTreeMaxSlots ? slots : 2 * kTreeMaxSlots;
    p->k_slots = (slots + 1) / 2;
    p->v_slots = slots / 2;
    p->off_k = (uint32_t)q;
    p->off_v = (uint32_t)(p->off_k + p->k_slots * C::kSlotBytes);
    p->off_raw = (uint32_t)(p->off_v + p->v_slots * C::kSlotBytes);
    p->off_misc = (uint32_t)(p->off_raw + 2 * p->raw_slots * C::kRawBytes);
    c->smem_bytes = p->off_misc + misc;
}

int slot_rows_of(int rows, int tree_rows) { return tree_rows < rows ? tree_rows : rows; }

// Query rows of a segment: both softmax groups get rows of their own when there are more than 128.
int segment_rows(int tree_rows, int d) { return d != 256 && tree_rows > 128 ? 256 : 128; }

struct TreeWorkspace {
    size_t cost, lse, o, sums, total;
};
TreeWorkspace tree_workspace(int batch, int tree_rows, int d)
{
    const size_t partials = 2 * kTreeMaxCtas, rows = partials * slot_rows_of(segment_rows(tree_rows, d), tree_rows);
    // the statistics of as many rows as any head dim's segment has, so that the
    // size grows with the head dim too
    const size_t lse_rows = partials * slot_rows_of(256, tree_rows);
    TreeWorkspace w;
    w.cost = 256;
    w.lse = align_up(w.cost + sizeof(long long) * ((size_t)batch + 1), 256);
    w.o = align_up(w.lse + sizeof(float) * lse_rows, 256);
    w.sums = align_up(w.o + sizeof(float) * rows * d, 256);
    w.total = align_up(w.sums + sizeof(float) * kTreeMaxCtas * tree_groups(d) * slot_rows_of(128, tree_rows) * d, 256);
    return w;
}

fd_status launch(TreeParams p, int head_dim, float scale, const fd_options *opts, void *workspace, fd_stream_t stream)
{
    DeviceInfo dev;
    fd_status st = device_info(&dev);
    if (st != FD_OK)
        return st;
    const bool f16 = opts && opts->dtype == FD_DTYPE_F16;
    const int kv_dtype = opts ? opts->kv_dtype : FD_KV_AS_Q;
    const int kv = kv_dtype == FD_KV_FP8_E4M3 ? kKvE4m3
                   : kv_dtype == FD_KV_FP8_E5M2 ? kKvE5m2 : (f16 ? kKvF16 : kKvBf16);
    const bool fp8 = kv_is_fp8(kv);
    // an FP8 cache's k_scale multiplies every score; a negative scale changes q's sign
    scale *= fp8 && opts->k_scale != 0.f ? opts->k_scale : 1.f;
    p.q_f16 = f16;
    p.negate_q = scale < 0.f;
    p.scale_log2 = (p.negate_q ? -scale : scale) * 1.4426950408889634f;
    if (p.scale_log2 < kTreeLeastScale)
        p.scale_log2 = kTreeLeastScale;
    p.v_scale = fp8 && opts->v_scale != 0.f ? opts->v_scale : 1.f;
    p.words = (p.tree_len + 63) / 64;
    p.group = p.hq / p.hkv;
    p.timeout_ns = opts && opts->wait_timeout_ns ? opts->wait_timeout_ns : 2000000000ull;
    p.starve = opts && (opts->flags & FD_FLAG_TEST_STARVE_FIRST_TILE) ? 1 : 0;
    p.rows = segment_rows(p.tree_len * p.group, head_dim);
    p.slot_rows = slot_rows_of(p.rows, p.tree_len * p.group);
    const TreeWorkspace w = tree_workspace(p.batch, p.tree_len * p.group, head_dim);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.ws_err = reinterpret_cast<unsigned int *>(ws);
    p.ws_cost = reinterpret_cast<long long *>(ws + w.cost);
    p.ws_lse = reinterpret_cast<float *>(ws + w.lse);
    p.ws_o = reinterpret_cast<float *>(ws + w.o);
    p.ws_sums = reinterpret_cast<float *>(ws + w.sums);
    p.sum_rows = slot_rows_of(128, p.tree_len * p.group);

    TreeLaunch c;
    c.grid = opts && opts->num_ctas > 0 ? opts->num_ctas : dev.sms < kTreeMaxCtas ? dev.sms : kTreeMaxCtas;
    c.smem_optin = (size_t)dev.smem_optin;
    c.stream = reinterpret_cast<cudaStream_t>(stream);
    const int load = p.block_table && p.page_size < 8 ? kTreeCopy : fp8 ? kTreeConvert : kTreeTma;
    if (head_dim == 64)
        plan_tree_smem<64>(&p, &c, load);
    else if (head_dim == 128)
        plan_tree_smem<128>(&p, &c, load);
    else
        plan_tree_smem<256>(&p, &c, load);
    if (p.v_slots < 2 || (load == kTreeConvert && p.raw_slots < 1))
        return FD_ERR_UNSUPPORTED;
    p.box_rows = p.block_table && p.page_size < kTileTokens ? p.page_size : kTileTokens;
    alignas(64) CUtensorMap tmk, tmv;
    std::memset(&tmk, 0, sizeof tmk);
    std::memset(&tmv, 0, sizeof tmv);
    if (load != kTreeCopy) {
        long long rows = p.block_table ? (long long)p.num_pages * p.page_size : (long long)p.batch * p.page_size;
        rows = rows > 0 ? rows : 1;
        if ((st = encode_kv_map(&tmk, p.k, p.hkv, rows, p.box_rows, !fp8, kv, head_dim)) != FD_OK ||
            (st = encode_kv_map(&tmv, p.v, p.hkv, rows, p.box_rows, !fp8, kv, head_dim)) != FD_OK)
            return st;
    }
    cudaEvent_t ev0 = opts ? static_cast<cudaEvent_t>(opts->split_start_event) : nullptr;
    cudaEvent_t ev1 = opts ? static_cast<cudaEvent_t>(opts->split_end_event) : nullptr;
    if (ev0 && !record_event(ev0, c.stream))
        return FD_ERR_CUDA;
    cudaError_t e = cudaErrorInvalidValue;
#define FD_PICK_TREE(D, F16, KV, LOAD)                              \
    if (head_dim == D && kv == KV && load == LOAD)                  \
        e = launch_tree_variant<D, F16, KV, LOAD>(p, tmk, tmv, c);
    FD_TREE_VARIANTS(FD_PICK_TREE)
#undef FD_PICK_TREE
    if (e != cudaSuccess)
        return FD_ERR_CUDA;
    if (ev1 && !record_event(ev1, c.stream))
        return FD_ERR_CUDA;
    return launch_tree_merge(head_dim, p, c.grid, c.stream) == cudaSuccess ? FD_OK : FD_ERR_CUDA;
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
    return tree_workspace(batch, num_q_heads / num_kv_heads * tree_len, head_dim).total;
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
    p.cap = s_max;
    p.page_size = s_max;
    p.o = o;
    p.lse = lse;
    return launch(p, head_dim, scale, opts, workspace, stream);
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
    p.cap = (int)cap;
    p.o = o;
    p.lse = lse;
    return launch(p, head_dim, scale, opts, workspace, stream);
}

}  // extern "C"
