// fd_cache.cu -- what a speculative decoding step does to a KV cache around
// its attention: block tables and slot maps from request lengths
// (fd_build_tables), new rows into their slots (fd_cache_write), and the
// accepted path to the front of the drafted tail (fd_cache_compact).
#include <cstdint>

#include <cuda_runtime.h>

#include "fd.h"
#include "fd_device.cuh"
#include "fd_sched.h"

namespace fd {
namespace {

// ---------------------------------------------------------------- tables

struct TablesParams {
    const int32_t *seq_lens, *new_lens, *held_pages, *free_pages, *free_count;
    int max_free, batch, page_size, num_pages, max_blocks, max_tokens;
    int page_shift;   // page_size = 2^page_shift, or -1
    int32_t *block_table;
    int64_t *slot_map;
    int32_t *cu_new_lens, *seq_lens_out, *held_out, *free_out;
    unsigned int *status;
};

constexpr int kTablesThreads = 256;
constexpr int kTablesTokensPerThread = 4;
// CTAs an SM: more hide the slots' chains of loads, and each scans the lengths
// once more.  1.6 M tokens of 384 requests: 2, 4, 8, 16 an SM 15.1, 11.8, 13.6,
// 15.0 us; 512 threads a CTA are slower at either end (15.4 us, and 64 tokens
// of 64 requests 4.7 instead of 4.5).
constexpr int kTablesCtasPerSm = 4;

// Shared memory of the kernel: cu and pages [batch + 1], old and held [batch].
constexpr size_t tables_smem(int batch) { return sizeof(int) * (4 * (size_t)batch + 2); }

// Sum of v over the threads before this one, and over all of them in *total.
template <class T>
__device__ __forceinline__ T block_exclusive_scan(T v, T *tmp, T *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off)
            x += y;
    }
    if (lane == 31)
        tmp[warp] = x;
    __syncthreads();
    T before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kTablesThreads / 32; ++w) {
        const T s = tmp[w];
        before += w < warp ? s : 0;
        all += s;
    }
    __syncthreads();   // tmp may be written again
    *total = all;
    return before + x - v;
}

// Request b's numbers before the token limit: length, new tokens (both inside
// the table), pages held.  Out-of-range values are clamped; *bad says so.
struct TableReq {
    int old, fresh, held;
};
__device__ __forceinline__ TableReq table_req(const TablesParams &p, int b, bool *bad)
{
    const int cap = p.max_blocks * p.page_size;   // < 2^31 (checked on the host)
    const int o = p.seq_lens[b], n = p.new_lens[b];
    TableReq r;
    r.old = min(max(o, 0), cap);
    r.fresh = min(max(n, 0), cap - r.old);
    const int least = (int)(((unsigned)r.old + p.page_size - 1u) / (unsigned)p.page_size);
    const int h = p.held_pages ? p.held_pages[b] : least;
    r.held = min(max(h, least), p.max_blocks);
    *bad = *bad || r.old != o || r.fresh != n || r.held != h;
    return r;
}

__device__ __forceinline__ int pages_needed(const TablesParams &p, int tokens, int held)
{
    const int all = (int)(((unsigned)tokens + p.page_size - 1u) / (unsigned)p.page_size);
    return max(0, all - held);
}

// The free page with ordinal `ord`, counted from the end of the stack; -1 when
// there is none left.  *bad: the stack holds a page outside the pool.
__device__ __forceinline__ int free_page(const TablesParams &p, int count, int ord, bool *bad)
{
    if (ord >= count)
        return -1;
    const int page = p.free_pages[count - 1 - ord];
    *bad = *bad || (unsigned)page >= (unsigned)p.num_pages;
    return page;
}

// One launch and no waits between CTAs: every CTA scans the lengths itself
// (they are a few KB in L2) into prefix sums in shared memory, new tokens and
// new pages of the requests before b, beside the requests' lengths and held
// pages; then it takes its share of the slots and of the new table entries.  A
// slot in a new page reads the free stack, not the table entry that another CTA
// may still have to write.  Small calls are one chain of dependent loads; large
// ones are bound by it too (a search, then a page per slot), hence several
// independent slots a thread.
__global__ void __launch_bounds__(kTablesThreads) build_tables_kernel(const __grid_constant__ TablesParams p)
{
    extern __shared__ int s_req[];
    int *cu = s_req, *pages = cu + p.batch + 1, *old = pages + p.batch + 1, *held = old + p.batch;
    __shared__ long long s_tmp_l[kTablesThreads / 32];
    __shared__ int s_tmp_i[kTablesThreads / 32];
    const int tid = threadIdx.x;
    const bool first_cta = blockIdx.x == 0;
    const int per = ceil_div(p.batch, kTablesThreads);   // batch <= kMaxBatch
    const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
    const int count_in = *p.free_count;
    bool bad = false;

    long long mine = 0, total_l;
    for (int b = tid; b < p.batch; b += kTablesThreads) {
        const TableReq r = table_req(p, b, &bad);
        old[b] = r.old;
        held[b] = r.held;
        cu[b] = r.fresh;   // for now
    }
    __syncthreads();
    for (int b = b0; b < b1; ++b)
        mine += cu[b];
    long long at = block_exclusive_scan(mine, s_tmp_l, &total_l);
    bad = bad || total_l > p.max_tokens;
    // tokens past max_tokens do not exist: the prefix stops there
    int need = 0, total_pages;
    for (int b = b0; b < b1; ++b) {
        const int c0 = (int)min(at, (long long)p.max_tokens);
        at += cu[b];
        const int c1 = (int)min(at, (long long)p.max_tokens);
        cu[b] = c0;
        pages[b] = pages_needed(p, old[b] + c1 - c0, held[b]);   // for now
        need += pages[b];
    }
    const int total_tokens = (int)min(total_l, (long long)p.max_tokens);
    int pg = block_exclusive_scan(need, s_tmp_i, &total_pages);
    const int count = min(max(count_in, 0), p.max_free);
    bad = bad || count != count_in;
    for (int b = b0; b < b1; ++b) {
        const int n = pages[b];
        pages[b] = pg;
        pg += n;
    }
    if (tid == 0) {
        cu[p.batch] = total_tokens;
        pages[p.batch] = total_pages;
    }
    if (first_cta && bad && p.status)
        atomicOr(p.status, FD_DEVICE_STATUS_BAD_LENGTH);
    __syncthreads();
    if (first_cta) {
        for (int b = tid; b <= p.batch; b += kTablesThreads) {
            p.cu_new_lens[b] = cu[b];
            if (b == p.batch)
                break;
            const int n = pages[b + 1] - pages[b], granted = min(n, max(0, count - pages[b]));
            const int tokens = old[b] + cu[b + 1] - cu[b];
            p.held_out[b] = held[b] + granted;
            p.seq_lens_out[b] = granted < n ? min(tokens, (held[b] + granted) * p.page_size) : tokens;
        }
        if (tid == 0) {
            p.free_out[0] = max(0, count - total_pages);
            if (p.status && total_pages > count)
                atomicOr(p.status, FD_DEVICE_STATUS_NO_PAGES);
        }
    }

    const int gthreads = gridDim.x * kTablesThreads, gid = blockIdx.x * kTablesThreads + tid;
    bool bad_page = false;
    // new table entries
    for (long long ord = gid; ord < total_pages; ord += gthreads) {
        const int b = request_of_tile(pages, p.batch, (int)ord);
        p.block_table[(long long)b * p.max_blocks + held[b] + ((int)ord - pages[b])] = free_page(p, count, (int)ord, &bad_page);
    }
    // slots: a warp takes 32 x kTablesTokensPerThread consecutive ones
    const int lane = tid & 31;
    const long long step = (long long)gthreads * kTablesTokensPerThread;
    for (long long w0 = (long long)(gid >> 5) * 32 * kTablesTokensPerThread; w0 < p.max_tokens; w0 += step) {
        int page[kTablesTokensPerThread], in[kTablesTokensPerThread];
        int b = -1;
#pragma unroll
        for (int k = 0; k < kTablesTokensPerThread; ++k) {
            const long long i = w0 + 32 * k + lane;
            page[k] = -1;
            in[k] = 0;
            if (i < total_tokens) {
                if (b < 0 || i >= cu[b + 1])
                    b = request_of_tile(cu, p.batch, (int)i);
                const unsigned pos = (unsigned)(old[b] + ((int)i - cu[b]));
                const int blk = (int)(p.page_shift >= 0 ? pos >> p.page_shift : pos / (unsigned)p.page_size);
                in[k] = (int)(pos - (unsigned)blk * (unsigned)p.page_size);
                if (blk < held[b]) {
                    page[k] = p.block_table[(long long)b * p.max_blocks + blk];
                    bad_page = bad_page || (unsigned)page[k] >= (unsigned)p.num_pages;
                } else
                    page[k] = free_page(p, count, pages[b] + blk - held[b], &bad_page);
            }
        }
#pragma unroll
        for (int k = 0; k < kTablesTokensPerThread; ++k) {
            const long long i = w0 + 32 * k + lane;
            if (i < p.max_tokens)
                p.slot_map[i] = (unsigned)page[k] < (unsigned)p.num_pages ? (long long)page[k] * p.page_size + in[k] : -1;
        }
    }
    if (bad_page && p.status)
        atomicOr(p.status, FD_DEVICE_STATUS_BAD_SLOT);
}

// ---------------------------------------------------------------- write

struct WriteParams {
    const uint8_t *src[2];        // K and V rows
    long long stride[2];          // bytes between token rows
    uint8_t *dst[2];
    float scale[2];
    const int64_t *slots;
    unsigned int *status;
    long long num_slots, row_bytes;   // bytes of a cache row
    int num_tokens, tokens_per_cta, units;   // units: pieces of a row, one thread's work each
    unsigned int units_magic;                // floor(2^32 / units) + 1: __umulhi(x, magic) = x / units for x * units < 2^32
};

constexpr int kWriteThreads = 256;
constexpr int kWriteUnitsPerThread = 4;

enum : int { kWriteCopy = 0, kWriteE4m3 = 1, kWriteE5m2 = 2 };

// Four fp32 values to four FP8 codes, nearest even, saturating, NaN kept.
template <int MODE, bool FAST>
__device__ __forceinline__ uint32_t quantise4(float2 a, float2 b, float scale, float r)
{
    a.x = quotient<FAST>(a.x, scale, r);
    a.y = quotient<FAST>(a.y, scale, r);
    b.x = quotient<FAST>(b.x, scale, r);
    b.y = quotient<FAST>(b.y, scale, r);
    if constexpr (MODE == kWriteE4m3)
        return (uint32_t)pack_e4m3x2(a.x, a.y) | ((uint32_t)pack_e4m3x2(b.x, b.y) << 16);
    else
        return (uint32_t)pack_e5m2x2(a.x, a.y) | ((uint32_t)pack_e5m2x2(b.x, b.y) << 16);
}

// A CTA takes tokens_per_cta tokens of K (blockIdx.y = 0) or V; a unit is 16
// bytes of the cache row, so every store is a full 16-byte one: 8 elements
// copied, or 16 elements (two loads) quantised.
template <int MODE, bool F16, bool FAST>
__global__ void __launch_bounds__(kWriteThreads) cache_write_kernel(const __grid_constant__ WriteParams p)
{
    const int t0 = blockIdx.x * p.tokens_per_cta;   // < num_tokens: fits an int
    const int n = min(p.tokens_per_cta, p.num_tokens - t0);
    const unsigned total = (unsigned)n * (unsigned)p.units;
    const int which = blockIdx.y;
    const uint8_t *src = p.src[which];
    uint8_t *dst = p.dst[which];
    const float scale = p.scale[which], r = __frcp_rn(scale);
    constexpr int kLoads = MODE == kWriteCopy ? 1 : 2;
    for (unsigned u0 = threadIdx.x; u0 < total; u0 += kWriteThreads * kWriteUnitsPerThread) {
        uint4 x[kWriteUnitsPerThread][kLoads];
        uint8_t *to[kWriteUnitsPerThread];
#pragma unroll
        for (int k = 0; k < kWriteUnitsPerThread; ++k) {
            const unsigned u = u0 + k * kWriteThreads;
            to[k] = nullptr;
            if (u < total) {
                const unsigned t = p.tokens_per_cta == 1 ? 0u : __umulhi(u, p.units_magic);   // u / units
                const unsigned c = u - t * (unsigned)p.units;
                const long long slot = p.slots[t0 + t];
                if (slot >= 0 && slot < p.num_slots) {
                    to[k] = dst + slot * p.row_bytes + (size_t)c * 16;
                    const uint8_t *from = src + (long long)(t0 + t) * p.stride[which] + (size_t)c * 16 * kLoads;
#pragma unroll
                    for (int i = 0; i < kLoads; ++i)
                        x[k][i] = ldg128_nc(from + 16 * i);
                } else if (slot >= 0 && p.status)
                    atomicOr(p.status, FD_DEVICE_STATUS_BAD_SLOT);
            }
        }
#pragma unroll
        for (int k = 0; k < kWriteUnitsPerThread; ++k) {
            if (!to[k])
                continue;
            uint4 y = x[k][0];
            if constexpr (MODE != kWriteCopy) {
                uint32_t y4[4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 w = x[k][i];
                    y4[2 * i] = quantise4<MODE, FAST>(x2_to_float2<F16>(w.x), x2_to_float2<F16>(w.y), scale, r);
                    y4[2 * i + 1] = quantise4<MODE, FAST>(x2_to_float2<F16>(w.z), x2_to_float2<F16>(w.w), scale, r);
                }
                y = make_uint4(y4[0], y4[1], y4[2], y4[3]);
            }
            *reinterpret_cast<uint4 *>(to[k]) = y;
        }
    }
}

template <bool FAST>
void launch_quantise(bool e4m3, bool f16, dim3 grid, cudaStream_t s, const WriteParams &p)
{
    if (e4m3 && f16)
        cache_write_kernel<kWriteE4m3, true, FAST><<<grid, kWriteThreads, 0, s>>>(p);
    else if (e4m3)
        cache_write_kernel<kWriteE4m3, false, FAST><<<grid, kWriteThreads, 0, s>>>(p);
    else if (f16)
        cache_write_kernel<kWriteE5m2, true, FAST><<<grid, kWriteThreads, 0, s>>>(p);
    else
        cache_write_kernel<kWriteE5m2, false, FAST><<<grid, kWriteThreads, 0, s>>>(p);
}

// ---------------------------------------------------------------- compact

constexpr int kMaxPath = 256;
constexpr int kCompactThreads = 128;
constexpr int kCompactBatch = 8;

struct CompactParams {
    uint8_t *cache[2];
    const int32_t *block_table, *seq_lens, *tree_lens, *accepted, *accept_lens;
    int32_t *seq_lens_out;
    unsigned int *status;
    long long row_bytes;
    int max_blocks, page_size, num_pages, tree_len, max_accept;
};

// Row of position t of request b, or -1 when its page is out of range.
__device__ __forceinline__ long long cache_row(const CompactParams &p, int b, int t)
{
    if (!p.block_table)
        return (long long)b * p.page_size + t;
    const unsigned blk = (unsigned)t / (unsigned)p.page_size;
    const int page = p.block_table[(long long)b * p.max_blocks + blk];
    return (unsigned)page < (unsigned)p.num_pages ? (long long)page * p.page_size + ((unsigned)t - blk * (unsigned)p.page_size) : -1;
}

// grid: (request, 2 KB column of the row, K or V).  A thread owns 16 bytes of
// every row and moves them down the path in order.  The path ascends, so row
// base + j is never read after it was written (accepted[i] >= i > j for the
// later i), and the next kCompactBatch rows can be loaded together before any
// of them is stored.
__global__ void __launch_bounds__(kCompactThreads) cache_compact_kernel(const __grid_constant__ CompactParams p)
{
    __shared__ long long s_src[kMaxPath], s_dst[kMaxPath];
    __shared__ int s_end;
    const int b = blockIdx.x, tid = threadIdx.x;
    const bool reports = blockIdx.y == 0 && blockIdx.z == 0;
    const int cap = p.block_table ? p.max_blocks * p.page_size : p.page_size;
    const int Lin = p.seq_lens[b], tin = p.tree_lens ? p.tree_lens[b] : p.tree_len, nin = p.accept_lens[b];
    const int L = min(max(Lin, 0), cap);
    const int t = min(min(max(tin, 0), p.tree_len), L);
    const int n = min(min(max(nin, 0), p.max_accept), t);
    const int base = L - t;
    if (tid == 0)
        s_end = n;
    __syncthreads();
    for (int j = tid; j < n; j += kCompactThreads) {
        const int32_t *path = p.accepted + (long long)b * p.max_accept;
        const int a = path[j];
        long long src = -1, dst = -1;
        if (a >= j && a < t && (j == 0 || a > path[j - 1])) {
            src = cache_row(p, b, base + a);
            dst = cache_row(p, b, base + j);
        }
        s_src[j] = src;
        s_dst[j] = dst;
        if (src < 0 || dst < 0)
            atomicMin(&s_end, j);
    }
    __syncthreads();
    const int end = s_end;
    if (reports && tid == 0) {
        p.seq_lens_out[b] = base + end;
        if (p.status) {
            unsigned int bits = 0;
            if (L != Lin || t != tin || n != nin)
                bits |= FD_DEVICE_STATUS_BAD_LENGTH;
            if (end != n)
                bits |= FD_DEVICE_STATUS_BAD_SLOT;
            if (bits)
                atomicOr(p.status, bits);
        }
    }
    const long long col = ((long long)blockIdx.y * kCompactThreads + tid) * 16;
    if (col >= p.row_bytes)
        return;
    uint8_t *cache = p.cache[blockIdx.z] + col;
    for (int j0 = 0; j0 < end; j0 += kCompactBatch) {
        uint4 x[kCompactBatch];
#pragma unroll
        for (int k = 0; k < kCompactBatch; ++k)
            if (j0 + k < end && s_src[j0 + k] != s_dst[j0 + k])
                x[k] = *reinterpret_cast<const uint4 *>(cache + s_src[j0 + k] * p.row_bytes);
#pragma unroll
        for (int k = 0; k < kCompactBatch; ++k)
            if (j0 + k < end && s_src[j0 + k] != s_dst[j0 + k])
                *reinterpret_cast<uint4 *>(cache + s_dst[j0 + k] * p.row_bytes) = x[k];
    }
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && na && nb && x < y + nb && y < x + na;
}

bool supported_head_dim(int d) { return d == 64 || d == 128 || d == 256; }

bool cache_options_valid(const fd_options *o)
{
    if (!o)
        return true;
    auto scale_ok = [](float x) { return x == 0.f || (x > 0.f && x < __builtin_huge_valf()); };
    return o->dtype >= 0 && o->dtype <= 1 && o->kv_dtype >= FD_KV_AS_Q && o->kv_dtype <= FD_KV_FP8_E5M2 &&
           scale_ok(o->k_scale) && scale_ok(o->v_scale);
}

long long pieces(long long n, long long size) { return (n + size - 1) / size; }

int device_sms()
{
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return sms;
}

}  // namespace
}  // namespace fd

using namespace fd;

extern "C" {

fd_status fd_build_tables(const int32_t *seq_lens, const int32_t *new_lens, const int32_t *held_pages,
                          const int32_t *free_pages, const int32_t *free_count, int max_free, int batch,
                          int page_size, int num_pages, int max_blocks_per_seq, int max_tokens,
                          int32_t *block_table, int64_t *slot_map, int32_t *cu_new_lens, int32_t *seq_lens_out,
                          int32_t *held_pages_out, int32_t *free_count_out, unsigned int *device_status,
                          fd_stream_t stream)
{
    if (batch < 0 || page_size <= 0 || num_pages <= 0 || max_blocks_per_seq <= 0 || max_tokens < 0 || max_free < 0)
        return FD_ERR_INVALID_ARG;
    if ((batch > 0 && (!seq_lens || !new_lens || !block_table || !seq_lens_out || !held_pages_out)) ||
        (max_free > 0 && !free_pages) || !free_count || (max_tokens > 0 && !slot_map) || !cu_new_lens ||
        !free_count_out)
        return FD_ERR_INVALID_ARG;
    const void *ins[] = {seq_lens, new_lens, held_pages, free_pages, free_count, block_table, cu_new_lens,
                         seq_lens_out, held_pages_out, free_count_out, device_status};
    for (const void *q : ins)
        if (q && !aligned(q, 4))
            return FD_ERR_INVALID_ARG;
    if (slot_map && !aligned(slot_map, 8))
        return FD_ERR_INVALID_ARG;
    if (batch > kMaxBatch || (long long)max_blocks_per_seq * page_size >= (1ll << 31) ||
        (long long)batch * max_blocks_per_seq >= (1ll << 31))
        return FD_ERR_UNSUPPORTED;
    // the outputs are written while other CTAs may still read the inputs
    struct Range { const void *p; size_t n; };
    const size_t nb = 4 * (size_t)batch;
    const Range in[] = {{seq_lens, nb}, {new_lens, nb}, {held_pages, nb}, {free_pages, 4 * (size_t)max_free}, {free_count, 4}};
    const Range out[] = {{block_table, 4 * (size_t)batch * max_blocks_per_seq}, {slot_map, 8 * (size_t)max_tokens},
                         {cu_new_lens, nb + 4}, {seq_lens_out, nb}, {held_pages_out, nb}, {free_count_out, 4}};
    for (int i = 0; i < 6; ++i) {
        for (const Range &r : in)
            if (overlap(out[i].p, out[i].n, r.p, r.n))
                return FD_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n))
                return FD_ERR_INVALID_ARG;
    }
    const int sms = device_sms();
    if (sms <= 0)
        return FD_ERR_CUDA;
    TablesParams p;
    p.seq_lens = seq_lens;
    p.new_lens = new_lens;
    p.held_pages = held_pages;
    p.free_pages = free_pages;
    p.free_count = free_count;
    p.max_free = max_free;
    p.batch = batch;
    p.page_size = page_size;
    p.page_shift = (page_size & (page_size - 1)) == 0 ? __builtin_ctz((unsigned)page_size) : -1;
    p.num_pages = num_pages;
    p.max_blocks = max_blocks_per_seq;
    p.max_tokens = max_tokens;
    p.block_table = block_table;
    p.slot_map = slot_map;
    p.cu_new_lens = cu_new_lens;
    p.seq_lens_out = seq_lens_out;
    p.held_out = held_pages_out;
    p.free_out = free_count_out;
    p.status = device_status;
    const long long want = pieces(max_tokens, kTablesThreads * kTablesTokensPerThread);
    const int grid = (int)(want < 1 ? 1 : want > kTablesCtasPerSm * sms ? kTablesCtasPerSm * sms : want);
    // beside the kernel's static part, large batches only: the limit is the
    // largest batch's, so that no call lowers it under another thread's launch
    const size_t smem = tables_smem(batch);
    if (smem > 48 * 1024 - 256 &&
        cudaFuncSetAttribute(build_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)tables_smem(kMaxBatch)) != cudaSuccess)
        return FD_ERR_CUDA;
    build_tables_kernel<<<grid, kTablesThreads, smem, reinterpret_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

fd_status fd_cache_write(const void *k_new, const void *v_new, long long k_stride, long long v_stride,
                         const int64_t *slot_map, int num_tokens, int num_kv_heads, int head_dim, void *k_cache,
                         void *v_cache, long long num_slots, const fd_options *opts, unsigned int *device_status,
                         fd_stream_t stream)
{
    if (num_tokens < 0 || num_kv_heads <= 0 || num_slots < 0 || !cache_options_valid(opts))
        return FD_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim) || num_kv_heads > (1 << 20))
        return FD_ERR_UNSUPPORTED;
    if (num_tokens == 0)
        return FD_OK;
    const long long row = (long long)num_kv_heads * head_dim;
    if (!k_new || !v_new || !slot_map || (num_slots > 0 && (!k_cache || !v_cache)) || !aligned(k_new, 16) ||
        !aligned(v_new, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(slot_map, 8) ||
        (device_status && !aligned(device_status, 4)))
        return FD_ERR_INVALID_ARG;
    if (num_tokens > 1 && (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8))
        return FD_ERR_INVALID_ARG;
    const int kv = opts ? opts->kv_dtype : FD_KV_AS_Q;
    const bool f16 = opts && opts->dtype == FD_DTYPE_F16;
    WriteParams p;
    p.src[0] = static_cast<const uint8_t *>(k_new);
    p.src[1] = static_cast<const uint8_t *>(v_new);
    p.stride[0] = num_tokens > 1 ? 2 * k_stride : 0;
    p.stride[1] = num_tokens > 1 ? 2 * v_stride : 0;
    p.dst[0] = static_cast<uint8_t *>(k_cache);
    p.dst[1] = static_cast<uint8_t *>(v_cache);
    p.scale[0] = opts && opts->k_scale != 0.f ? opts->k_scale : 1.f;
    p.scale[1] = opts && opts->v_scale != 0.f ? opts->v_scale : 1.f;
    p.slots = slot_map;
    p.status = device_status;
    p.num_slots = num_slots;
    p.row_bytes = row * (kv == FD_KV_AS_Q ? 2 : 1);
    p.num_tokens = num_tokens;
    p.units = (int)(p.row_bytes / 16);
    p.units_magic = (unsigned int)((1ull << 32) / (unsigned)p.units) + 1u;
    const int per_pass = kWriteThreads * kWriteUnitsPerThread;
    p.tokens_per_cta = p.units >= per_pass ? 1 : per_pass / p.units;
    const dim3 grid((unsigned)pieces(num_tokens, p.tokens_per_cta), 2);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto fast = [](float x) { return x >= 0x1p-60f && x <= 0x1p60f; };
    if (kv == FD_KV_AS_Q)
        cache_write_kernel<kWriteCopy, false, true><<<grid, kWriteThreads, 0, s>>>(p);
    else if (fast(p.scale[0]) && fast(p.scale[1]))
        launch_quantise<true>(kv == FD_KV_FP8_E4M3, f16, grid, s, p);
    else
        launch_quantise<false>(kv == FD_KV_FP8_E4M3, f16, grid, s, p);
    return cudaGetLastError() == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

fd_status fd_cache_compact(void *k_cache, void *v_cache, const int32_t *block_table, int max_blocks_per_seq,
                           int page_size, int num_pages, const int32_t *seq_lens, const int32_t *tree_lens,
                           int tree_len, const int32_t *accepted, const int32_t *accept_lens, int max_accept,
                           int batch, int num_kv_heads, int head_dim, int32_t *seq_lens_out, const fd_options *opts,
                           unsigned int *device_status, fd_stream_t stream)
{
    if (batch < 0 || num_kv_heads <= 0 || page_size <= 0 || tree_len <= 0 || max_accept <= 0 ||
        !cache_options_valid(opts) || (block_table && (max_blocks_per_seq <= 0 || num_pages <= 0)))
        return FD_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim) || batch > kMaxBatch || tree_len > kMaxPath || max_accept > kMaxPath ||
        num_kv_heads > (1 << 20) || (block_table && (long long)max_blocks_per_seq * page_size >= (1ll << 31)))
        return FD_ERR_UNSUPPORTED;
    if (batch == 0)
        return FD_OK;
    if (!k_cache || !v_cache || !seq_lens || !accepted || !accept_lens || !seq_lens_out || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16))
        return FD_ERR_INVALID_ARG;
    const void *ints[] = {block_table, seq_lens, tree_lens, accepted, accept_lens, seq_lens_out, device_status};
    for (const void *q : ints)
        if (q && !aligned(q, 4))
            return FD_ERR_INVALID_ARG;
    const size_t nb = 4 * (size_t)batch;
    if (overlap(seq_lens_out, nb, seq_lens, nb) || overlap(seq_lens_out, nb, tree_lens, nb) ||
        overlap(seq_lens_out, nb, accept_lens, nb) || overlap(seq_lens_out, nb, accepted, nb * max_accept))
        return FD_ERR_INVALID_ARG;
    const bool fp8 = opts && opts->kv_dtype != FD_KV_AS_Q;
    CompactParams p;
    p.cache[0] = static_cast<uint8_t *>(k_cache);
    p.cache[1] = static_cast<uint8_t *>(v_cache);
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.tree_lens = tree_lens;
    p.accepted = accepted;
    p.accept_lens = accept_lens;
    p.seq_lens_out = seq_lens_out;
    p.status = device_status;
    p.row_bytes = (long long)num_kv_heads * head_dim * (fp8 ? 1 : 2);
    p.max_blocks = max_blocks_per_seq;
    p.page_size = page_size;
    p.num_pages = num_pages;
    p.tree_len = tree_len;
    p.max_accept = max_accept;
    const long long cols = pieces(p.row_bytes, kCompactThreads * 16);
    if (cols > 65535)
        return FD_ERR_UNSUPPORTED;
    cache_compact_kernel<<<dim3((unsigned)batch, (unsigned)cols, 2), kCompactThreads, 0,
                           reinterpret_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

}  // extern "C"
