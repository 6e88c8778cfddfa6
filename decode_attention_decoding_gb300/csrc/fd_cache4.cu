// fd_cache4.cu -- rows into a 4-bit cache and back (fd_cache_write4,
// fd_cache_read4).
//
// A row's 16 consecutive dims are a block with an E4M3 scale s; an element is
// code * s * t, code in E2M1 and t the tensor's scale.  Both calls move 2 + 9/16
// bytes an element.  A thread has one block of K or V: 32 bytes of a 16-bit
// row, 8 bytes of codes and the scale's byte.
//
// What bounds them (GB300, 32768 rows of 8 heads of 128 dims, 172 MB, 25.4 us
// at a copy's rate; written 37, read 34 to 35): the instructions, then latency.
// The schedulers issue in 74% of the write's cycles and 60% of the read's, and
// the memory moves little more than it must: written, 138 MB read and 26
// written (134 and 38, the rest still in L2); read, 60 MB read and 77 written
// (38 and 134).  The slots' order hardly matters: random, whole pages at random
// and in order 37.1, 37.2 and 37.0 written, 35.5, 34.4 and 33.8 read.
#include <cstdint>

#include <cuda_runtime.h>

#include "fd.h"
#include "fd_device.cuh"

namespace fd {
namespace {

struct Cache4Params {
    const int64_t *slots;
    unsigned int *status;
    uint8_t *codes[2], *scales[2];    // K and V: [pages, hkv, page, D / 2] and [.., D / 16]
    uint8_t *rows[2];                 // 16-bit rows, read or written
    long long stride[2];              // bytes between token rows
    float scale[2];
    long long num_slots;
    int num_tokens, tokens_per_cta, hkv, page_size;
    int blocks_log2;                  // blocks of a kv head's row: D / 16
    int units;                        // blocks of a token: hkv * D / 16
    unsigned int units_magic;         // floor(2^32 / units) + 1: __umulhi(x, magic) = x / units for x * units < 2^32
    int page_shift;                   // page_size = 2^page_shift, or -1
    int wide;                         // rows of 32-byte pieces: base and stride are multiples of 32
};

// Measured on GB300 (32768 rows of 8 heads into random slots, and back; us): 128 threads with one block each 35.5 and
// 33.5; two blocks a thread 35.9 and 34.2, four 37.1 and 40.6; 256 threads 35.7 and 34.2, 64 35.7 and 35.9.  With these at 37.1
// and 35.5: two 16-byte accesses in place of one of 32 bytes (rows that 32 bytes do not divide) 37.6 and
// 37.5, in order 37.2 and 38.6; rows read after their slots 38.1 written.
constexpr int kCache4Threads = 128;

// 32 bytes of a row, as one access where they are aligned.
__device__ __forceinline__ void load_piece(const uint8_t *p, bool wide, uint32_t (&w)[8])
{
    if (wide) {
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(p));
    } else {
        const uint4 a = ldg128_nc(p), b = ldg128_nc(p + 16);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w; w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
}
__device__ __forceinline__ void store_piece(uint8_t *p, bool wide, const uint32_t (&w)[8])
{
    if (wide)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                     "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    else {
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4 *>(p + 16) = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

__device__ __forceinline__ uint32_t pack_e2m1x8(const float (&x)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}
__device__ __forceinline__ void e2m1x2_to_f16x2(uint32_t w, uint32_t (&r)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}
template <bool F16>
__device__ __forceinline__ uint32_t max_nan_x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    if constexpr (F16)
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// One block of a row: 16 elements, two a word, to 8 bytes of codes and a scale.
template <bool F16>
__device__ __forceinline__ uint2 quantise_block(const uint32_t (&w)[8], float t, uint32_t *scale_code)
{
    uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 8; ++i)
        m = max_nan_x2<F16>(m, w[i] & 0x7FFF7FFFu);
    const float top = x2_to_float2<F16>(max_nan_x2<F16>(m, m >> 16)).x;
    const uint32_t code = pack_e4m3x2(__fdiv_rn(top, 6.f * t), 0.f) & 0xFFu;
    *scale_code = code;
    const float unit = fp8x2_to_float2<kKvE4m3>((uint16_t)code).x * t;
    if (!(unit > 0.f))   // 0, or NaN
        return make_uint2(0u, 0u);
    uint32_t out[2];
    if (code < 0x7Eu && unit >= 0x1p-60f && unit <= 0x1p60f) {
        // below the largest scale the quotients are finite, so this is quotient<true> without its limits: at most 6.4, 9 where s is
        // subnormal and rounded down by a third; the conversion saturates
        const float r = __frcp_rn(unit);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 x2 = x2_to_float2<F16>(w[4 * h + i / 2]);
                const float x = i % 2 ? x2.y : x2.x, q = x * r;
                y[i] = copysignf(fmaf(fmaf(-q, unit, x), r, q), x);
            }
            out[h] = pack_e2m1x8(y);
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float y[8];
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                const float2 x = x2_to_float2<F16>(w[4 * h + i]);
                y[2 * i] = quotient<false>(x.x, unit, 0.f);
                y[2 * i + 1] = quotient<false>(x.y, unit, 0.f);
            }
            out[h] = pack_e2m1x8(y);
        }
    }
    return make_uint2(out[0], out[1]);
}

// A CTA takes tokens_per_cta tokens of K (blockIdx.y = 0) or V.
template <bool WRITE, bool F16>
__global__ void __launch_bounds__(kCache4Threads) cache4_kernel(const __grid_constant__ Cache4Params p)
{
    const int t0 = blockIdx.x * p.tokens_per_cta, n = min(p.tokens_per_cta, p.num_tokens - t0);
    const unsigned total = (unsigned)n * (unsigned)p.units;
    const int which = blockIdx.y;
    const float scale = p.scale[which];
    uint8_t *all_codes = p.codes[which], *all_scales = p.scales[which], *rows = p.rows[which];
    const long long stride = p.stride[which];
    for (unsigned u = threadIdx.x; u < total; u += kCache4Threads) {
        const unsigned t = p.tokens_per_cta == 1 ? 0u : __umulhi(u, p.units_magic);   // u / units
        const unsigned unit = u - t * (unsigned)p.units, h = unit >> p.blocks_log2, in = unit & ((1u << p.blocks_log2) - 1);
        const long long slot = p.slots[t0 + t];
        uint8_t *row = rows + (long long)(t0 + t) * stride + (size_t)unit * 32;
        uint32_t x[8];
        if constexpr (WRITE)   // read while the slot is on its way
            load_piece(row, p.wide, x);
        if (slot < 0 || slot >= p.num_slots) {
            if (slot >= 0 && p.status)
                atomicOr(p.status, FD_DEVICE_STATUS_BAD_SLOT);
            continue;
        }
        const long long page = p.page_shift >= 0 ? slot >> p.page_shift
                               : slot >> 32 == 0 ? (long long)((unsigned)slot / (unsigned)p.page_size) : slot / p.page_size;
        const long long at = (((page * p.hkv + h) * p.page_size + (slot - page * p.page_size)) << p.blocks_log2) + in;   // the block's place
        if constexpr (WRITE) {
            uint32_t code;
            *reinterpret_cast<uint2 *>(all_codes + at * 8) = quantise_block<F16>(x, scale, &code);
            all_scales[at] = (uint8_t)code;
        } else {
            const uint2 codes = *reinterpret_cast<const uint2 *>(all_codes + at * 8);
            const float s = fp8x2_to_float2<kKvE4m3>((uint16_t)all_scales[at]).x;
            const uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t f[4];
                e2m1x2_to_f16x2(w[i], f);
                // code * s is exact; the product with t is rounded to fp32, and that to 16 bits
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 y = f16x2_to_float2(f[e]);
                    x[4 * i + e] = pack_x2<F16>(y.x * s * scale, y.y * s * scale);
                }
            }
            store_piece(row, p.wide, x);
        }
    }
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool scale_ok(float x) { return x == 0.f || (x > 0.f && x < __builtin_huge_valf()); }

// Both calls: checks and launch.
template <bool WRITE>
fd_status run(const fd_cache4 *cache, int page_size, long long num_slots, const void *k, const void *v, long long k_stride,
              long long v_stride, const int64_t *slot_map, int num_tokens, int hkv, int head_dim, const fd_options *opts,
              unsigned int *device_status, fd_stream_t stream)
{
    if (!cache || num_tokens < 0 || hkv <= 0 || num_slots < 0 || page_size <= 0 || num_slots % page_size ||
        (opts && (opts->dtype < 0 || opts->dtype > 1 || opts->kv_dtype != FD_KV_AS_Q || !scale_ok(opts->k_scale) || !scale_ok(opts->v_scale))))
        return FD_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || hkv > (1 << 20))
        return FD_ERR_UNSUPPORTED;
    if (num_tokens == 0)
        return FD_OK;
    const long long row = (long long)hkv * head_dim;
    const void *tensors[] = {cache->k_codes, cache->k_scales, cache->v_codes, cache->v_scales};
    for (const void *t : tensors)
        if ((num_slots > 0 && !t) || !aligned(t, 16))
            return FD_ERR_INVALID_ARG;
    if (!k || !v || !slot_map || !aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 8) || !aligned(device_status, 4))
        return FD_ERR_INVALID_ARG;
    if (num_tokens > 1 && (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8))
        return FD_ERR_INVALID_ARG;
    Cache4Params p;
    p.slots = slot_map;
    p.status = device_status;
    p.codes[0] = cache->k_codes;
    p.codes[1] = cache->v_codes;
    p.scales[0] = cache->k_scales;
    p.scales[1] = cache->v_scales;
    p.rows[0] = static_cast<uint8_t *>(const_cast<void *>(k));
    p.rows[1] = static_cast<uint8_t *>(const_cast<void *>(v));
    p.stride[0] = num_tokens > 1 ? 2 * k_stride : 0;
    p.stride[1] = num_tokens > 1 ? 2 * v_stride : 0;
    p.scale[0] = opts && opts->k_scale != 0.f ? opts->k_scale : 1.f;
    p.scale[1] = opts && opts->v_scale != 0.f ? opts->v_scale : 1.f;
    p.num_slots = num_slots;
    p.num_tokens = num_tokens;
    p.hkv = hkv;
    p.page_size = page_size;
    p.blocks_log2 = head_dim == 64 ? 2 : head_dim == 128 ? 3 : 4;
    p.units = hkv << p.blocks_log2;
    p.units_magic = (unsigned int)((1ull << 32) / (unsigned)p.units) + 1u;
    p.page_shift = (page_size & (page_size - 1)) == 0 ? __builtin_ctz((unsigned)page_size) : -1;
    p.wide = aligned(k, 32) && aligned(v, 32) && p.stride[0] % 32 == 0 && p.stride[1] % 32 == 0;
    p.tokens_per_cta = p.units >= kCache4Threads ? 1 : kCache4Threads / p.units;
    const dim3 grid((unsigned)((num_tokens + (long long)p.tokens_per_cta - 1) / p.tokens_per_cta), 2);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (opts && opts->dtype == FD_DTYPE_F16)
        cache4_kernel<WRITE, true><<<grid, kCache4Threads, 0, s>>>(p);
    else
        cache4_kernel<WRITE, false><<<grid, kCache4Threads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? FD_OK : FD_ERR_CUDA;
}

}  // namespace
}  // namespace fd

using namespace fd;

extern "C" {

fd_status fd_cache_write4(const void *k_new, const void *v_new, long long k_stride, long long v_stride,
                          const int64_t *slot_map, int num_tokens, int num_kv_heads, int head_dim,
                          const fd_cache4 *cache, int page_size, long long num_slots, const fd_options *opts,
                          unsigned int *device_status, fd_stream_t stream)
{
    return run<true>(cache, page_size, num_slots, k_new, v_new, k_stride, v_stride, slot_map, num_tokens, num_kv_heads, head_dim, opts,
                     device_status, stream);
}

fd_status fd_cache_read4(const int64_t *slot_map, int num_tokens, int num_kv_heads, int head_dim, const fd_cache4 *cache,
                         int page_size, long long num_slots, void *k_out, void *v_out, long long k_stride,
                         long long v_stride, const fd_options *opts, unsigned int *device_status, fd_stream_t stream)
{
    return run<false>(cache, page_size, num_slots, k_out, v_out, k_stride, v_stride, slot_map, num_tokens, num_kv_heads, head_dim, opts,
                      device_status, stream);
}

}  // extern "C"
