// fd_cache4.cu -- rows into a 4-bit cache and back (fd_cache_write4,
// fd_cache_read4).
//
// A row's 16 consecutive dims are a block with an E4M3 scale s; an element is
// code * s * t, code in E2M1 and t the tensor's scale.  Both calls move 2 + 9/16
// bytes an element and are bound by that.  A thread has one block of K or V:
// 32 bytes of a 16-bit row, 8 bytes of codes and the scale's byte.
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
};

constexpr int kCache4Threads = 256;
constexpr int kCache4Units = 2;   // blocks a thread has in flight

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
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// One block of a row: 16 fp32 values to 8 bytes of codes and a scale.
__device__ __forceinline__ uint2 quantise_block(const float (&x)[16], float t, uint32_t *scale_code)
{
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        top = max_nan(top, fabsf(x[i]));
    const uint32_t code = pack_e4m3x2(__fdiv_rn(top, 6.f * t), 0.f) & 0xFFu;
    *scale_code = code;
    const float unit = fp8x2_to_float2<kKvE4m3>((uint16_t)code).x * t;
    if (!(unit > 0.f))   // 0, or NaN
        return make_uint2(0u, 0u);
    float y[2][8];
    if (unit >= 0x1p-60f && unit <= 0x1p60f) {
        const float r = __frcp_rn(unit);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            y[i / 8][i % 8] = quotient<true>(x[i], unit, r);
    } else {
#pragma unroll 1
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y[h][i] = quotient<false>(x[8 * h + i], unit, 0.f);
    }
    return make_uint2(pack_e2m1x8(y[0]), pack_e2m1x8(y[1]));
}

// A CTA takes tokens_per_cta tokens of K (blockIdx.y = 0) or V.
template <bool WRITE, bool F16>
__global__ void __launch_bounds__(kCache4Threads) cache4_kernel(const __grid_constant__ Cache4Params p)
{
    const int t0 = blockIdx.x * p.tokens_per_cta, n = min(p.tokens_per_cta, p.num_tokens - t0);
    const unsigned total = (unsigned)n * (unsigned)p.units;
    const int which = blockIdx.y;
    const float scale = p.scale[which];
    for (unsigned u0 = threadIdx.x; u0 < total; u0 += kCache4Threads * kCache4Units) {
        uint4 x[kCache4Units][2];
        uint2 codes[kCache4Units];
        uint32_t s[kCache4Units];
        long long blk[kCache4Units];      // the block's place in the cache, or -1
        uint8_t *row[kCache4Units];
#pragma unroll
        for (int k = 0; k < kCache4Units; ++k) {
            const unsigned u = u0 + k * kCache4Threads;
            blk[k] = -1;
            if (u < total) {
                const unsigned t = u / (unsigned)p.units, c = u - t * (unsigned)p.units;
                const long long slot = p.slots[t0 + t];
                if (slot >= 0 && slot < p.num_slots) {
                    const unsigned h = c >> p.blocks_log2, in = c & ((1u << p.blocks_log2) - 1);
                    const long long page = slot < (1ll << 32) ? (long long)((unsigned)slot / (unsigned)p.page_size) : slot / p.page_size;
                    const long long at = (page * p.hkv + h) * p.page_size + (slot - page * p.page_size);
                    blk[k] = (at << p.blocks_log2) + in;
                    row[k] = p.rows[which] + (long long)(t0 + t) * p.stride[which] + (size_t)c * 32;
                    if constexpr (WRITE) {
                        x[k][0] = ldg128_nc(row[k]);
                        x[k][1] = ldg128_nc(row[k] + 16);
                    } else {
                        codes[k] = *reinterpret_cast<const uint2 *>(p.codes[which] + blk[k] * 8);
                        s[k] = p.scales[which][blk[k]];
                    }
                } else if (slot >= 0 && p.status)
                    atomicOr(p.status, FD_DEVICE_STATUS_BAD_SLOT);
            }
        }
#pragma unroll
        for (int k = 0; k < kCache4Units; ++k) {
            if (blk[k] < 0)
                continue;
            if constexpr (WRITE) {
                float v[16];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t w[4] = {x[k][i].x, x[k][i].y, x[k][i].z, x[k][i].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 y = x2_to_float2<F16>(w[e]);
                        v[8 * i + 2 * e] = y.x;
                        v[8 * i + 2 * e + 1] = y.y;
                    }
                }
                uint32_t code;
                *reinterpret_cast<uint2 *>(p.codes[which] + blk[k] * 8) = quantise_block(v, scale, &code);
                p.scales[which][blk[k]] = (uint8_t)code;
            } else {
                const float sc = fp8x2_to_float2<kKvE4m3>((uint16_t)s[k]).x;
                const uint32_t w[2] = {codes[k].x, codes[k].y};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t f[4];
                    e2m1x2_to_f16x2(w[i], f);
                    // code * s is exact; the product with t is rounded to fp32, and that to 16 bits
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 y = f16x2_to_float2(f[e]);
                        f[e] = pack_x2<F16>(y.x * sc * scale, y.y * sc * scale);
                    }
                    *reinterpret_cast<uint4 *>(row[k] + 16 * i) = make_uint4(f[0], f[1], f[2], f[3]);
                }
            }
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
    const int per_pass = kCache4Threads * kCache4Units;
    p.tokens_per_cta = p.units >= per_pass ? 1 : per_pass / p.units;
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
