// fd_window_kernel.cuh -- split kernel of the window attention (fd_window.cuh).
//
// Every warp is a worker of its own: it takes a run of tiles of the schedule
// (fd_sched.h), copies their rows into a ring of its own with cp.async, and
// multiplies with warp MMAs; nothing but the end of the kernel synchronises
// the warps of a CTA.
//
//   S^T = K Q^T     A: 16 rows of K, B: 8 query columns
//   O^T += V^T P^T  A: 16 dims of V^T, B: the weights of 16 rows
//
// So every lane has rows and dims of its own, whatever the cache's type, and
// the conversion of FP8 and 4-bit codes works on the words as they lie in
// shared memory: of K, lane (g, c) holds the pieces c, c + 4, .. of rows
// window_row(g) and + 8, any four elements of which are its part of a k step
// (the query's dims are permuted to match); of V, the pieces g, g + 8, .. of
// rows c, 4 + (c ^ 1), 8 + c, 12 + (c ^ 1), whose elements are paired row by
// row, for 4-bit codes before they are converted, eight at a time.
//
// An E2M1 code times its E4M3 scale has 6 significant bits and is an fp16
// value, so K and V of a 4-bit cache enter the MMAs exactly.
#pragma once

#include <atomic>

#include "fd_window.cuh"

namespace fd {

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Copy BYTES from src, or write zeros (size 0).
template <int BYTES>
__device__ __forceinline__ void cp_async_or_zero(uint32_t dst, const void *src, uint32_t size, uint64_t policy)
{
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(size), "l"(policy)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global.L2::cache_hint [%0], [%1], %4, %2, %3;" ::"r"(dst), "l"(src), "r"(size), "l"(policy),
                     "n"(BYTES)
                     : "memory");
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

// The four bytes of w, each two E2M1 codes (the first in the low half), as
// four pairs of fp16.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&r)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <bool F16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
{
    uint32_t r;
    if constexpr (F16)
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Two fp32 values rounded towards zero to 16 bits.
template <bool F16>
__device__ __forceinline__ uint32_t pack_rz_x2(float lo, float hi)
{
    uint32_t r;
    if constexpr (F16)
        asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Row of a 16-row tile that MMA row (and k index) g < 8 stands for; g + 8: 8
// more.  The rows of k indices 2c are four in a row, and so are those of 2c +
// 1, and the rows of k indices 2c, 2c + 1 differ in parity: with the swizzle
// below every load of K or V from shared memory is free of bank conflicts
// (except K rows of 32 bytes: two lanes a bank).
__device__ __forceinline__ int window_row(int g) { return g & 1 ? 4 + ((g >> 1) ^ 1) : g >> 1; }
// Piece x of row r lies at piece x ^ window_swizzle(r).
template <int GRAN>
__device__ __forceinline__ int window_swizzle(int r) { return (((r & 1) << 2) | (r & 2)) & (GRAN - 1); }

// One warp's place in the schedule.
struct WindowCursor {
    int b, h, j, nb;     // request, launch head, tile of the segment, tiles of a segment
    WindowReq req;
};

template <class C, int NT, bool PACK>
struct WindowWarp {
    static constexpr int D = C::D, KV = C::KV, kTile = C::kTile, kRow = C::kRow, kGran = C::kGran;
    static constexpr int KT = kTile / 16;          // k steps of a tile
    static constexpr int kSteps = D / 16;          // k steps of a row, and 16-dim blocks of the output
    static constexpr int kParts = PACK ? 1 : C::kParts;   // MMAs a block (PACK: both parts in one)
    static constexpr float kShift = C::kShift;
    static constexpr int kColMask = PACK ? 3 : 8 * NT - 1;

    uint32_t qf[NT][kSteps][2];
    float mult[NT][2];         // score of column 2c, 2c + 1 of an MMA's eight -> log2 units
    float acc[kSteps][NT][4];
    float m[NT][2], l[NT][2];

    // Load the query of segment (b, head) as the B operand of S^T.
    __device__ __forceinline__ void start(const WindowParams &p, int b, int head, int g, int c)
    {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int col = (nt * 8 + g) & kColMask;
            const int i = col / p.group;
            const bool real = col < p.cols;
            const uint16_t *src = p.q + ((long long)(b * p.q_len + (real ? i : 0)) * p.hq + head * p.group + (real ? col - i * p.group : 0)) * D;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                // elements of a piece, and the lane's four in step s
                constexpr int kEl = kRow >= 64 ? 16 * D / kRow : 16, kPer = kEl / 4;
                const int dim = (c + 4 * (s / kPer)) * kEl + 4 * (s % kPer);
                uint2 w = make_uint2(0u, 0u);
                if (real)
                    w = *reinterpret_cast<const uint2 *>(src + dim);
                qf[nt][s][0] = w.x;
                qf[nt][s][1] = w.y;
            }
            float f = p.scale_log2;
            if (KV >= kKvE4m3 && !p.q_f16) {
                // bf16 as fp16 times a power of two: the row's largest element goes to [2^14, 2^15), so that
                // what fp16 cannot hold is below 2^-39 of it
                float top = 0.f;
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 x = bf16x2_to_float2(qf[nt][s][e]);
                        top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
                    }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                int e = ((int)(__float_as_uint(top) >> 23) & 255) - 127;     // top in [2^e, 2^(e + 1))
                e = top > 0.f && e < 128 ? min(max(14 - e, -126), 126) : 0;
                const float up = __uint_as_float((uint32_t)(e + 127) << 23), down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const float2 x = bf16x2_to_float2(qf[nt][s][w]);
                        qf[nt][s][w] = pack_f16x2(x.x * up, x.y * up);
                    }
                f *= down;
            }
            mult[nt][0] = __shfl_sync(0xffffffffu, f, 8 * c);
            mult[nt][1] = __shfl_sync(0xffffffffu, f, 8 * c + 4);
            m[nt][0] = m[nt][1] = -__builtin_huge_valf();
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[s][nt][e] = 0.f;
        }
    }

    // S^T of a tile in log2 units: sc[kt][nt] = rows window_row(g), + 8 of 16-row step kt times columns 2c, 2c + 1.
    __device__ __forceinline__ void scores(uint32_t k, uint32_t ks, int g, int c, float (&sc)[KT][NT][4]) const
    {
        const int r = window_row(g), sw = window_swizzle<kGran>(r);
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sc[kt][nt][e] = 0.f;
            constexpr int kPieces = kRow >= 64 ? kRow / 64 : 1, kWords = kRow >= 64 ? 4 : 2;
#pragma unroll
            for (int x = 0; x < kPieces; ++x) {
                uint32_t a[2][4], s16[2][2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t row = (uint32_t)(kt * 16 + r + 8 * i);
                    if constexpr (kRow >= 64) {
                        const uint4 w = lds128(k + row * kRow + (((c + 4 * x) ^ sw) << 4));
                        a[i][0] = w.x; a[i][1] = w.y; a[i][2] = w.z; a[i][3] = w.w;
                    } else {
                        const uint2 w = lds64(k + row * kRow + 8 * c);
                        a[i][0] = w.x; a[i][1] = w.y;
                    }
                    if constexpr (C::kFp4) {
                        if constexpr (kRow >= 64) {
                            const uint32_t b = fp8x2_to_f16x2<kKvE4m3>((uint16_t)lds16(ks + row * C::kScaleRow + 2 * (c + 4 * x)));
                            s16[i][0] = prmt(b, b, 0x1010);
                            s16[i][1] = prmt(b, b, 0x3232);
                        } else {
                            const uint32_t b = fp8x2_to_f16x2<kKvE4m3>((uint16_t)lds8(ks + row * C::kScaleRow + c));
                            s16[i][0] = prmt(b, b, 0x1010);
                        }
                    }
                }
                if constexpr (C::kFp4) {
#pragma unroll
                    for (int w = 0; w < kWords; ++w) {
                        uint32_t f[2][4];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            e2m1x8_to_f16x2(a[i][w], f[i]);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                f[i][e] = hmul2(f[i][e], s16[i][w / 2]);
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int s = (x * kWords + w) * 2 + e;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_16816<C::kF16>(sc[kt][nt], f[0][2 * e], f[1][2 * e], f[0][2 * e + 1], f[1][2 * e + 1], qf[nt][s][0], qf[nt][s][1]);
                        }
                    }
                } else if constexpr (C::kFp8) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t a0 = fp8x2_to_f16x2<KV>(lo16(a[0][w])), a1 = fp8x2_to_f16x2<KV>(lo16(a[1][w]));
                        const uint32_t a2 = fp8x2_to_f16x2<KV>(hi16(a[0][w])), a3 = fp8x2_to_f16x2<KV>(hi16(a[1][w]));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_16816<C::kF16>(sc[kt][nt], a0, a1, a2, a3, qf[nt][x * 4 + w][0], qf[nt][x * 4 + w][1]);
                    }
                } else {
#pragma unroll
                    for (int w = 0; w < 2; ++w)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_16816<C::kF16>(sc[kt][nt], a[0][2 * w], a[1][2 * w], a[0][2 * w + 1], a[1][2 * w + 1],
                                               qf[nt][x * 2 + w][0], qf[nt][x * 2 + w][1]);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sc[kt][nt][e] *= mult[nt][e & 1];
        }
    }

    // Hide what a column's token does not see in the tile from row `row0` of the request.
    __device__ __forceinline__ void mask(const WindowParams &p, const WindowReq &req, int row0, int g, int c, float (&sc)[KT][NT][4]) const
    {
        const int r = window_row(g);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = ((nt * 8 + 2 * c + e) & kColMask) / p.group;
                const int own = req.L - p.q_len + min(i, p.q_len - 1);
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                    for (int a = 0; a < 2; ++a)
                        if (!visible(p, req, row0 + kt * 16 + r + 8 * a, own))
                            sc[kt][nt][2 * a + e] = -__builtin_huge_valf();
            }
    }
    // Whether the token at position `own` sees row v of the request.
    __device__ __forceinline__ static bool visible(const WindowParams &p, const WindowReq &req, int v, int own)
    {
        const int pos = window_pos(req, v);
        return v < req.rows && pos <= own && (!p.window || pos < p.sinks || own - pos < p.window);
    }

    // The scores' softmax weights against the running maximum, in parts, as the B operand of O^T: pf[kt][part][nt][2];
    // alpha: the factor of what was summed before.
    __device__ __forceinline__ void weights(float (&sc)[KT][NT][4], int c, uint32_t (&pf)[KT][kParts][NT][2], float (&alpha)[NT][2])
    {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float ref[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float top = -__builtin_huge_valf();
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    top = fmaxf(top, fmaxf(sc[kt][nt][e], sc[kt][nt][e + 2]));
                }
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                const float now = fmaxf(m[nt][e], top);
                ref[e] = now == -__builtin_huge_valf() ? 0.f : now;
                // at least fp32's least normal number: an infinite sum stays infinite
                alpha[nt][e] = fmaxf(exp2_approx(m[nt][e] - ref[e]), 1.1754944e-38f);
                m[nt][e] = now;
                l[nt][e] *= alpha[nt][e];
                ref[e] -= kShift;
            }
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    float x = exp2_approx(sc[kt][nt][2 * a] - ref[0]), y = exp2_approx(sc[kt][nt][2 * a + 1] - ref[1]);
                    l[nt][0] += x;
                    l[nt][1] += y;
                    if constexpr (PACK) {
                        // columns 0 to 3: the weight rounded down, 4 to 7: its remainder
                        uint32_t w = pack_rz_x2<true>(x, y);
                        const float2 top = f16x2_to_float2(w);
                        const uint32_t rest = pack_f16x2(x - top.x, y - top.y);
                        w = c & 2 ? rest : w;
                        if constexpr (C::kInf)
                            w = max2<true>(w, 0x00010001u);
                        pf[kt][0][nt][a] = movmatrix_trans(w);
                    } else {
#pragma unroll
                        for (int part = 0; part < kParts; ++part) {
                            uint32_t w;
                            if (part == kParts - 1)
                                w = pack_x2<C::kF16>(x, y);
                            else {
                                w = pack_rz_x2<C::kF16>(x, y);
                                const float2 top = x2_to_float2<C::kF16>(w);
                                x -= top.x;
                                y -= top.y;
                            }
                            // an infinite V element times a part that is 0 would be NaN: parts of what is seen
                            // are at least 2^-38 (fp16) or 2^-126 of the largest weight
                            if constexpr (C::kInf)
                                w = max2<C::kF16>(w, C::kF16 ? 0x00010001u : 0x00800080u);
                            pf[kt][part][nt][a] = movmatrix_trans(w);
                        }
                    }
                }
        }
    }

    // acc = acc * alpha + V^T P^T.  TOKEN: only the weights of token `token`'s columns, and of V only the rows that it
    // sees, whatever the others hold.
    template <bool TOKEN>
    __device__ __forceinline__ void values(const WindowParams &p, const WindowReq &req, int row0, int token, uint32_t v, uint32_t vs,
                                           int g, int c, const uint32_t (&pin)[KT][kParts][NT][2], const float (&alpha)[NT][2])
    {
        constexpr int kLane = kRow / 8;                        // bytes of a row that a lane takes
        constexpr int kLoad = kLane < 16 ? kLane : 16, kPieces = kLane / kLoad, kWords = kLoad / 4;
        constexpr int kBlocks = C::kFp4 ? 4 : C::kFp8 ? 2 : 1; // 16-dim output blocks of a word
        const int r[4] = {c, 4 + (c ^ 1), 8 + c, 12 + (c ^ 1)};
        uint32_t pf[KT][kParts][NT][2], keep[KT][2];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
            for (int part = 0; part < kParts; ++part)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const bool mine = !TOKEN || ((nt * 8 + g) & kColMask) / p.group == token;
                    pf[kt][part][nt][0] = mine ? pin[kt][part][nt][0] : 0u;
                    pf[kt][part][nt][1] = mine ? pin[kt][part][nt][1] : 0u;
                }
            if constexpr (TOKEN) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int own = req.L - p.q_len + token;
                    keep[kt][i] = (visible(p, req, row0 + kt * 16 + r[2 * i], own) ? 0x0000FFFFu : 0u) |
                                  (visible(p, req, row0 + kt * 16 + r[2 * i + 1], own) ? 0xFFFF0000u : 0u);
                }
            }
        }
#pragma unroll
        for (int x = 0; x < kPieces; ++x) {
            uint32_t w[KT][4][kWords];
            uint32_t s16[KT][2][2];   // [row pair][block scale]: fp16 pairs
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t at = v + (uint32_t)(kt * 16 + r[i]) * kRow;
                    const int sw = window_swizzle<kGran>(r[i]);
                    if constexpr (kLoad == 16) {
                        const uint4 y = lds128(at + (((g + 8 * x) ^ sw) << 4));
                        w[kt][i][0] = y.x; w[kt][i][1] = y.y; w[kt][i][2] = y.z; w[kt][i][3] = y.w;
                    } else if constexpr (kLoad == 8) {
                        const uint2 y = lds64(at + ((((g >> 1)) ^ sw) << 4) + 8 * (g & 1));
                        w[kt][i][0] = y.x; w[kt][i][1] = y.y;
                    } else
                        w[kt][i][0] = lds32(at + 4 * g);
                }
                if constexpr (C::kFp4) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t a = vs + (uint32_t)(kt * 16 + r[2 * i]) * C::kScaleRow, b = vs + (uint32_t)(kt * 16 + r[2 * i + 1]) * C::kScaleRow;
                        if constexpr (D == 256) {
                            const uint32_t y = prmt(lds16(a + 2 * g), lds16(b + 2 * g), 0x5140);
                            s16[kt][i][0] = fp8x2_to_f16x2<kKvE4m3>(lo16(y));
                            s16[kt][i][1] = fp8x2_to_f16x2<kKvE4m3>(hi16(y));
                        } else {
                            const int blk = D == 128 ? g : g >> 1;
                            s16[kt][i][0] = fp8x2_to_f16x2<kKvE4m3>((uint16_t)(lds8(a + blk) | lds8(b + blk) << 8));
                        }
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kWords; ++j) {
                uint32_t a[KT][kBlocks][4];
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    const uint32_t w0 = w[kt][0][j], w1 = w[kt][1][j], w2 = w[kt][2][j], w3 = w[kt][3][j];
                    if constexpr (C::kFp4) {
                        // even and odd dims of two rows side by side, then to fp16
                        constexpr uint32_t kLo = 0x0F0F0F0Fu;
                        uint32_t f[4];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t y = i ? w2 : w0, z = i ? w3 : w1, s = s16[kt][i][D == 256 ? j / 2 : 0];
                            e2m1x8_to_f16x2((y & kLo) | ((z << 4) & ~kLo), f);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                a[kt][e][2 * i] = hmul2(f[e], s);
                            e2m1x8_to_f16x2(((y >> 4) & kLo) | (z & ~kLo), f);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                a[kt][e][2 * i + 1] = hmul2(f[e], s);
                        }
                    } else if constexpr (C::kFp8) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t y = i ? w2 : w0, z = i ? w3 : w1;
                            const uint32_t lo = prmt(y, z, 0x5140), hi = prmt(y, z, 0x7362);
                            a[kt][0][2 * i] = fp8x2_to_f16x2<KV>(lo16(lo));
                            a[kt][0][2 * i + 1] = fp8x2_to_f16x2<KV>(hi16(lo));
                            a[kt][1][2 * i] = fp8x2_to_f16x2<KV>(lo16(hi));
                            a[kt][1][2 * i + 1] = fp8x2_to_f16x2<KV>(hi16(hi));
                        }
                    } else {
                        a[kt][0][0] = prmt(w0, w1, 0x5410);
                        a[kt][0][1] = prmt(w0, w1, 0x7632);
                        a[kt][0][2] = prmt(w2, w3, 0x5410);
                        a[kt][0][3] = prmt(w2, w3, 0x7632);
                    }
                    if constexpr (TOKEN) {
#pragma unroll
                        for (int e = 0; e < kBlocks; ++e)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                a[kt][e][i] &= keep[kt][i / 2];
                    }
                }
                // The tile's sums start from 0 and are added in fp32: the tensor cores' additions truncate.
#pragma unroll
                for (int e = 0; e < kBlocks; ++e) {
                    const int blk = (x * kWords + j) * kBlocks + e;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                            for (int part = 0; part < kParts; ++part)
                                mma_16816<C::kF16>(t, a[kt][e][0], a[kt][e][1], a[kt][e][2], a[kt][e][3], pf[kt][part][nt][0], pf[kt][part][nt][1]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            // 0 times a row that only `token` sees may be NaN
                            const bool mine = !TOKEN || ((nt * 8 + 2 * c + (i & 1)) & kColMask) / p.group == token;
                            acc[blk][nt][i] = fmaf(acc[blk][nt][i], alpha[nt][i & 1], mine ? t[i] : 0.f);
                        }
                    }
                }
            }
        }
    }

    // First of the two dims that the lane holds of output block blk (rows g and g + 8 of the MMA).
    __device__ __forceinline__ static int block_dim(int blk, int g)
    {
        constexpr int kLane = kRow / 8, kLoad = kLane < 16 ? kLane : 16;
        constexpr int kEl = kLoad * D / kRow, kBlk = kEl / 2;   // elements and blocks of a lane's piece
        return (g + 8 * (blk / kBlk)) * kEl + 2 * (blk % kBlk);
    }

    // Add up what the lanes hold apart: sums of weights, and the two parts of PACK.
    __device__ __forceinline__ void finish()
    {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], off);
        if constexpr (PACK) {
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[s][0][e] += __shfl_xor_sync(0xffffffffu, acc[s][0][e], 2);
        }
    }
};

// Place in o / lse of column col of kv head `head`.
__device__ __forceinline__ long long window_out_row(const WindowParams &p, int b, int head, int col)
{
    const int i = col / p.group;
    return (long long)(b * p.q_len + i) * p.hq + head * p.group + (col - i * p.group);
}
// LSE from the reference exponent (log2) and the sum of weights.
__device__ __forceinline__ float window_lse(float m, float l)
{
    return l == 0.f ? -__builtin_huge_valf() : ((m == -__builtin_huge_valf() ? 0.f : m) + log2f(l)) * 0.6931471805599453f;
}

// The CTA's copy of the schedule: prefix and non-empty requests in shared memory.
template <int TILE>
__device__ __forceinline__ void window_schedule(const WindowParams &p, int *prefix, int *nonempty, int *tmp, bool report)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int heads = p.hkv / p.team;
    int run = 0, live = 0;
    for (int b0 = 0; b0 < p.batch; b0 += blockDim.x) {
        const int b = b0 + threadIdx.x;
        int n = 0;
        if (b < p.batch)
            n = (window_req(p, b, report ? p.ws_err : nullptr).rows + TILE - 1) / TILE;
        int x = n * heads, y = n > 0 ? 1 : 0;
        const int mx = x, my = y;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, x, off), c = __shfl_up_sync(0xffffffffu, y, off);
            if (lane >= off) {
                x += a;
                y += c;
            }
        }
        if (lane == 31) {
            tmp[2 * warp] = x;
            tmp[2 * warp + 1] = y;
        }
        __syncthreads();
        int bx = 0, by = 0, ax = 0, ay = 0;
        for (int w = 0; w < warps; ++w) {
            if (w == warp) {
                bx = ax;
                by = ay;
            }
            ax += tmp[2 * w];
            ay += tmp[2 * w + 1];
        }
        if (b < p.batch) {
            prefix[b] = run + bx + x - mx;
            nonempty[b] = live + by + y - my;
        }
        run += ax;
        live += ay;
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        prefix[p.batch] = run;
        nonempty[p.batch] = live;
    }
    __syncthreads();
}

// Shared memory: the warps' rings, then prefix and non-empty [batch + 1], then scratch.
constexpr int kWindowScratch = 2 * kWindowMaxWarps + 2 * kWindowMaxWarps;   // ints: the scan's sums; the warps' last segments
template <class C>
constexpr size_t window_smem(int batch)
{
    return (size_t)C::kWarps * C::kRing + sizeof(int) * (2 * ((size_t)batch + 1) + kWindowScratch);
}

template <class C, int NT, bool PACK>
__global__ void __launch_bounds__(32 * C::kWarps) window_kernel(const __grid_constant__ WindowParams p)
{
    using Warp = WindowWarp<C, NT, PACK>;
    constexpr int D = C::D, kTile = C::kTile, kRow = C::kRow, kGran = C::kGran, kStages = C::kStages;
    constexpr int kMl = NT * 8 * 2;   // floats of (m, l) in front of a warp's sums
    static_assert(C::kRing >= (int)sizeof(float) * (kMl + NT * 8 * D), "the ring holds a warp's sums at the end");
    extern __shared__ __align__(128) uint8_t smem[];
    int *prefix = reinterpret_cast<int *>(smem + C::kWarps * C::kRing);
    int *nonempty = prefix + p.batch + 1, *tmp = nonempty + p.batch + 1, *s_last = tmp + 2 * kWindowMaxWarps;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;

    pdl_launch_dependents();
    pdl_wait_prior_grid();
    window_schedule<kTile>(p, prefix, nonempty, tmp, blockIdx.x == 0);
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < 2 * (p.batch + 1); i += blockDim.x)
            p.ws_prefix[i] = prefix[i];

    const int heads = p.hkv / p.team;
    Schedule sch = {prefix, nonempty, p.batch, heads, kWindowSegCost, 0};
    const int teams = window_workers(sch.cost(), gridDim.x, C::kWarps / p.team);
    sch.P = gridDim.x * teams;
    const int team = warp / p.team, lead = warp - team * p.team;   // the warp's kv head of the team's
    const int worker = blockIdx.x * teams + team;
    int t0 = 0, t1 = 0;
    if (team < teams)
        sch.range(worker, &t0, &t1);

    Warp w;
    int last = -1;   // the segment of the sums that the warp still holds
    if (t0 < t1) {
        const uint32_t ring = smem_addr(smem) + warp * C::kRing;
        const uint64_t policy = l2_policy_evict_first();

        // A tile's rows of the cache: lane r has row r's number, or none.
        constexpr uint32_t kNone = 0xFFFFFFFFu;
        WindowCursor ld;
        ld.b = request_of_tile(prefix, p.batch, t0);
        ld.nb = (prefix[ld.b + 1] - prefix[ld.b]) / heads;
        ld.h = (t0 - prefix[ld.b]) / ld.nb;
        ld.j = t0 - prefix[ld.b] - ld.h * ld.nb;
        ld.req = window_req(p, ld.b, nullptr);
        WindowCursor use = ld;
        auto advance = [&](WindowCursor &x) {
            if (++x.j < x.nb)
                return;
            x.j = 0;
            if (++x.h < heads)
                return;
            x.h = 0;
            do
                ++x.b;
            while (prefix[x.b + 1] == prefix[x.b]);
            x.nb = (prefix[x.b + 1] - prefix[x.b]) / heads;
            x.req = window_req(p, x.b, nullptr);
        };
        // The page and slot of lane's row of the tile at ld; one tile ahead of the copies, which wait for them.
        int page = -1, slot = 0, head = 0;
        auto look_up = [&]() {
            const int v = ld.j * kTile + lane;
            page = -1;
            head = ld.h * p.team + lead;
            if (lane < kTile && v < ld.req.rows) {
                const int pos = window_pos(ld.req, v);
                if (p.block_table) {
                    const int blk = (unsigned)pos / (unsigned)p.page_size;
                    slot = pos - blk * p.page_size;
                    page = p.block_table[(long long)ld.b * p.max_blocks + blk];
                    if ((unsigned)page >= (unsigned)p.num_pages) {
                        page = 0;
                        atomicOr(p.ws_err, kErrPage);
                    }
                } else {
                    page = ld.b;
                    slot = pos;
                }
            }
        };
        auto copy = [&](int stage) {
            const uint32_t row = page < 0 ? kNone : (uint32_t)page * p.row_page + (uint32_t)slot * p.row_token + (uint32_t)head * p.row_head;
            const uint32_t k = ring + stage * C::kStage, v = k + kTile * kRow;
            constexpr int kCopies = kTile * kGran / 32, kRows = 32 / kGran;   // copies of a lane, rows of a copy
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int r = i * kRows + lane / kGran, x = lane % kGran;
                const uint32_t from = __shfl_sync(0xffffffffu, row, r);
                const uint32_t size = from == kNone ? 0u : 16u;
                const size_t at = from == kNone ? 0 : (size_t)from * kRow + 16 * x;
                const uint32_t to = r * kRow + ((x ^ window_swizzle<kGran>(r)) << 4);
                cp_async_or_zero<16>(k + to, p.k + at, size, policy);
                cp_async_or_zero<16>(v + to, p.v + at, size, policy);
            }
            if constexpr (C::kFp4) {
                constexpr int kS = C::kScaleRow;
                const uint32_t ks = v + kTile * kRow, vs = ks + kTile * kS;
                if (kTile == 32 || lane < kTile) {
                    const uint32_t size = row == kNone ? 0u : (uint32_t)kS;
                    const size_t at = row == kNone ? 0 : (size_t)row * kS;
                    cp_async_or_zero<kS>(ks + lane * kS, p.ks + at, size, policy);
                    cp_async_or_zero<kS>(vs + lane * kS, p.vs + at, size, policy);
                }
            }
        };

        int ahead = t0;   // tile at ld
        look_up();
        auto fetch = [&](int stage) {
            if (ahead < t1) {
                copy(stage);
                if (++ahead < t1) {
                    advance(ld);
                    look_up();
                }
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i)
            fetch(i);

        int stage = 0;
        bool whole = false;   // the segment's first tile was the warp's
        for (int t = t0; t < t1; ++t) {
            const int seg = use.b * heads + use.h, head_now = use.h * p.team + lead;
            if (seg != last) {
                w.start(p, use.b, head_now, g, c);
                last = seg;
                whole = use.j == 0;
            }
            cp_async_wait<kStages - 2>();
            __syncwarp();
            fetch(stage == 0 ? kStages - 1 : stage - 1);
            const uint32_t k = ring + stage * C::kStage, v = k + kTile * kRow, ks = v + kTile * kRow, vs = ks + kTile * C::kScaleRow;
            stage = stage + 1 == kStages ? 0 : stage + 1;
            const int row0 = use.j * kTile;
            // every row of the tile visible to every new token?
            bool plain = row0 + kTile <= use.req.rows && window_pos(use.req, row0 + kTile - 1) <= use.req.L - p.q_len;
            if (p.window && p.q_len > 1) {
                const int from = max(window_pos(use.req, row0), use.req.first);   // the tile's first row behind the sinks
                plain = plain && (row0 + kTile <= use.req.head || from < p.sinks || use.req.L - 1 - from < p.window);
            }
            float sc[Warp::KT][NT][4], alpha[NT][2];
            uint32_t pf[Warp::KT][Warp::kParts][NT][2];
            w.scores(k, ks, g, c, sc);
            if (!plain)
                w.mask(p, use.req, row0, g, c, sc);
            w.weights(sc, c, pf, alpha);
            if (plain || p.q_len == 1)
                w.template values<false>(p, use.req, row0, 0, v, vs, g, c, pf, alpha);
            else {
                float one[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    one[nt][0] = one[nt][1] = 1.f;
                for (int i = 0; i < p.q_len; ++i) {
                    w.template values<true>(p, use.req, row0, i, v, vs, g, c, pf, alpha);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        alpha[nt][0] = alpha[nt][1] = 1.f;
                }
            }
            if (use.j + 1 == use.nb && (whole || t + 1 < t1)) {
                // the segment ends inside the run: its output, or a partial of a segment that others began
                w.finish();
                const long long slot_o = (long long)(2 * worker) * p.team + lead;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int col = nt * 8 + 2 * c + e;
                        if (col >= p.cols || (PACK && c >= 2))
                            continue;
                        float *dst;
                        float f = 1.f;
                        if (whole) {
                            const long long row = window_out_row(p, use.b, head_now, col);
                            dst = p.o + row * D;
                            f = w.l[nt][e] == 0.f ? 0.f : p.v_scale / w.l[nt][e];
                            if (g == 0 && p.lse)
                                p.lse[row] = window_lse(w.m[nt][e] - Warp::kShift, w.l[nt][e]);
                        } else {
                            dst = p.ws_o + (slot_o * p.cols + col) * D;
                            if (g == 0)
                                p.ws_ml[slot_o * p.cols + col] = make_float2(w.m[nt][e], w.l[nt][e]);
                        }
#pragma unroll
                        for (int s = 0; s < Warp::kSteps; s += 2)
                            *reinterpret_cast<float4 *>(dst + Warp::block_dim(s, g)) =
                                make_float4(w.acc[s][nt][e] * f, w.acc[s][nt][e + 2] * f, w.acc[s + 1][nt][e] * f, w.acc[s + 1][nt][e + 2] * f);
                    }
                last = -1;
            }
            if (t + 1 < t1)
                advance(use);
        }
        cp_async_wait<0>();
        __syncwarp();
    }

    // Sums that warps still hold: those of the same segment are added up over the CTA.  A warp leaves (m, l) and its
    // sums in its own ring.
    if (last >= 0) {
        w.finish();
        float *ml = reinterpret_cast<float *>(smem + warp * C::kRing), *sum = ml + kMl;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int col = nt * 8 + 2 * c + e;
                if (col >= p.cols || (PACK && c >= 2))
                    continue;
                if (g == 0) {
                    ml[2 * col] = w.m[nt][e];
                    ml[2 * col + 1] = w.l[nt][e];
                }
#pragma unroll
                for (int s = 0; s < Warp::kSteps; s += 2)
                    *reinterpret_cast<float4 *>(sum + col * D + Warp::block_dim(s, g)) =
                        make_float4(w.acc[s][nt][e], w.acc[s][nt][e + 2], w.acc[s + 1][nt][e], w.acc[s + 1][nt][e + 2]);
            }
    }
    if (lane == 0)
        s_last[warp] = last;
    __syncthreads();
    for (int a = 0; a < C::kWarps; ++a) {   // a: the group's first warp (of its kv head of the team's)
        const int seg = s_last[a];
        if (seg < 0 || (a >= p.team && s_last[a - p.team] == seg))
            continue;
        int n = 1;
        while (a + n * p.team < C::kWarps && s_last[a + n * p.team] == seg)
            ++n;
        const int b = seg / heads, head = (seg - b * heads) * p.team + a % p.team;
        // did the group have the whole segment?
        const long long pos = sch.seg_pos(b, seg - b * heads);
        const int nb = (prefix[b + 1] - prefix[b]) / heads, w0 = blockIdx.x * teams + a / p.team;
        const bool all = sch.cta_at(pos) == w0 && sch.cta_at(pos + nb - 1) == w0 + n - 1;
        const long long slot_o = (long long)(2 * w0 + 1) * p.team + a % p.team;
        for (int i = threadIdx.x; i < p.cols * (D / 4); i += blockDim.x) {
            const int col = i / (D / 4), d = 4 * (i - col * (D / 4));
            float top = -__builtin_huge_valf();
            for (int k = 0; k < n; ++k)
                top = fmaxf(top, reinterpret_cast<const float *>(smem + (a + k * p.team) * C::kRing)[2 * col]);
            const float ref = top == -__builtin_huge_valf() ? 0.f : top;
            float sum = 0.f;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < n; ++k) {
                const float *ml = reinterpret_cast<const float *>(smem + (a + k * p.team) * C::kRing);
                const float4 y = *reinterpret_cast<const float4 *>(ml + kMl + col * D + d);
                const float f = fmaxf(exp2_approx(ml[2 * col] - ref), 1.1754944e-38f);
                sum = fmaf(f, ml[2 * col + 1], sum);
                x.x = fmaf(f, y.x, x.x);
                x.y = fmaf(f, y.y, x.y);
                x.z = fmaf(f, y.z, x.z);
                x.w = fmaf(f, y.w, x.w);
            }
            if (all) {
                const long long row = window_out_row(p, b, head, col);
                const float f = sum == 0.f ? 0.f : p.v_scale / sum;
                *reinterpret_cast<float4 *>(p.o + row * D + d) = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
                if (d == 0 && p.lse)
                    p.lse[row] = window_lse(top - Warp::kShift, sum);
            } else {
                *reinterpret_cast<float4 *>(p.ws_o + (slot_o * p.cols + col) * D + d) = x;
                if (d == 0)
                    p.ws_ml[slot_o * p.cols + col] = make_float2(top, sum);
            }
        }
    }
}

template <class C, int NT, bool PACK>
cudaError_t launch_window_t(const WindowParams &p, const WindowLaunch &c)
{
    auto kernel = window_kernel<C, NT, PACK>;
    // Raise the kernel's shared-memory limit once per device, so that later calls may be captured; again if a launch
    // is refused (the device's context was reset since).
    static std::atomic<unsigned long long> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const unsigned long long bit = 1ull << (dev & 63);
    auto configure = [&]() -> cudaError_t {
        const cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)c.smem_optin);
        if (r == cudaSuccess)
            configured.fetch_or(bit, std::memory_order_release);
        return r;
    };
    if (!(configured.load(std::memory_order_acquire) & bit) && (e = configure()) != cudaSuccess)
        return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)c.grid);
    cfg.blockDim = dim3(32 * C::kWarps);
    cfg.dynamicSmemBytes = window_smem<C>(p.batch);
    cfg.stream = c.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, p);
    if (e == cudaErrorInvalidValue) {
        (void)cudaGetLastError();
        if ((e = configure()) != cudaSuccess)
            return e;
        e = cudaLaunchKernelEx(&cfg, kernel, p);
    }
    return e;
}

template <int D, int KV>
cudaError_t launch_window_variant(const WindowParams &p, const WindowLaunch &c)
{
    using C = WindowCfg<D, KV>;
    static_assert(window_smem<C>(kMaxBatch) <= 232448, "fits the 227 KB of a CTA");
    cudaError_t e;
    if (p.cols > 8)
        e = launch_window_t<C, 2, false>(p, c);
    else if constexpr (C::kF16)
        e = p.cols <= 4 ? launch_window_t<C, 1, true>(p, c) : launch_window_t<C, 1, false>(p, c);
    else
        e = launch_window_t<C, 1, false>(p, c);
    return e;
}

}  // namespace fd
