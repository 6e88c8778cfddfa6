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
//
// Softmax in one pass: with x_t = scale q . k_t in log2 units and a reference
// m that only rises, l = sum 2^(x_t - m), O = sum 2^(x_t - m) v_t / l, LSE =
// (m + log2 l) ln 2; sums of two warps with references m, m' join after
// factors of 2^(m - max), 2^(m' - max).  A weight is two fp16 or three bf16
// parts, so that it is off by 2^-22 of itself at most, of fp16 parts by 2^-39
// of the reference's weight where that is more (a weight's remainder ends at
// half of fp16's least step, 2^-25, and the reference's weight is 2^14); up to
// four fp16 columns have both parts as columns of one MMA.
//
// What bounds it (GB300, contexts of hundreds of MB): 16-bit and FP8 caches
// memory: 64 requests of GQA-4 and a window of 4096 in bf16 162 us = 6.5 TB/s,
// 96% of a copy; E4M3 314 us = 96%.  9 to 16 columns over FP8 caches are not
// there (400 MB, 128 dims: 93 us of 59): two MMAs for each converted operand.
// 4-bit caches the warps' arithmetic: 604 MB in 122 us = 4.9 TB/s, 73%, the
// same with the pages in L2, and 96 us for the loads alone.  An MMA of 2048
// products a scheduler takes 8 cycles, each conversion or multiplication of a
// code pair 2, and HMUL2 shares the MMAs' pipe: 14.3 cycles for the MMA with
// its four pairs.  V does not go to tcgen05: the scales of its blocks run along
// the output's dims, not along the sum, so each code would have to be written
// to shared memory in 16 bits and read again, for 1 to 16 columns of 128 rows.
// K's codes and scales as they lie are operands of tcgen05's block-scaled FP4
// MMAs (16 elements a scale, along the sum), with the query in several 4-bit
// parts; that has been neither built nor measured.
#pragma once

#include <atomic>
#include <type_traits>

#include "fd_window.cuh"

namespace fd {

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int BYTES>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src, uint64_t policy)
{
    if constexpr (BYTES == 16)
        cp_async_16(dst, src, policy);
    else
        asm volatile("cp.async.ca.shared.global.L2::cache_hint [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "l"(policy), "n"(BYTES)
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

// Byte I of w, two E2M1 codes (the first in the low half), as a pair of fp16.
template <int I>
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t w)
{
    uint32_t r;
    if constexpr (I == 0)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
    else if constexpr (I == 1)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
    else if constexpr (I == 2)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(w));
    else
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t e2m1x2_at(uint32_t w, int i)   // i known to the compiler
{
    return i == 0 ? e2m1x2_to_f16x2<0>(w) : i == 1 ? e2m1x2_to_f16x2<1>(w) : i == 2 ? e2m1x2_to_f16x2<2>(w) : e2m1x2_to_f16x2<3>(w);
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// As mma_16816 with C = 0.
template <bool F16>
__device__ __forceinline__ void mma_16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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

// Where a lane finds its pieces in a tile, in bytes: of K row window_row(g), the even pieces x (place ke + 64 x) and the
// odd ones (ko + 64 x); of V the rows c and 4 + (c ^ 1) (v[] + 128 x); of the block scales of either.  Rows 8 further are
// 8 rows of bytes further.
template <class C>
struct WindowPlaces {
    uint32_t ke, ko, ks, v[2], vs[2];
    __device__ __forceinline__ WindowPlaces(int g, int c)
    {
        constexpr int kRow = C::kRow, kLane = kRow / 8;
        const int r = window_row(g), sw = window_swizzle<C::kGran>(r);
        ke = ko = r * kRow + (kRow >= 64 ? (c ^ (sw & 3)) << 4 : 8 * c);
        if (kRow >= 128) {
            ke += 16 * (sw & 4);
            ko -= 16 * (sw & 4);
        }
        ks = r * C::kScaleRow + (kRow >= 64 ? 2 * c : c);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = i ? 4 + (c ^ 1) : c, s = window_swizzle<C::kGran>(row);
            v[i] = row * kRow + (kLane >= 16 ? (g ^ s) << 4 : kLane == 8 ? (((g >> 1) ^ s) << 4) + 8 * (g & 1) : 4 * g);
            vs[i] = row * C::kScaleRow + (C::D == 256 ? 2 * g : C::D == 128 ? g : g >> 1);
        }
    }
};

// A tile's flags; above them its rows.
enum : int { kTilePlain = 1, kTileFirst = 2, kTileLast = 4, kTileN = 8 };   // kTileN: a shift

__device__ __forceinline__ void sts128(uint32_t addr, int x, int y, int z, int w)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// The rows that new token i of a request sees: [0, below) and [from, to).
struct WindowSight {
    int below, from, to;
    __device__ __forceinline__ WindowSight(const WindowParams &p, const WindowReq &req, int i)
    {
        const int own = req.L - p.q_len + i, skip = req.first - req.head;
        below = min(req.head, own + 1);
        from = req.head;
        if (p.window)
            from = (int)max((long long)req.head, (long long)own - p.window - skip + 1);
        to = own - skip + 1;
    }
    // v may pass 2^31 in a tile's last rows
    __device__ __forceinline__ bool sees(int v) const { return v >= 0 && (v < below || (v >= from && v < to)); }
};

// One warp's place in the schedule.
struct WindowCursor {
    int b, h, j, nb;        // request, launch head, tile of the segment, tiles of a segment
    int rows, head, skip;   // row v of the request is position v, + skip from row head on
    const int32_t *pages;   // the request's block table
};

template <class C, bool PACK>
struct WindowWarp {
    static constexpr int NT = C::NT, D = C::D, KV = C::KV, kTile = C::kTile, kRow = C::kRow, kGran = C::kGran;
    static constexpr int KT = kTile / 16;          // k steps of a tile
    static constexpr int kSteps = D / 16;          // k steps of a row, and 16-dim blocks of the output
    static constexpr int kParts = PACK ? 1 : C::kParts;   // MMAs a block (PACK: both parts in one)
    static constexpr float kShift = C::kShift;
    static constexpr int kColMask = PACK ? 3 : 8 * NT - 1;

    // The query as the B operand of S^T, two words of each k step: in registers, or in shared memory (every lane its own).
    static constexpr int kHeld = C::kQueryShared ? 1 : kSteps;
    uint32_t qf[kHeld][NT][2];
    uint32_t q_at;
    float mult[NT][2];         // score of column 2c, 2c + 1 of an MMA's eight -> log2 units
    float acc[kSteps][NT][4];
    // Of columns 2c, 2c + 1: the largest score so far (the reference) times -1, fp32's largest number if there is none, and
    // the sum of weights.  A weight is worked out from the difference of two scores: score * mult less the reference's,
    // in one step, leaves the rounding of the reference, and that passes fp16's range for references from 2^25 on and
    // fp32's from 2^31 on (the difference takes an addition a weight: 131072 positions of 32 heads in 4 bits 120.3 -> 122.3
    // us, 64 ragged requests 126.2 -> 128.1, 16-bit and FP8 caches alike).
    float minus[NT][2], l[NT][2];

    // Load the query of segment (b, head) as the B operand of S^T.
    __device__ __forceinline__ void start(const WindowParams &p, int b, int head, int g, int c)
    {
        const uint32_t sign = p.negate_q ? 0x80008000u : 0u;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int col = (nt * 8 + g) & kColMask;
            const int i = col / p.group;
            const bool real = col < p.cols;
            const uint16_t *src = p.q + ((long long)(b * p.q_len + (real ? i : 0)) * p.hq + head * p.group + (real ? col - i * p.group : 0)) * D;
            uint2 words[kSteps];
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                // elements of a piece, and the lane's four in step s
                constexpr int kEl = kRow >= 64 ? 16 * D / kRow : 16, kPer = kEl / 4;
                const int dim = (c + 4 * (s / kPer)) * kEl + 4 * (s % kPer);
                words[s] = make_uint2(0u, 0u);
                if (real)
                    words[s] = *reinterpret_cast<const uint2 *>(src + dim);
                words[s].x ^= sign;
                words[s].y ^= sign;
            }
            float f = p.scale_log2;
            if (KV >= kKvE4m3 && !p.q_f16) {
                // bf16 as fp16 times a power of two: the row's largest element goes to [2^14, 2^15), so that
                // what fp16 cannot hold is below 2^-39 of it
                float top = 0.f;
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    const float2 x = bf16x2_to_float2(words[s].x), y = bf16x2_to_float2(words[s].y);
                    top = fmaxf(top, fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(y.x), fabsf(y.y))));
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                int e = ((int)(__float_as_uint(top) >> 23) & 255) - 127;     // top in [2^e, 2^(e + 1))
                e = top > 0.f && e < 128 ? min(max(14 - e, -126), 126) : 0;
                const float up = __uint_as_float((uint32_t)(e + 127) << 23), down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    const float2 x = bf16x2_to_float2(words[s].x), y = bf16x2_to_float2(words[s].y);
                    words[s] = make_uint2(pack_f16x2(x.x * up, x.y * up), pack_f16x2(y.x * up, y.y * up));
                }
                f = fmaxf(f * down, 1.1754944e-38f);
            }
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                if constexpr (C::kQueryShared)
                    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(q_at + (s * NT + nt) * 256), "r"(words[s].x), "r"(words[s].y) : "memory");
                else {
                    qf[s][nt][0] = words[s].x;
                    qf[s][nt][1] = words[s].y;
                }
            }
            mult[nt][0] = __shfl_sync(0xffffffffu, f, 8 * c);
            mult[nt][1] = __shfl_sync(0xffffffffu, f, 8 * c + 4);
            minus[nt][0] = minus[nt][1] = 3.4028235e38f;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[s][nt][e] = 0.f;
        }
    }

    // S^T of a tile, without the scale: sc[kt][nt] = rows window_row(g), + 8 of 16-row step kt times columns 2c, 2c + 1.
    __device__ __forceinline__ void scores(const WindowPlaces<C> &at, uint32_t k, uint32_t ks, float (&sc)[KT][NT][4]) const
    {
        const uint32_t ke = k + at.ke, ko = k + at.ko, kscale = ks + at.ks;
        constexpr int kPieces = kRow >= 64 ? kRow / 64 : 1;
        constexpr int kPer = kSteps / kPieces;   // k steps of a piece
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sc[kt][nt][e] = 0.f;
#pragma unroll
        for (int x = 0; x < kPieces; ++x) {
            uint32_t a[KT][2][4], s16[KT][2][2];   // rows window_row(g) and + 8 of each 16: words; block scales as fp16 pairs
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t from = (x & 1 ? ko : ke) + (kt * 16 + 8 * i) * kRow + 64 * x;
                    if constexpr (kRow >= 64) {
                        const uint4 w = lds128(from);
                        a[kt][i][0] = w.x; a[kt][i][1] = w.y; a[kt][i][2] = w.z; a[kt][i][3] = w.w;
                    } else {
                        const uint2 w = lds64(from);
                        a[kt][i][0] = w.x; a[kt][i][1] = w.y;
                    }
                    if constexpr (C::kFp4) {
                        const uint32_t place = kscale + (kt * 16 + 8 * i) * C::kScaleRow + 8 * x;
                        const uint32_t b = fp8x2_to_f16x2<kKvE4m3>((uint16_t)(kRow >= 64 ? lds16(place) : lds8(place)));
                        s16[kt][i][0] = prmt(b, b, 0x1010);
                        s16[kt][i][1] = prmt(b, b, 0x3232);
                    }
                }
#pragma unroll
            for (int s = 0; s < kPer; ++s) {
                uint32_t q[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if constexpr (C::kQueryShared) {
                        const uint2 w = lds64(q_at + ((x * kPer + s) * NT + nt) * 256);
                        q[nt][0] = w.x;
                        q[nt][1] = w.y;
                    } else {
                        q[nt][0] = qf[x * kPer + s][nt][0];
                        q[nt][1] = qf[x * kPer + s][nt][1];
                    }
                }
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    uint32_t f[2][2];   // [row][pair of the lane's four elements]
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if constexpr (C::kFp4) {
                            const uint32_t w = a[kt][i][s / 2], sc16 = s16[kt][i][s / 4];
                            f[i][0] = hmul2(e2m1x2_at(w, 2 * (s & 1)), sc16);
                            f[i][1] = hmul2(e2m1x2_at(w, 2 * (s & 1) + 1), sc16);
                        } else if constexpr (C::kFp8) {
                            f[i][0] = fp8x2_to_f16x2<KV>(lo16(a[kt][i][s]));
                            f[i][1] = fp8x2_to_f16x2<KV>(hi16(a[kt][i][s]));
                        } else {
                            f[i][0] = a[kt][i][2 * s];
                            f[i][1] = a[kt][i][2 * s + 1];
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_16816<C::kF16>(sc[kt][nt], f[0][0], f[1][0], f[0][1], f[1][1], q[nt][0], q[nt][1]);
                }
            }
        }
    }

    // Hide the rows from n on.
    __device__ __forceinline__ void cut(int n, int g, float (&sc)[KT][NT][4]) const
    {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (kt * 16 + window_row(g) + 8 * (e / 2) >= n)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        sc[kt][nt][e] = -__builtin_huge_valf();
    }
    // Hide what a column's token does not see in the tile from row `row0` of the request.
    __device__ __forceinline__ void mask(const WindowParams &p, const WindowReq &req, int row0, int g, int c, float (&sc)[KT][NT][4]) const
    {
        const int r = window_row(g);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const WindowSight sight(p, req, min(((nt * 8 + 2 * c + e) & kColMask) / p.group, p.q_len - 1));
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                    for (int a = 0; a < 2; ++a)
                        if (!sight.sees(row0 + kt * 16 + r + 8 * a))
                            sc[kt][nt][2 * a + e] = -__builtin_huge_valf();
            }
    }

    // Move the references up to the tile's scores if one passes its own, which is rare after the first tiles.
    __device__ __forceinline__ void rescale(const float (&sc)[KT][NT][4])
    {
        float top[NT][2];
        bool over = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = fmaxf(sc[0][nt][e], sc[0][nt][e + 2]);
#pragma unroll
                for (int kt = 1; kt < KT; ++kt)
                    x = fmaxf(x, fmaxf(sc[kt][nt][e], sc[kt][nt][e + 2]));
                top[nt][e] = x;
                over = over || x > -minus[nt][e];
            }
        if (!__any_sync(0xffffffffu, over))
            return;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = top[nt][e];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
                // 0 times an infinite sum: NaN, and window_repair looks for what made it
                const float now = fminf(minus[nt][e], -x), alpha = exp2_approx((now - minus[nt][e]) * mult[nt][e]);
                minus[nt][e] = now;
                l[nt][e] *= alpha;
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    acc[s][nt][e] *= alpha;
                    acc[s][nt][e + 2] *= alpha;
                }
            }
    }
    // The reference of a column in log2 units.
    __device__ __forceinline__ float reference(int nt, int e) const { return -minus[nt][e] * mult[nt][e]; }

    // The scores' softmax weights in parts, as the B operand of O^T: pf[kt][part][nt][2].
    __device__ __forceinline__ void weights(const float (&sc)[KT][NT][4], int c, uint32_t (&pf)[KT][kParts][NT][2])
    {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    float x = exp2_approx(fmaf(sc[kt][nt][2 * a] + minus[nt][0], mult[nt][0], kShift));
                    float y = exp2_approx(fmaf(sc[kt][nt][2 * a + 1] + minus[nt][1], mult[nt][1], kShift));
                    l[nt][0] += x;
                    l[nt][1] += y;
                    if constexpr (PACK) {
                        // columns 0 to 3: the weight rounded down, 4 to 7: its remainder
                        uint32_t w = pack_rz_x2<true>(x, y);
                        const float2 top = f16x2_to_float2(w);
                        const uint32_t rest = pack_f16x2(x - top.x, y - top.y);
                        w = c & 2 ? rest : w;
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
                            pf[kt][part][nt][a] = movmatrix_trans(w);
                        }
                    }
                }
        }
    }

    // acc += V^T P^T
    __device__ __forceinline__ void values(const WindowPlaces<C> &at, uint32_t v, uint32_t vs, const uint32_t (&pf)[KT][kParts][NT][2])
    {
        const uint32_t from[2] = {v + at.v[0], v + at.v[1]}, scale[2] = {vs + at.vs[0], vs + at.vs[1]};
        constexpr int kLane = kRow / 8;                        // bytes of a row that a lane takes
        constexpr int kLoad = kLane < 16 ? kLane : 16, kPieces = kLane / kLoad, kWords = kLoad / 4;
        constexpr int kBlocks = C::kFp4 ? 4 : C::kFp8 ? 2 : 1; // 16-dim output blocks of a word
#pragma unroll
        for (int x = 0; x < kPieces; ++x) {
            uint32_t w[KT][4][kWords];
            uint32_t s16[KT][2][2];   // [row pair][block scale]: fp16 pairs
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t place = from[i & 1] + (kt * 16 + 8 * (i / 2)) * kRow + 128 * x;
                    if constexpr (kLoad == 16) {
                        const uint4 y = lds128(place);
                        w[kt][i][0] = y.x; w[kt][i][1] = y.y; w[kt][i][2] = y.z; w[kt][i][3] = y.w;
                    } else if constexpr (kLoad == 8) {
                        const uint2 y = lds64(place);
                        w[kt][i][0] = y.x; w[kt][i][1] = y.y;
                    } else
                        w[kt][i][0] = lds32(place);
                }
                if constexpr (C::kFp4) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t a = scale[0] + (kt * 16 + 8 * i) * C::kScaleRow, b = scale[1] + (kt * 16 + 8 * i) * C::kScaleRow;
                        if constexpr (D == 256) {
                            const uint32_t y = prmt(lds16(a), lds16(b), 0x5140);
                            s16[kt][i][0] = fp8x2_to_f16x2<kKvE4m3>(lo16(y));
                            s16[kt][i][1] = fp8x2_to_f16x2<kKvE4m3>(hi16(y));
                        } else {
                            s16[kt][i][0] = fp8x2_to_f16x2<kKvE4m3>((uint16_t)(lds8(a) | lds8(b) << 8));
                        }
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kWords; ++j) {
                // the words of two rows each, paired row by row: even and odd dims apart (4 bits), or as bytes and halves
                uint32_t y[KT][4];
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t a = w[kt][2 * i][j], b = w[kt][2 * i + 1][j];
                        if constexpr (C::kFp4) {
                            constexpr uint32_t kLo = 0x0F0F0F0Fu;
                            y[kt][2 * i] = (a & kLo) | ((b << 4) & ~kLo);
                            y[kt][2 * i + 1] = ((a >> 4) & kLo) | (b & ~kLo);
                        } else {
                            y[kt][2 * i] = prmt(a, b, C::kFp8 ? 0x5140 : 0x5410);
                            y[kt][2 * i + 1] = prmt(a, b, C::kFp8 ? 0x7362 : 0x7632);
                        }
                    }
#pragma unroll
                for (int e = 0; e < kBlocks; ++e) {
                    uint32_t a[KT][4];
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if constexpr (C::kFp4) {
                                const uint32_t s = s16[kt][i][D == 256 ? j / 2 : 0];
                                a[kt][2 * i] = hmul2(e2m1x2_at(y[kt][2 * i], e), s);
                                a[kt][2 * i + 1] = hmul2(e2m1x2_at(y[kt][2 * i + 1], e), s);
                            } else if constexpr (C::kFp8) {
                                a[kt][2 * i] = fp8x2_to_f16x2<KV>(lo16(y[kt][2 * i + e]));
                                a[kt][2 * i + 1] = fp8x2_to_f16x2<KV>(hi16(y[kt][2 * i + e]));
                            } else {
                                a[kt][2 * i] = y[kt][2 * i];
                                a[kt][2 * i + 1] = y[kt][2 * i + 1];
                            }
                        }
                    const int blk = (x * kWords + j) * kBlocks + e;
                    // The tile's sums start from 0 and are added in fp32: the tensor cores' additions truncate.
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float t[4];
#pragma unroll
                        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                            for (int part = 0; part < kParts; ++part)
                                if (kt == 0 && part == 0)
                                    mma_16816_zero<C::kF16>(t, a[kt][0], a[kt][1], a[kt][2], a[kt][3], pf[kt][part][nt][0], pf[kt][part][nt][1]);
                                else
                                    mma_16816<C::kF16>(t, a[kt][0], a[kt][1], a[kt][2], a[kt][3], pf[kt][part][nt][0], pf[kt][part][nt][1]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[blk][nt][i] += t[i];
                    }
                }
            }
        }
    }

    // Of a tile that some columns see in part: what V holds that is not finite becomes 0 in the tile, so that weights of 0
    // do not make it NaN.  True if there was some; window_repair has to account for it.
    __device__ __forceinline__ static bool screen(uint32_t v, uint32_t vs, int lane)
    {
        constexpr int kBytes = C::kFp4 ? kTile * C::kScaleRow : kTile * kRow;
        const uint32_t at = C::kFp4 ? vs : v;
        bool bad = false;
#pragma unroll 2
        for (int i = 16 * lane; i < kBytes; i += 512) {
            const uint4 w = lds128(at + i);
            bad = bad || (not_finite(w.x) | not_finite(w.y) | not_finite(w.z) | not_finite(w.w));
        }
        if (!__any_sync(0xffffffffu, bad))
            return false;
#pragma unroll 1
        for (int i = 4 * lane; i < kBytes; i += 128) {
            uint32_t w = lds32(at + i);
            constexpr int kTop = C::kFp4 || C::kFp8 ? 7 : 15;
            w &= ~((not_finite(w) >> kTop) * (kTop == 7 ? 0xFFu : 0xFFFFu));
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + i), "r"(w) : "memory");
        }
        __syncwarp();
        return true;
    }
    // The top bits of the elements (scales of a 4-bit cache) in w that are infinities or NaN.
    __device__ __forceinline__ static uint32_t not_finite(uint32_t w)
    {
        constexpr uint32_t kExp = C::kFp4 || KV == kKvE4m3 ? 0x7F7F7F7Fu : KV == kKvE5m2 ? 0x7C7C7C7Cu : KV == kKvF16 ? 0x7C007C00u : 0x7F807F80u;
        constexpr uint32_t kTop = C::kFp4 || C::kFp8 ? 0x80808080u : 0x80008000u;
        constexpr uint32_t kStep = C::kFp4 || KV == kKvE4m3 ? 0x01010101u : KV == kKvE5m2 ? 0x04040404u : KV == kKvF16 ? 0x04000400u : 0x00800080u;
        return ((w & kExp) + kStep) & kTop;
    }
    // Whether some sum is NaN (a type without infinities has NaN only beside NaN) of a column whose weights are numbers.
    __device__ __forceinline__ bool broken() const
    {
        bool any = false;
        if constexpr (C::kInf) {
            // a sum of them is NaN if one of them is (or needlessly)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = 0.f;
#pragma unroll
                    for (int s = 0; s < kSteps; ++s)
                        x += acc[s][nt][e] + acc[s][nt][e + 2];
                    any = any || (x != x && l[nt][e] == l[nt][e]);
                }
        }
        return any;
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
// V's element d of row v of a request.
template <class C>
__device__ __forceinline__ float window_element(const WindowParams &p, const WindowReq &req, int b, int head, int v, int d)
{
    int slot = window_pos(req, v), page = b;
    if (p.block_table) {
        const int blk = slot / p.page_size;
        slot -= blk * p.page_size;
        page = p.block_table[(long long)b * p.max_blocks + blk];
        page = (unsigned)page < (unsigned)p.num_pages ? page : 0;
    }
    const size_t row = (uint32_t)page * p.row_page + (uint32_t)slot * p.row_token + (uint32_t)head * p.row_head;
    if constexpr (C::kFp4) {
        const uint32_t w = p.v[row * C::kRow + d / 2];
        return f16x2_to_float2(e2m1x2_to_f16x2<0>(d & 1 ? w >> 4 : w)).x *
               fp8x2_to_float2<kKvE4m3>((uint16_t)p.vs[row * C::kScaleRow + d / 16]).x;
    } else if constexpr (C::kFp8)
        return fp8x2_to_float2<C::KV>((uint16_t)p.v[row * C::kRow + d]).x;
    else
        return x2_to_float2<C::kF16>(reinterpret_cast<const uint16_t *>(p.v + row * C::kRow)[d]).x;
}
// An infinite V element times a weight's part that is 0 or less than 0 is NaN, and in tiles that are seen in part V's
// elements that are not finite were left out.  Here a warp looks for them in rows [from, to) of a request, whose sums (or
// output, base null) it has just written, and adds those that a token sees to its columns with a bit in `ok` (columns whose
// weights are numbers; 0: there is nothing to do): what else was summed there does not matter.
template <class C>
__device__ __noinline__ void window_repair(const WindowParams &p, int b, int head, int from, int to, uint32_t ok, float *base)
{
    constexpr int D = C::D, kMine = D / 32;
    const int lane = threadIdx.x & 31;
    const WindowReq req = window_req(p, b, nullptr);
    __syncwarp();
    uint32_t found[kMine];   // of the lane's dims: bit i, token i sees infinity or NaN; bit 16 + i, -infinity or NaN
#pragma unroll
    for (int e = 0; e < kMine; ++e)
        found[e] = 0;
#pragma unroll 4
    for (int v = from; v < to; ++v) {
        float x[kMine];
        bool any = false;
#pragma unroll
        for (int e = 0; e < kMine; ++e) {
            x[e] = window_element<C>(p, req, b, head, v, lane + 32 * e);
            any = any || !(fabsf(x[e]) < __builtin_huge_valf());
        }
        if (any) {
            uint32_t who = 0;
#pragma unroll 1
            for (int i = 0; i < p.q_len; ++i)
                who |= WindowSight(p, req, i).sees(v) ? 1u << i : 0u;
#pragma unroll
            for (int e = 0; e < kMine; ++e) {
                if (fabsf(x[e]) < __builtin_huge_valf())
                    continue;
                found[e] |= x[e] < 0.f ? 0u : who;           // NaN: both
                found[e] |= x[e] > 0.f ? 0u : who << 16;
            }
        }
    }
#pragma unroll 1
    for (int col = 0; col < p.cols; ++col) {
        if (!(ok >> col & 1))
            continue;
        const int i = col / p.group;
#pragma unroll
        for (int e = 0; e < kMine; ++e) {
            float *at = (base ? base + col * D : p.o + window_out_row(p, b, head, col) * D) + lane + 32 * e;
            const bool plus = found[e] >> i & 1, minus = found[e] >> (16 + i) & 1;
            if (plus || minus) {
                const float x = (plus ? __builtin_huge_valf() : 0.f) - (minus ? __builtin_huge_valf() : 0.f);
                *at = *at != *at ? x : *at + x;
            }
        }
    }
}
// LSE from the reference exponent (log2) and the sum of weights.
__device__ __forceinline__ float window_lse(float m, float l)
{
    return l == 0.f ? -__builtin_huge_valf() : ((m == -__builtin_huge_valf() ? 0.f : m) + log2f(l)) * 0.6931471805599453f;
}

// The CTA's copy of the schedule: prefix and non-empty requests in shared memory.  Returns the tiles of the longest
// segment.
template <int TILE>
__device__ __forceinline__ int window_schedule(const WindowParams &p, int *prefix, int *nonempty, int *tmp, bool report)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int heads = p.hkv / p.team;
    int run = 0, live = 0, most = 0;
    if (p.batch <= 32) {   // every warp for itself
        const int n = lane < p.batch ? (int)(((unsigned)window_req(p, lane, report && warp == 0 ? p.ws_err : nullptr).rows + TILE - 1) / TILE) : 0;
        const uint32_t full = __ballot_sync(0xffffffffu, n > 0);
        int x = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off)
                x += a;
        }
        if (warp == 0) {
            if (lane < p.batch) {
                prefix[lane + 1] = x * heads;
                nonempty[lane + 1] = __popc(full & (2u << lane) - 1);
            }
            if (lane == 0)
                prefix[0] = nonempty[0] = 0;
        }
        __syncthreads();
        return __reduce_max_sync(0xffffffffu, n);
    }
    for (int b0 = 0; b0 < p.batch; b0 += blockDim.x) {
        const int b = b0 + threadIdx.x;
        int n = 0;
        if (b < p.batch)
            n = (int)(((unsigned)window_req(p, b, report ? p.ws_err : nullptr).rows + TILE - 1) / TILE);   // rows may be close to 2^31
        int x = n * heads, y = n > 0 ? 1 : 0;
        const int mx = x, my = y, top = __reduce_max_sync(0xffffffffu, n);
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, x, off), c = __shfl_up_sync(0xffffffffu, y, off);
            if (lane >= off) {
                x += a;
                y += c;
            }
        }
        if (lane == 31) {
            tmp[3 * warp] = x;
            tmp[3 * warp + 1] = y;
            tmp[3 * warp + 2] = top;
        }
        __syncthreads();
        int bx = 0, by = 0, ax = 0, ay = 0;
        for (int w = 0; w < warps; ++w) {
            if (w == warp) {
                bx = ax;
                by = ay;
            }
            ax += tmp[3 * w];
            ay += tmp[3 * w + 1];
            most = max(most, tmp[3 * w + 2]);
        }
        if (b < p.batch) {
            prefix[b] = run + bx + x - mx;
            nonempty[b] = live + by + y - my;
        }
        run += ax;
        live += ay;
        if (b0 + blockDim.x < p.batch)
            __syncthreads();   // tmp is written again
    }
    if (threadIdx.x == 0) {
        prefix[p.batch] = run;
        nonempty[p.batch] = live;
    }
    __syncthreads();
    return most;
}

// The partials of a segment that workers w0 .. w1 share: one of each CTA, and one more of w1 if it went on to another
// segment.  n is 1 if one CTA (or worker) has it whole.
struct WindowParts {
    int w0, w1, c0, c1, n;
    bool apart;
    WindowParts() = default;
    __device__ __forceinline__ WindowParts(const WindowSchedule &s, int teams, int seg)
    {
        const int b = seg / s.hkv;
        const long long pos = s.seg_pos(b, seg - b * s.hkv), end = pos + (s.prefix[b + 1] - s.prefix[b]) / s.hkv;
        w0 = s.cta_at(pos);
        w1 = s.cta_at(end - 1);
        apart = w0 != w1 && end + s.w < s.total && s.cta_at(end + s.w) == w1;
        c0 = w0 / teams;
        c1 = (apart ? w1 - 1 : w1) / teams;
        n = c1 - c0 + 1 + (apart ? 1 : 0);
    }
    // Where partial k lies (in units of a team).
    __device__ __forceinline__ int slot(int teams, int k) const
    {
        return c0 + k > c1 ? 2 * w1 : 2 * max(w0, (c0 + k) * teams) + 1;
    }
};

// The segment of tile t.
__device__ __forceinline__ int segment_of_tile(const int *prefix, int batch, int heads, int t)
{
    const int b = request_of_tile(prefix, batch, t);
    return b * heads + (t - prefix[b]) / ((prefix[b + 1] - prefix[b]) / heads);
}

// Shared memory: the warps' rings, then prefix and non-empty [batch + 1], then scratch: the scan's sums,
// and what the warps hold at the end.
constexpr int kWindowScratch = kWindowMaxWarps * (3 + 2 * (2 + (int)(sizeof(WindowParts) / sizeof(int))));
template <class C>
constexpr size_t window_smem(int batch)
{
    return (size_t)C::kWarps * C::kRing + sizeof(int) * (2 * ((size_t)batch + 1) + kWindowScratch);
}

// Partials that a thread reads and adds together, 4 where no more are left.  Measured on GB300 with 4, 8, 16 and with both 4
// and 16 (us): 16 columns of one kv head over 65536 positions in 4 bits 37.4, 32.9, 30.8, 30.8; 29 requests of up to 4001
// positions, 12 columns of 64 dims in fp16 28.7, 28.8, 29.9, 28.9.
constexpr int kWindowTogether = 16;

template <class At>
__device__ __noinline__ float4 window_infinities(float4 sum, int n, At at)
{
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
        const float4 x = at(k);
        s.x += fabsf(x.x) < __builtin_huge_valf() ? 0.f : x.x;
        s.y += fabsf(x.y) < __builtin_huge_valf() ? 0.f : x.y;
        s.z += fabsf(x.z) < __builtin_huge_valf() ? 0.f : x.z;
        s.w += fabsf(x.w) < __builtin_huge_valf() ? 0.f : x.w;
    }
    return make_float4(sum.x == sum.x || s.x == 0.f ? sum.x : s.x, sum.y == sum.y || s.y == 0.f ? sum.y : s.y,
                       sum.z == sum.z || s.z == 0.f ? sum.z : s.z, sum.w == sum.w || s.w == 0.f ? sum.w : s.w);
}

// Sums of weights and of weighted V rows (4 dims) against the reference exponent `top`.
struct WindowSum {
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    float top = -__builtin_huge_valf(), l = 0.f;
    // Add N sums x with their references and weights ml (reference -inf: nothing).
    template <int N>
    __device__ __forceinline__ void add(const float2 (&ml)[N], const float4 (&x)[N])
    {
        float higher = top;
#pragma unroll
        for (int e = 0; e < N; ++e)
            higher = fmaxf(higher, ml[e].x);
        const float ref = higher == -__builtin_huge_valf() ? 0.f : higher, f = exp2_approx(top - ref);
        top = higher;
        l *= f;
        sum = make_float4(sum.x * f, sum.y * f, sum.z * f, sum.w * f);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float w = exp2_approx(ml[e].x - ref);
            l = fmaf(w, ml[e].y, l);
            sum.x = fmaf(w, x[e].x, sum.x);
            sum.y = fmaf(w, x[e].y, sum.y);
            sum.z = fmaf(w, x[e].z, sum.z);
            sum.w = fmaf(w, x[e].w, sum.w);
        }
    }
    // After sums at(0) .. at(n - 1) were added: an infinite one whose factor fp32 does not hold has made the sum NaN; the
    // sum is what the infinite ones (and NaN) come to.  (Factors of fp32's least normal number in place of 0 would keep
    // infinities too, but also 2^-14 of finite bf16 sums of 2^112; looking for them in each addition took 0.5 us of a short
    // call's 10.1 and 3.4 of the 26.3 of 5 requests of 16 columns, one kv head.)
    template <bool INF, class At>
    __device__ __forceinline__ void infinities(int n, At at)
    {
        if constexpr (INF) {
            const float any = (sum.x + sum.y) + (sum.z + sum.w);   // NaN if one of them is, or needlessly
            if (any != any)
                sum = window_infinities(sum, n, at);
        }
    }
    template <int D>
    __device__ __forceinline__ void store(const WindowParams &p, int b, int head, int col, int d, float shift) const
    {
        const long long row = window_out_row(p, b, head, col);
        const float f = l == 0.f ? 0.f : p.v_scale / l;
        *reinterpret_cast<float4 *>(p.o + row * D + d) = make_float4(sum.x * f, sum.y * f, sum.z * f, sum.w * f);
        if (d == 0 && p.lse)
            p.lse[row] = window_lse(top - shift, l);
    }
};

template <class C, bool PACK>
__global__ void __launch_bounds__(32 * C::kWarps, 1) window_kernel(const __grid_constant__ WindowParams p)
{
    using Warp = WindowWarp<C, PACK>;
    constexpr int NT = C::NT, D = C::D, kTile = C::kTile, kRow = C::kRow, kGran = C::kGran, kStages = C::kStages;
    constexpr int kMl = NT * 8 * 2;   // floats of (m, l) in front of a warp's sums
    static_assert(C::kRing >= C::kSums, "the ring holds a warp's sums at the end");
    extern __shared__ __align__(128) uint8_t smem[];
    int *prefix = reinterpret_cast<int *>(smem + C::kWarps * C::kRing);
    int *nonempty = prefix + p.batch + 1, *tmp = nonempty + p.batch + 1;
    int *s_seg = tmp + 3 * kWindowMaxWarps, *s_size = s_seg + 2 * kWindowMaxWarps;
    WindowParts *s_parts = reinterpret_cast<WindowParts *>(s_size + 2 * kWindowMaxWarps);
    int *s_list = tmp, *s_count = tmp + 2 * kWindowMaxWarps;   // the scan's sums are used up
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;

    pdl_launch_dependents();
    pdl_wait_prior_grid();
    const int most = window_schedule<kTile>(p, prefix, nonempty, tmp, blockIdx.x == 0);
    const int heads = p.hkv / p.team;
    for (int b = blockIdx.x; b < p.batch && nonempty[p.batch] < p.batch; b += gridDim.x)   // requests that see nothing
        if (prefix[b] == prefix[b + 1])
            for (int i = threadIdx.x; i < p.q_len * p.hq * (D / 4); i += blockDim.x) {
                const long long row = (long long)b * p.q_len * p.hq + i / (D / 4);
                *reinterpret_cast<float4 *>(p.o + row * D + i % (D / 4) * 4) = make_float4(0.f, 0.f, 0.f, 0.f);
                if (p.lse && i % (D / 4) == 0)
                    p.lse[row] = -__builtin_huge_valf();
            }
    WindowSchedule sch;
    sch.prefix = prefix;
    sch.nonempty = nonempty;
    sch.batch = p.batch;
    sch.hkv = heads;
    sch.w = kWindowSegCost;
    sch.total = sch.cost();
    const int team = warp / p.team, lead = warp - team * p.team;   // the warp's kv head of the team's
    // Short segments: a CTA has some whole, each shared by some of its warps, and nothing is left to join.
    const int segments = nonempty[p.batch] * heads, all_teams = C::kWarps / p.team;
    const int together = (segments + gridDim.x - 1) / gridDim.x, each = together > 0 && together <= all_teams ? all_teams / together : 0;
    const bool by_segment = each > 0 && (most + each - 1) / each <= prefix[p.batch] / (int)(gridDim.x * all_teams) + window_join_tiles(p.cols, D);
    const int grid = window_ctas(gridDim.x, segments, prefix[p.batch] / all_teams, p.cols, D);
    const int teams = by_segment ? all_teams : window_workers(sch.total, grid, all_teams);
    sch.P = grid * teams;
    sch.busy = sch.total < sch.P ? (int)sch.total : sch.P;
    const int worker = blockIdx.x * teams + team;
    int t0 = 0, t1 = 0;
    if (by_segment) {
        const int mine = blockIdx.x * together + team / each;
        if (team < each * together && mine < segments) {
            const int b = request_of_tile(nonempty, p.batch, mine / heads);
            const int nb = (prefix[b + 1] - prefix[b]) / heads, share = (nb + each - 1) / each, of = team % each;
            const int begin = prefix[b] + mine % heads * nb;
            t0 = begin + min(nb, of * share);
            t1 = begin + min(nb, (of + 1) * share);
        }
    } else if (team < teams && worker < sch.busy) {
        // odd lanes find the run's end
        const int t = sch.first_tile(worker + (lane & 1));
        t0 = __shfl_sync(0xffffffffu, t, 0);
        t1 = __shfl_sync(0xffffffffu, t, 1);
    }

    Warp w;
    w.q_at = smem_addr(smem) + warp * C::kRing + C::kStages * (C::kStage + kWindowAbout) + 8 * lane;
    int last = -1, begun = -1;   // the segments of the sums in the warp's ring, and of a partial that it ended
    if (t0 < t1) {
        const uint32_t ring = smem_addr(smem) + warp * C::kRing;
        const uint32_t meta = ring + kStages * C::kStage;   // of each tile: request, launch head, first row, kTile* and its rows; the request's rows, head, skip
        const uint64_t policy = l2_policy_evict_first();

        WindowCursor ld;
        auto request = [&](int b) {   // the request's tiles and rows
            const WindowReq r = window_req(p, b, nullptr);
            ld.b = b;
            ld.nb = (prefix[b + 1] - prefix[b]) / heads;
            ld.rows = r.rows;
            ld.head = r.head;
            ld.skip = r.first - r.head;
            ld.pages = p.block_table + (long long)b * p.max_blocks;
        };
        request(request_of_tile(prefix, p.batch, t0));
        ld.h = (t0 - prefix[ld.b]) / ld.nb;
        ld.j = t0 - prefix[ld.b] - ld.h * ld.nb;
        auto advance = [&]() {
            if (++ld.j < ld.nb)
                return;
            ld.j = 0;
            if (++ld.h < heads)
                return;
            ld.h = 0;
            int b = ld.b + 1;
            while (prefix[b + 1] == prefix[b])
                ++b;
            request(b);
        };
        // Lane's rows of the tile at ld: their pages, and their numbers within a page's rows.  Looked up one tile ahead of
        // the copies, which wait for them.  Rows behind the last are copies of it: their weights are 0.
        constexpr int kMine = kTile > 32 ? kTile / 32 : 1;
        int page[kMine];
        uint32_t in_page[kMine];
        auto position = [&](int row) { return row < ld.head ? row : row + ld.skip; };
        auto look_up = [&]() {
            const uint32_t head_row = (uint32_t)(ld.h * p.team + lead) * p.row_head;
#pragma unroll
            for (int m = 0; m < kMine; ++m) {
                int slot = position((int)min((unsigned)(ld.j * kTile + 32 * m + (lane & (kTile - 1))), (unsigned)(ld.rows - 1)));
                page[m] = ld.b;
                if (p.block_table) {
                    const int blk = p.page_shift >= 0 ? slot >> p.page_shift : (int)((unsigned)slot / (unsigned)p.page_size);
                    slot -= blk * p.page_size;
                    page[m] = ld.pages[blk];
                }
                in_page[m] = (uint32_t)slot * p.row_token + head_row;
            }
        };
        // Places of the lane's pieces: the first of a copy, and of every other copy.
        constexpr int kCopies = kTile * kGran / 32, kRows = 32 / kGran;   // copies of a lane, rows of a copy
        const uint8_t *from_k = p.k + 16 * (lane % kGran), *from_v = p.v + 16 * (lane % kGran);
        const uint32_t to_even = lane / kGran * kRow + ((lane % kGran ^ window_swizzle<kGran>(lane / kGran)) << 4);
        const uint32_t to_odd = lane / kGran * kRow + ((lane % kGran ^ window_swizzle<kGran>(lane / kGran + kRows)) << 4);
        auto copy = [&](int stage) {
            uint32_t row[kMine];
#pragma unroll
            for (int m = 0; m < kMine; ++m) {
                if ((unsigned)page[m] >= (unsigned)p.num_pages) {
                    page[m] = 0;
                    atomicOr(p.ws_err, kErrPage);
                }
                row[m] = (uint32_t)page[m] * p.row_page + in_page[m];
            }
            const int row0 = ld.j * kTile, n = min(kTile, ld.rows - row0);
            // is every row visible to every new token?
            bool plain = n == kTile;
            if (p.q_len > 1) {
                plain = plain && position(row0 + kTile - 1) <= ld.rows + ld.skip - p.q_len;
                if (p.window) {
                    const int behind = max(position(row0), ld.head + ld.skip);   // the first row behind the sinks
                    plain = plain && (row0 + kTile <= ld.head || ld.rows + ld.skip - 1 - behind < p.window);
                }
            }
            if (p.q_len > 1)
                sts128(meta + kWindowAbout * stage + 16, ld.rows, ld.head, ld.skip, 0);
            sts128(meta + kWindowAbout * stage, ld.b, ld.h, row0, n << kTileN | (plain ? kTilePlain : 0) | (ld.j == 0 ? kTileFirst : 0) |
                                                            (ld.j + 1 == ld.nb ? kTileLast : 0));
            const uint32_t k = ring + stage * C::kStage, even = k + to_even, odd = k + to_odd;
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const size_t at = (size_t)__shfl_sync(0xffffffffu, row[i * kRows / 32], (i * kRows + lane / kGran) & 31) * kRow;
                // the swizzle has a period of 4 rows: of 1, 2 or 4 copies
                const uint32_t to = kRows >= 4 ? even + i * kRows * kRow : kRows == 2 ? (i & 1 ? odd : even) + i * kRows * kRow
                                               : k + i * kRow + ((lane % kGran ^ window_swizzle<kGran>(i)) << 4);
                cp_async_16(to, from_k + at, policy);
                cp_async_16(to + kTile * kRow, from_v + at, policy);
            }
            if constexpr (C::kFp4) {
                constexpr int kS = C::kScaleRow;
                const uint32_t ks = k + 2 * kTile * kRow, vs = ks + kTile * kS;
                if constexpr (kTile >= 32) {
#pragma unroll
                    for (int m = 0; m < kMine; ++m) {
                        cp_async_small<kS>(ks + (32 * m + lane) * kS, p.ks + (size_t)row[m] * kS, policy);
                        cp_async_small<kS>(vs + (32 * m + lane) * kS, p.vs + (size_t)row[m] * kS, policy);
                    }
                } else   // rows of K for half the lanes, of V for the others
                    cp_async_small<kS>((lane < 16 ? ks : vs - 16 * kS) + lane * kS, (lane < 16 ? p.ks : p.vs) + (size_t)row[0] * kS, policy);
            }
        };

        int ahead = t0;   // tile at ld
        look_up();
        auto fetch = [&](int stage) {
            if (ahead < t1) {
                copy(stage);
                if (++ahead < t1) {
                    advance();
                    look_up();
                }
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i)
            fetch(i);
        // Who else has parts of the run's first and last segment is worked out while the tiles are on their way.
        if (lane < 2 && !by_segment)
            s_parts[lane * C::kWarps + warp] = WindowParts(sch, teams, segment_of_tile(prefix, p.batch, heads, lane ? t1 - 1 : t0));
        const WindowPlaces<C> places(g, c);
        int stage = 0, seg = -1;             // the tile's slot; the segment of the sums
        bool whole = false, dirty = false;   // the segment's first tile was the warp's; V was not finite in a tile seen in part
        int from = 0;                        // the first of the segment's rows that the warp has
        for (int t = t0; t < t1; ++t) {
            const uint32_t about = meta + kWindowAbout * stage;
            __syncwarp();
            const uint4 tile = lds128(about);
            if ((int)(tile.x * heads + tile.y) != seg) {   // the query is loaded while the tile is on its way
                seg = tile.x * heads + tile.y;
                w.start(p, tile.x, tile.y * p.team + lead, g, c);
                whole = tile.w & kTileFirst;
                dirty = false;
                from = tile.z;
            }
            cp_async_wait<kStages - 2>();
            __syncwarp();
            const uint32_t k = ring + stage * C::kStage, v = k + kTile * kRow, ks = v + kTile * kRow, vs = ks + kTile * C::kScaleRow;
            stage = stage + 1 == kStages ? 0 : stage + 1;
            fetch(stage);
            const int row0 = (int)tile.z, flags = (int)tile.w;
            float sc[Warp::KT][NT][4];
            uint32_t pf[Warp::KT][Warp::kParts][NT][2];
            w.scores(places, k, ks, sc);
            if (!(flags & kTilePlain)) {
                if (p.q_len == 1)
                    w.cut(flags >> kTileN, g, sc);
                else {
                    const uint4 what = lds128(about + 16);
                    const WindowReq req = {(int)(what.x + what.z), (int)what.y, (int)(what.y + what.z), (int)what.x};
                    w.mask(p, req, row0, g, c, sc);
                    dirty |= w.screen(v, vs, lane);
                }
            }
            w.rescale(sc);
            w.weights(sc, c, pf);
            w.values(places, v, vs, pf);
            const bool ends = flags & kTileLast;
            if (!ends && t + 1 < t1)
                continue;
            // The end of the segment, or of the run.  A segment that the warp has whole: its output.  One that it found
            // begun and whose end is inside the run: a partial.  Else: sums, left in the warp's own ring.
            const int b = (int)tile.x, head = (int)tile.y * p.team + lead;
            float *sums = nullptr, *ml = nullptr;
            if (!ends || (!whole && t + 1 == t1)) {
                ml = reinterpret_cast<float *>(smem + warp * C::kRing);
                sums = ml + kMl;
                last = seg;
                __syncwarp();   // the tile has been read
            } else if (!whole) {
                const long long slot = (long long)(2 * worker) * p.team + lead;
                ml = reinterpret_cast<float *>(p.ws_ml + slot * p.cols);
                sums = p.ws_o + slot * p.cols * D;
                begun = seg;
            }
            w.finish();
            uint32_t ok = 0;   // columns whose sums of weights are numbers
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int col = nt * 8 + 2 * c + e;
                    const float l = w.l[nt][e], ref = w.reference(nt, e);
                    ok |= l == l ? 1u << col : 0u;
                    if (col >= p.cols || (PACK && c >= 2))
                        continue;
                    float *dst = sums + col * D;
                    float f = 1.f;
                    if (!sums) {
                        const long long row = window_out_row(p, b, head, col);
                        dst = p.o + row * D;
                        f = l == 0.f ? 0.f : p.v_scale / l;
                        if (g == 0 && p.lse)
                            p.lse[row] = window_lse(ref - Warp::kShift, l);
                    } else if (g == 0)
                        *reinterpret_cast<float2 *>(ml + 2 * col) = make_float2(ref, l);
#pragma unroll
                    for (int s = 0; s < Warp::kSteps; s += 2)
                        *reinterpret_cast<float4 *>(dst + Warp::block_dim(s, g)) =
                            make_float4(w.acc[s][nt][e] * f, w.acc[s][nt][e + 2] * f, w.acc[s + 1][nt][e] * f, w.acc[s + 1][nt][e + 2] * f);
                }
            if (__any_sync(0xffffffffu, dirty || w.broken())) {
                ok = __reduce_or_sync(0xffffffffu, ok) & ((1u << p.cols) - 1);
                if (ok)
                    window_repair<C>(p, b, head, from, row0 + (flags >> kTileN), ok, sums);
            }
            seg = -1;
        }
    }

    // What the CTA has of segments that others share: the partials of segments that its warps found begun (entries 0 ..
    // kWarps - 1), and its groups of warps that left sums of one segment (kWarps .. 2 kWarps - 1, at the group's first).
    if (lane == 0) {
        s_seg[warp] = begun;
        s_seg[C::kWarps + warp] = last;
        if (by_segment)
            s_parts[C::kWarps + warp].n = 1;
    }
    __syncthreads();
    if (warp == 0) {
        const int a = lane, seg = a < 2 * C::kWarps ? s_seg[a] : -1;
        int n = seg >= 0 && (a < C::kWarps || a < C::kWarps + p.team || s_seg[a - p.team] != seg) ? 1 : 0;
        const bool group = n && a >= C::kWarps;
        if (group)
            while (a + n * p.team < 2 * C::kWarps && s_seg[a + n * p.team] == seg)
                ++n;
        if (a < 2 * C::kWarps)
            s_size[a] = n;
        const uint32_t all = __ballot_sync(0xffffffffu, group);
        if (group)
            s_list[__popc(all & ((1u << lane) - 1))] = a;
        if (lane == 0)
            *s_count = __popc(all);
    }
    __syncthreads();
    const int items = p.cols * (D / 4);   // 4 dims of a column
    for (int i = threadIdx.x, end = *s_count * items; i < end; i += blockDim.x) {   // the groups' sums
        const int a = s_list[i / items], n = s_size[a], first = a - C::kWarps, of = first % p.team, seg = s_seg[a], b = seg / heads;
        const int col = i % items / (D / 4), d = 4 * (i % (D / 4));
        WindowSum x;
#pragma unroll 1
        for (int k0 = 0; k0 < n; k0 += 4) {
            float2 ml[4];
            float4 y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float *at = reinterpret_cast<const float *>(smem + (first + min(k0 + e, n - 1) * p.team) * C::kRing);
                ml[e] = k0 + e < n ? *reinterpret_cast<const float2 *>(at + 2 * col) : make_float2(-__builtin_huge_valf(), 0.f);
                y[e] = k0 + e < n ? *reinterpret_cast<const float4 *>(at + kMl + col * D + d) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            x.add(ml, y);
        }
        const float *sums = reinterpret_cast<const float *>(smem + first * C::kRing) + kMl + col * D + d;
        const int step = p.team * C::kRing / (int)sizeof(float);
        x.infinities<C::kInf>(n, [=](int k) { return *reinterpret_cast<const float4 *>(sums + k * step); });
        if (s_parts[a].n == 1)
            x.store<D>(p, b, (seg - b * heads) * p.team + of, col, d, Warp::kShift);
        else {
            const long long slot = (long long)(2 * (blockIdx.x * teams + first / p.team) + 1) * p.team + of;
            *reinterpret_cast<float4 *>(p.ws_o + (slot * p.cols + col) * D + d) = x.sum;
            if (d == 0)
                p.ws_ml[slot * p.cols + col] = make_float2(x.top, x.l);
        }
    }

    // The CTA that writes the last partial of a segment adds them up, in the order of the workers.
    __syncthreads();
    if (warp == 0) {
        bool merge = false;
        if (lane < 2 * C::kWarps && s_size[lane] > 0 && s_parts[lane].n > 1) {
            unsigned int *count = p.ws_counts + s_parts[lane].w0 * p.team + lane % C::kWarps % p.team;
            __threadfence();   // the CTA's partials before the count, and the others' after it
            merge = atomicAdd(count, 1u) == (unsigned)s_parts[lane].n - 1;
            __threadfence();
            if (merge)
                *count = 0;
        }
        const uint32_t all = __ballot_sync(0xffffffffu, merge);
        if (merge)
            s_list[__popc(all & ((1u << lane) - 1))] = lane;
        if (lane == 0)
            *s_count = __popc(all);
    }
    __syncthreads();
    const int merges = *s_count;
    if (merges == 0)
        return;
    // Threads share the (segment, 4 dims) pairs, or several share the partials of one.
    const int total = merges * items, per = min(total, (int)blockDim.x), split = blockDim.x / per, mine = threadIdx.x / per;
    WindowSum *shared = reinterpret_cast<WindowSum *>(smem);
    for (int i0 = 0; i0 < total; i0 += per) {
        const int i = i0 + threadIdx.x - mine * per;
        const bool active = mine < split && i < total;
        int a = 0, b = 0, head = 0, col = 0, d = 0;
        WindowSum x;
        if (active) {
            a = s_list[i / items];
            const WindowParts parts = s_parts[a];
            const int seg = s_seg[a], of = a % C::kWarps % p.team;
            b = seg / heads;
            head = (seg - b * heads) * p.team + of;
            col = i % items / (D / 4);
            d = 4 * (i % (D / 4));
#pragma unroll 1
            for (int k0 = mine; k0 < parts.n;) {
                auto join = [&](auto width) {
                    constexpr int N = decltype(width)::value;
                    float2 ml[N];
                    float4 y[N];
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        ml[e] = make_float2(-__builtin_huge_valf(), 0.f);
                        y[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (k0 + e * split < parts.n) {
                            const long long slot = (long long)parts.slot(teams, k0 + e * split) * p.team + of;
                            ml[e] = __ldcg(p.ws_ml + slot * p.cols + col);
                            y[e] = __ldcg(reinterpret_cast<const float4 *>(p.ws_o + (slot * p.cols + col) * D + d));
                        }
                    }
                    x.add(ml, y);
                    k0 += N * split;
                };
                if (parts.n - k0 > 4 * split)
                    join(std::integral_constant<int, kWindowTogether>());
                else
                    join(std::integral_constant<int, 4>());
            }
        }
        if (split > 1) {   // then total < blockDim: one pass
            __syncthreads();
            if (active)
                shared[mine * per + i] = x;
            __syncthreads();
            if (active && mine == 0)
                for (int k = 1; k < split; ++k) {
                    const WindowSum &y = shared[k * per + i];
                    const float2 ml[1] = {make_float2(y.top, y.l)};
                    const float4 of[1] = {y.sum};
                    x.add(ml, of);
                }
        }
        if (active && mine == 0) {
            const WindowParts *parts = s_parts + a;
            const long long step = (long long)p.team * p.cols * D;
            const float *sums = p.ws_o + ((long long)(a % C::kWarps % p.team) * p.cols + col) * D + d;
            x.infinities<C::kInf>(parts->n, [=](int k) { return __ldcg(reinterpret_cast<const float4 *>(sums + parts->slot(teams, k) * step)); });
            x.store<D>(p, b, head, col, d, Warp::kShift);
        }
    }
}

template <class C, bool PACK>
cudaError_t launch_window_t(const WindowParams &p, const WindowLaunch &c)
{
    auto kernel = window_kernel<C, PACK>;
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
    if (c.start_event && !record_event(c.start_event, c.stream))
        return cudaErrorInvalidValue;
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
    if (e != cudaSuccess)
        return e;
    if (c.end_event && !record_event(c.end_event, c.stream))
        return cudaErrorInvalidValue;
    return cudaSuccess;
}

template <int D, int KV>
cudaError_t launch_window_variant(const WindowParams &p, const WindowLaunch &c)
{
    using One = WindowCfg<D, KV, 1>;
    using Two = WindowCfg<D, KV, 2>;
    static_assert(window_smem<One>(kMaxBatch) <= 232448 && window_smem<Two>(kMaxBatch) <= 232448, "fits the 227 KB of a CTA");
    if (p.cols > 8)
        return launch_window_t<Two, false>(p, c);
    if constexpr (One::kF16)
        if (p.cols <= 4)
            return launch_window_t<One, true>(p, c);
    return launch_window_t<One, false>(p, c);
}

}  // namespace fd
