// fd_tree_kernel.cuh -- the split kernel of the tree attention (sm_103a).
//
// One persistent CTA per SM takes a run of tiles (fd_tree.cuh).  Per tile of N
// positions and 128 query rows:
//
//     S = Q K^T        128 x N,  tcgen05, Q and K in shared memory, S in tensor memory
//     P = exp2(S scale log2(e) - m)   a thread per row: a running maximum m and sum l
//     O = O + P V      128 x D,  tcgen05, P in tensor memory, V in shared memory
//
//   * K and V tiles come into rings of shared-memory slots, in the 128-byte
//     swizzled layout that the MMAs read: parts of 64 dims, a part being N rows
//     of 128 bytes.  A warp for K and one for V load 16-bit caches by TMA.  FP8
//     codes come by TMA into rings of their own, and four warps convert them to
//     fp16 (every FP8 value is one), the type of that call's MMAs; a bf16 query
//     is then scaled by a power of two a row, so that fp16 holds it: an element
//     of less than 2^-29 of its row's largest loses bits, by at most 2^-40 of
//     that largest.  Pages under 8 tokens are copied by the four warps;
//   * one thread issues the MMAs; their completion releases the slots;
//   * two groups of 128 threads (one for D = 256, whose accumulator fills half
//     the tensor memory) hold one query row a thread and turn S into P in
//     place.  With up to 128 rows both groups have the same rows, and each takes
//     64 positions of every tile into an accumulator of its own; the two are
//     added at the end of the segment, and the next tile's scores are formed in
//     the other of two buffers meanwhile.  (With the groups on whole tiles in
//     turn, a score buffer each: 64K tokens of MHA 182 us instead of 171, 64
//     dims 154 instead of 136, 64-token pages 187 instead of 180.)  With more
//     rows, each group has 128 of its own and a score buffer, and takes every
//     tile: one group's exponentials run beside the other's MMAs.
//
// P is taken as a 16-bit part and its 16-bit remainder (two MMAs): outputs are
// fp32, and one bf16 part alone would leave an error of 2^-8.  The two parts
// of 32 positions, 16 + 16 columns, overwrite those positions' 32 columns of S.
//
// The accumulator is rescaled only when a row's maximum grew by more than
// 2^kSlack; until then the weights may exceed 1.
//
// The tensor cores cut an accumulator's low bits off at every MMA, towards
// zero: measured, 1.7e-8 of it a step, 2.9e-5 after 108 tiles of 16 MMAs.  So
// after kTreeFlush units an accumulator is added to fp32 sums that the CTA
// keeps in the workspace (in L2: a thread's row is its own), and starts again.
//
// What a row must not see must not reach it: a score outside the row's mask is
// dropped before the maximum, and V rows behind the last position are zeroed
// in shared memory.  Among the nodes, a V element that is not finite is zeroed
// too and added afterwards, to the rows that see its node (the end of
// tree_softmax).  In the context it goes through the MMAs: every row sees it.
// NaN comes out as NaN, but an infinity as itself or as NaN, by the signs of
// the weights' remainders and by what is rescaled by 0 (tree_infinities).
#pragma once

#include <atomic>

#include "fd_tree.cuh"

namespace fd {

// ---------------------------------------------------------------- PTX

__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 32 consecutive 32-bit columns of this thread's tensor-memory lane.  The
// registers are valid after tmem_wait_ld32, which takes them so that no use
// moves ahead of it.  These instructions want the whole warp together: behind
// code that lanes may take differently stands a __syncwarp.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                   "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
                   "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
// The same 32 columns and, per lane, the largest of them that is a number (NaN
// if none is).  Of a tile's 64 columns that takes 87 cycles with two warps a
// scheduler, and 257 with the maximum formed by three-way instructions.
__device__ __forceinline__ float tmem_ld32_max(uint32_t addr, uint32_t (&r)[32])
{
    float m;
    asm volatile("tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, %32, [%33];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                   "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
                   "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=f"(m)
                 : "r"(addr)
                 : "memory");
    return m;
}
__device__ __forceinline__ void tmem_wait_max(float &a, float &b)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+f"(a), "+f"(b) : : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
                 "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                 "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
                 "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
                 "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
                 : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                 "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Instruction descriptor of a dense kind::f16 MMA (A and B both fp16, or both
// bf16), fp32 accumulator: D format 1 = F32 (bits 4-5), A and B formats
// (7-9, 10-12; 0 = fp16, 1 = bf16), B major (16; 1 = N contiguous), N >> 3
// (17-22), M >> 4 (24-28).
__host__ __device__ constexpr uint32_t umma_idesc_f16(int m, int n, bool f16, bool b_n_major)
{
    return (1u << 4) | ((f16 ? 0u : 1u) << 7) | ((f16 ? 0u : 1u) << 10) | ((b_n_major ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Descriptor of an operand whose N (not K) is contiguous, in the 128-byte
// swizzled layout: a part holds 64 elements of N a row, one row a K index;
// groups of 8 rows are 1024 bytes apart (stride offset), parts part_bytes apart
// (leading offset).  Other fields as in umma_desc_sw128.
__device__ __forceinline__ uint64_t umma_desc_sw128_n_major(uint32_t addr, uint32_t part_bytes)
{
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(part_bytes >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// D[tmem] (+)= A B^T for one K step of 16 elements, A in shared or in tensor memory.
__device__ __forceinline__ void umma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
                 : "memory");
}
__device__ __forceinline__ void umma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
                 : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most N of this thread's groups of copies are in flight.
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void red_add_v4(float *at, float4 x)
{
    asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(at), "f"(x.x), "f"(x.y), "f"(x.z), "f"(x.w) : "memory");
}

// x minus the packed 16-bit pair w, exact when w is x rounded.
template <bool F16>
__device__ __forceinline__ float2 minus_x2(float2 x, uint32_t w)
{
    float2 r;
    if constexpr (F16)
        asm("{\n\t.reg .b16 lo, hi, m;\n\tmov.b32 {lo, hi}, %2;\n\tmov.b16 m, 0xBC00;\n\t"
            "fma.rn.f32.f16 %0, lo, m, %3;\n\tfma.rn.f32.f16 %1, hi, m, %4;\n\t}"
            : "=f"(r.x), "=f"(r.y)
            : "r"(w), "f"(x.x), "f"(x.y));
    else
        asm("{\n\t.reg .b16 lo, hi, m;\n\tmov.b32 {lo, hi}, %2;\n\tmov.b16 m, 0xBF80;\n\t"
            "fma.rn.f32.bf16 %0, lo, m, %3;\n\tfma.rn.f32.bf16 %1, hi, m, %4;\n\t}"
            : "=f"(r.x), "=f"(r.y)
            : "r"(w), "f"(x.x), "f"(x.y));
    return r;
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// A thread's register limit; all warps of a warpgroup execute it.
template <int N>
__device__ __forceinline__ void regs_more()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_fewer()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ uint64_t l2_policy_evict_normal()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

// ---------------------------------------------------------------- layout

constexpr int kTreeMaxSlots = 6;
constexpr int kTreeMaxRaw = 4;

template <int D, int LOAD>
struct TreeCfg {
    static constexpr int kN = tree_tile(D);
    static constexpr int kGroups = tree_groups(D);
    static constexpr int kSoftWarps = 4 * kGroups;
    static constexpr int kSoftThreads = 32 * kSoftWarps;
    static constexpr int kCopyWarps = LOAD == kTreeTma ? 0 : 4;   // they convert, or copy small pages
    static constexpr int kCopyThreads = 32 * kCopyWarps;
    static constexpr int kLoadWarp = kSoftWarps + kCopyWarps;     // K by TMA; the next one V
    static constexpr int kMmaWarp = kLoadWarp + 2;
    static constexpr int kWarps = kLoadWarp + 4;                  // whole warpgroups
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kParts = D / 64;
    static constexpr int kPartBytes = kN * 128;                   // of a K or V tile
    static constexpr int kSlotBytes = kParts * kPartBytes;
    static constexpr int kRawBytes = kN * D;                      // of a tile of FP8 codes
    static constexpr int kQBytes = 128 * D * 2;                   // 128 query rows
    static constexpr int kHalves = kN / 64;                       // of a tile's weights
    // Units between flushes: with shared rows an accumulator gets 64 positions of a unit, else all of them.
    static constexpr int kFlush = kTreeFlush, kFlushShared = 2 * kTreeFlush;
    // Registers.  A softmax thread wants some 160, more than an even share of
    // a block with the copying warps, which give some of theirs up (setmaxnreg).
    static constexpr bool kSplitRegs = kGroups == 2 && LOAD != kTreeTma;
    static constexpr int kLaunchRegs = 128, kSoftRegs = 160, kOtherRegs = 96;
    static_assert(!kSplitRegs || kSoftRegs * kSoftThreads + kOtherRegs * (kThreads - kSoftThreads) <= kLaunchRegs * kThreads,
                  "the shares come out of what the block was launched with");
    // tensor memory: two score buffers, then the accumulators
    static constexpr uint32_t kTmemO = 256;
    static constexpr uint32_t kTmemCols = 512;
};

struct TreeMisc {
    uint64_t kfull[kTreeMaxSlots], kempty[kTreeMaxSlots], vfull[kTreeMaxSlots], vempty[kTreeMaxSlots];
    uint64_t rkfull[kTreeMaxRaw], rkempty[kTreeMaxRaw], rvfull[kTreeMaxRaw], rvempty[kTreeMaxRaw];
    uint64_t sfull[2], pfull[2][2], pvdone[2], qfull, ofree, pair, drain;
    long long scan[18];
    long long segpos, x1;
    int b, seg, j, abort;
    uint32_t tmem;
    unsigned int bad[2][kMaxTree / 32];   // nodes whose V row is not finite, of even and odd segments
    int8_t power[2][128];                 // FP8: exponents of the powers of two that the rows were divided by
    // a softmax thread's maximum and sum at the end of a segment, when both groups have some of it
    float2 ml[2][128];
};

// A CTA's walk over its tiles, segment by segment; every role makes its own.
template <int D>
struct TreeWalk {
    int b, seg, j0, n;      // request, segment of it, its tiles [j0, j0 + n) are this CTA's
    long long segpos, x1;   // position of the segment's first tile, end of the CTA's positions
    TreeReq r;
    TreeSeg s;

    __device__ __forceinline__ void load(const TreeParams &p)
    {
        r = tree_req(p, b, nullptr);
        s = tree_seg<D>(p, r);
    }
    __device__ __forceinline__ void count()
    {
        const long long left = x1 - segpos;
        n = (int)(left < s.nb ? (left < 0 ? 0 : left) : s.nb) - j0;
    }
    __device__ __forceinline__ void start(const TreeParams &p, const TreeMisc &m)
    {
        b = m.b;
        seg = m.seg;
        j0 = m.j;
        segpos = m.segpos;
        x1 = m.x1;
        n = 0;
        if (b < p.batch) {
            load(p);
            count();
        }
    }
    __device__ __forceinline__ void next(const TreeParams &p)
    {
        segpos += s.nb + kTreeSegCost;
        j0 = 0;
        ++seg;
        while (seg >= s.segs) {
            seg = 0;
            if (++b >= p.batch) {
                n = 0;
                return;
            }
            load(p);
        }
        count();
    }
};

// Pool row of position pos of request b (contiguous or paged); a page out of range is page 0.
__device__ __forceinline__ int tree_page(const TreeParams &p, int b, int blk, bool report)
{
    int page = p.block_table[(long long)b * p.max_blocks + blk];
    if ((unsigned)page >= (unsigned)p.num_pages) {
        if (report)
            atomicOr(p.ws_err, kErrPage);
        page = 0;
    }
    return page;
}
__device__ __forceinline__ int tree_row(const TreeParams &p, int b, int pos, bool report)
{
    if (!p.block_table)
        return b * p.page_size + pos;
    const unsigned blk = (unsigned)pos / (unsigned)p.page_size;
    return tree_page(p, b, (int)blk, report) * p.page_size + (int)((unsigned)pos - blk * (unsigned)p.page_size);
}

// Which of the nodes n0 .. n0 + 31 row i sees, as bits; n0 < 0 are positions of
// the context, seen by every row.  Nodes from t on do not exist.
__device__ __forceinline__ uint32_t tree_bits(const TreeParams &p, const uint64_t *mask_row, int i, int n0, int t)
{
    if (n0 <= -32)
        return 0xffffffffu;
    const int s = max(n0, 0);
    uint32_t w = 0;
    if (s < t) {
        if (mask_row) {
            const int k = s >> 6, sh = s & 63;
            uint64_t x = mask_row[k] >> sh;
            if (sh > 32 && k + 1 < p.words)
                x |= mask_row[k + 1] << (64 - sh);
            w = (uint32_t)x;
        } else {
            const int seen = i - s + 1;   // nodes s .. i
            w = seen >= 32 ? 0xffffffffu : seen <= 0 ? 0u : (1u << seen) - 1u;
        }
        if (t - s < 32)
            w &= (1u << (t - s)) - 1u;
    }
    return n0 < 0 ? (w << -n0) | ((1u << -n0) - 1u) : w;
}

// ---------------------------------------------------------------- roles

// A ring of slots as one of its sides sees it.
struct TreeRing {
    int slot;
    uint32_t ph;
    __device__ __forceinline__ void next(int slots)
    {
        if (++slot == slots) {
            slot = 0;
            ph ^= 1u;
        }
    }
};

// K or V tiles by TMA, 16-bit ones as (box, part) pairs, FP8 codes as whole
// rows; a lane issues one copy.
template <int D, int LOAD, bool IS_K>
__device__ __forceinline__ void tree_load_tma(const TreeParams &p, TreeMisc &m, const CUtensorMap *map, uint32_t ring,
                                              int slots, int lane)
{
    using C = TreeCfg<D, LOAD>;
    constexpr bool kRaw = LOAD == kTreeConvert;
    constexpr int kParts = kRaw ? 1 : C::kParts, kRowBytes = kRaw ? D : 128;
    uint64_t *full = kRaw ? (IS_K ? m.rkfull : m.rvfull) : (IS_K ? m.kfull : m.vfull);
    uint64_t *empty = kRaw ? (IS_K ? m.rkempty : m.rvempty) : (IS_K ? m.kempty : m.vempty);
    volatile int *abort_flag = &m.abort;
    const int box = lane / kParts, part = lane % kParts;
    TreeRing r = {0, 0};
    int issued = 0;
    TreeWalk<D> w;
    bool ok = true;
    for (w.start(p, m); ok && w.n > 0; w.next(p)) {
        const int g = w.seg / w.s.groups;
        // row groups read the same tiles: those stay in L2
        const uint64_t policy = w.s.groups > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
        for (int j = w.j0; j < w.j0 + w.n; ++j) {
            const int t0 = j * C::kN;
            const int boxes = (min(C::kN, w.r.L - t0) + p.box_rows - 1) / p.box_rows;
            int row = 0;
            if (box < boxes)
                row = tree_row(p, w.b, t0 + box * p.box_rows, IS_K);
            ok = mbar_wait_bounded(smem_addr(&empty[r.slot]), r.ph ^ 1u, p.timeout_ns, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok)
                break;
            const uint32_t bar = smem_addr(&full[r.slot]);
            if (lane == 0)
                mbar_arrive_expect_tx(bar, (uint32_t)(boxes * kParts * p.box_rows * kRowBytes) +
                                               (IS_K && p.starve && issued == 0 && blockIdx.x == 0 ? 16u : 0u));
            __syncwarp();
            if (box < boxes)
                tma_load_3d(ring + r.slot * (kRaw ? C::kRawBytes : C::kSlotBytes) + part * C::kPartBytes +
                                box * p.box_rows * kRowBytes,
                            map, bar, part * 64, g, row, policy);
            ++issued;
            r.next(slots);
        }
    }
    if (lane == 0) {
        // Every release has arrived: nothing signals this CTA's barriers any
        // more.  Having given up, wait (bounded) for the copies in flight instead.
        for (int k = 0; ok && k < slots; ++k, r.next(slots))
            ok = mbar_wait_bounded(smem_addr(&empty[r.slot]), r.ph ^ 1u, p.timeout_ns, abort_flag);
        if (!ok) {
            atomicOr(p.ws_err, kErrTimeout);
            *abort_flag = 1;
            for (int k = max(0, issued - slots); k < issued; ++k)
                mbar_wait_bounded(smem_addr(&full[k % slots]), (uint32_t)(k / slots) & 1u, p.timeout_ns, nullptr);
        }
    }
    __syncwarp();
}

// One tile of FP8 codes (rows of D bytes) to the swizzled fp16 tile.  A unit is
// 16 codes; eight lanes that store together take 4 units of 2 rows, whose
// chunks fall into different banks.
template <int D, int KV>
__device__ __forceinline__ void tree_convert(uint32_t raw, uint32_t tile, int tid)
{
    using C = TreeCfg<D, kTreeConvert>;
    constexpr int kRowUnits = D / 16, kUnits = C::kN * kRowUnits;
    static_assert(kUnits % C::kCopyThreads == 0, "whole rounds");
    constexpr int kRounds = kUnits / C::kCopyThreads, kBatch = 4;
    // 8 lanes: units 4 n .. 4 n + 3 of rows 2 k, 2 k + 1.  From round to round a
    // thread stays on its unit and moves on by a multiple of 8 rows, so its
    // addresses move by constants.
    constexpr int kQuads = kRowUnits / 4, kRowStep = 2 * (C::kCopyThreads / 8) / kQuads;
    static_assert(kRounds % kBatch == 0 && kRowStep % 8 == 0, "whole batches and swizzle periods");
    const int row = 2 * (tid / 8 / kQuads) + ((tid & 7) >> 2), unit = 4 * (tid / 8 % kQuads) + (tid & 3), c = 2 * (unit & 3);
    const uint32_t from = raw + row * D + unit * 16;
    const uint32_t at = tile + (unit / 4) * C::kPartBytes + row * 128;
    const uint32_t to0 = at + ((c ^ (row & 7)) << 4), to1 = at + (((c + 1) ^ (row & 7)) << 4);
#pragma unroll
    for (int n = 0; n < kRounds; n += kBatch) {
        uint4 x[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            x[k] = lds128(from + (n + k) * kRowStep * D);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const uint4 lo = make_uint4(fp8x2_to_f16x2<KV>(lo16(x[k].x)), fp8x2_to_f16x2<KV>(hi16(x[k].x)),
                                        fp8x2_to_f16x2<KV>(lo16(x[k].y)), fp8x2_to_f16x2<KV>(hi16(x[k].y)));
            const uint4 hi = make_uint4(fp8x2_to_f16x2<KV>(lo16(x[k].z)), fp8x2_to_f16x2<KV>(hi16(x[k].z)),
                                        fp8x2_to_f16x2<KV>(lo16(x[k].w)), fp8x2_to_f16x2<KV>(hi16(x[k].w)));
            sts128(to0 + (n + k) * kRowStep * 128, lo);
            sts128(to1 + (n + k) * kRowStep * 128, hi);
        }
    }
}

// Small pages: one tile's rows by 128 threads, converted on the way if they
// are FP8 codes; 16-bit rows by asynchronous copies, complete after
// cp_async_wait.  A warp takes a quarter of the tile's rows; `rows` holds the
// pool row of its row `lane`.  Rows from `valid` on are left as they are.
template <int D, int KV>
__device__ __forceinline__ void tree_copy_rows(const TreeParams &p, const uint8_t *cache, int g, bool once, int rows,
                                               int valid, uint32_t tile, int warp, int lane)
{
    using C = TreeCfg<D, kTreeCopy>;
    constexpr int kRows = C::kN / C::kCopyWarps, kPieces = kv_is_fp8(KV) ? D / 16 : D / 8, kStep = 32 / kPieces;
    static_assert(kRows <= 32 && 32 % kPieces == 0, "a lane a row");
    const int piece = lane % kPieces;
    const uint8_t *base = cache + (size_t)g * D * (kv_is_fp8(KV) ? 1 : 2) + piece * 16;
    const size_t row_bytes = (size_t)p.hkv * D * (kv_is_fp8(KV) ? 1 : 2);
    if constexpr (kv_is_fp8(KV)) {
        constexpr int kBatch = 4;
        const int c = 2 * (piece & 3);
#pragma unroll 1
        for (int r0 = 0; r0 < kRows; r0 += kStep * kBatch) {
            uint4 x[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int r = r0 + k * kStep + lane / kPieces, from = __shfl_sync(0xffffffffu, rows, r & 31);
                x[k] = make_uint4(0, 0, 0, 0);
                if (r < kRows && warp * kRows + r < valid)
                    x[k] = ldg128_nc(base + (size_t)from * row_bytes);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int r = r0 + k * kStep + lane / kPieces, row = warp * kRows + r;
                if (r >= kRows || row >= valid)
                    continue;
                const uint32_t at = tile + (piece / 4) * C::kPartBytes + row * 128;
                sts128(at + ((c ^ (row & 7)) << 4),
                       make_uint4(fp8x2_to_f16x2<KV>(lo16(x[k].x)), fp8x2_to_f16x2<KV>(hi16(x[k].x)),
                                  fp8x2_to_f16x2<KV>(lo16(x[k].y)), fp8x2_to_f16x2<KV>(hi16(x[k].y))));
                sts128(at + (((c + 1) ^ (row & 7)) << 4),
                       make_uint4(fp8x2_to_f16x2<KV>(lo16(x[k].z)), fp8x2_to_f16x2<KV>(hi16(x[k].z)),
                                  fp8x2_to_f16x2<KV>(lo16(x[k].w)), fp8x2_to_f16x2<KV>(hi16(x[k].w))));
            }
        }
    } else {
        const uint64_t policy = once ? l2_policy_evict_first() : l2_policy_evict_normal();
#pragma unroll 4
        for (int r0 = 0; r0 < kRows; r0 += kStep) {
            const int r = r0 + lane / kPieces, from = __shfl_sync(0xffffffffu, rows, r & 31), row = warp * kRows + r;
            if (row < valid)
                cp_async_16(tile + (piece / 8) * C::kPartBytes + row * 128 + (((piece & 7) ^ (row & 7)) << 4),
                            base + (size_t)from * row_bytes, policy);
        }
    }
}

// The four warps that convert FP8 tiles, or copy small pages: K and V tiles in
// turn.  Copies of one tile run while the next one's are issued.
template <int D, int KV, int LOAD>
__device__ __forceinline__ void tree_copy(const TreeParams &p, TreeMisc &m, uint32_t k_ring, uint32_t v_ring,
                                          uint32_t raw_k, uint32_t raw_v, int tid)
{
    using C = TreeCfg<D, LOAD>;
    constexpr bool kAsync = LOAD == kTreeCopy && !kv_is_fp8(KV);
    volatile int *abort_flag = &m.abort;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        const bool r = mbar_wait_bounded(smem_addr(bar), parity, p.timeout_ns, abort_flag);
        return __all_sync(0xffffffffu, r) != 0;
    };
    TreeRing rk = {0, 0}, rv = {0, 0}, rr = {0, 0};
    uint64_t *pending = nullptr;   // the full barrier of a tile whose copies are in flight (the same in every thread)
    bool starve = LOAD == kTreeCopy && p.starve && blockIdx.x == 0 && tid == 0;
    auto finish = [&]() {
        fence_async_shared();      // the MMAs read what these threads wrote
        if (!starve)               // the test hook leaves out an arrival, so that the first tile never becomes full
            mbar_arrive(smem_addr(pending));
        starve = false;
        pending = nullptr;
    };
    bool ok = true;
    TreeWalk<D> w;
    for (w.start(p, m); ok && w.n > 0; w.next(p))
        for (int j = w.j0; ok && j < w.j0 + w.n; ++j) {
            const int t0 = j * C::kN, valid = min(C::kN, w.r.L - t0);
            [[maybe_unused]] int rows = 0;   // small pages: the pool row of this warp's row `lane`
            if constexpr (LOAD == kTreeCopy) {
                const int r = (tid >> 5) * (C::kN / C::kCopyWarps) + (tid & 31);
                if ((tid & 31) < C::kN / C::kCopyWarps && r < valid)
                    rows = tree_row(p, w.b, t0 + r, true);
            }
#pragma unroll 1
            for (int half = 0; ok && half < 2; ++half) {
                TreeRing &r = half ? rv : rk;
                uint64_t *full = half ? &m.vfull[r.slot] : &m.kfull[r.slot], *empty = half ? &m.vempty[r.slot] : &m.kempty[r.slot];
                const uint32_t tile = (half ? v_ring : k_ring) + r.slot * C::kSlotBytes;
                if (kAsync && pending && !__all_sync(0xffffffffu, mbar_try_wait(smem_addr(empty), r.ph ^ 1u))) {
                    // do not hold a tile back while waiting for a slot
                    cp_async_wait<0>();
                    finish();
                }
                if (!(ok = wait(empty, r.ph ^ 1u)))
                    break;
                if constexpr (LOAD == kTreeConvert) {
                    if (!(ok = wait(half ? &m.rvfull[rr.slot] : &m.rkfull[rr.slot], rr.ph)))
                        break;
                    tree_convert<D, KV>((half ? raw_v : raw_k) + rr.slot * C::kRawBytes, tile, tid);
                    mbar_arrive(smem_addr(half ? &m.rvempty[rr.slot] : &m.rkempty[rr.slot]));
                } else
                    tree_copy_rows<D, KV>(p, half ? p.v : p.k, w.seg / w.s.groups, w.s.groups == 1, rows, valid, tile,
                                          tid >> 5, tid & 31);
                if constexpr (kAsync) {
                    cp_async_commit();
                    if (pending) {
                        cp_async_wait<1>();
                        finish();
                    }
                    pending = full;
                } else {
                    pending = full;
                    finish();
                }
                r.next(half ? p.v_slots : p.k_slots);
            }
            if (LOAD == kTreeConvert)
                rr.next(p.raw_slots);
        }
    if (kAsync) {
        cp_async_wait<0>();
        if (ok && pending)
            finish();
    }
    // every release has arrived: nothing signals this CTA's barriers any more
    for (int k = 0; ok && k < p.k_slots; ++k, rk.next(p.k_slots))
        ok = wait(&m.kempty[rk.slot], rk.ph ^ 1u);
    for (int k = 0; ok && k < p.v_slots; ++k, rv.next(p.v_slots))
        ok = wait(&m.vempty[rv.slot], rv.ph ^ 1u);
    if (!ok) {
        atomicOr(p.ws_err, kErrTimeout);
        *abort_flag = 1;
    }
    __syncwarp();
}

// Groups with rows of their own in segment w; 0: both (or the only one) have the same rows.
template <int D>
__device__ __forceinline__ int tree_active(const TreeParams &p, const TreeWalk<D> &w)
{
    return p.rows == 128 ? 0 : (w.seg % w.s.groups) * 256 + 128 < w.r.t * p.group ? 2 : 1;
}

// How the MMAs of a segment follow one another.  With the same rows in both
// groups (or one group) unit u is tile u, in score buffer u & 1; with rows of
// their own, tile u / active for group u % active, each with a buffer.  (An
// issuer for each of the two groups, so that neither waits for the other's
// weights: 64 nodes x 8 heads over 4 x 32768 positions 337 us instead of 297.
// The groups then fall into step and the tensor core waits for both at once.)
struct TreeUnits {
    int active;
    __device__ __forceinline__ int buf(int u) const { return active == 1 ? 0 : u & 1; }
    __device__ __forceinline__ int ahead() const { return active == 1 ? 1 : 2; }
    __device__ __forceinline__ bool last_of_tile(int u) const { return active != 2 || (u & 1); }
    __device__ __forceinline__ bool first_of_tile(int u) const { return active != 2 || !(u & 1); }
};

// The MMA issuer: one warp, whose lanes all run the loop (so that addresses and
// descriptors stay in uniform registers) and whose elected lane issues.
template <int D, bool F16, int LOAD>
__device__ __forceinline__ void tree_mma(const TreeParams &p, TreeMisc &m, uint32_t q_smem, uint32_t k_ring,
                                         uint32_t v_ring, uint32_t tmem)
{
    using C = TreeCfg<D, LOAD>;
    constexpr uint32_t kIdescS = umma_idesc_f16(128, C::kN, F16, false);
    constexpr uint32_t kIdescO = umma_idesc_f16(128, D, F16, true);
    volatile int *abort_flag = &m.abort;
    const bool leader = elect_one();
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        const bool r = mbar_wait_bounded(smem_addr(bar), parity, p.timeout_ns, abort_flag);
        return __all_sync(0xffffffffu, r) != 0;
    };
    const uint32_t sfull0 = smem_addr(m.sfull), pvdone0 = smem_addr(m.pvdone), kempty0 = smem_addr(m.kempty),
                   vempty0 = smem_addr(m.vempty);
    // descriptors: the high words are constants, an address enters the low word
    const uint64_t desc_k = umma_desc_sw128(0), desc_v = umma_desc_sw128_n_major(0, C::kPartBytes);
    int ks = 0, vs = 0, segs = 0;   // the slot of the newest S's tile, and of the next P V's
    uint32_t kph = 0, vph = 0, pph = 0;
    TreeWalk<D> w;
    bool ok = true;
    for (w.start(p, m); ok && w.n > 0; w.next(p), ++segs) {
        const int active = tree_active<D>(p, w), units = active == 2 ? 2 * w.n : w.n;
        const TreeUnits un = {active};
        const int ahead = un.ahead();
        if (!(ok = wait(&m.qfull, segs & 1)))
            break;
        tc_fence_after();
        auto scores = [&](int u) {
            if (un.first_of_tile(u) && !wait(&m.kfull[ks], kph))
                return false;
            tc_fence_after();
            const int buf = un.buf(u);
            const bool last = un.last_of_tile(u);
            if (leader) {
                const uint64_t a = desc_k + ((q_smem + (active == 2 ? buf * C::kQBytes : 0)) >> 4);
                const uint64_t b = desc_k + ((k_ring + ks * C::kSlotBytes) >> 4);
                const uint32_t d = tmem + buf * C::kN;
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    umma_f16_ss(d, a + (((k / 4) * (128 * 128) + (k % 4) * 32) >> 4),
                                b + (((k / 4) * C::kPartBytes + (k % 4) * 32) >> 4), kIdescS, k > 0);
                umma_commit(sfull0 + 8 * buf);
                if (last)
                    umma_commit(kempty0 + 8 * ks);
            }
            __syncwarp();
            if (last && ++ks == p.k_slots) {
                ks = 0;
                kph ^= 1u;
            }
            return true;
        };
        for (int u = 0; ok && u < ahead && u < units; ++u)
            ok = scores(u);
        int nth = 0;   // of the accumulators: a unit that starts them, and one after a flush, overwrites
        for (int u = 0; ok && u < units; ++u) {
            const int buf = un.buf(u);
            const bool last = un.last_of_tile(u), halves = active == 0 && C::kGroups == 2;
            const uint32_t a = tmem + buf * C::kN;
            const uint64_t b = desc_v + ((v_ring + vs * C::kSlotBytes) >> 4);
#pragma unroll 1
            for (int half = 0; ok && half < C::kHalves; ++half) {
                if (!(ok = wait(&m.pfull[buf][half], (pph >> buf) & 1u)))
                    break;
                if (half == 0 && un.first_of_tile(u) && !(ok = wait(&m.vfull[vs], vph)))
                    break;
                // the accumulators of the last segment have been read
                if (half == 0 && u == 0 && segs > 0 && !(ok = wait(&m.ofree, (segs - 1) & 1)))
                    break;
                tc_fence_after();
                // each half has its group's accumulator, or both that of the unit's group
                const int acc = C::kGroups == 1 ? 0 : halves ? half : buf;
                const bool fresh = nth == 0 && (halves || half == 0);
                if (leader) {
                    const uint32_t d = tmem + C::kTmemO + acc * D, ah = a + 64 * half;
                    const uint64_t bh = b + (uint32_t)(half * 64 * 128 >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        umma_f16_ts(d, ah + (k / 2) * 32 + (k % 2) * 8, bh + (k * 16 * 128 >> 4), kIdescO, k > 0 || !fresh);
                        umma_f16_ts(d, ah + (k / 2) * 32 + (k % 2) * 8 + 16, bh + (k * 16 * 128 >> 4), kIdescO, true);
                    }
                    if (halves || half == C::kHalves - 1)
                        umma_commit(pvdone0 + 8 * acc);
                    if (last && half == C::kHalves - 1)
                        umma_commit(vempty0 + 8 * vs);
                }
                __syncwarp();
            }
            if (!ok)
                break;
            pph ^= 1u << buf;
            if (last && ++vs == p.v_slots) {
                vs = 0;
                vph ^= 1u;
            }
            if (active != 2 || (u & 1))
                nth = nth + 1 == (active == 0 ? C::kFlushShared : C::kFlush) ? 0 : nth + 1;
            if (u + ahead < units)
                ok = scores(u + ahead);
        }
    }
    if (!ok && leader) {
        atomicOr(p.ws_err, kErrTimeout);
        *abort_flag = 1;
        // gave up: the MMAs in flight end before the tensor memory is freed
        umma_commit(smem_addr(&m.drain));
        mbar_wait_bounded(smem_addr(&m.drain), 0, p.timeout_ns, nullptr);
    }
    __syncwarp();
}

// Query rows of a segment on their way into the swizzled operand: rows
// [first_row, first_row + 128) by THREADS threads, 8 (or fewer) 16-byte pieces
// of each in registers between fetch and store, BATCHES times.  Rows without a
// node are zero.  For FP8 caches (TO_F16) bf16 rows become fp16 ones divided by
// a power of two that brings their largest element to [2^14, 2^15).
template <int D, int THREADS, bool TO_F16>
struct TreeQuery {
    static constexpr int kChunks = D / 8, kStep = THREADS / kChunks, kRounds = 128 / kStep;
    static constexpr int kBatch = kRounds < 8 ? kRounds : 8, kBatches = kRounds / kBatch;
    uint4 x[kBatch];

    __device__ __forceinline__ void fetch(const TreeParams &p, const TreeWalk<D> &w, int first_row, int tid, int batch)
    {
        const int g = w.seg / w.s.groups, chunk = tid % kChunks;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int row = first_row + tid / kChunks + (batch * kBatch + k) * kStep, i = row / p.group, h = row - i * p.group;
            x[k] = make_uint4(0, 0, 0, 0);
            if (i < w.r.t)
                x[k] = __ldg(reinterpret_cast<const uint4 *>(
                                 p.q + (((long long)w.b * p.tree_len + i) * p.hq + g * p.group + h) * D) + chunk);
        }
    }
    // power, power2: where the rows' exponents go
    __device__ __forceinline__ void store(const TreeParams &p, uint32_t q_smem, int tid, int batch,
                                          [[maybe_unused]] int8_t *power, [[maybe_unused]] int8_t *power2)
    {
        const uint32_t flip = p.negate_q ? 0x80008000u : 0u;
        const int chunk = tid % kChunks;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int r = tid / kChunks + (batch * kBatch + k) * kStep;
            uint32_t v[4] = {x[k].x ^ flip, x[k].y ^ flip, x[k].z ^ flip, x[k].w ^ flip};
            if constexpr (TO_F16) {
                int ex = 0;
                if (!p.q_f16) {
                    float top = 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = bf16x2_to_float2(v[e]);
                        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
#pragma unroll
                    for (int off = kChunks / 2; off; off >>= 1)
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                    // kept where 2^(+-ex) are normal numbers (infinite: as the largest number)
                    ex = min(max((__float_as_int(top) >> 23 & 255) - 127 - 14, -120), 113);
                    const float down = __int_as_float((127 - ex) << 23);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = bf16x2_to_float2(v[e]);
                        v[e] = pack_f16x2(f.x * down, f.y * down);
                    }
                }
                if (chunk == 0) {
                    power[r] = (int8_t)ex;
                    power2[r] = (int8_t)ex;
                }
            }
            sts128(q_smem + (chunk / 8) * (128 * 128) + r * 128 + (((chunk & 7) ^ (r & 7)) << 4), make_uint4(v[0], v[1], v[2], v[3]));
        }
    }
};

// V tile rows [from, upto): those at or past `valid` become zero, and in the
// others (tree nodes) elements that are not finite do, their node marked in bad.
template <int D, bool F16, int LOAD>
__device__ __forceinline__ void tree_clean_v(uint32_t tile, int from, int upto, int valid, int node0, unsigned int *bad, int tid)
{
    using C = TreeCfg<D, LOAD>;
    constexpr int kChunks = D / 8;
    constexpr uint32_t kExp = F16 ? 0x7c00u : 0x7f80u;
    for (int e = from * kChunks + tid; e < upto * kChunks; e += 128) {
        const int row = e / kChunks, chunk = e % kChunks;
        const uint32_t at = tile + (chunk / 8) * C::kPartBytes + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
        if (row >= valid) {
            sts128(at, make_uint4(0, 0, 0, 0));
            continue;
        }
        const uint4 v = lds128(at);
        uint32_t x[4] = {v.x, v.y, v.z, v.w};
        bool hit = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if ((x[k] & kExp) == kExp) {
                x[k] &= 0xffff0000u;
                hit = true;
            }
            if ((x[k] & (kExp << 16)) == kExp << 16) {
                x[k] &= 0x0000ffffu;
                hit = true;
            }
        }
        if (hit) {
            sts128(at, make_uint4(x[0], x[1], x[2], x[3]));
            const int node = node0 + row;
            atomicOr(&bad[node >> 5], 1u << (node & 31));
        }
    }
}

// Element e of a K or V row as fp32, for values that are not finite.
template <bool F16, int KV>
__device__ __forceinline__ float tree_element(const uint8_t *cache, long long e)
{
    if constexpr (kv_is_fp8(KV))
        return fp8x2_to_float2<KV>(cache[e]).x;
    else
        return x2_to_float2<F16>(reinterpret_cast<const uint16_t *>(cache)[e]).x;
}

// Infinities of the context.  An infinite V element takes an infinite amount
// into its dim, whatever its weight; in the MMAs that is infinity times a
// weight's two parts, one of which may be 0 or of the other sign, and NaN then.
// So when an output is NaN though no score was, a warp looks through the V rows
// [from, to) of its CTA's part of the context for what is not finite, and the
// rows' outputs in those dims (c0 to c1) are set to what all of it adds up to.
// cache: V's rows of the kv head, of the whole pool with the request's blocks in
// table, of the request without.
// Nothing is read otherwise; when it is (or for a NaN), each warp reads it all,
// 4 KB at a time: 1 M positions in one CTA take 84 ms instead of 9.  Not inlined,
// so that the code that every segment runs stays together (one short request 17.4
// us, inlined 17.65).
template <int D, bool F16, int KV>
__device__ __noinline__ void tree_infinities(const uint8_t *cache, long long row_bytes, const int32_t *table, int page_size,
                                             int num_pages, int from, int to, int c0, int c1, bool mine, float *dst, int stride)
{
    constexpr int kBytes = kv_is_fp8(KV) ? 1 : 2, kPer = 16 / kBytes, kPieces = D / kPer, kRows = 32 / kPieces;
    constexpr uint32_t kExp = kv_is_fp8(KV) ? 0x7cu : F16 ? 0x7c00u : 0x7f80u, kSign = kv_is_fp8(KV) ? 0x80u : 0x8000u;
    // in every element of a word: its sign bit; what carries an exponent of ones into it
    constexpr uint32_t kOnes = kv_is_fp8(KV) ? 0x01010101u : 0x00010001u, kSigns = kOnes * kSign, kCarry = kOnes * (kSign - kExp);
    constexpr int kBatch = 8;   // steps whose loads are in flight together
    static_assert(KV != kKvE4m3 && kPieces <= 32, "E4M3 has no infinities");
    uint32_t plus = 0, minus = 0, nan = 0;   // a bit for each element of this lane's piece of a row
    const int lane = threadIdx.x & 31;
    const uint8_t *piece = cache + lane % kPieces * 16;
    const unsigned end = max(to, 0);
#pragma unroll 1
    for (unsigned n = from + lane / kPieces; n < end; n += kRows * kBatch) {
        uint4 v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const unsigned pos = min(n + k * kRows, end - 1);   // the last row more than once does no harm
            long long row = pos;
            if (table) {
                const unsigned blk = pos / (unsigned)page_size, page = (unsigned)table[blk];
                row = (long long)(page < (unsigned)num_pages ? page : 0u) * page_size + (pos - blk * (unsigned)page_size);
            }
            v[k] = ldg128_nc(piece + row * row_bytes);
        }
        auto odd = [&](uint32_t x) { return (x & ~kSigns) + kCarry; };
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const uint32_t x[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
            if (!((odd(x[0]) | odd(x[1]) | odd(x[2]) | odd(x[3])) & kSigns))
                continue;
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const uint32_t y = x[e * kBytes / 4] >> (e * kBytes % 4 * 8) & (kSign * 2 - 1);
                if ((y & kExp) == kExp)
                    (y & (kExp ^ (kSign - 1)) ? nan : y & kSign ? minus : plus) |= 1u << e;
            }
        }
    }
    __syncwarp();
    for (int off = kPieces; off < 32; off <<= 1) {
        plus |= __shfl_xor_sync(0xffffffffu, plus, off);
        minus |= __shfl_xor_sync(0xffffffffu, minus, off);
        nan |= __shfl_xor_sync(0xffffffffu, nan, off);
    }
    for (int k = c0 / kPer; k < c1 / kPer; ++k) {
        const uint32_t up = __shfl_sync(0xffffffffu, plus, k), down = __shfl_sync(0xffffffffu, minus, k),
                       none = __shfl_sync(0xffffffffu, nan, k) | (up & down);
        for (uint32_t left = up | down | none; mine && left; left &= left - 1) {
            const int e = __ffs(left) - 1, d = k * kPer + e;
            dst[(d / 4) * stride + d % 4] = __uint_as_float(none >> e & 1u ? 0x7fffffffu : up >> e & 1u ? 0x7f800000u : 0xff800000u);
        }
    }
}

// A group of 128 threads, one query row each.
template <int D, bool F16, int KV, int LOAD>
__device__ __forceinline__ void tree_softmax(const TreeParams &p, TreeMisc &m, uint32_t q_smem, uint32_t v_ring,
                                             uint32_t tmem)
{
    using C = TreeCfg<D, LOAD>;
    // fp16 weights: 2^8 more keeps weights down to 2^-33 of the largest among
    // the 16-bit parts (fp16 ends at 2^-25), and 2^7 of slack ends at 2^15.
    constexpr float kShift = F16 ? 8.f : 0.f, kSlack = F16 ? 7.f : 8.f;
    // A weight's remainder by fused instructions that take the 16-bit part as it
    // is, or widened first, which is two instructions more a pair on another
    // pipe.  The first way costs 67.8 us instead of 69.7 for 16 ragged requests,
    // 293 instead of 298 for 512 rows, 275 instead of 280 for 4-token pages; but
    // 203 instead of 200 beside the converting warps, and 141 instead of 137 for 64 dims.
    constexpr bool kMixed = D > 64 && !kv_is_fp8(KV);
    constexpr float kNegInf = -__builtin_huge_valf();
    const int tid = threadIdx.x & 127, group = threadIdx.x >> 7, lane_base = (threadIdx.x >> 5 & 3) << 5;
    volatile int *abort_flag = &m.abort;
    const bool own_rows = p.rows == 256;             // each group has its own 128 rows
    const bool shared_rows = C::kGroups == 2 && !own_rows;
    const uint32_t t_lane = tmem + ((uint32_t)lane_base << 16);
    const uint32_t t_o = t_lane + C::kTmemO + (C::kGroups == 2 ? group * D : 0);
    float sl = p.scale_log2;                         // FP8: times the row's power of two
    uint32_t qph = 0, sph = 0, pvph = 0, pairph = 0;
    int vcount = 0;                                  // tiles before the current segment
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        // all lanes take part; a lane that gives up takes its warp with it
        const bool r = mbar_wait_bounded(smem_addr(bar), parity, p.timeout_ns, abort_flag);
        return __all_sync(0xffffffffu, r) != 0;
    };
    auto pair_sync = [&]() {
        mbar_arrive(smem_addr(&m.pair));
        const bool r = wait(&m.pair, pairph);
        pairph ^= 1u;
        return r;
    };
    // this thread's sums of the units before the last flush, relative to the maximum then
    float *sums = p.ws_sums + ((long long)(blockIdx.x * C::kGroups + group) * (D / 4) * p.sum_rows + tid) * 4;
    const bool has_sums = tid < p.sum_rows;
    float ref = kNegInf;   // the maximum that the sums are relative to: the one at the segment's first flush
    // sums += accumulator * 2^((now - ref) scale), by reductions that nothing waits
    // for: the rows are this thread's own, so their order is the program's
    auto flush_sums = [&](bool fresh, float now) {
        if (fresh || ref == kNegInf)
            ref = now;   // nothing was added yet, or only zeros
        float up = now == kNegInf ? 0.f : (now - ref) * sl;
        if (!fresh && __any_sync(0xffffffffu, up > 60.f)) {   // rare: move the reference
            const float corr = exp2_approx(-up);
            if (has_sums)
#pragma unroll 1
                for (int c = 0; c < D / 4; ++c) {
                    float4 *at = reinterpret_cast<float4 *>(sums + (long long)c * p.sum_rows * 4);
                    const float4 x = __ldcg(at);
                    *at = make_float4(x.x * corr, x.y * corr, x.z * corr, x.w * corr);
                }
            ref = now;
            up = 0.f;
        }
        const float scale = exp2_approx(up);
        __syncwarp();
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(t_o + 32 * c, o);
            tmem_wait_ld32(o);
            if (has_sums) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    float *at = sums + (long long)(8 * c + k) * p.sum_rows * 4;
                    const float4 x = make_float4(__uint_as_float(o[4 * k]) * scale, __uint_as_float(o[4 * k + 1]) * scale,
                                                 __uint_as_float(o[4 * k + 2]) * scale, __uint_as_float(o[4 * k + 3]) * scale);
                    if (fresh)
                        *reinterpret_cast<float4 *>(at) = x;
                    else
                        red_add_v4(at, x);
                }
            }
            __syncwarp();
        }
        tc_fence_before();
    };
    TreeWalk<D> w;
    w.start(p, m);
    // the rows of a segment, fetched early (with one set of rows, by all
    // threads) and stored when the MMAs are done with those before
    auto first_row = [&](const TreeWalk<D> &of) { return (of.seg % of.s.groups) * p.rows; };
    TreeQuery<D, C::kSoftThreads, kv_is_fp8(KV)> q_all;
    auto fetch_q = [&](const TreeWalk<D> &of) {
        if (!own_rows)
            q_all.fetch(p, of, first_row(of), threadIdx.x, 0);
    };
    auto store_q = [&](const TreeWalk<D> &of) {
        if (!own_rows) {
            q_all.store(p, q_smem, threadIdx.x, 0, m.power[0], m.power[1]);
            if constexpr (q_all.kBatches > 1) {
#pragma unroll 1
                for (int n = 1; n < q_all.kBatches; ++n) {
                    q_all.fetch(p, of, first_row(of), threadIdx.x, n);
                    q_all.store(p, q_smem, threadIdx.x, n, m.power[0], m.power[1]);
                }
            }
        } else {
            TreeQuery<D, 128, kv_is_fp8(KV)> q_own;
#pragma unroll 1
            for (int n = 0; n < q_own.kBatches; ++n) {
                q_own.fetch(p, of, first_row(of) + group * 128, tid, n);
                q_own.store(p, q_smem + group * C::kQBytes, tid, n, m.power[group], m.power[group]);
            }
        }
        fence_async_shared();
        mbar_arrive(smem_addr(&m.qfull));
    };
    if (w.n > 0) {
        fetch_q(w);
        store_q(w);
    }
    int odd = 0;   // segments, modulo 2
    while (w.n > 0) {
        const int L = w.r.L, t = w.r.t, base = L - t;
        const int row = (w.seg % w.s.groups) * p.rows + (own_rows ? group * 128 : 0) + tid;
        const int i = row / p.group, h = row - i * p.group;
        const bool in_call = i < p.tree_len, live = i < t && base + i >= 0;
        const bool warp_live = __any_sync(0xffffffffu, live);
        const uint64_t *mask_row = p.mask && in_call ? p.mask + w.b * p.mask_stride + (long long)i * p.words : nullptr;
        if constexpr (kv_is_fp8(KV)) {
            if (!(ok = wait(&m.qfull, qph)))
                break;
            qph ^= 1u;
            sl = fmaxf(p.scale_log2 * __int_as_float((127 + m.power[group][tid]) << 23), kTreeLeastScale);
        }
        float mx = kNegInf, l = 0.f;
        int since = 0;                               // units since the start or the last flush
        bool flushed = false;
        // own rows: whole tiles; shared: this group's 64 positions of every tile
        const int end = own_rows && group >= tree_active<D>(p, w) ? 0 : w.n;
        const int columns = own_rows ? C::kN : 64, col0 = shared_rows ? 64 * group : 0;
        const int flush_every = own_rows ? C::kFlush : C::kFlushShared;
        uint64_t *pvdone = &m.pvdone[C::kGroups == 2 ? group : 0];
        for (int u = 0; u < end; ++u, ++since) {   // tiles
            const int buf = own_rows ? group : u & 1;
            const int t0 = (w.j0 + u) * C::kN + col0;   // the first position of this group's
            const uint32_t t_s = t_lane + buf * C::kN + col0;
            const bool tail = columns > base - t0;   // t0 + columns may be 2^31
            if (!(ok = wait(&m.sfull[buf], (sph >> buf) & 1u)))
                break;
            sph ^= 1u << buf;
            tc_fence_after();
            const bool flush = since == flush_every;
            if (!own_rows && flush && !(ok = wait(pvdone, pvph ^ 1u)))
                break;
            if (flush) {
                tc_fence_after();
                if (warp_live)
                    flush_sums(!flushed, mx);
                since = 0;
                flushed = true;
            }
            float mx_off = 0.f;
            if (warp_live) {
                // Two passes over the row's scores: the maximum, which the loads
                // form, then the weights, 32 columns at a time.  The loops stay
                // small for the instruction cache (with a tile unrolled and its
                // scores in registers, a third of the cycles went to fetching
                // instructions).  What the row does not see becomes -inf in
                // tensor memory, so neither pass needs a mask.
                if (tail) {
#pragma unroll 1
                    for (int c = 0; c < columns / 32; ++c) {
                        uint32_t s[32];
                        tmem_ld32(t_s + 32 * c, s);
                        const uint32_t bits = live ? tree_bits(p, mask_row, i, t0 + 32 * c - base, t) : 0u;
                        __syncwarp();
                        tmem_wait_ld32(s);
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            s[k] = bits >> k & 1u ? s[k] : 0xff800000u;
                        tmem_st32(t_s + 32 * c, s);
                    }
                    tmem_wait_st();
                }
                float tm = kNegInf;
#pragma unroll 1
                for (int c = 0; c < columns; c += 64) {
                    uint32_t s0[32], s1[32];
                    float m0 = tmem_ld32_max(t_s + c, s0), m1 = tmem_ld32_max(t_s + c + 32, s1);
                    tmem_wait_max(m0, m1);
                    tm = fmaxf(tm, fmaxf(m0, m1));
                }
                const bool grow = tm > mx && (mx == kNegInf || (tm - mx) * sl > kSlack);
                if (__any_sync(0xffffffffu, grow)) {
                    const float corr = grow ? (mx == kNegInf ? 0.f : exp2_approx((mx - tm) * sl)) : 1.f;
                    if (grow)
                        mx = tm;
                    l *= corr;
                    if (since > 0) {   // at the start, and after a flush there is nothing to rescale
                        // with own rows the score that was waited for follows this
                        // accumulator's last MMAs; with two score buffers the last unit's
                        // may still run
                        if (!own_rows && !(ok = wait(pvdone, pvph ^ 1u)))
                            break;
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t o[16];
                            tmem_ld16(t_o + 16 * c, o);
                            tmem_wait_ld16(o);
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                o[k] = __float_as_uint(__uint_as_float(o[k]) * corr);
                            tmem_st16(t_o + 16 * c, o);
                        }
                    }
                }
                mx_off = kShift - (mx == kNegInf ? 0.f : mx * sl);
            }
            if (tail && (!own_rows || group == 0)) {
                // the V rows of these weights (with own rows the first group cleans for both)
                const int vs = (vcount + u) % p.v_slots;
                if (!(ok = wait(&m.vfull[vs], ((vcount + u) / p.v_slots) & 1)))
                    break;
                tree_clean_v<D, F16, LOAD>(v_ring + vs * C::kSlotBytes, col0 + max(0, base - t0), col0 + columns,
                                           L - t0 + col0, t0 - col0 - base, m.bad[odd], tid);
                fence_async_shared();
                __syncwarp();
            }
            // A barrier's phases are told apart by parity alone: each has to be waited
            // for before the next but one can end.  The last unit's MMAs are waited
            // for below; those before them here, as long as the last cannot run.
            if (!own_rows && u > 0 && u + 1 == end && !(ok = wait(pvdone, pvph ^ 1u)))
                break;
            // The weights, 64 positions at a time: the MMAs of the first half
            // run beside the exponentials of the second.
            const float2 sl2 = make_float2(sl, sl), off2 = make_float2(mx_off, mx_off), one2 = make_float2(1.f, 1.f),
                         neg2 = make_float2(-1.f, -1.f);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            auto weights = [&](int c, uint32_t (&s)[32]) {
                float2 x[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    x[k] = fma2(make_float2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), sl2, off2);
                    x[k].x = exp2_approx(x[k].x);
                    x[k].y = exp2_approx(x[k].y);
                }
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    sum[k & 1] = fma2(x[k], one2, sum[k & 1]);
                    s[k] = pack_x2<F16>(x[k].x, x[k].y);
                    const float2 rest = kMixed ? minus_x2<F16>(x[k], s[k]) : fma2(x2_to_float2<F16>(s[k]), neg2, x[k]);
                    s[16 + k] = pack_x2<F16>(rest.x, rest.y);
                }
                tmem_st32(t_s + 32 * c, s);
            };
#pragma unroll 1
            for (int half = 0; half < columns / 64; ++half) {
                if (warp_live) {
                    uint32_t s0[32], s1[32];
                    tmem_ld32(t_s + 64 * half, s0);
                    tmem_wait_ld32(s0);
                    tmem_ld32(t_s + 64 * half + 32, s1);
                    weights(2 * half, s0);
                    tmem_wait_ld32(s1);
                    weights(2 * half + 1, s1);
                    tmem_wait_st();
                }
                tc_fence_before();
                mbar_arrive(smem_addr(&m.pfull[buf][shared_rows ? group : half]));
            }
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            pvph ^= 1u;
        }
        if (!ok)
            break;
        // the accumulator's last MMAs (those before: with own rows the last score
        // followed them, else they were waited for)
        if (end > 0 && !(ok = wait(pvdone, pvph ^ 1u)))
            break;
        tc_fence_after();
        vcount += w.n;
        TreeWalk<D> next = w;
        next.next(p);
        if (next.n > 0)
            fetch_q(next);

        // the segment's result: O / l and the log-sum-exp (base 2), final or partial
        if (flushed && warp_live) {
            flush_sums(false, mx);   // the segment's whole sum, relative to ref
            if (mx != kNegInf) {
                l *= exp2_approx((mx - ref) * sl);
                mx = ref;
            }
            __threadfence_block();   // with shared rows the other group reads half of it
        }
        if (!live) {
            mx = kNegInf;
            l = 0.f;
        }
        if (shared_rows)
            m.ml[group][tid] = make_float2(mx, l);
        tc_fence_before();
        if (!(ok = pair_sync()))
            break;
        tc_fence_after();
        // both groups' units are done: the next rows may come, and their scores
        // be formed beside what follows.  (ml of the next segment is written by
        // groups with units, after their MMAs, which wait for ofree.)
        if (threadIdx.x < kMaxTree / 32)
            m.bad[odd ^ 1][threadIdx.x] = 0;         // the last segment's, read before its end
        if (next.n > 0)
            store_q(next);
        float a0 = 1.f, a1 = 0.f;
        if (shared_rows) {
            const float2 x = m.ml[0][tid], y = m.ml[1][tid];
            mx = fmaxf(x.x, y.x);
            a0 = x.x == kNegInf ? 0.f : exp2_approx((x.x - mx) * sl);
            a1 = y.x == kNegInf ? 0.f : exp2_approx((y.x - mx) * sl);
            // scores of NaN leave no maximum, but a sum of NaN
            l = x.y * (x.x == kNegInf ? 1.f : a0) + y.y * (y.x == kNegInf ? 1.f : a1);
        }
        const bool any = live && l != 0.f;           // true for NaN
        const float inv = any ? p.v_scale / l : 0.f;
        const float lse2 = any ? (mx == kNegInf ? 0.f : mx * sl) + log2f(l) - kShift : kNegInf;
        const int g = w.seg / w.s.groups;
        const long long o_row = ((long long)w.b * p.tree_len + i) * p.hq + g * p.group + h;
        const bool whole = w.j0 == 0 && w.n == w.s.nb;
        const int slot = 2 * (int)blockIdx.x + (w.j0 > 0 ? 0 : 1);
        const int srow = (own_rows ? group * 128 : 0) + tid;   // row of the partial
        const int c0 = shared_rows ? group * (D / 2) : 0, c1 = shared_rows ? c0 + D / 2 : D;
        // dim d of this row's output, or partial: out[d / 4 * stride + d % 4]
        float *out = whole ? p.o + o_row * D : p.ws_o + ((long long)slot * (D / 4) * p.slot_rows + srow) * 4;
        const int stride = whole ? 4 : p.slot_rows * 4;
        [[maybe_unused]] float2 every = make_float2(0.f, 0.f);   // the outputs' sums: NaN if an output is
        __syncwarp();
        for (int c = c0; c < c1; c += 32) {
            float v[32];
            [[maybe_unused]] uint32_t x[32];
#pragma unroll
            for (int k = 0; k < 32; ++k)
                v[k] = 0.f;
            if (end > 0 && warp_live) {
                // columns c .. c + 31 of a group's sum: in the workspace once it was flushed
                auto add = [&](int of, bool flushed, float weight) {
                    if (flushed) {
                        if (has_sums) {
                            const float *src = p.ws_sums + (((long long)(blockIdx.x * C::kGroups + of) * (D / 4) + c / 4) * p.sum_rows + tid) * 4;
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const float4 o = __ldcg(reinterpret_cast<const float4 *>(src + (long long)k * p.sum_rows * 4));
                                v[4 * k] = fmaf(o.x, weight, v[4 * k]);
                                v[4 * k + 1] = fmaf(o.y, weight, v[4 * k + 1]);
                                v[4 * k + 2] = fmaf(o.z, weight, v[4 * k + 2]);
                                v[4 * k + 3] = fmaf(o.w, weight, v[4 * k + 3]);
                            }
                        }
                        __syncwarp();
                    } else {
                        tmem_ld32(t_lane + C::kTmemO + of * D + c, x);
                        tmem_wait_ld32(x);
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            v[k] = fmaf(__uint_as_float(x[k]), weight, v[k]);
                    }
                };
                if (shared_rows) {
                    add(0, flushed, a0);
                    add(1, flushed, a1);
                } else
                    add(C::kGroups == 1 ? 0 : group, flushed, 1.f);
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    v[k] = any ? v[k] * inv : 0.f;
                if constexpr (KV != kKvE4m3) {   // a tree of sums: as a chain they cost a short call 0.1 us
                    const float2 one = make_float2(1.f, 1.f);
                    float2 y[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        y[k] = fma2(make_float2(v[2 * k], v[2 * k + 1]), one, make_float2(v[2 * k + 16], v[2 * k + 17]));
#pragma unroll
                    for (int n = 4; n; n >>= 1)
#pragma unroll
                        for (int k = 0; k < n; ++k)
                            y[k] = fma2(y[k], one, y[k + n]);
                    every = fma2(y[0], one, every);
                }
            }
            if (in_call && (whole || any)) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    *reinterpret_cast<float4 *>(out + (c / 4 + k) * stride) = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            }
            __syncwarp();
        }
        tc_fence_before();
        mbar_arrive(smem_addr(&m.ofree));
        if (in_call && (!shared_rows || group == 0)) {
            if (!whole)
                p.ws_lse[slot * p.slot_rows + srow] = lse2;
            else if (p.lse)
                p.lse[o_row] = any ? lse2 * 0.6931471805599453f : kNegInf;
        }
        // values that are not finite: of the context, then of nodes in this CTA's tiles
        if constexpr (KV != kKvE4m3) {
            const float all = every.x + every.y;
            const bool mine = any && l == l && all != all;
            if (__builtin_expect(__any_sync(0xffffffffu, mine), 0)) {
                const long long row_bytes = (long long)p.hkv * D * (kv_is_fp8(KV) ? 1 : 2), row0 = p.block_table ? 0 : (long long)w.b * p.page_size;
                tree_infinities<D, F16, KV>(p.v + (row0 * p.hkv + g) * D * (kv_is_fp8(KV) ? 1 : 2), row_bytes,
                                            p.block_table ? p.block_table + (long long)w.b * p.max_blocks : nullptr, p.page_size,
                                            p.num_pages, w.j0 * C::kN, (int)min((long long)(w.j0 + w.n) * C::kN, (long long)base), c0, c1, mine, out, stride);
            }
        }
        for (int wd = 0; wd < kMaxTree / 32; ++wd) {
            uint32_t nodes = m.bad[odd][wd];
            for (; nodes; nodes &= nodes - 1) {
                const int node = 32 * wd + __ffs(nodes) - 1;
                if (!any || !(tree_bits(p, mask_row, i, node, t) & 1u))
                    continue;
                const long long at = ((long long)tree_row(p, w.b, base + node, false) * p.hkv + g) * D;
                float s = 0.f;
                for (int d = 0; d < D; ++d)
                    s = fmaf(p.q_f16 ? f16x2_to_float2(p.q[o_row * D + d]).x : bf16x2_to_float2(p.q[o_row * D + d]).x,
                             tree_element<F16, KV>(p.k, at + d), s);
                // an infinity stays one when its weight is too small for fp32 (a weight of NaN has made the row NaN)
                const float weight = fmaxf(exp2_approx((p.negate_q ? -s : s) * p.scale_log2 - lse2), 1.1754944e-38f);
                for (int d = c0; d < c1; ++d) {
                    const float x = tree_element<F16, KV>(p.v, at + d);
                    if (fabsf(x) <= 3.4028235e38f)
                        continue;
                    float *dst = out + (d / 4) * stride + d % 4;
                    *dst = fmaf(weight, x, *dst);
                }
            }
        }
        w = next;
        odd ^= 1;
    }
    if (!ok) {
        atomicOr(p.ws_err, kErrTimeout);
        *abort_flag = 1;
    }
    __syncwarp();
}

// ---------------------------------------------------------------- kernel

template <int D, bool F16, int KV, int LOAD>
__global__ void __launch_bounds__(TreeCfg<D, LOAD>::kThreads, 1)
tree_split_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ CUtensorMap tmk,
                  const __grid_constant__ CUtensorMap tmv)
{
    using C = TreeCfg<D, LOAD>;
    extern __shared__ __align__(1024) uint8_t smem[];
    TreeMisc &m = *reinterpret_cast<TreeMisc *>(smem + p.off_misc);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    if (smem_addr(smem) & 1023u) {   // the swizzled layout and its descriptors count on it
        if (tid == 0)
            atomicOr(p.ws_err, kErrTimeout);
        return;
    }
    if (warp == C::kMmaWarp)
        tmem_alloc(smem_addr(&m.tmem), C::kTmemCols);
    if (tid == 0) {
        const int copies = LOAD == kTreeTma ? 1 : C::kCopyThreads;   // arrivals that fill a K or V slot
        for (int s = 0; s < kTreeMaxSlots; ++s) {
            mbar_init(smem_addr(&m.kfull[s]), copies);
            mbar_init(smem_addr(&m.vfull[s]), copies);
            mbar_init(smem_addr(&m.kempty[s]), 1);
            mbar_init(smem_addr(&m.vempty[s]), 1);
        }
        for (int s = 0; s < kTreeMaxRaw; ++s) {
            mbar_init(smem_addr(&m.rkfull[s]), 1);
            mbar_init(smem_addr(&m.rvfull[s]), 1);
            mbar_init(smem_addr(&m.rkempty[s]), copies);
            mbar_init(smem_addr(&m.rvempty[s]), copies);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_addr(&m.sfull[s]), 1);
            mbar_init(smem_addr(&m.pfull[s][0]), 128);
            mbar_init(smem_addr(&m.pfull[s][1]), 128);
            mbar_init(smem_addr(&m.pvdone[s]), 1);
        }
        mbar_init(smem_addr(&m.qfull), C::kSoftThreads);
        mbar_init(smem_addr(&m.ofree), C::kSoftThreads);
        mbar_init(smem_addr(&m.pair), C::kSoftThreads);
        mbar_init(smem_addr(&m.drain), 1);
        mbar_init_fence();
        m.abort = 0;
        m.b = p.batch;
        if (LOAD != kTreeCopy) {
            tma_prefetch_desc(&tmk);
            tma_prefetch_desc(&tmv);
        }
    }
    if (tid < 2 * (kMaxTree / 32))
        (&m.bad[0][0])[tid] = 0;
    pdl_wait_prior_grid();
    pdl_launch_dependents();

    // This CTA's run: a scan of the requests' costs, and the thread whose
    // requests hold the run's first position looks it up.
    const int per = (p.batch + C::kThreads - 1) / C::kThreads;
    const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
    long long mine = 0;
    for (int b = b0; b < b1; ++b)
        mine += tree_cost(tree_seg<D>(p, tree_req(p, b, blockIdx.x == 0 ? p.ws_err : nullptr)));
    long long x = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off)
            x += y;
    }
    if (lane == 31)
        m.scan[warp] = x;
    __syncthreads();
    long long before = x - mine, total = 0;
    for (int k = 0; k < C::kWarps; ++k) {
        before += k < warp ? m.scan[k] : 0;
        total += m.scan[k];
    }
    const TreeSplit split = tree_split(total, gridDim.x);
    const int cta = blockIdx.x;
    const bool works = cta < split.ctas;
    const long long x0 = works ? split.begin(cta) : 0;
    if (tid == 0)
        m.x1 = works ? split.begin(cta + 1) : 0;
    long long at = before;
    for (int b = b0; b < b1 && (cta == 0 || works); ++b) {
        const TreeSeg s = tree_seg<D>(p, tree_req(p, b, nullptr));
        if (cta == 0)
            p.ws_cost[b] = at;
        const long long cost = tree_cost(s);
        if (works && at <= x0 && x0 < at + cost) {
            const long long rel = x0 - at - kTreeSegCost;
            long long seg = rel < 0 ? 0 : TreeSplit::quotient(rel, s.nb + kTreeSegCost);
            long long j = rel < 0 ? 0 : rel - seg * (s.nb + kTreeSegCost);
            if (j >= s.nb) {   // the gap before the next segment (there is one: the last ends with its tiles)
                ++seg;
                j = 0;
            }
            m.b = b;
            m.seg = (int)seg;
            m.j = (int)j;
            m.segpos = at + seg * (s.nb + kTreeSegCost) + kTreeSegCost;
        }
        at += cost;
    }
    if (cta == 0 && tid == 0)
        p.ws_cost[p.batch] = total;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = m.tmem;
    const uint32_t q_smem = smem_addr(smem), k_ring = smem_addr(smem + p.off_k), v_ring = smem_addr(smem + p.off_v);
    if (warp < C::kSoftWarps) {
        if constexpr (C::kSplitRegs)
            regs_more<C::kSoftRegs>();
        tree_softmax<D, F16, KV, LOAD>(p, m, q_smem, v_ring, tmem);
    } else {
        if constexpr (C::kSplitRegs)
            regs_fewer<C::kOtherRegs>();
        const uint32_t raw_k = smem_addr(smem + p.off_raw), raw_v = raw_k + p.raw_slots * C::kRawBytes;
        if (C::kCopyWarps > 0 && warp < C::kLoadWarp) {
            if constexpr (LOAD != kTreeTma)
                tree_copy<D, KV, LOAD>(p, m, k_ring, v_ring, raw_k, raw_v, tid - C::kSoftThreads);
        } else if (warp == C::kMmaWarp)
            tree_mma<D, F16, LOAD>(p, m, q_smem, k_ring, v_ring, tmem);
        else if (LOAD != kTreeCopy && warp == C::kLoadWarp)
            tree_load_tma<D, LOAD, true>(p, m, &tmk, LOAD == kTreeConvert ? raw_k : k_ring,
                                         LOAD == kTreeConvert ? p.raw_slots : p.k_slots, lane);
        else if (LOAD != kTreeCopy && warp == C::kLoadWarp + 1)
            tree_load_tma<D, LOAD, false>(p, m, &tmv, LOAD == kTreeConvert ? raw_v : v_ring,
                                          LOAD == kTreeConvert ? p.raw_slots : p.v_slots, lane);
    }
    // every role returns, its waits being bounded
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == C::kMmaWarp)
        tmem_dealloc(tmem, C::kTmemCols);
}

template <int D, bool F16, int KV, int LOAD>
cudaError_t launch_tree_variant(const TreeParams &p, const CUtensorMap &tmk, const CUtensorMap &tmv, const TreeLaunch &c)
{
    // the shared-memory limit is raised once per device, so that later calls
    // may be captured; again if a launch is refused (the context was reset)
    static std::atomic<unsigned long long> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const unsigned long long bit = 1ull << (dev & 63);
    auto configure = [&]() -> cudaError_t {
        const cudaError_t r = cudaFuncSetAttribute(tree_split_kernel<D, F16, KV, LOAD>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)c.smem_optin);
        // the warps' register shares come out of the launch's: no launch with fewer
        cudaFuncAttributes fa;
        if (r == cudaSuccess && TreeCfg<D, LOAD>::kSplitRegs &&
            (cudaFuncGetAttributes(&fa, tree_split_kernel<D, F16, KV, LOAD>) != cudaSuccess ||
             fa.numRegs != TreeCfg<D, LOAD>::kLaunchRegs))
            return cudaErrorInvalidConfiguration;
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
    cfg.blockDim = dim3(TreeCfg<D, LOAD>::kThreads);
    cfg.dynamicSmemBytes = c.smem_bytes;
    cfg.stream = c.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, tree_split_kernel<D, F16, KV, LOAD>, p, tmk, tmv);
    if (e == cudaErrorInvalidValue) {
        (void)cudaGetLastError();
        if ((e = configure()) != cudaSuccess)
            return e;
        e = cudaLaunchKernelEx(&cfg, tree_split_kernel<D, F16, KV, LOAD>, p, tmk, tmv);
    }
    return e;
}

}  // namespace fd
