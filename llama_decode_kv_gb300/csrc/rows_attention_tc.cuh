// rows_attention_tc.cuh -- attention of packed bf16 rows on the 5th-generation tensor cores,
// heads of up to 128, over a paged cache or packed prompts: the kernel, compiled for plain causal
// scores by rows_attention_tc.cu and for scored ones by rows_scored_tc_*.cu.
//
// out = sum_{t <= p} softmax_t(q . k_t / sqrt(hd)) v_t for every row (token, query head).
// The G query heads of a kv head and TT = 128 / G tokens make a tile of up to 128 rows (row =
// token * G + head), so keys and values are read once for the whole group, and a decode step is
// the same kernel with one tile that is mostly empty.  An item is two such tiles, one behind
// the other, over the same keys: while the softmax of one runs, the tensor core works for the
// other.  An item of 64-wide heads with one tile only (a decode step, the end of a chunk) is
// worked on twice over: the first softmax group takes its even blocks, the second the odd ones,
// each with its own S, O, maximum and sum, added up at the end.  Items are cut into equal ranges of
// 128-position blocks (rows_plan.h), one persistent CTA per SM; pieces of items leave as partial
// states for rows_join_kernel.
//
// Long prompts and chunks are bound by the chain S, softmax, P V of a tile, which two tiles do not
// hide altogether: prompts of 8,192 and fewer tokens, 32 / 8 heads of 128, 366 us = 1.54 PFLOP/s in a
// short run (82% of cuBLAS's burst rate; tensor pipe 64% busy by its counter) and 396 us = 1.42 back to
// back under the power cap (85% of its sustained rate).  64-wide heads take nearly the same chain for
// half the operations: 2,048 tokens 35 us = 0.49 PFLOP/s.  Decode steps are bound by HBM: 64 sequences
// of up to 8,000 positions 164 us = 6.3 TB/s, 94% of the copy rate.  Short calls are bound by one
// dependent chain: one token over 262 positions 8.5 us.
//
// Heads of 72 to 112 run as 128-wide ones in P V and in shared memory (their S leaves the missing
// columns out), so up to 44% of their P V and of their ring is padding.
//
// Scored rows (SCORE):  x_t = scale q . k_t,  cap tanh(x_t / cap),  - slope_h |p - t|,  over the t that
// the row sees, [from, to) by row_span (window, document, prefix); a row that sees none is 0.  An item
// walks the blocks that some row of it sees (MaskedWalk), and its softmax groups mask where a block
// holds a key that some row of the warp does not see.  What is different from plain rows, and why:
//   * Both heads' widths work on one-tile items twice over, and items of up to 32 rows (a decode
//     step) are split: their queries stand in the tile four times, 32 rows for each warp of a group, so
//     the four warps take 32 of a block's keys each in place of one warp all 128.  With one warp at work
//     a capped block cost more than its bytes took to come (64 sequences, 32 / 8 heads of 128, window
//     4,096, cap 30: 334 us; split 182, with quarters in loops 163 = 5.8 TB/s, 86% of the copy rate).
//   * A quarter of 32 keys is the body of a loop.  The scored softmax as straight code pushes the other
//     roles' instructions out of the cache (no_instruction was the first stall by far), and these
//     then feed the tensor core late: documents of up to 1,500 in prompts of up to 6,000, 250 us as
//     straight code, 205 in quarters (183 now).  Long items get over it, so they have a variant with straight code
//     for blocks without masks (kStraight; the rule and its figures stand in rows_op.cu).
//   * tanh is a polynomial while |x| is at most the cap, its degree by the warp's largest |x|
//     (cap_tier), the branch outside the loops: inside, the compiler computes both sides for every key
//     (64 sequences as above 992 us, outside 334).
//   * The maximum is the score of the largest product plus a bound of the distance's term, so that one
//     pass over a quarter finds it; slopes too steep for that take it key by key.  Without distances the
//     cap of the largest |product|, which cap_tier needs anyhow, serves where it is small (documents 193 us
//     -> 183, a prompt of 8,192 588 -> 548).
// What bounds them now: decode steps HBM; prompts and chunks with masks the same chain of hand-offs as
// plain rows, its softmax part longer by the cap's five to seven instructions for two keys (a prompt of
// 8,192: 535 us with a cap, 436 without, plain 356), joining the items that ranges cut (12 of the 106 us of
// windowed chunks, 13 of the 183 of documents), and items' ends where documents are short.
//
//   warps 0-3, 4-7  softmax of tile 0 and of tile 1, a thread per row: S from tensor memory, the
//                   causal mask where the block needs one, the running maximum, P = 2^(S - m) as
//                   bf16 back into tensor memory, the sum in fp32; at the end O / l to global
//                   memory.  O stays where it is: it is rescaled (by the same threads) only when
//                   a row's maximum grew by more than 2^8, so P stays below 2^8 and the final
//                   division takes the stale maximum out again.
//   warp 8          tcgen05.mma issuer: S = Q K^T (both operands in shared memory, K-major),
//                   O += P V (P from tensor memory, V as it lies in memory: head_dim contiguous,
//                   which is the MN-major operand).  Also zeroes the rows of the last block's V
//                   that no row sees, since 0 * NaN is NaN.
//   warp 9          TMA producer: the tile's queries as one box {64, G, TT} per 64 columns, keys
//                   and values as boxes of up to 128 positions, one per page where pages are
//                   shorter, into a ring of 128-byte-swizzled [128][64] panels.  Head widths
//                   that are no multiple of 64 are filled up with zeros by the copy.
//
// Rounding: q, k, v as given; S, maxima, sums and O in fp32; P to bf16 (at most 2^-8 relative:
// the tensor core takes 16-bit operands), the result to bf16.
//
// Every wait is bounded; the first to run out stops all roles.  The MMA warp and the producer end
// only when what they issued has run (bounded too), whoever gave up and whenever; then tensor memory
// is freed.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "device_common.cuh"
#include "gemm_tc.cuh"
#include "rows.cuh"

namespace slm {

// Threads of a CTA: ten warps; with kStraight twelve (two of them idle), so that the softmax groups can
// take registers over from the other roles: 2 x 128 x 216 + 128 x 72 = 384 x 168, what such a CTA is
// launched with (a prompt of 8,192 with a cap 535 us; with 224 / 56 549, 208 / 88 548, 192 / 120 578).
__host__ __device__ constexpr int tc_threads(int score) { return score & kStraight ? 384 : 320; }
constexpr int kTcBlk = 128;                 // positions per block
constexpr int kPanel = 128 * 128;           // bytes of [128 rows][64 bf16]
constexpr int kTcCols = 512;                // tensor memory columns
constexpr float kNear = 40.0f;              // log2 scores this near 0 take a bound for their maximum
constexpr float kTcSlack = 8.0f;            // log2 growth of a maximum that O is not rescaled for

struct RowsTcArgs {
    CUtensorMap q, k, v;
    CUtensorMap q_few;  // queries of 32 / G tokens (split items)
    RowsArgs a;
    int TT;      // tokens per tile
    int box;     // positions per key / value box
    int stages;  // ring depth
    int wide;    // output heads begin on 32-byte boundaries and are multiples of 16 long
};

struct TcBars {
    uint64_t kv_full[16], kv_empty[16];
    uint64_t q_full[2], q_empty[2], s_full[2], p_half[2], p_ready[2], o_full[2], drain;
    uint64_t quarter[2];      // split items: the four warps of a group have handed something over
    uint64_t x_full, x_free;  // twin items: group 1's statistics stand in shared memory; group 0 is done
    uint32_t tmem;
    int stop;
};

// ------------------------------------------------------------------ PTX wrappers

__device__ __forceinline__ void tma_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void tma_4d(void *dst, const CUtensorMap *map, int x, int y, int z, int w, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory operand descriptors, 128-byte swizzle, rows of 128 bytes in groups of 8 (1024
// bytes apart).  K-major (Q, K): the groups run along M / N.  MN-major (V): the groups run along
// K, and panels of 64 columns are kPanel apart.  The upper word is the same for all: the group
// stride, version 1, the swizzle.  The lower word is the address and the panel stride (`lead`), in
// units of 16 bytes; offsets are added to it.
constexpr uint32_t kDescHi = (1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_lo(const void *p, uint32_t lead) {
    return (smem_addr(p) >> 4) | (lead >> 4) << 16;
}

// kind::f16, fp32 accumulator, bf16 operands; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t tc_idesc(int m, int n, int b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, "
        "%5};\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "r"(kDescHi)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(idesc), "r"(acc), "r"(kDescHi)
        : "memory");
}

__device__ __forceinline__ void tc_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

#define SLM_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define SLM_I8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])

// Columns of this thread's lane.  The wait stands in the same statement: the registers are not
// valid before it, and between two statements the compiler may copy them and give them to others.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : SLM_R8(r, 0), SLM_R8(r, 8), SLM_R8(r, 16), SLM_R8(r, 24)
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld1(uint32_t addr, uint32_t &r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;" : "=r"(r) : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_ld64(uint32_t addr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : SLM_R8(r, 0), SLM_R8(r, 8), SLM_R8(r, 16), SLM_R8(r, 24), SLM_R8(r, 32), SLM_R8(r, 40), SLM_R8(r, 48),
          SLM_R8(r, 56)
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        SLM_I8(r, 0), SLM_I8(r, 8), SLM_I8(r, 16), SLM_I8(r, 24)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(addr),
        SLM_I8(r, 0), SLM_I8(r, 8)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// fp32 pairs in one register pair: one instruction for two results.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Keys from `lim` on become -infinity (or `hidden`).  `all` (at most any lane's lim): no lane's key before
// it does, so groups of 16 below it are left alone (two instructions an element at half rate: a diagonal
// block took twice as long as the others).
constexpr uint32_t kHidden = 0xff800000u, kIgnored = 0x7fffffffu;  // -infinity; a NaN, which a maximum passes over
template <int N> __device__ __forceinline__ void mask_from(uint32_t (&s)[N], int lim, int all, uint32_t hidden = kHidden) {
#pragma unroll
    for (int k0 = 0; k0 < N; k0 += 16)
        if (k0 + 16 > all) {
#pragma unroll
            for (int k = k0; k < k0 + 16; k++)
                if (k >= lim) s[k] = hidden;
        }
}

template <int N> __device__ __forceinline__ float max_of(const uint32_t (&s)[N]) {
    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int k = 0; k < N; k += 8)
#pragma unroll
        for (int q = 0; q < 4; q++) m[q] = max3(m[q], __uint_as_float(s[k + 2 * q]), __uint_as_float(s[k + 2 * q + 1]));
    return fmaxf(max3(m[0], m[1], m[2]), m[3]);
}

// Keys before `low` do.  `all`: at least any lane's low.
template <int N> __device__ __forceinline__ void mask_to(uint32_t (&s)[N], int low, int all, uint32_t hidden = kHidden) {
#pragma unroll
    for (int k0 = 0; k0 < N; k0 += 16)
        if (k0 < all) {
#pragma unroll
            for (int k = k0; k < k0 + 16; k++)
                if (k < low) s[k] = hidden;
        }
}

template <int N> __device__ __forceinline__ float absmax(const uint32_t (&s)[N]) {
    float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < N; k += 8)
#pragma unroll
        for (int q = 0; q < 4; q++)
            m[q] = max3(m[q], fabsf(__uint_as_float(s[k + 2 * q])), fabsf(__uint_as_float(s[k + 2 * q + 1])));
    return fmaxf(max3(m[0], m[1], m[2]), m[3]);
}

// Capped scores.  tanh(y) = y (1 + z Q(z)), z = y^2: with Q of degree 2 where |y| <= 1/2 and of degree 4
// where |y| <= 1 (least largest relative error, by reweighted least squares: 2^-20.5 both), and beyond
// 1 - 2 / (1 + e^(2 |y|)) with the SFU's exponential and reciprocal, 2^-22 off.  A relative error, so the
// cap may be as large as it likes.  Scale, cap and log2(e) are multiplied into the polynomial's
// coefficients (RowsScores), so that a score is s P(s^2) + off of the product s = q . k.
__device__ __forceinline__ float tanh_large(float y) {
    float e = fast_exp2(2.8853900817779268f * fabsf(y)), r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return copysignf(fmaf(-2.0f, r, 1.0f), y);
}
// 0: every |s| of the warp is below half the cap (in its units), 1: below it, 2: some are above.  `most`
// counts products of the batch's rows with keys that they see and no others: what lies behind a
// sequence's last key or row differs from call to call, and the bits of a call must not.
__device__ __forceinline__ int cap_tier(const RowsScores &sc, float most) {
    return __all_sync(0xffffffffu, most <= sc.half_cap) ? 0 : __all_sync(0xffffffffu, most <= sc.one_cap) ? 1 : 2;
}
template <int TIER> __device__ __forceinline__ uint64_t cap_poly(const RowsScores &sc, float c, uint64_t v) {
    const uint64_t z = mul2(v, v);
    uint64_t q;
    if (TIER == 0) {
        q = pack2(sc.poly3[2], sc.poly3[2]);
#pragma unroll
        for (int i = 1; i >= 0; i--) q = fma2(z, q, pack2(sc.poly3[i], sc.poly3[i]));
    } else {
        q = pack2(sc.poly5[4], sc.poly5[4]);
#pragma unroll
        for (int i = 3; i >= 0; i--) q = fma2(z, q, pack2(sc.poly5[i], sc.poly5[i]));
    }
    return fma2(z, q, pack2(c, c));  // of s
}
__device__ __forceinline__ float cap_any(const RowsScores &sc, float c, float v) {
    if (fabsf(v) > sc.one_cap) return sc.cap_log2 * tanh_large(v * sc.cap_in);
    float a, b;
    unpack2(cap_poly<1>(sc, c, pack2(v, v)), a, b);
    return v * a;
}

// The scores of N keys in the log2 domain plus `off`, from q . k.  d0: the first key's position minus
// the row's; sl: slope log2(e); BOTH: some key may stand behind its row.
template <int SCORE, int TIER, bool BOTH, int N>
__device__ __forceinline__ void score_pairs(uint32_t (&s)[N], const RowsScores &sc, float c, float sl, float d0, float off) {
    const float base = SCORE & kBiased ? fmaf(sl, d0, off) : off;
    const uint64_t c2 = pack2(c, c), base2 = pack2(base, base);
#pragma unroll
    for (int k = 0; k < N; k += 2) {
        float a = __uint_as_float(s[k]), b = __uint_as_float(s[k + 1]);
        uint64_t v = pack2(a, b), f = c2, add = base2;
        if (SCORE & kCapped) {
            if (TIER == 2) {
                v = pack2(cap_any(sc, c, a), cap_any(sc, c, b));
                f = pack2(1.f, 1.f);
            } else {
                f = cap_poly<TIER>(sc, c, v);
            }
        }
        if (SCORE & kBiased) {
            if (BOTH)  // -sl |d|
                add = pack2(fmaf(-sl, fabsf(d0 + (float)k), off), fmaf(-sl, fabsf(d0 + (float)(k + 1)), off));
            else       // d <= 0 wherever it counts
                add = pack2(fmaf((float)k, sl, base), fmaf((float)(k + 1), sl, base));
        }
        unpack2(fma2(v, f, add), a, b);
        s[k] = __float_as_uint(a);
        s[k + 1] = __float_as_uint(b);
    }
}
template <int SCORE, int N>
__device__ __forceinline__ void scores(uint32_t (&s)[N], const RowsScores &sc, float c, float sl, float d0, int tier, bool both,
                                       float off) {
    // the branches stand outside the loops: within, both sides of them would be computed for every key
    auto tiers = [&](auto b) {
        constexpr bool BOTH = decltype(b)::value;
        if (!(SCORE & kCapped) || tier == 0)
            score_pairs<SCORE, 0, BOTH>(s, sc, c, sl, d0, off);
        else if (tier == 1)
            score_pairs<SCORE, 1, BOTH>(s, sc, c, sl, d0, off);
        else
            score_pairs<SCORE, 2, BOTH>(s, sc, c, sl, d0, off);
    };
    if ((SCORE & kBiased) && both)
        tiers(std::true_type{});
    else
        tiers(std::false_type{});
}

// The most that a distance's term comes to in the N keys from d0 (their first position minus the row's) on.
template <int N> __device__ __forceinline__ float bias_most(float sl, float d0) {
    const float a = fabsf(d0), b = fabsf(d0 + (float)(N - 1)), far = fmaxf(a, b);
    const float near = d0 > 0.f || d0 < (float)(1 - N) ? fminf(a, b) : 0.f;
    return -sl * (sl > 0.f ? near : far);
}

// P = 2^S (DONE) or 2^(S c - m c) of 32 keys: added to the sums, and as bf16 pairs.
template <bool DONE>
__device__ __forceinline__ void weights32(const uint32_t (&s)[32], uint64_t c2, uint64_t mc2, uint64_t (&sum)[2], uint32_t (&pk)[16]) {
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
        float a = __uint_as_float(s[k]), b = __uint_as_float(s[k + 1]);
        if (!DONE) unpack2(fma2(pack2(a, b), c2, mc2), a, b);
        a = fast_exp2(a);
        b = fast_exp2(b);
        sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], pack2(a, b));
        pk[k / 2] = pack_bf16x2(a, b);
    }
}

// The same of 64 keys, the pairs to tensor memory.
template <bool DONE>
__device__ __forceinline__ void straight_weights(const uint32_t (&s)[64], uint64_t c2, uint64_t mc2, uint64_t (&sum)[2], uint32_t addr) {
#pragma unroll
    for (int k0 = 0; k0 < 64; k0 += 32) {
        uint32_t pk[16];
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
            float a = __uint_as_float(s[k0 + k]), b = __uint_as_float(s[k0 + k + 1]);
            if (!DONE) unpack2(fma2(pack2(a, b), c2, mc2), a, b);
            a = fast_exp2(a);
            b = fast_exp2(b);
            sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], pack2(a, b));
            pk[k / 2] = pack_bf16x2(a, b);
        }
        tmem_st16(addr + k0 / 2, pk);
    }
}

// P = 2^(S c - m c) of 64 keys: added to the sums, and as bf16 pairs to tensor memory.
__device__ __forceinline__ void weights64(const uint32_t (&s)[64], uint64_t c2, uint64_t mc2, uint64_t (&sum)[2], uint32_t addr) {
#pragma unroll
    for (int k0 = 0; k0 < 64; k0 += 32) {
        uint32_t pk[16];
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
            float a, b;
            unpack2(fma2(pack2(__uint_as_float(s[k0 + k]), __uint_as_float(s[k0 + k + 1])), c2, mc2), a, b);
            a = fast_exp2(a);
            b = fast_exp2(b);
            sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], pack2(a, b));
            pk[k / 2] = pack_bf16x2(a, b);
        }
        tmem_st16(addr + k0 / 2, pk);
    }
}

__device__ __forceinline__ void st_global32(void *p, const uint32_t (&h)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), SLM_I8(h, 0) : "memory");
}

// One lane of the (converged) warp, always the same.  Behind this predicate the compiler keeps the
// operands of the asynchronous instructions in uniform registers; behind `lane == 0` it moved them
// there one by one, ~100 cycles an MMA, which bound the kernel.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

// Bounded wait of a whole warp for the phase of the given parity; the first wait of the CTA to run
// out raises stop, and every later wait gives up at once.  The warp is together again behind it
// (the roles keep warp-uniform state, and tcgen05 instructions are warp-wide).
__device__ __forceinline__ bool tc_wait(uint64_t *bar, uint32_t parity, int *status, volatile int *stop) {
    bool ok = mbar_try_wait(bar, parity);
    if (!__all_sync(0xffffffffu, ok)) {
        const unsigned long long t0 = global_ns();
        while (true) {
            ok = mbar_try_wait(bar, parity);
            if (__all_sync(0xffffffffu, ok)) break;
            const bool late = *stop || global_ns() - t0 > kWaitLimitNs;
            if (__any_sync(0xffffffffu, late)) {
                if (!*stop) atomicOr(status, SLM_ROWS_TIMEOUT);
                *stop = 1;
                return false;
            }
        }
    }
    return true;
}

// The blocks of a piece that softmax group i works on, and its tokens: its own tile's, or (twin)
// every second block of tile 0's.
struct TileView {
    bool twin, split;
    int n, tok0, ntok;  // blocks; first token in the sequence; tokens
    int first, step;    // block j is first + j step
};
// prefix: positions that all rows see (masked items).
__device__ __forceinline__ TileView tile_view(const SeqRows &sr, const RowsPiece &p, int TT, int PT, int i, int prefix,
                                              bool twin) {
    TileView v;
    const int left = sr.n - p.t * PT;  // tokens from the item's first on, at least 1
    v.twin = twin && left <= TT;
    v.split = false;
    if (v.twin) {
        v.tok0 = p.t * PT;
        v.ntok = left;
        v.n = (p.kb1 - p.kb0 + 1 - i) >> 1;
        v.first = p.kb0 + i;
        v.step = 2;
    } else {
        v.tok0 = p.t * PT + i * TT;
        v.ntok = max(0, min(TT, sr.n - v.tok0));
        v.n = v.ntok > 0 ? max(0, min(p.kb1, (int)(((unsigned)max(sr.ctx + v.tok0 + v.ntok, prefix) + kTcBlk - 1) / kTcBlk)) - p.kb0) : 0;
        v.first = p.kb0;
        v.step = 1;
    }
    return v;
}

inline size_t tc_lengths_bytes(int nseq, bool spans) {
    return (size_t)nseq * sizeof(SeqRows) + (size_t)(nseq + 1) * 8 + (spans ? masked_bytes() : 0);
}

__host__ __device__ constexpr size_t tc_fixed_bytes(int HDP, int stages, bool spans) {
    return 1024 + (size_t)(2 + stages) * (HDP / 64) * kPanel + (sizeof(TcBars) + 15) / 16 * 16 +
           (HDP == 64 ? 1024 + (spans ? 2 * 384 * sizeof(float) : 0) : spans ? 256 : 0);
}

// ------------------------------------------------------------------ the kernel

template <int HDP, bool PAGED, int SCORE>
__global__ void __launch_bounds__(tc_threads(SCORE), 1) rows_tc_kernel(const __grid_constant__ RowsTcArgs T) {
    constexpr int NP = HDP / 64;  // 64-column panels of a [128][head_dim] operand
    // Tensor memory columns: S 128 i, O 256 + HDP i.  P (64 columns) has its own where O leaves
    // room, else the upper half of S, which the softmax holds in registers by then.
    constexpr uint32_t kO = 256, kP = HDP == 64 ? 384 : 64, kPStep = HDP == 64 ? 64 : 128;
    // One-tile items twice over only where it pays: a block of 64-wide heads arrives faster than one
    // group's chain of S, softmax and P V (4 x 32,768 positions: 72 us with one group, 52 with two);
    // 128-wide ones come at 95% of the copy rate with one group, and joining the halves costs 4%.
    constexpr bool kTwin = HDP == 64;
    // Masked items have blocks of their own, rows see spans; capped or biased scores are worked out in
    // the log2 domain (kX), plain ones stay q . k and take their factor with the exponential.
    constexpr bool kSpans = SCORE != 0, kCap = (SCORE & kCapped) != 0, kBias = (SCORE & kBiased) != 0, kX = kCap || kBias;
    constexpr bool kAbs = kCap && !kBias;  // the largest |product| may stand for the maximum
    constexpr bool kLong = (SCORE & kStraight) != 0;
    using Walk = std::conditional_t<kSpans, RowsMaskedWalk, RowsWalk>;
    const RowsArgs &A = T.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *sq = base;                             // [2 tiles][NP][128][64]
    uint8_t *ring = base + 2 * NP * kPanel;         // [stages][NP][128][64]
    // Split items (kSpans) put their weights where the second tile's queries go: of group i from
    // kSplitP i on, [2 panels of 64 keys][32 rows], swizzled like the other operands.
    constexpr int kSplitP = 8192;
    uint8_t *split_p = sq + NP * kPanel;
    TcBars *B = (TcBars *)(ring + (size_t)T.stages * NP * kPanel);
    float *xm = (float *)((uint8_t *)B + (sizeof(TcBars) + 15) / 16 * 16);  // maxima and sums of a twin item's rows
    // split items: of each group maxima [2][4 warps][32] and sums [4][32]; for 128-wide heads behind the
    // weights
    float *split_x = kTwin ? xm + 256 : (float *)(split_p + 24576);
    constexpr int kXm = kTwin ? 128 : 32;  // rows of a twin item
    long long *wstart = (long long *)(xm + (kTwin ? 256 + (kSpans ? 2 * 384 : 0) : kSpans ? 2 * kXm : 0));
    SeqRows *seq = (SeqRows *)(wstart + A.nseq + 1);
    volatile int *stop = &B->stop;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int TT = T.TT, PT = A.geom.PT, G = A.G;

    if (tid == 0) {
        // test hook (slm_debug_rows_faults): a barrier that waits for one more arrival never completes
        const uint32_t kv_arrivals = 1 + (A.lost == 1), o_arrivals = 1 + (A.lost == 2);
        for (int s = 0; s < T.stages; s++) {
            mbar_init(&B->kv_full[s], kv_arrivals);
            mbar_init(&B->kv_empty[s], 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&B->q_full[i], 1);
            mbar_init(&B->q_empty[i], 1);
            mbar_init(&B->s_full[i], 1);
            mbar_init(&B->p_half[i], 4);
            mbar_init(&B->p_ready[i], 4);
            mbar_init(&B->o_full[i], o_arrivals);
        }
        mbar_init(&B->drain, 1);
        mbar_init(&B->quarter[0], 4);
        mbar_init(&B->quarter[1], 4);
        mbar_init(&B->x_full, 4);
        mbar_init(&B->x_free, 4);
        B->stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&B->tmem)),
                     "r"(kTcCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    pdl_wait();  // what stands above touches no memory of an earlier kernel
    pdl_trigger();
    Walk w;
    if constexpr (kSpans) {
        RowsStart *start = (RowsStart *)(((uintptr_t)(seq + A.nseq) + 15) & ~(uintptr_t)15);
        masked_layout(A, seq, wstart, start, (int *)ring, w, tid, tc_threads(SCORE));
        const long long unit = range_units(wstart[A.nseq], A.P);
        w.begin(seq, wstart[A.nseq], A.nseq, A.geom, unit * blockIdx.x, unit * (blockIdx.x + 1), *start);
    } else {
        rows_layout(A, seq, wstart, tid, tc_threads(SCORE));  // ends with a __syncthreads()
    }
    // an item of at most 32 rows is split by keys over the four warps of a group, and worked on twice
    // over whatever its heads' width
    auto view = [&](const SeqRows &sr, const RowsPiece &p, int i, int prefix) {
        const bool split = kSpans && fits_rows(sr.n - p.t * PT, G, 32);
        TileView v = tile_view(sr, p, TT, PT, i, prefix, kTwin || split);
        v.split = split;
        return v;
    };
    auto prefix_of = [&](int s) {  // positions that all rows of the sequence see
        if constexpr (kSpans)
            return w.mask.prefix(s);
        else
            return 0;
    };
    // positions [from, to) that an item sees
    auto item_from = [&](const SeqRows &sr, const RowsPiece &p) {
        if constexpr (kSpans)
            return row_from(w.mask(p.s), sr.ctx, p.t * PT);
        else
            return 0;
    };
    auto item_to = [&](const SeqRows &sr, const RowsPiece &p) {
        const int end = sr.ctx + min(p.t * PT + PT, sr.n);
        return kSpans ? max(end, prefix_of(p.s)) : end;
    };
    tc_after();
    const uint32_t tmem = B->tmem;
    const long long unit = range_units(wstart[A.nseq], A.P);
    if constexpr (!kSpans) w.begin(seq, wstart, A.nseq, A.geom, unit * blockIdx.x, unit * (blockIdx.x + 1));
    RowsPiece p;

    if (warp < 8) {
        if constexpr (kLong) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        // ---------------------------------------------------------------- softmax, a thread per row
        const int i = warp >> 2, r = tid & 127;                 // tile, row
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lanes + 128 * i, tP = tmem + lanes + kP + kPStep * i, tO = tmem + lanes + kO + HDP * i;
        const int tile_tok = r / G, few_tok = lane / G;  // the row's token; in a split item
        const float c = A.scale_log2;
        const float mu = kX ? 1.0f : c;   // of m, to the log2 domain
        uint32_t sp = 0, op = 0, xp = 0;  // phases of s_full; of both o_full (bit i); of x_full, x_free
        bool lent = false;                // group 1: group 0 may still read O and xm, xl of a twin item
        bool joined = false;
        const int wq = warp & 3;  // split items: the warp's quarter of a block's keys
        uint32_t hp = 0;          // phase of `quarter`
        RowsPiece ahead;  // the next piece, found while the tensor core finishes this one
        bool more = w.next(seq, A.nseq, A.geom, ahead);
        while (more) {
            p = ahead;
            const SeqRows sr = seq[p.s];
            const int pre = prefix_of(p.s);
            const TileView v = view(sr, p, i, pre);
            const bool whole = p.begins() && p.ends();
            const int tok = kSpans && v.split ? few_tok : tile_tok, head = (kSpans && v.split ? lane : r) - tok * G;
            const bool valid = tok < v.ntok && (kSpans && v.split ? lane < v.ntok * G : r < TT * G);
            const bool busy = __any_sync(0xffffffffu, valid);    // else only the hand-offs
            const int pos = sr.ctx + v.tok0 + tok;
            int from = 0, seen = pos + 1;  // the row sees positions [from, seen)
            float sl = 0.f;                // the head's slope, times log2(e)
            if constexpr (kSpans) {
                if (valid) row_span(A, w.mask(p.s), sr, v.tok0 + tok, p.g == 0 && head == 0 && p.begins(), from, seen);
                if (kBias && valid) sl = 1.4426950408889634f * __ldg(A.sc.slopes + p.g * G + head);
            }
            const bool sees = seen > p.kb0 * kTcBlk && (!kSpans || from < min(seen, p.kb1 * kTcBlk));  // some of the piece's
            const bool blind = kSpans && from >= seen;                                                // nothing at all
            // over the warp's rows: the least and the most that they see, their first position
            int seen_all = 0, seen_any = 0, from_all = 0, from_any = 0, pos_any = 0;
            bool steep = false;
            if constexpr (kSpans) {
                seen_all = __reduce_min_sync(0xffffffffu, valid ? seen : 0x7fffffff);
                seen_any = __reduce_max_sync(0xffffffffu, valid ? seen : 0);
                from_all = __reduce_max_sync(0xffffffffu, valid ? from : 0);
                from_any = __reduce_min_sync(0xffffffffu, valid ? from : 0x7fffffff);
                if (kBias) {
                    pos_any = __reduce_min_sync(0xffffffffu, valid ? pos : 0x7fffffff);
                    steep = __any_sync(0xffffffffu, fabsf(sl) > 96.f / 63.f);
                }
            }
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            const uint32_t op0 = op;  // phases that this piece's O completes
            if (v.twin) {
                op ^= p.kb1 - p.kb0 > 1 ? 3u : (uint32_t)(!kSpans || p.kb1 > p.kb0);
            } else {
                const TileView u = view(sr, p, 1 - i, pre);
                op ^= (uint32_t)(v.n > 0) << i | (uint32_t)(u.n > 0) << (1 - i);
            }
            if (i == 1 && lent && v.n > 0) {
                if (!tc_wait(&B->x_free, xp, A.status, stop)) break;
                xp ^= 1;
                lent = false;
            }
            if (!whole && p.begins()) {
                joined = true;
                if (tid == 0) write_join(A, blockIdx.x, seq, unit, &p);
            }
            for (int j = 0; j < v.n; j++) {
                if (!(ok = tc_wait(&B->s_full[i], sp, A.status, stop))) break;
                sp ^= 1;
                if constexpr (kSpans) {
                    // With kStraight, a block that all of the warp's rows see whole goes through straight code, keys
                    // 0-63 for the maximum only, keys 64-127 to stay, then 0-63 once more: long items run faster
                    // by it, short ones slower, whose instructions it pushes out of the cache (rows_op.cu has
                    // the figures).  The others go by quarters of 32 keys, in loops whose bodies fit the instruction cache beside the other roles': first for the
                    // maximum, then, the last quarter first (P of a quarter takes the place of keys behind it), for
                    // the weights.  In a split item the four warps hold the same 32 rows, and each has one quarter:
                    // their maxima and, at the end, sums meet in shared memory, and their weights, which the tensor
                    // core takes from there.
                    const int t0 = (v.first + j * v.step) * kTcBlk;
                    const int qa = v.split ? wq : 0, qb = v.split ? wq : 3;
                    float *xs = split_x + 384 * i;
                    float mb = -INFINITY, most = 0.f;
                    int tier = 0;
                    // keys [lo, hi) of the quarter are those that the row sees; `some`: any row of the warp does
                    auto mask = [&](uint32_t (&x)[32], int k0, uint32_t hidden) {
                        if (seen_all < k0 + 32) mask_from(x, seen - k0, seen_all - k0, hidden);
                        if (from_all > k0) mask_to(x, from - k0, from_all - k0, hidden);
                    };
                    auto some = [&](int k0) { return seen_any > k0 && from_any < k0 + 32; };
                    const bool both = kBias && pre > 0 && t0 + kTcBlk - 1 > pos_any;
                    const bool clear = kLong && busy && !v.split && seen_all >= t0 + kTcBlk && from_all <= t0 && !steep;
                    // The running maximum after a block's; O and l follow it where it grew by too much.
                    auto follow = [&](float top) {
                        if (j == 0) {
                            m = top;
                            return;
                        }
                        const bool grow = m == -INFINITY ? top > m : (top - m) * mu > kTcSlack;
                        if (!__any_sync(0xffffffffu, grow)) return;
                        const float f = grow ? fast_exp2((m - top) * mu) : 1.0f;
                        if (grow) m = top;
                        l *= f;
                        if (v.split && wq > 0) return;
#pragma unroll 1
                        for (int d = 0; d < HDP; d += 32) {
                            uint32_t o[32];
                            tmem_ld32(tO + d, o);
#pragma unroll
                            for (int k = 0; k < 32; k++) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                            tmem_st32(tO + d, o);
                        }
                        tmem_wait_st();
                    };
                    // The largest |product| is wanted for the cap's tier.  Without distances it serves for the maximum
                    // too, where no score can be far from 0: the cap of it is then a bound, at most 2 kNear above the
                    // largest score, and weights of 2^-24 of the largest stay normal numbers.  That holds for a row
                    // that sees some of these keys; of one that does not, `most` says nothing and there is no maximum.
                    auto bound = [&] {
                        if (!__all_sync(0xffffffffu, !valid || fminf(most * c, A.sc.cap_log2) <= kNear)) return false;
                        if (max(from, t0 + 32 * qa) < min(seen, t0 + 32 * qb + 32)) mb = cap_any(A.sc, c, most);
                        return true;
                    };
                    bool straight = false;  // the block is done
                    bool have = false;      // mb is
                    if (kLong && clear) {
                        tc_after();
                        __syncwarp();
                        // The largest score is the largest product's: tanh is monotone, and a distance's term is at
                        // most bias_most, a bound at most 63 |sl| above (`steep` has no more than 96, so that
                        // weights of 2^-24 of the largest stay normal numbers).
                        auto largest = [&](uint32_t (&x)[64], int k0) {
                            if (kCap) most = fmaxf(most, absmax(x));
                            if (kAbs) return -INFINITY;
                            float y = max_of(x);
                            if (kX) y = kCap ? cap_any(A.sc, c, y) : y * c;
                            if (kBias) y += bias_most<64>(sl, (float)(k0 - pos));
                            return y;
                        };
                        uint32_t lo[64], hi[64];
                        tmem_ld64(tS, lo);
                        mb = largest(lo, t0);
                        tmem_ld64(tS + 64, hi);
                        mb = fmaxf(mb, largest(hi, t0 + 64));
                        if (kCap) tier = cap_tier(A.sc, valid ? most : 0.f);
                        have = !kAbs || bound();
                        straight = have && tier == 0 && !both;
                        if (straight) {
                            follow(mb);
                            const float mc = m == -INFINITY ? 0.f : m * mu;
                            const uint64_t c2 = pack2(mu, mu), mc2 = pack2(-mc, -mc);
                            uint64_t sum[2] = {0, 0};
                            if (kX) score_pairs<SCORE, 0, false>(hi, A.sc, c, sl, (float)(t0 + 64 - pos), -mc);
                            straight_weights<kX>(hi, c2, mc2, sum, tP + 32);
                            tmem_wait_st();  // keys 64-127: the tensor core can begin
                            tc_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&B->p_half[i]);
                            __syncwarp();
                            tmem_ld64(tS, lo);
                            if (kX) score_pairs<SCORE, 0, false>(lo, A.sc, c, sl, (float)(t0 - pos), -mc);
                            straight_weights<kX>(lo, c2, mc2, sum, tP);
                            float a, b;
                            unpack2(add2(sum[0], sum[1]), a, b);
                            l += a + b;
                        }
                    } else if (busy) {
                        tc_after();
                        __syncwarp();
                        if constexpr (kAbs) {
#pragma unroll 1
                            for (int q = qa; q <= qb; q++) {
                                const int k0 = t0 + 32 * q;
                                if (!some(k0)) continue;
                                uint32_t x[32];
                                tmem_ld32(tS + 32 * q, x);
                                mask(x, k0, kIgnored);
                                most = fmaxf(most, absmax(x));
                            }
                            tier = cap_tier(A.sc, valid ? most : 0.f);
                            have = bound();
                        }
                    }
                    if (busy && !have) {
#pragma unroll 1
                        for (int q = qa; q <= qb; q++) {
                            const int k0 = t0 + 32 * q;
                            if (!some(k0)) continue;
                            uint32_t x[32];
                            tmem_ld32(tS + 32 * q, x);
                            mask(x, k0, kIgnored);
                            if (kCap && !kAbs) most = fmaxf(most, absmax(x));
                            // Of the products, the largest: tanh is monotone, and a distance's term is at most
                            // bias_most.  That bound of the maximum is at most 31 |sl| above it (96 where it is
                            // taken, so that weights of 2^-24 of the largest stay normal numbers).
                            float y = max_of(x);
                            if (kX && y != -INFINITY) {
                                y = kCap ? cap_any(A.sc, c, y) : y * c;
                                if (kBias) y += bias_most<32>(sl, (float)(k0 - pos));
                            }
                            mb = fmaxf(mb, y);
                        }
                        if (kCap && !kAbs) tier = cap_tier(A.sc, valid ? most : 0.f);
                        if (kBias && steep) {  // key by key
                            mb = -INFINITY;
#pragma unroll 1
                            for (int k = 32 * qa; k < 32 * qb + 32; k++) {
                                uint32_t x1;
                                tmem_ld1(tS + k, x1);
                                const float y = kCap ? cap_any(A.sc, c, __uint_as_float(x1)) : __uint_as_float(x1) * c;
                                if (t0 + k < seen && t0 + k >= from) mb = fmaxf(mb, fmaf(-sl, fabsf((float)(t0 + k - pos)), y));
                            }
                        }
                    }
                    if (v.split) {
                        xs[(j & 1) * 128 + 32 * wq + lane] = mb;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&B->quarter[i]);
                        if (!(ok = tc_wait(&B->quarter[i], hp, A.status, stop))) break;
                        hp ^= 1;
                        const float *xr = xs + (j & 1) * 128 + lane;
                        mb = fmaxf(fmaxf(xr[0], xr[32]), fmaxf(xr[64], xr[96]));
                    }
                    if (busy && !straight) {
                        follow(mb);
                        const float mc = m == -INFINITY ? 0.f : m * mu;
                        uint64_t sum[2] = {0, 0};
#pragma unroll 1
                        for (int q = qb; q >= qa; q--) {
                            const int k0 = t0 + 32 * q;
                            uint32_t x[32], pk[16];
                            if (some(k0)) {
                                tmem_ld32(tS + 32 * q, x);
                                if (kX) scores<SCORE>(x, A.sc, c, sl, (float)(k0 - pos), tier, both, -mc);
                                mask(x, k0, kHidden);
                                weights32<kX>(x, pack2(mu, mu), pack2(-mc, -mc), sum, pk);
                            } else {
#pragma unroll
                                for (int k = 0; k < 16; k++) pk[k] = 0;
                            }
                            if (v.split) {
                                // row `lane`, 16-byte chunk 4 (wq & 1) + e of its 128 bytes in panel wq >> 1
                                const uint32_t dst = smem_addr(split_p) + kSplitP * i + 4096 * (wq >> 1) + 128 * lane;
#pragma unroll
                                for (int e = 0; e < 4; e++)
                                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + (((4 * (wq & 1) + e) ^ (lane & 7)) << 4)),
                                                 "r"(pk[4 * e]), "r"(pk[4 * e + 1]), "r"(pk[4 * e + 2]), "r"(pk[4 * e + 3])
                                                 : "memory");
                            } else {
                                tmem_st16(tP + 16 * q, pk);
                                if (q == 2) {  // keys 64-127: the tensor core can begin
                                    tmem_wait_st();
                                    tc_before();
                                    __syncwarp();
                                    if (lane == 0) mbar_arrive(&B->p_half[i]);
                                    __syncwarp();
                                }
                            }
                        }
                        float a, b;
                        unpack2(add2(sum[0], sum[1]), a, b);
                        l += a + b;
                    }
                    if (v.split) {
                        if (j == v.n - 1) {  // before the last weights go: then this memory may be the producer's
                            xs[256 + 32 * wq + lane] = l;
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&B->quarter[i]);
                            if (!(ok = tc_wait(&B->quarter[i], hp, A.status, stop))) break;
                            hp ^= 1;
                            l = (xs[256 + lane] + xs[288 + lane]) + (xs[320 + lane] + xs[352 + lane]);
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    } else if (busy) {
                        tmem_wait_st();
                    }
                    tc_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (v.split || !busy) mbar_arrive(&B->p_half[i]);
                        mbar_arrive(&B->p_ready[i]);
                    }
                    continue;
                }
                if (busy) {
                    tc_after();
                    __syncwarp();
                    // Keys 0-63 for the maximum only, keys 64-127 to stay, then 0-63 once more: the
                    // row fits the registers in halves, and tensor memory is quick to read twice.
                    const int lim = seen - (v.first + j * v.step) * kTcBlk;  // keys of the block that the row sees
                    const int all = __reduce_min_sync(0xffffffffu, lim);
                    const bool cut = all < kTcBlk;
                    uint32_t lo[64], hi[64];
                    tmem_ld64(tS, lo);
                    if (cut) mask_from(lo, lim, all);
                    float mb = max_of(lo);
                    tmem_ld64(tS + 64, hi);
                    if (cut) mask_from(hi, lim - 64, all - 64);
                    mb = fmaxf(mb, max_of(hi));
                    if (j == 0) {
                        m = mb;
                    } else {
                        const bool grow = m == -INFINITY ? mb > m : (mb - m) * c > kTcSlack;
                        if (__any_sync(0xffffffffu, grow)) {
                            const float f = grow ? fast_exp2((m - mb) * c) : 1.0f;
                            if (grow) m = mb;
                            l *= f;
#pragma unroll 1
                            for (int d = 0; d < HDP; d += 32) {
                                uint32_t o[32];
                                tmem_ld32(tO + d, o);
#pragma unroll
                                for (int k = 0; k < 32; k++) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                                tmem_st32(tO + d, o);
                            }
                        }
                    }
                    const float mc = m == -INFINITY ? 0.f : m * c;
                    const uint64_t c2 = pack2(c, c), mc2 = pack2(-mc, -mc);
                    uint64_t sum[2] = {0, 0};  // two packed pairs of fp32 zeros
                    weights64(hi, c2, mc2, sum, tP + 32);
                    tmem_wait_st();  // keys 64-127: the tensor core can begin
                    tc_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&B->p_half[i]);
                    __syncwarp();
                    tmem_ld64(tS, lo);
                    if (cut) mask_from(lo, lim, all);
                    weights64(lo, c2, mc2, sum, tP);
                    float a, b;
                    unpack2(add2(sum[0], sum[1]), a, b);
                    l += a + b;
                    tmem_wait_st();
                    tc_before();
                } else {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&B->p_half[i]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&B->p_ready[i]);
            }
            if (!ok) break;
            more = w.next(seq, A.nseq, A.geom, ahead);
            // twin: group 1 hands its statistics over, group 0 adds both halves up
            const bool both = v.twin && p.kb1 - p.kb0 > 1;
            float f0 = 1.0f, f1 = 0.0f;
            if (both && i == 1) {
                if (!kSpans || !v.split || wq == 0) {
                    xm[r] = m;
                    xm[kXm + r] = l;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&B->x_full);
                lent = true;
                continue;
            }
            if (v.n > 0 && !tc_wait(&B->o_full[i], op0 >> i & 1, A.status, stop)) break;
            if (both) {
                if (!tc_wait(&B->o_full[1], op0 >> 1 & 1, A.status, stop)) break;
                if (!tc_wait(&B->x_full, xp, A.status, stop)) break;
                xp ^= 1;
                if (!kSpans || !v.split || wq == 0) {
                    const float m1 = xm[r], M = fmaxf(m, m1);
                    f0 = m == -INFINITY ? 0.f : fast_exp2((m - M) * mu);
                    f1 = m1 == -INFINITY ? 0.f : fast_exp2((m1 - M) * mu);
                    l = l * f0 + xm[kXm + r] * f1;
                    m = M;
                }
            }
            if (!busy || (v.twin && i == 1) || (kSpans && v.split && wq > 0)) {
                __syncwarp();
                if (both && lane == 0) mbar_arrive(&B->x_free);
                continue;
            }
            tc_after();
            __syncwarp();
            // O of this row, 32 columns at a time
            auto row_o = [&](int d, uint32_t (&o)[32]) {
                tmem_ld32(tO + d, o);
                if (both) {
                    uint32_t o1[32];
                    tmem_ld32(tO + HDP + d, o1);
#pragma unroll
                    for (int k = 0; k < 32; k++)
                        o[k] = __float_as_uint(__uint_as_float(o[k]) * f0 + __uint_as_float(o1[k]) * f1);
                }
            };
            if (whole) {
                const float inv = blind ? 0.f : 1.0f / l;
                uint16_t *dst = (uint16_t *)A.out + (size_t)(sr.row0 + v.tok0 + tok) * A.out_ld + (size_t)(p.g * G + head) * A.hd;
#pragma unroll 1
                for (int d = 0; d < HDP; d += 32) {
                    uint32_t o[32];
                    if (!kSpans || v.n > 0) row_o(d, o);
                    if (blind) {
#pragma unroll
                        for (int k = 0; k < 32; k++) o[k] = 0;
                    }
#pragma unroll
                    for (int k = 0; k < 32; k += 16) {
                        uint32_t h[8];
#pragma unroll
                        for (int q = 0; q < 8; q++)
                            h[q] = pack_bf16x2(__uint_as_float(o[k + 2 * q]) * inv, __uint_as_float(o[k + 2 * q + 1]) * inv);
                        if (!valid) continue;
                        if (T.wide) {  // whole 32-byte sectors: a lane writes its own row
                            if (d + k < A.hd) st_global32(dst + d + k, h);
                        } else {
                            if (d + k < A.hd) *(uint4 *)(dst + d + k) = make_uint4(h[0], h[1], h[2], h[3]);
                            if (d + k + 8 < A.hd) *(uint4 *)(dst + d + k + 8) = make_uint4(h[4], h[5], h[6], h[7]);
                        }
                    }
                    __syncwarp();
                }
            } else {
                float *part = slot_ptr(A, piece_slot(blockIdx.x, p));
                const int row = (v.twin ? 0 : i) * TT * G + r;
                if (v.n > 0) {
#pragma unroll 1
                    for (int d = 0; d < HDP; d += 32) {
                        uint32_t o[32];
                        row_o(d, o);
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            if (valid && d + k < A.hd)
                                *(uint4 *)(part + ((size_t)((d + k) / 4) * A.slot_rows + row) * 4) =
                                    make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                        __syncwarp();
                    }
                }
                if (valid) {  // the maximum in the log2 domain, as the join takes it
                    float *pm = part + (size_t)A.slot_rows * A.hd + row;
                    pm[0] = piece_max(m * mu, sees);
                    pm[A.slot_rows] = l;
                }
            }
            tc_before();
            __syncwarp();
            if (both && lane == 0) mbar_arrive(&B->x_free);
        }
        if (!joined && tid == 0) write_join(A, blockIdx.x, seq, unit, nullptr);
    } else if (kLong && warp >= 10) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    } else if (warp == 8) {
        if constexpr (kLong) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        // ---------------------------------------------------------------- tensor core
        constexpr uint32_t idS = tc_idesc(128, kTcBlk, 0), idO = tc_idesc(128, HDP, 1);
        const int ksteps = (A.hd + 15) / 16;
        // descriptors of the query tiles and of ring stage 0
        const uint32_t dq = desc_lo(sq, 16), dk = desc_lo(ring, 16), dv = desc_lo(ring, kPanel);
        // the ring stages of the next block's K and V (K, V, K, V, ... in the ring), and their phases
        uint32_t ks = 0, kph = 0, vs = 1, vph = 0;
        uint32_t qph = 0, pph = 0;  // phases of q_full and of p_half, p_ready: bit i
        bool ok = true, ran = false;  // ran: something was issued
        auto forward = [&](uint32_t &st, uint32_t &ph) {
            st += 2;
            if (st >= (uint32_t)T.stages) {
                st -= T.stages;
                ph ^= 1;
            }
        };
        auto issue_s = [&](int i, int qi) {  // S_i = Q_qi K^T
            const uint32_t a = dq + qi * (NP * kPanel / 16), b = dk + ks * (NP * kPanel / 16);
#pragma unroll
            for (int k = 0; k < HDP / 16; k++) {
                const int off = (k >> 2) * (kPanel / 16) + (k & 3) * 2;
                if (k < ksteps) mma_ss(tmem + 128 * i, a + off, b + off, idS, k != 0);
            }
        };
        auto issue_o = [&](int i, int half, bool first) {  // O_i (+)= P_i V, 64 keys
            const uint32_t b = dv + vs * (NP * kPanel / 16);
            const uint32_t a = tmem + kP + kPStep * i;
#pragma unroll
            for (int k = 0; k < 4; k++)
                mma_ts(tmem + kO + HDP * i, a + 8 * (4 * half + k), b + (4 * half + k) * 128, idO, !(first && k == 0));
        };
        auto issue_split_o = [&](int i, bool first) {  // O_i (+)= P_i V, all keys, P_i in shared memory
            const uint32_t b = dv + vs * (NP * kPanel / 16), a = desc_lo(split_p + kSplitP * i, 16);
#pragma unroll
            for (int k = 0; k < 8; k++)
                mma_ss(tmem + kO + HDP * i, a + (k >> 2) * (4096 / 16) + (k & 3) * 2, b + k * 128, idO, !(first && k == 0));
        };
        // P_i V for one block of group i; `last`: O_i is complete
        auto weigh = [&](int i, bool first, bool last) {
            if (!tc_wait(&B->p_half[i], pph >> i & 1, A.status, stop)) return false;
            tc_after();
            if (elect_one()) issue_o(i, 1, first);
            if (!tc_wait(&B->p_ready[i], pph >> i & 1, A.status, stop)) return false;
            pph ^= 1u << i;
            tc_after();
            if (elect_one()) {
                issue_o(i, 0, false);
                if (last) tc_commit(&B->o_full[i]);
            }
            return true;
        };
        auto weigh_split = [&](int i, bool first, bool last) {
            if (!tc_wait(&B->p_half[i], pph >> i & 1, A.status, stop)) return false;
            if (!tc_wait(&B->p_ready[i], pph >> i & 1, A.status, stop)) return false;
            pph ^= 1u << i;
            tc_after();
            if (elect_one()) {
                issue_split_o(i, first);
                if (last) tc_commit(&B->o_full[i]);
            }
            return true;
        };
        // V of the next block; the rows before `head` and from `tail` on are nobody's and become zero:
        // whole 128-byte rows, so the swizzle does not matter
        auto zero_v = [&](int r0, int r1) {
            const uint32_t v0 = smem_addr(ring) + vs * NP * kPanel + r0 * 128;
            for (int pn = 0; pn < NP; pn++)
                for (int x = lane * 16; x < (r1 - r0) * 128; x += 512)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(v0 + pn * kPanel + x), "r"(0) : "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
        };
        auto take_v = [&](int head, int tail) {
            if (!tc_wait(&B->kv_full[vs], vph, A.status, stop)) return false;
            if (tail < kTcBlk) zero_v(tail, kTcBlk);
            if (kSpans && head > 0) zero_v(0, head);
            return true;
        };
        auto drop_v = [&] {
            if (elect_one()) tc_commit(&B->kv_empty[vs]);
            forward(vs, vph);
        };
        auto drop_k = [&] {
            if (elect_one()) tc_commit(&B->kv_empty[ks]);
            forward(ks, kph);
        };
        RowsPiece ahead;  // the next piece, found while the softmax of this one's first block runs
        bool another = w.next(seq, A.nseq, A.geom, ahead);
        while (ok && another) {
            p = ahead;
            const SeqRows sr = seq[p.s];
            const int n = p.kb1 - p.kb0;
            if (kSpans && n == 0) {  // an item that sees nothing
                another = w.next(seq, A.nseq, A.geom, ahead);
                continue;
            }
            const int tail = p.ends() ? item_to(sr, p) - (p.kb1 - 1) * kTcBlk : kTcBlk;  // of the last block
            const int head = kSpans && p.begins() ? item_from(sr, p) - p.kb0 * kTcBlk : 0;  // of the first one
            const int pre = prefix_of(p.s);
            const TileView v0 = view(sr, p, 0, pre);
            if (kSpans && v0.split) {  // the second tile's place holds weights
                if (!(ok = tc_wait(&B->q_full[1], qph >> 1 & 1, A.status, stop))) break;
                qph ^= 2;
            }
            if (v0.twin) {
                // one tile: block b belongs to group b & 1
                auto score = [&](int b) {
                    if (!tc_wait(&B->kv_full[ks], kph, A.status, stop)) return false;
                    tc_after();
                    ran = true;
                    if (elect_one()) {
                        issue_s(b & 1, 0);
                        tc_commit(&B->s_full[b & 1]);
                        if (b == n - 1) tc_commit(&B->q_empty[0]);
                    }
                    drop_k();
                    return true;
                };
                if (!(ok = tc_wait(&B->q_full[0], qph & 1, A.status, stop))) break;
                qph ^= 1;
                if (!(ok = score(0)) || (n > 1 && !(ok = score(1)))) break;
                another = w.next(seq, A.nseq, A.geom, ahead);
                for (int b = 0; b < n; b++) {
                    if (!(ok = take_v(b == 0 ? head : 0, b == n - 1 ? tail : kTcBlk)) || !(ok = (kSpans && v0.split ? weigh_split(b & 1, b < 2, b + 2 >= n) : weigh(b & 1, b < 2, b + 2 >= n)))) break;
                    drop_v();
                    if (b + 2 < n && !(ok = score(b + 2))) break;
                }
                if (kSpans && ok && v0.split && elect_one()) tc_commit(&B->q_empty[1]);
                continue;
            }
            const int nt[2] = {v0.n, view(sr, p, 1, pre).n};
            if (!(ok = tc_wait(&B->kv_full[ks], kph, A.status, stop))) break;
#pragma unroll
            for (int i = 0; i < 2; i++) {
                if (nt[i] == 0) continue;
                if (!(ok = tc_wait(&B->q_full[i], qph >> i & 1, A.status, stop))) break;
                qph ^= 1u << i;
                tc_after();
                ran = true;
                if (elect_one()) {
                    issue_s(i, i);
                    tc_commit(&B->s_full[i]);
                    if (nt[i] == 1) tc_commit(&B->q_empty[i]);
                }
            }
            if (!ok) break;
            drop_k();
            another = w.next(seq, A.nseq, A.geom, ahead);
            for (int j = 0; j < n; j++) {
                if (!(ok = take_v(j == 0 ? head : 0, j == n - 1 ? tail : kTcBlk))) break;
                const bool more = j + 1 < n;
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    if (j < nt[i] && !(ok = weigh(i, j == 0, j == nt[i] - 1))) break;
                    if (i == 1) drop_v();
                    if (i == 0 && more) {
                        if (!(ok = tc_wait(&B->kv_full[ks], kph, A.status, stop))) break;
                        tc_after();
                    }
                    if (j + 1 < nt[i] && elect_one()) {
                        issue_s(i, i);
                        tc_commit(&B->s_full[i]);
                        if (j + 2 == nt[i]) tc_commit(&B->q_empty[i]);
                    }
                }
                if (!ok) break;
                if (more) drop_k();
            }
        }
        // What was issued has run, and its commits have arrived, before the CTA gives up its tensor and
        // shared memory -- in an abandoned call too, whoever gives up and however late.
        if (ran && elect_one()) {
            tc_commit(&B->drain);
            const unsigned long long t0 = global_ns();
            while (!mbar_try_wait(&B->drain, 0) && global_ns() - t0 < kWaitLimitNs) {
            }
        }
        __syncwarp();
    } else if (warp == 9) {
        if constexpr (kLong) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        // ---------------------------------------------------------------- TMA producer
        if constexpr (kSpans) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // masked_layout's scratch
        uint32_t st = 0, ph = 0, issued = 0;  // ring position; stages filled so far
        uint32_t qn[2] = {0, 0};              // query tiles loaded so far
        bool ok = true;
        const int shift = A.kv.page_shift, box = T.box;
        const int bshift = 31 - __clz(box);   // a box is the power of two that a page is, or a block
        const int per = kTcBlk >> bshift;     // boxes of a block
        while (ok && w.next(seq, A.nseq, A.geom, p)) {
            const SeqRows sr = seq[p.s];
            const int L = item_to(sr, p), from = item_from(sr, p), pre = prefix_of(p.s);
            // the page (lane: box) of a block, read a block ahead and not looked at before it is used
            auto page_of = [&](int kb) {
                const int pos = kb * kTcBlk + (lane << bshift);
                if (!PAGED || lane >= per || pos >= L || kb >= p.kb1 || (kSpans && pos + box <= from)) return 0;
                return __ldg(A.kv.table + (size_t)p.s * A.kv.table_ld + (pos >> shift));
            };
            int page = page_of(p.kb0);
            for (int kb = p.kb0; kb < p.kb1 && ok; kb++) {
                const int after = page_of(kb + 1);
                const int pos0 = kb * kTcBlk;
                const int nbox = PAGED ? min(per, (L - pos0 + box - 1) >> bshift) : 1;
                const int box0 = kSpans && PAGED ? max(0, from - pos0) >> bshift : 0;  // boxes that no row sees a position of
                if (PAGED && lane < nbox && lane >= box0 && (page < 0 || page >= A.kv.n_pages)) {  // becomes page 0
                    atomicOr(A.status, SLM_ROWS_PAGE);
                    page = 0;
                }
                for (int is_v = 0; is_v < 2; is_v++) {
                    if (issued >= (uint32_t)T.stages && !(ok = tc_wait(&B->kv_empty[st], ph ^ 1, A.status, stop))) break;
                    uint64_t *bar = &B->kv_full[st];
                    uint8_t *dst = ring + (size_t)st * NP * kPanel;
                    const CUtensorMap *map = is_v ? &T.v : &T.k;
                    if (lane == 0) mbar_expect_tx(bar, (uint32_t)((nbox - box0) << bshift) * (128 * NP));
                    __syncwarp();
                    if (lane < nbox && lane >= box0)
#pragma unroll
                        for (int pn = 0; pn < NP; pn++) {
                            if (PAGED)
                                tma_4d(dst + pn * kPanel + lane * box * 128, map, pn * 64, (pos0 + lane * box) & ((1 << shift) - 1),
                                       p.g, page, bar);
                            else
                                tma_3d(dst + pn * kPanel, map, pn * 64, p.g, sr.row0 + pos0, bar);
                        }
                    issued++;
                    if (++st == (uint32_t)T.stages) {
                        st = 0;
                        ph ^= 1;
                    }
                    if (kb == p.kb0 && is_v == 0) {  // the queries, behind the first keys
#pragma unroll
                        for (int i = 0; i < 2; i++) {
                            const TileView v = view(sr, p, i, pre);
                            if (kSpans && v.split) {
                                if (qn[i] > 0 && !(ok = tc_wait(&B->q_empty[i], (qn[i] - 1) & 1, A.status, stop))) break;
                                qn[i]++;
                                if (i == 1) {  // lent to the weights
                                    if (lane == 0) mbar_arrive(&B->q_full[1]);
                                } else if (lane == 0) {  // the rows once for each warp
                                    const int few = 32 / G;
                                    mbar_expect_tx(&B->q_full[0], (uint32_t)(NP * 4 * few * G * 128));
#pragma unroll
                                    for (int pn = 0; pn < NP; pn++)
#pragma unroll
                                        for (int q = 0; q < 4; q++)
                                            tma_3d(sq + (size_t)pn * kPanel + q * 4096, &T.q_few, pn * 64, p.g * G, sr.row0 + v.tok0,
                                                   &B->q_full[0]);
                                }
                                __syncwarp();
                                continue;
                            }
                            if (v.n == 0 || (v.twin && i == 1)) continue;
                            if (qn[i] > 0 && !(ok = tc_wait(&B->q_empty[i], (qn[i] - 1) & 1, A.status, stop))) break;
                            qn[i]++;
                            if (lane == 0) {
                                mbar_expect_tx(&B->q_full[i], (uint32_t)(NP * TT * G * 128));
#pragma unroll
                                for (int pn = 0; pn < NP; pn++)
                                    tma_3d(sq + (size_t)(i * NP + pn) * kPanel, &T.q, pn * 64, p.g * G, sr.row0 + v.tok0,
                                           &B->q_full[i]);
                            }
                        }
                        if (!ok) break;
                    }
                }
                page = after;
            }
        }
        // The copies have landed before the shared memory goes, as above.
        const unsigned long long t0 = global_ns();
        const uint32_t back = min(issued, (uint32_t)T.stages);
        for (uint32_t b = 1; b <= back; b++) {
            const uint32_t q = issued - b;
            while (!mbar_try_wait(&B->kv_full[q % T.stages], (q / T.stages) & 1) && global_ns() - t0 < kWaitLimitNs) {
            }
        }
        for (int i = 0; i < 2; i++)
            while (qn[i] > 0 && !mbar_try_wait(&B->q_full[i], (qn[i] - 1) & 1) && global_ns() - t0 < kWaitLimitNs) {
            }
    }
    tc_before();
    __syncthreads();
    if (warp == 8) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTcCols) : "memory");
    }
}

// ------------------------------------------------------------------ host side

static int tc_stages(int hd, int nseq, bool spans) {
    // ring stages: up to 10 of 16 KB or 5 of 32 KB, fewer where the batch's lengths need the room (1,024
    // sequences: 20 KB)
    const int HDP = hd <= 64 ? 64 : 128;
    int n = HDP == 64 ? 10 : 5;
    while (tc_fixed_bytes(HDP, n, spans) + tc_lengths_bytes(nseq, spans) > kSmemLimit) n--;
    return n;
}

// The attribute comes first: it is the runtime call that makes the device's context current on a
// host thread that has made none yet, and tensor maps are encoded by a driver call, which fails
// without one.
template <int HDP, bool PAGED, int SCORE> static cudaError_t launch_tc(RowsTcArgs &t, cudaStream_t s) {
    const RowsArgs &a = t.a;
    const size_t smem = tc_fixed_bytes(HDP, t.stages, SCORE != 0) + tc_lengths_bytes(a.nseq, SCORE != 0);
    cudaError_t e = allow_smem((const void *)rows_tc_kernel<HDP, PAGED, SCORE>);
    const uint64_t hb = (uint64_t)a.hd * 2;  // bytes of a head
    const uint64_t qd[] = {(uint64_t)a.hd, (uint64_t)a.H, (uint64_t)a.rows}, qs[] = {hb, (uint64_t)a.q_ld * 2};
    const uint32_t qb[] = {64, (uint32_t)a.G, (uint32_t)t.TT}, qf[] = {64, (uint32_t)a.G, (uint32_t)std::max(1, 32 / a.G)};
    if (e == cudaSuccess) e = make_bf16_map_nd(&t.q, a.q, 3, qd, qs, qb);
    if (e == cudaSuccess && SCORE) e = make_bf16_map_nd(&t.q_few, a.q, 3, qd, qs, qf);
    if (PAGED) {
        const uint64_t page = 1ull << a.kv.page_shift;
        t.box = page < kTcBlk ? (int)page : kTcBlk;
        const uint64_t d[] = {(uint64_t)a.hd, page, (uint64_t)a.KV, (uint64_t)a.kv.n_pages};
        const uint64_t st[] = {hb, hb * page, hb * page * a.KV};
        const uint32_t b[] = {64, (uint32_t)t.box, 1, 1};
        if (e == cudaSuccess) e = make_bf16_map_nd(&t.k, a.kv.k, 4, d, st, b);
        if (e == cudaSuccess) e = make_bf16_map_nd(&t.v, a.kv.v, 4, d, st, b);
    } else {
        t.box = kTcBlk;
        const uint64_t d[] = {(uint64_t)a.hd, (uint64_t)a.KV, (uint64_t)a.rows};
        const uint64_t ks[] = {hb, (uint64_t)a.kv.k_ld * 2}, vs[] = {hb, (uint64_t)a.kv.v_ld * 2};
        const uint32_t b[] = {64, 1, (uint32_t)t.box};
        if (e == cudaSuccess) e = make_bf16_map_nd(&t.k, a.kv.k, 3, d, ks, b);
        if (e == cudaSuccess) e = make_bf16_map_nd(&t.v, a.kv.v, 3, d, vs, b);
    }
    if (e != cudaSuccess) return e;
    return launch_pdl(rows_tc_kernel<HDP, PAGED, SCORE>, dim3(a.P), dim3(tc_threads(SCORE)), smem, s, t);
}

static RowsTcArgs tc_args(const RowsArgs &a, bool spans) {
    RowsTcArgs t{};
    t.a = a;
    t.TT = a.geom.PT / 2;
    t.stages = tc_stages(a.hd, a.nseq, spans);
    t.wide = ((uintptr_t)a.out & 31) == 0 && a.hd % 16 == 0 && a.out_ld % 16 == 0;
    return t;
}

}  // namespace slm
