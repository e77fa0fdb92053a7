// rows_attention_tc.cu -- attention of packed bf16 rows on the 5th-generation tensor cores,
// heads of up to 128, over a paged cache or packed prompts.
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
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "device_common.cuh"
#include "gemm_tc.cuh"
#include "rows.cuh"

namespace slm {

constexpr int kTcThreads = 320;
constexpr int kTcBlk = 128;                 // positions per block
constexpr int kPanel = 128 * 128;           // bytes of [128 rows][64 bf16]
constexpr int kTcCols = 512;                // tensor memory columns
constexpr float kTcSlack = 8.0f;            // log2 growth of a maximum that O is not rescaled for

struct RowsTcArgs {
    CUtensorMap q, k, v;
    RowsArgs a;
    int TT;      // tokens per tile
    int box;     // positions per key / value box
    int stages;  // ring depth
    int wide;    // output heads begin on 32-byte boundaries and are multiples of 16 long
};

struct TcBars {
    uint64_t kv_full[16], kv_empty[16];
    uint64_t q_full[2], q_empty[2], s_full[2], p_half[2], p_ready[2], o_full[2], drain;
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
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Keys from `lim` on become -infinity.  `all` (at most any lane's lim): no lane's key before it does,
// so groups of 16 below it are left alone (two instructions an element at half rate: a diagonal
// block took twice as long as the others).
__device__ __forceinline__ void mask64(uint32_t (&s)[64], int lim, int all) {
#pragma unroll
    for (int k0 = 0; k0 < 64; k0 += 16)
        if (k0 + 16 > all) {
#pragma unroll
            for (int k = k0; k < k0 + 16; k++)
                if (k >= lim) s[k] = 0xff800000u;
        }
}

__device__ __forceinline__ float max64(const uint32_t (&s)[64]) {
    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int k = 0; k < 64; k += 8)
#pragma unroll
        for (int q = 0; q < 4; q++) m[q] = max3(m[q], __uint_as_float(s[k + 2 * q]), __uint_as_float(s[k + 2 * q + 1]));
    return fmaxf(max3(m[0], m[1], m[2]), m[3]);
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
    bool twin;
    int n, tok0, ntok;  // blocks; first token in the sequence; tokens
    int first, step;    // block j is first + j step
};
template <bool TWIN>
__device__ __forceinline__ TileView tile_view(const SeqRows &sr, const RowsPiece &p, int TT, int PT, int i) {
    TileView v;
    const int left = sr.n - p.t * PT;  // tokens from the item's first on, at least 1
    v.twin = TWIN && left <= TT;
    if (v.twin) {
        v.tok0 = p.t * PT;
        v.ntok = left;
        v.n = (p.kb1 - p.kb0 + 1 - i) >> 1;
        v.first = p.kb0 + i;
        v.step = 2;
    } else {
        v.tok0 = p.t * PT + i * TT;
        v.ntok = max(0, min(TT, sr.n - v.tok0));
        v.n = v.ntok > 0 ? max(0, min(p.kb1, (sr.ctx + v.tok0 + v.ntok + kTcBlk - 1) / kTcBlk) - p.kb0) : 0;
        v.first = p.kb0;
        v.step = 1;
    }
    return v;
}

__host__ __device__ constexpr size_t tc_fixed_bytes(int HDP, int stages) {
    return 1024 + (size_t)(2 + stages) * (HDP / 64) * kPanel + (sizeof(TcBars) + 15) / 16 * 16 + (HDP == 64 ? 1024 : 0);
}

// ------------------------------------------------------------------ the kernel

template <int HDP, bool PAGED>
__global__ void __launch_bounds__(kTcThreads, 1) rows_tc_kernel(const __grid_constant__ RowsTcArgs T) {
    constexpr int NP = HDP / 64;  // 64-column panels of a [128][head_dim] operand
    // Tensor memory columns: S 128 i, O 256 + HDP i.  P (64 columns) has its own where O leaves
    // room, else the upper half of S, which the softmax holds in registers by then.
    constexpr uint32_t kO = 256, kP = HDP == 64 ? 384 : 64, kPStep = HDP == 64 ? 64 : 128;
    // One-tile items twice over only where it pays: a block of 64-wide heads arrives faster than one
    // group's chain of S, softmax and P V (4 x 32,768 positions: 72 us with one group, 52 with two);
    // 128-wide ones come at 95% of the copy rate with one group, and joining the halves costs 4%.
    constexpr bool kTwin = HDP == 64;
    const RowsArgs &A = T.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *sq = base;                             // [2 tiles][NP][128][64]
    uint8_t *ring = base + 2 * NP * kPanel;         // [stages][NP][128][64]
    TcBars *B = (TcBars *)(ring + (size_t)T.stages * NP * kPanel);
    float *xm = (float *)((uint8_t *)B + (sizeof(TcBars) + 15) / 16 * 16);  // [128] maxima, [128] sums
    long long *wstart = (long long *)(xm + (kTwin ? 256 : 0));
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
    rows_layout(A, seq, wstart, tid, kTcThreads);  // ends with a __syncthreads()
    tc_after();
    const uint32_t tmem = B->tmem;
    const long long unit = range_units(wstart[A.nseq], A.P);
    RowsWalk w;
    w.begin(seq, wstart, A.nseq, A.geom, unit * blockIdx.x, unit * (blockIdx.x + 1));
    RowsPiece p;

    if (warp < 8) {
        // ---------------------------------------------------------------- softmax, a thread per row
        const int i = warp >> 2, r = tid & 127;                 // tile, row
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lanes + 128 * i, tP = tmem + lanes + kP + kPStep * i, tO = tmem + lanes + kO + HDP * i;
        const int tok = r / G, head = r - tok * G;
        const float c = A.scale_log2;
        uint32_t sp = 0, op = 0, xp = 0;  // phases of s_full; of both o_full (bit i); of x_full, x_free
        bool lent = false;                // group 1: group 0 may still read O and xm, xl of a twin item
        bool joined = false;
        RowsPiece ahead;  // the next piece, found while the tensor core finishes this one
        bool more = w.next(seq, A.nseq, A.geom, ahead);
        while (more) {
            p = ahead;
            const SeqRows sr = seq[p.s];
            const TileView v = tile_view<kTwin>(sr, p, TT, PT, i);
            const bool whole = p.kb0 == 0 && p.kb1 == p.nb;
            const bool valid = tok < v.ntok && r < TT * G;
            const bool busy = __any_sync(0xffffffffu, valid);    // else only the hand-offs
            const int seen = sr.ctx + v.tok0 + tok + 1;          // positions the row sees
            const bool sees = seen > p.kb0 * kTcBlk;             // some of the piece's
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            const uint32_t op0 = op;  // phases that this piece's O completes
            if (v.twin) {
                op ^= (p.kb1 - p.kb0 > 1) ? 3u : 1u;
            } else {
                const TileView u = tile_view<kTwin>(sr, p, TT, PT, 1 - i);
                op ^= (uint32_t)(v.n > 0) << i | (uint32_t)(u.n > 0) << (1 - i);
            }
            if (i == 1 && lent && v.n > 0) {
                if (!tc_wait(&B->x_free, xp, A.status, stop)) break;
                xp ^= 1;
                lent = false;
            }
            if (!whole && p.kb0 == 0) {
                joined = true;
                if (tid == 0) write_join(A, blockIdx.x, seq, unit, &p);
            }
            for (int j = 0; j < v.n; j++) {
                if (!(ok = tc_wait(&B->s_full[i], sp, A.status, stop))) break;
                sp ^= 1;
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
                    if (cut) mask64(lo, lim, all);
                    float mb = max64(lo);
                    tmem_ld64(tS + 64, hi);
                    if (cut) mask64(hi, lim - 64, all - 64);
                    mb = fmaxf(mb, max64(hi));
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
                    if (cut) mask64(lo, lim, all);
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
                xm[r] = m;
                xm[128 + r] = l;
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
                const float m1 = xm[r], M = fmaxf(m, m1);
                f0 = m == -INFINITY ? 0.f : fast_exp2((m - M) * c);
                f1 = m1 == -INFINITY ? 0.f : fast_exp2((m1 - M) * c);
                l = l * f0 + xm[128 + r] * f1;
                m = M;
            }
            if (!busy || (v.twin && i == 1)) {
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
                const float inv = 1.0f / l;
                uint16_t *dst = (uint16_t *)A.out + (size_t)(sr.row0 + v.tok0 + tok) * A.out_ld + (size_t)(p.g * G + head) * A.hd;
#pragma unroll 1
                for (int d = 0; d < HDP; d += 32) {
                    uint32_t o[32];
                    row_o(d, o);
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
                    pm[0] = piece_max(m * c, sees);
                    pm[A.slot_rows] = l;
                }
            }
            tc_before();
            __syncwarp();
            if (both && lane == 0) mbar_arrive(&B->x_free);
        }
        if (!joined && tid == 0) write_join(A, blockIdx.x, seq, unit, nullptr);
    } else if (warp == 8) {
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
        // V of the next block; the rows from `tail` on are nobody's and become zero: whole 128-byte
        // rows, so the swizzle does not matter
        auto take_v = [&](int tail) {
            if (!tc_wait(&B->kv_full[vs], vph, A.status, stop)) return false;
            if (tail < kTcBlk) {
                const uint32_t v0 = smem_addr(ring) + vs * NP * kPanel + tail * 128;
                for (int pn = 0; pn < NP; pn++)
                    for (int x = lane * 16; x < (kTcBlk - tail) * 128; x += 512)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(v0 + pn * kPanel + x), "r"(0)
                                     : "memory");
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
            }
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
            const int L = sr.ctx + min(p.t * PT + PT, sr.n);  // positions the item sees
            const int tail = p.kb1 == p.nb ? L - (p.nb - 1) * kTcBlk : kTcBlk;  // of the last block
            const TileView v0 = tile_view<kTwin>(sr, p, TT, PT, 0);
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
                    if (!(ok = take_v(b == n - 1 ? tail : kTcBlk)) || !(ok = weigh(b & 1, b < 2, b + 2 >= n))) break;
                    drop_v();
                    if (b + 2 < n && !(ok = score(b + 2))) break;
                }
                continue;
            }
            const int nt[2] = {v0.n, tile_view<kTwin>(sr, p, TT, PT, 1).n};
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
                if (!(ok = take_v(j == n - 1 ? tail : kTcBlk))) break;
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
        // ---------------------------------------------------------------- TMA producer
        uint32_t st = 0, ph = 0, issued = 0;  // ring position; stages filled so far
        uint32_t qn[2] = {0, 0};              // query tiles loaded so far
        bool ok = true;
        const int shift = A.kv.page_shift, box = T.box;
        const int per = kTcBlk / box;         // boxes of a block
        while (ok && w.next(seq, A.nseq, A.geom, p)) {
            const SeqRows sr = seq[p.s];
            const int L = sr.ctx + min(p.t * PT + PT, sr.n);
            // the page (lane: box) of a block; a bad id becomes page 0
            auto page_of = [&](int kb) {
                const int pos = kb * kTcBlk + lane * box;
                if (!PAGED || lane >= per || pos >= L || kb >= p.kb1) return -1;
                int pg = __ldg(A.kv.table + (size_t)p.s * A.kv.table_ld + (pos >> shift));
                if (pg < 0 || pg >= A.kv.n_pages) {
                    atomicOr(A.status, SLM_ROWS_PAGE);
                    pg = 0;
                }
                return pg;
            };
            int page = page_of(p.kb0);
            for (int kb = p.kb0; kb < p.kb1 && ok; kb++) {
                const int after = page_of(kb + 1);
                const int pos0 = kb * kTcBlk;
                const int nbox = PAGED ? min(per, (L - pos0 + box - 1) / box) : 1;
                for (int is_v = 0; is_v < 2; is_v++) {
                    if (issued >= (uint32_t)T.stages && !(ok = tc_wait(&B->kv_empty[st], ph ^ 1, A.status, stop))) break;
                    uint64_t *bar = &B->kv_full[st];
                    uint8_t *dst = ring + (size_t)st * NP * kPanel;
                    const CUtensorMap *map = is_v ? &T.v : &T.k;
                    if (lane == 0) mbar_expect_tx(bar, (uint32_t)(nbox * box * 128 * NP));
                    __syncwarp();
                    if (lane < nbox)
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
                            const TileView v = tile_view<kTwin>(sr, p, TT, PT, i);
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

static int tc_stages(int hd, int nseq) {
    // ring stages: up to 10 of 16 KB or 5 of 32 KB, fewer where the batch's lengths need the room (1,024
    // sequences: 20 KB)
    const int HDP = hd <= 64 ? 64 : 128;
    int n = HDP == 64 ? 10 : 5;
    while (tc_fixed_bytes(HDP, n) + (size_t)nseq * sizeof(SeqRows) + (size_t)(nseq + 1) * 8 > kSmemLimit) n--;
    return n;
}

// The attribute comes first: it is the runtime call that makes the device's context current on a
// host thread that has made none yet, and tensor maps are encoded by a driver call, which fails
// without one.
template <int HDP, bool PAGED> static cudaError_t launch_tc(RowsTcArgs &t, cudaStream_t s) {
    const RowsArgs &a = t.a;
    const size_t smem = tc_fixed_bytes(HDP, t.stages) + (size_t)a.nseq * sizeof(SeqRows) + (size_t)(a.nseq + 1) * 8;
    cudaError_t e = allow_smem((const void *)rows_tc_kernel<HDP, PAGED>);
    const uint64_t hb = (uint64_t)a.hd * 2;  // bytes of a head
    const uint64_t qd[] = {(uint64_t)a.hd, (uint64_t)a.H, (uint64_t)a.rows}, qs[] = {hb, (uint64_t)a.q_ld * 2};
    const uint32_t qb[] = {64, (uint32_t)a.G, (uint32_t)t.TT};
    if (e == cudaSuccess) e = make_bf16_map_nd(&t.q, a.q, 3, qd, qs, qb);
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
    return launch_pdl(rows_tc_kernel<HDP, PAGED>, dim3(a.P), dim3(kTcThreads), smem, s, t);
}

cudaError_t rows_tc_launch(const RowsArgs &a, cudaStream_t s) {
    RowsTcArgs t{};
    t.a = a;
    t.TT = a.geom.PT / 2;
    t.stages = tc_stages(a.hd, a.nseq);
    t.wide = ((uintptr_t)a.out & 31) == 0 && a.hd % 16 == 0 && a.out_ld % 16 == 0;
    const bool paged = a.kv.table != nullptr;
    if (a.hd <= 64) return paged ? launch_tc<64, true>(t, s) : launch_tc<64, false>(t, s);
    return paged ? launch_tc<128, true>(t, s) : launch_tc<128, false>(t, s);
}

}  // namespace slm
