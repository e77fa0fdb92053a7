// rows.cuh -- what the packed-row operators share: arguments, lengths in shared memory, the
// addresses of cached rows, the workspace of partial states.
#pragma once

#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include "rows_plan.h"
#include "slm_internal.h"

namespace slm {

// Keys and values of an attention call: a paged cache, or (table null) packed rows.
struct RowsKv {
    const uint8_t *k, *v;
    const int *table;      // [nseq][table_ld]
    int table_ld, n_pages, page_shift;
    long long k_ld, v_ld;  // packed rows: elements from one row to the next
};

struct RowsArgs {
    const int *row_start, *ctx_len;  // ctx_len null: no cached positions
    int nseq, rows;
    int H, KV, G, hd;
    long long cap;                   // positions a sequence may reach
    const uint8_t *q;
    uint8_t *out;
    long long q_ld, out_ld;          // elements
    RowsKv kv;
    int *status;
    float scale_log2;                // log2(e) / sqrt(hd)
    // partial states (rows_ws_bytes); P = CTAs of the attention launch
    uint8_t *ws;
    int P, slot_rows;
    RowsGeom geom;
    int lost;                        // test hook: a hand-off that never completes (slm_debug_rows_faults)
};

// Workspace: one RowsJoin per CTA, then 2 P slots of slot_rows unnormalised output rows
// (fp32, [hd / 4][slot_rows] quads), their running maxima (log2 domain) and their sums.
struct RowsJoin {
    int pieces;               // of the item that this CTA starts and another one finishes; 0: none
    int row0, tokens, head0;  // the item's first packed row, its tokens, its first query head
};

__host__ __device__ inline size_t join_bytes(int P) { return ((size_t)P * sizeof(RowsJoin) + 255) / 256 * 256; }
__host__ __device__ inline size_t slot_floats(int slot_rows, int hd) {
    return ((size_t)slot_rows * (hd + 2) + 63) / 64 * 64;
}
__host__ __device__ inline size_t rows_ws_bytes(int P, int slot_rows, int hd) {
    return join_bytes(P) + 2 * (size_t)P * slot_floats(slot_rows, hd) * sizeof(float);
}

#ifdef __CUDACC__

// Check every sequence's lengths and lay the units out: seq[nseq], wstart[nseq + 1] in
// shared memory.  Called by all `threads` threads of the CTA (tid from 0); ends with a
// __syncthreads().  A length out of bounds sets SLM_ROWS_LENGTH.
__device__ __forceinline__ void rows_layout(const RowsArgs &A, SeqRows *seq, long long *wstart, int tid, int threads) {
    for (int s = tid; s < A.nseq; s += threads) {
        SeqRows r;
        const int a = __ldg(A.row_start + s), b = __ldg(A.row_start + s + 1);
        const int c = A.ctx_len ? __ldg(A.ctx_len + s) : 0;
        if (!seq_rows(a, b, c, A.rows, A.cap, r) && blockIdx.x == 0) atomicOr(A.status, SLM_ROWS_LENGTH);
        seq[s] = r;
        wstart[s + 1] = r.n > 0 ? head_units(A.geom, r.ctx, r.n, item_count(A.geom, r.n)) * A.KV : 0;
    }
    if (tid == 0) wstart[0] = 0;
    __syncthreads();
    if (tid < 32) {  // inclusive scan of wstart[1 ..]
        long long carry = 0;
        for (int s0 = 0; s0 < A.nseq; s0 += 32) {
            const int s = s0 + tid;
            long long v = s < A.nseq ? wstart[s + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(0xffffffffu, v, o);
                if (tid >= o) v += u;
            }
            if (s < A.nseq) wstart[s + 1] = carry + v;
            carry += __shfl_sync(0xffffffffu, v, 31);
        }
    }
    __syncthreads();
}

// What the joining kernel needs to know about the item that this CTA starts and another
// finishes (p null: none).  unit: units of a range.
__device__ __forceinline__ void write_join(const RowsArgs &A, int cta, const SeqRows *seq, long long unit,
                                           const RowsPiece *p) {
    RowsJoin j{};
    if (p) {
        const SeqRows r = seq[p->s];
        j.pieces = (int)udiv(p->base + A.geom.cost + p->nb - 1, unit) - cta + 1;
        j.row0 = r.row0 + p->t * A.geom.PT;
        j.tokens = min(A.geom.PT, r.n - p->t * A.geom.PT);
        j.head0 = p->g * A.G;
    }
    ((RowsJoin *)A.ws)[cta] = j;
}

// The maximum of a row's partial state (log2 domain).  -infinity tells the join that the row sees
// none of the piece's positions; a row that sees some has a finite one, also where every score is
// NaN (maxima skip those) or -infinity.
__device__ __forceinline__ float piece_max(float m, bool sees) { return sees ? fmaxf(m, -FLT_MAX) : -INFINITY; }

__device__ __forceinline__ float *slot_ptr(const RowsArgs &A, int slot) {
    return (float *)(A.ws + join_bytes(A.P)) + (size_t)slot * slot_floats(A.slot_rows, A.hd);
}

#endif  // __CUDACC__

// ---- host side, shared by the entry points (rows_op.cu)

int attn_fail(int code, const char *fmt, ...);  // records the text, returns the code

// Let the launches of `kernel` ask for up to kSmemLimit bytes of shared memory.  The attribute is
// the function's, on the current device, not the launch's: with the same value from every call, no
// other host thread's launch can find it lowered between here and there.
inline cudaError_t allow_smem(const void *kernel) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemLimit);
}

// The joining launch: every item that several CTAs share, from its partial states.
cudaError_t rows_join_launch(const RowsArgs &a, bool bf16, cudaStream_t s);

// CUDA-core attention: fp32, and bf16 heads wider than 128.
constexpr int kSimtSmallTile = 16;                      // query rows (token, head) per item: of the small tile,
int rows_simt_wide_tile(int hd);                        // of the wide one,
int rows_simt_tile(int rows, int nseq, int G, int hd);  // and of the one that a call takes
int rows_simt_ctas(int sms, int hd, int R, int nseq);
cudaError_t rows_simt_launch(const RowsArgs &a, bool bf16, cudaStream_t s);

// Tensor-core attention: bf16, head_dim up to 128; items of two tiles of 128 / G tokens.
cudaError_t rows_tc_launch(const RowsArgs &a, cudaStream_t s);

struct AppendArgs {
    const int *row_start, *ctx_len;
    int nseq, rows;
    int H, KV, hd;
    long long cap;
    const uint8_t *q, *k, *v;
    uint8_t *q_out, *kc, *vc;
    long long q_ld, k_ld, v_ld, q_out_ld;
    const float *rope;
    int rope_len;
    const int *table;
    int table_ld, n_pages, page_shift;
    int *status;
};
cudaError_t rows_append_launch(const AppendArgs &a, bool in_bf16, bool cache_bf16, cudaStream_t s);

}  // namespace slm
