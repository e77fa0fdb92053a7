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

// Scores and masks besides the plain causal ones (slm_scores); all null and zero: those.
struct RowsScores {
    const float *slopes;         // [H]
    const int *prefix, *first;   // [nseq], [rows]
    int window;
    float cap_in, cap_log2;      // scale / cap, cap log2(e)
    // the tensor-core kernel's tanh (rows_attention_tc.cuh): |q . k| up to half the cap and up to it, and the
    // polynomials' coefficients of powers of (q . k)^2
    float half_cap, one_cap, poly3[3], poly5[5];
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
    float scale_log2;                // log2(e) / sqrt(hd), or log2(e) times the caller's scale
    RowsScores sc;
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

// Masked items: the mask of sequence s, its prefix cut to the sequence.
struct SeqMasks {
    const SeqRows *seq;
    const int *prefixes, *first;
    int window;
    __device__ __forceinline__ int prefix(int s) const {
        return prefixes ? min(max(__ldg(prefixes + s), 0), seq[s].ctx + seq[s].n) : 0;
    }
    __device__ __forceinline__ RowsMask operator()(int s) const {
        return RowsMask{first ? first + seq[s].row0 : nullptr, prefix(s), window};
    }
};
typedef MaskedWalk<SeqMasks> RowsMaskedWalk;

// Shared memory that masked_layout takes after seq and wstart (aligned to 16 bytes); besides, nseq + 1
// ints of scratch that it is done with at its end.
__host__ __device__ inline size_t masked_bytes() { return sizeof(RowsStart) + 16; }

// The last s with a[s] <= x, of n.
template <typename T> __device__ __forceinline__ int last_upto(const T *a, int n, T x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a[mid] <= x)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// a[1 .. n] become their inclusive sums times `times`, none above `most`; the last sum, uncut.  One warp.
template <typename T> __device__ __forceinline__ long long running_sums(T *a, int n, long long times, long long most, int lane) {
    long long carry = 0;
    for (int s0 = 0; s0 < n; s0 += 32) {
        const int s = s0 + lane;
        long long v = s < n ? a[s + 1] * times : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        if (s < n) a[s + 1] = (T)min(carry + v, most);
        carry += __shfl_sync(0xffffffffu, v, 31);
    }
    return carry;
}

// rows_layout for masked items.  A sequence of one item has its units at once (a decode step); those of
// several are added up item by item, an equal share of them per thread (8,192 rows of 4 heads per kv
// head are 128 items).  Warp 0 looks for the item that this CTA's range begins in.  Ends with a
// __syncthreads().
__device__ __forceinline__ void masked_layout(const RowsArgs &A, SeqRows *seq, long long *wstart, RowsStart *start, int *items,
                                              RowsMaskedWalk &w, int tid, int threads) {
    w.mask = SeqMasks{seq, A.sc.prefix, A.sc.first, A.sc.window};
    bool several = false;
    for (int s = tid; s < A.nseq; s += threads) {
        SeqRows r;
        const int a = __ldg(A.row_start + s), b = __ldg(A.row_start + s + 1);
        const int c = A.ctx_len ? __ldg(A.ctx_len + s) : 0;
        if (!seq_rows(a, b, c, A.rows, A.cap, r) && blockIdx.x == 0) atomicOr(A.status, SLM_ROWS_LENGTH);
        seq[s] = r;
        const int n = r.n > 0 ? item_count(A.geom, r.n) : 0;
        several |= n > 1;
        items[s + 1] = n;
        wstart[s + 1] = n == 1 ? A.geom.cost + item_span(A.geom, r, w.mask(s), 0).nb : 0;
    }
    if (tid == 0) wstart[0] = items[0] = 0;
    if (__syncthreads_or(several)) {
        if (tid < 32) {
            // Row ranges that overlap (row_start descends somewhere, which has been reported) could
            // claim any number of items; ranges that do not have at most this many.
            const long long most = (long long)A.rows / A.geom.PT + A.nseq;
            if (running_sums(items, A.nseq, 1, most, tid) > most) {  // nobody has rows then
                __syncwarp();
                for (int s = tid; s < A.nseq; s += 32) {
                    seq[s].n = 0;
                    items[s + 1] = 0;
                    wstart[s + 1] = 0;
                }
            }
        }
        __syncthreads();
        const int all = items[A.nseq], share = (all + threads - 1) / threads;
        const int i1 = min(all, (tid + 1) * share);
        int i = min(all, tid * share);
        if (i < i1)
            for (int s = last_upto(items, A.nseq, i); i < i1; s++) {
                const int stop = min(i1, items[s + 1]);
                if (i >= stop) continue;
                const SeqRows r = seq[s];
                const RowsMask m = w.mask(s);
                unsigned long long units = 0;
                const bool one = items[s + 1] - items[s] == 1;  // has its units
                for (; i < stop; i++)
                    if (!one) units += A.geom.cost + item_span(A.geom, r, m, i - items[s]).nb;
                if (!one) atomicAdd((unsigned long long *)&wstart[s + 1], units);  // whole numbers: any order
            }
        __syncthreads();
    }
    if (tid < 32) {
        running_sums(wstart, A.nseq, A.KV, 0x7fffffffffffffffLL, tid);
        __syncwarp();
        const long long total = wstart[A.nseq], x = range_units(total, A.P) * blockIdx.x;
        if (x < total) {
            const int s = last_upto(wstart, A.nseq, x);
            const SeqRows r = seq[s];
            const RowsMask m = w.mask(s);
            const unsigned long long per = udiv(wstart[s + 1] - wstart[s], A.KV), g = udiv(x - wstart[s], per);
            long long at = wstart[s] + (long long)(g * per);  // units before item t0 of this kv head
            const int T = item_count(A.geom, r.n);
            if (T == 1) {
                if (tid == 0) *start = RowsStart{s, (int)g, 0, at};
            } else {
                for (int t0 = 0; t0 < T; t0 += 32) {
                    const int t = t0 + tid, u = t < T ? A.geom.cost + item_span(A.geom, r, m, t).nb : 0;
                    long long v = u;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const long long y = __shfl_up_sync(0xffffffffu, v, o);
                        if (tid >= o) v += y;
                    }
                    const bool mine = u > 0 && at + v - u <= x && x < at + v;
                    if (mine) *start = RowsStart{s, (int)g, t, at + v - u};
                    if (__any_sync(0xffffffffu, mine)) break;
                    at += __shfl_sync(0xffffffffu, v, 31);
                }
            }
        }
    }
    __syncthreads();
}

// The span that row i of sequence s sees; checks that `first` does not descend.
__device__ __forceinline__ void row_span(const RowsArgs &A, const RowsMask &m, const SeqRows &r, int i, bool check, int &lo,
                                         int &hi) {
    lo = row_from(m, r.ctx, i);
    hi = row_to(m, r.ctx, i);
    if (check && m.first && i > 0 && m.first[i] < m.first[i - 1]) atomicOr(A.status, SLM_ROWS_LENGTH);
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
cudaError_t rows_simt_scored_launch(const RowsArgs &a, bool bf16, cudaStream_t s);

// Tensor-core attention: bf16, head_dim up to 128; items of two tiles of 128 / G tokens.
cudaError_t rows_tc_launch(const RowsArgs &a, cudaStream_t s);
// head_dim up to 64, and from 72 to 128; `straight`: the same for long items.
cudaError_t rows_tc_scored_64(const RowsArgs &a, cudaStream_t s);
cudaError_t rows_tc_scored_128(const RowsArgs &a, cudaStream_t s);
cudaError_t rows_tc_scored_straight_64(const RowsArgs &a, cudaStream_t s);
cudaError_t rows_tc_scored_straight_128(const RowsArgs &a, cudaStream_t s);

// What a kernel does beyond the plain causal scores, as bits of a template argument.
// kStraight: how, not what (rows_attention_tc.cuh).
constexpr int kMasked = 1, kCapped = 2, kBiased = 4, kStraight = 8;

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

// The append whose pairs turn by positions of their own axes.
constexpr int kMaxAxes = 8;
struct AxesArgs {
    AppendArgs a;
    const int *positions;    // [n_axes][ld]
    long long ld;
    int n_axes;
    uint8_t axis[128];       // of every pair; 0xff: not turned
};
cudaError_t rows_append_axes_launch(const AxesArgs &a, bool in_bf16, bool cache_bf16, cudaStream_t s);

// The plan of a step.
struct StepArgs {
    const int *new_len, *seq_len, *free_count;
    int *page_table, *free_pages;
    int nseq, table_ld, n_pages, page_shift, rows;
    long long cap;
    int *row_start, *ctx_len, *positions, *seq_len_out, *free_count_out, *status;
    long long *slots;
};
cudaError_t rows_step_launch(const StepArgs &a, cudaStream_t s);

constexpr int kSampleMaxVocab = 1 << 22;  // weights of 2^40 at most add up below 2^62
// The draw of the next tokens with every row's own parameters (null: the default).
struct SampleRowsArgs {
    const uint8_t *logits;  // [rows][ld] of fp32 or bf16
    long long ld;
    int rows, vocab;
    const float *temperature, *top_p, *min_p, *uniforms;
    const int *top_k;
    int *next_ids;
};
cudaError_t sample_rows_launch(const SampleRowsArgs &a, bool bf16, int sms, cudaStream_t s);

}  // namespace slm
