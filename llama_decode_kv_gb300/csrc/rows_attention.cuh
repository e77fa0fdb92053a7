// rows_attention.cuh -- attention of packed rows on the CUDA cores (fp32, and bf16 heads wider
// than 128): the kernels, compiled for plain causal scores by rows_attention.cu and for scored ones
// by rows_scored.cu.
//
// For a row at position p and query head h of kv head g = h / G:
//     out = sum_{t <= p} softmax_t(q . k_t / sqrt(hd)) v_t.
// An item is up to R rows (token, head) of one kv head, so that keys and values are read once
// for the whole query group.  A CTA walks its blocks of 64 positions with one pass of a
// running softmax: S = Q K^T, the row's maximum m and sum l carried on in fp32 and
// O = 2^(m_old - m_new) O + P V, everything fp32 in the log2 domain (q . k times
// log2(e) / sqrt(hd)).  fp32 has no tensor-core format of its own precision, so the FMA pipe
// bounds prompts and large chunks (rows_fma_kernel: 64-row tiles); a decode step is bound by
// reading the cache, and takes the 16-row tile of rows_simt_kernel, where four thread groups share
// the keys of a block instead of multiplying rows that do not exist.  Seven prompts of up to 701
// tokens, 9 / 3 heads of 64: 76 us = 18 TFLOP/s of useful work, 30% of the FMA pipe's issue slots (a
// CTA has five blocks, and half of a diagonal block is masked).
//
// Scored rows are the same kernels with SCORED: a row's span (row_span) in place of [0, p], and simt_score
// on every product.  The prefixes make blocks above the diagonal count, which is why seven prompts
// of up to 700 tokens with prefixes and slopes take 141 us for twice the pairs.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "device_common.cuh"
#include "rows.cuh"

namespace slm {

constexpr int kSimtThreads = 256;
constexpr int kSimtBlk = 64;  // positions per block

template <typename T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// 16 bytes of T at p, widened to floats at d.
__device__ __forceinline__ void widen16(const float *p, float *d) { *(float4 *)d = *(const float4 *)p; }
__device__ __forceinline__ void widen16(const __nv_bfloat16 *p, float *d) {
    const uint4 w = *(const uint4 *)p;
    *(float4 *)d = make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
    *(float4 *)(d + 4) = make_float4(bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w), bf16_hi(w.w));
}

// Row of position `pos` of sequence s, kv head g, in elements from the cache's base.  A page id
// outside the pool is read as page 0 (and reported), so that nothing outside it is touched.
__device__ __forceinline__ size_t rows_kv_offset(const RowsArgs &A, bool is_v, int s, int row0, int g, int pos) {
    if (!A.kv.table) return (size_t)(row0 + pos) * (size_t)(is_v ? A.kv.v_ld : A.kv.k_ld) + (size_t)g * A.hd;
    int page = __ldg(A.kv.table + (size_t)s * A.kv.table_ld + (pos >> A.kv.page_shift));
    if (page < 0 || page >= A.kv.n_pages) {
        atomicOr(A.status, SLM_ROWS_PAGE);
        page = 0;
    }
    const size_t row = ((((size_t)page * A.KV + g) << A.kv.page_shift)) + (pos & ((1 << A.kv.page_shift) - 1));
    return row * A.hd;
}

// Two key / value buffers for fp32 heads of up to 128: the next block is copied (cp.async) while
// this one is multiplied.  bf16 has to be widened on the way and 256-wide heads fill the shared
// memory, so those load a block when they need it.
template <typename T, int HDP> constexpr bool kSimtAsync = sizeof(T) == 4 && HDP <= 128;
template <int HDP> constexpr int simt_ld() { return HDP + 4; }
// Scores in the log2 domain from q . k log2(e) / sqrt(hd) (x, with a cap: q . k scale / cap) of the
// position d after the row's.
__device__ __forceinline__ float simt_score(float x, const RowsScores &sc, float sl, int d) {
    if (sc.cap_log2 > 0.f) x = sc.cap_log2 * tanhf(x);
    if (sc.slopes) x = fmaf(-sl, fabsf((float)d), x);
    return x;
}
// The factor of q.
template <bool SCORED> __device__ __forceinline__ float simt_scale(const RowsArgs &A) {
    return SCORED && A.sc.cap_log2 > 0.f ? A.sc.cap_in : A.scale_log2;
}

template <typename T, int HDP, int R> constexpr size_t simt_smem(int nseq) {
    return (size_t)(R + 2 * kSimtBlk * (kSimtAsync<T, HDP> ? 2 : 1)) * simt_ld<HDP>() * 4 + (size_t)R * (kSimtBlk + 4) * 4 +
           3 * R * 4 + (size_t)nseq * sizeof(SeqRows) + (size_t)(nseq + 1) * 8 + 16;
}

template <typename T, int HDP, int R, bool SCORED>
__global__ void __launch_bounds__(kSimtThreads) rows_simt_kernel(const __grid_constant__ RowsArgs A) {
    constexpr int LD = simt_ld<HDP>(), PLD = kSimtBlk + 4;
    constexpr int KQ = 64 / R;           // thread groups that share a block's keys
    constexpr int KS = 4 / KQ;           // keys per thread in Q K^T
    constexpr int C = HDP / 64;          // float4 columns per thread in P V
    constexpr int TPR = kSimtThreads / R, KPT = kSimtBlk / TPR;  // softmax: threads per row, keys per thread
    constexpr int E = 16 / sizeof(T);    // elements per 16 bytes
    extern __shared__ __align__(16) uint8_t smem[];
    long long *wstart = (long long *)smem;
    SeqRows *seq = (SeqRows *)(wstart + A.nseq + 1);
    float *qs = (float *)(((uintptr_t)(seq + A.nseq) + 15) & ~(uintptr_t)15);
    constexpr bool ASYNC = kSimtAsync<T, HDP>;
    float *kv = qs + R * LD, *ps = kv + (ASYNC ? 4 : 2) * kSimtBlk * LD;  // [buffer][keys, values][64][LD]
    float *alpha = ps + R * PLD, *mrow = alpha + R, *lrow = mrow + R;
    const int tid = threadIdx.x;
    const int tx = tid & 15, kq = (tid >> 4) % KQ, ty = (tid >> 4) / KQ;
    const T *Q = (const T *)A.q;

    pdl_wait();
    pdl_trigger();
    constexpr bool kSpans = SCORED;
    std::conditional_t<kSpans, RowsMaskedWalk, RowsWalk> w;
    if constexpr (kSpans) {
        RowsStart *start = (RowsStart *)(((uintptr_t)(lrow + R) + 15) & ~(uintptr_t)15);
        masked_layout(A, seq, wstart, start, (int *)kv, w, tid, kSimtThreads);
        const long long unit = range_units(wstart[A.nseq], A.P);
        w.begin(seq, wstart[A.nseq], A.nseq, A.geom, unit * blockIdx.x, unit * (blockIdx.x + 1), *start);
    } else {
        rows_layout(A, seq, wstart, tid, kSimtThreads);
        const long long unit = range_units(wstart[A.nseq], A.P);
        w.begin(seq, wstart, A.nseq, A.geom, unit * blockIdx.x, unit * (blockIdx.x + 1));
    }
    const long long unit = range_units(wstart[A.nseq], A.P);
    RowsPiece p;
    bool joined = false;
    while (w.next(seq, A.nseq, A.geom, p)) {
        const SeqRows sr = seq[p.s];
        const int tok0 = p.t * A.geom.PT, ntok = min(A.geom.PT, sr.n - tok0), nr = ntok * A.G;
        int L = sr.ctx + tok0 + ntok, from = 0;  // the item sees positions [from, L)
        if constexpr (kSpans) {
            from = row_from(w.mask(p.s), sr.ctx, tok0);
            L = max(L, w.mask.prefix(p.s));
        }
        __syncthreads();  // the last piece is done with every buffer
        // queries, times log2(e) / sqrt(hd)
        for (int e = tid; e < R * (HDP / E); e += kSimtThreads) {
            const int r = e / (HDP / E), d = (e - r * (HDP / E)) * E;
            float x[E];
            if (r < nr && d < A.hd) {
                const int tok = r / A.G, h = p.g * A.G + (r - tok * A.G);
                widen16(Q + (size_t)(sr.row0 + tok0 + tok) * A.q_ld + (size_t)h * A.hd + d, x);
            } else {
#pragma unroll
                for (int i = 0; i < E; i++) x[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < E; i++) qs[r * LD + d + i] = x[i] * simt_scale<SCORED>(A);
        }
        if (tid < R) {
            mrow[tid] = -INFINITY;
            lrow[tid] = 0.f;
        }
        float4 o[4][C];
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int c = 0; c < C; c++) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
        const bool some = 4 * ty < nr;  // this thread's rows exist (else it only loads and keeps step)

        // keys and values of block kb into buffer b; rows that no row of the item sees are zero
        auto load = [&](int kb, int b) {
            float *ks = kv + (size_t)b * 2 * kSimtBlk * LD, *vs = ks + kSimtBlk * LD;
            const int k0 = kb * kSimtBlk;
            for (int e = tid; e < kSimtBlk * (HDP / E); e += kSimtThreads) {
                const int j = e / (HDP / E), d = (e - j * (HDP / E)) * E;
                float *kd = ks + j * LD + d, *vd = vs + j * LD + d;
                if (k0 + j < L && (!kSpans || k0 + j >= from) && d < A.hd) {
                    const T *k = (const T *)A.kv.k + rows_kv_offset(A, false, p.s, sr.row0, p.g, k0 + j) + d;
                    const T *v = (const T *)A.kv.v + rows_kv_offset(A, true, p.s, sr.row0, p.g, k0 + j) + d;
                    if (ASYNC) {
                        cp_async16(kd, k);
                        cp_async16(vd, v);
                    } else {
                        widen16(k, kd);
                        widen16(v, vd);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < E; i++) kd[i] = vd[i] = 0.f;
                }
            }
            if (ASYNC) cp_async_commit();
        };
        if (ASYNC && (!kSpans || p.kb1 > p.kb0)) load(p.kb0, 0);

        for (int kb = p.kb0; kb < p.kb1; kb++) {
            const int k0 = kb * kSimtBlk, buf = ASYNC ? (kb - p.kb0) & 1 : 0;
            float *ks = kv + (size_t)buf * 2 * kSimtBlk * LD, *vs = ks + kSimtBlk * LD;
            if (!ASYNC) {
                load(kb, 0);
            } else if (kb + 1 < p.kb1) {
                load(kb + 1, buf ^ 1);  // its last readers are behind the barrier that ended block kb - 1
                cp_async_wait_upto(1);
            } else {
                cp_async_wait_upto(0);
            }
            __syncthreads();
            // S: rows 4 ty + i, keys kq * 16 + tx (+ 16 j)
            if (some) {
                float s[4][KS];
#pragma unroll
                for (int i = 0; i < 4; i++)
#pragma unroll
                    for (int j = 0; j < KS; j++) s[i][j] = 0.f;
#pragma unroll 4
                for (int d = 0; d < HDP; d += 4) {
                    float4 a[4], b[KS];
#pragma unroll
                    for (int i = 0; i < 4; i++) a[i] = *(const float4 *)(qs + (4 * ty + i) * LD + d);
#pragma unroll
                    for (int j = 0; j < KS; j++) b[j] = *(const float4 *)(ks + (kq * 16 * KS + tx + 16 * j) * LD + d);
#pragma unroll
                    for (int i = 0; i < 4; i++)
#pragma unroll
                        for (int j = 0; j < KS; j++) {
                            s[i][j] = fmaf(a[i].x, b[j].x, s[i][j]);
                            s[i][j] = fmaf(a[i].y, b[j].y, s[i][j]);
                            s[i][j] = fmaf(a[i].z, b[j].z, s[i][j]);
                            s[i][j] = fmaf(a[i].w, b[j].w, s[i][j]);
                        }
                }
#pragma unroll
                for (int i = 0; i < 4; i++)
#pragma unroll
                    for (int j = 0; j < KS; j++) ps[(4 * ty + i) * PLD + kq * 16 * KS + tx + 16 * j] = s[i][j];
            }
            __syncthreads();
            // the row's new maximum, weights and sum
            {
                const int r = tid / TPR, c = tid % TPR;
                const int tok = r / A.G;
                const int pos = sr.ctx + tok0 + tok;
                int lim = pos + 1 - k0, low = 0;  // keys [low, lim) of the block are those that the row sees
                float sl = 0.f;
                if constexpr (kSpans) {
                    int lo = 0, hi = 0;
                    if (r < nr) row_span(A, w.mask(p.s), sr, tok0 + tok, false, lo, hi);
                    low = lo - k0;
                    lim = hi - k0;
                    if (A.sc.slopes && r < nr) sl = 1.4426950408889634f * __ldg(A.sc.slopes + p.g * A.G + (r - tok * A.G));
                }
                float x[KPT], mx = mrow[r];
#pragma unroll
                for (int j = 0; j < KPT; j++) {
                    const int k = c + j * TPR;
                    x[j] = k < lim && k >= low ? simt_score(ps[r * PLD + k], A.sc, sl, k0 + k - pos) : -INFINITY;
                    mx = fmaxf(mx, x[j]);
                }
#pragma unroll
                for (int off = TPR / 2; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                const float m0 = mx == -INFINITY ? 0.f : mx;  // nothing seen yet: every weight is 2^-inf = 0
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < KPT; j++) {
                    x[j] = exp2f(x[j] - m0);
                    sum += x[j];
                    ps[r * PLD + c + j * TPR] = x[j];
                }
#pragma unroll
                for (int off = TPR / 2; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                __syncwarp();
                if (c == 0) {
                    const float f = exp2f(mrow[r] - m0);
                    alpha[r] = f;
                    lrow[r] = lrow[r] * f + sum;
                    mrow[r] = mx;
                }
            }
            __syncthreads();
            // O = alpha O + P V: rows 4 ty + i, columns 4 tx + 64 c, keys of group kq
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; i++) f[i] = alpha[4 * ty + i];
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int c = 0; c < C; c++) {
                    o[i][c].x *= f[i];
                    o[i][c].y *= f[i];
                    o[i][c].z *= f[i];
                    o[i][c].w *= f[i];
                }
            const int jend = some ? (kq + 1) * (kSimtBlk / KQ) : 0;
#pragma unroll 2
            for (int j = kq * (kSimtBlk / KQ); j < jend; j += 4) {
                float4 pv[4];
#pragma unroll
                for (int i = 0; i < 4; i++) pv[i] = *(const float4 *)(ps + (4 * ty + i) * PLD + j);
#pragma unroll
                for (int jj = 0; jj < 4; jj++)
#pragma unroll
                    for (int c = 0; c < C; c++) {
                        const float4 v = *(const float4 *)(vs + (j + jj) * LD + 4 * tx + 64 * c);
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const float a = jj == 0 ? pv[i].x : jj == 1 ? pv[i].y : jj == 2 ? pv[i].z : pv[i].w;
                            o[i][c].x = fmaf(a, v.x, o[i][c].x);
                            o[i][c].y = fmaf(a, v.y, o[i][c].y);
                            o[i][c].z = fmaf(a, v.z, o[i][c].z);
                            o[i][c].w = fmaf(a, v.w, o[i][c].w);
                        }
                    }
            }
            __syncthreads();  // keys, values and weights are free again
        }
        // the key groups' sums of O (over the first key buffer: KQ R rows are exactly its length)
        float *ks = kv;
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int c = 0; c < C; c++)
                *(float4 *)(ks + ((size_t)kq * R + 4 * ty + i) * LD + 4 * tx + 64 * c) = o[i][c];
        __syncthreads();
        if (kq == 0) {
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int c = 0; c < C; c++) {
                    float4 a = o[i][c];
#pragma unroll
                    for (int q = 1; q < KQ; q++) {
                        const float4 b = *(const float4 *)(ks + ((size_t)q * R + 4 * ty + i) * LD + 4 * tx + 64 * c);
                        a.x += b.x;
                        a.y += b.y;
                        a.z += b.z;
                        a.w += b.w;
                    }
                    o[i][c] = a;
                }
        }
        const bool whole = p.begins() && p.ends();
        if (!whole && p.begins()) {
            joined = true;
            if (tid == 0) write_join(A, blockIdx.x, seq, unit, &p);
        }
        if (whole) {
            if (kq == 0)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int r = 4 * ty + i;
                    if (r >= nr) continue;
                    const int tok = r / A.G, h = p.g * A.G + (r - tok * A.G);
                    float inv = 1.0f / lrow[r];
                    if constexpr (kSpans) {
                        int lo, hi;
                        row_span(A, w.mask(p.s), sr, tok0 + tok, p.g == 0 && h == 0 && tx == 0, lo, hi);
                        if (lo >= hi) {  // nothing seen: zeros
                            inv = 0.f;
#pragma unroll
                            for (int c = 0; c < C; c++) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
                        }
                    }
                    T *dst = (T *)A.out + (size_t)(sr.row0 + tok0 + tok) * A.out_ld + (size_t)h * A.hd;
#pragma unroll
                    for (int c = 0; c < C; c++) {
                        const int d = 4 * tx + 64 * c;
                        if (d < A.hd) {
                            dst[d] = from_float<T>(o[i][c].x * inv);
                            dst[d + 1] = from_float<T>(o[i][c].y * inv);
                            dst[d + 2] = from_float<T>(o[i][c].z * inv);
                            dst[d + 3] = from_float<T>(o[i][c].w * inv);
                        }
                    }
                }
        } else {
            float *part = slot_ptr(A, piece_slot(blockIdx.x, p));
            float *pm = part + (size_t)A.slot_rows * A.hd;
            if (kq == 0)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int r = 4 * ty + i;
                    if (r >= nr) continue;
#pragma unroll
                    for (int c = 0; c < C; c++) {
                        const int d = 4 * tx + 64 * c;
                        if (d < A.hd) *(float4 *)(part + ((size_t)(d / 4) * A.slot_rows + r) * 4) = o[i][c];
                    }
                }
            if (tid < nr) {
                bool sees = sr.ctx + tok0 + tid / A.G + 1 > p.kb0 * kSimtBlk;
                if constexpr (kSpans) {
                    int lo, hi;
                    row_span(A, w.mask(p.s), sr, tok0 + tid / A.G, p.g == 0 && tid % A.G == 0 && p.begins(), lo, hi);
                    sees = max(lo, p.kb0 * kSimtBlk) < min(hi, p.kb1 * kSimtBlk);
                }
                pm[tid] = piece_max(mrow[tid], sees);
                pm[A.slot_rows + tid] = lrow[tid];
            }
        }
    }
    if (!joined && tid == 0) write_join(A, blockIdx.x, seq, unit, nullptr);
}

// ---- 64-row tiles (fp32 heads of up to 128): the same walk with every row inside one warp
//
// A warp owns 8 rows: thread (ty, tx) has rows 4 ty + i and keys tx + 16 j of S and columns 4 tx of
// O, so the softmax of a row stays within 16 lanes (its maximum by shuffles, its sum as 16 partial
// sums until the end) and the weights go through the warp's own piece of shared memory.  One block
// barrier per 64 positions is left, for the key / value buffers, so a warp's softmax runs beside the
// other warps' multiplications.
template <int HDP, bool SCORED>
__global__ void __launch_bounds__(kSimtThreads, HDP == 64 ? 2 : 1) rows_fma_kernel(const __grid_constant__ RowsArgs A) {
    constexpr int R = 64, LD = simt_ld<HDP>(), PLD = kSimtBlk + 4, C = HDP / 64;
    extern __shared__ __align__(16) uint8_t smem[];
    long long *wstart = (long long *)smem;
    SeqRows *seq = (SeqRows *)(wstart + A.nseq + 1);
    float *qs = (float *)(((uintptr_t)(seq + A.nseq) + 15) & ~(uintptr_t)15);
    float *kv = qs + R * LD, *ps = kv + 4 * kSimtBlk * LD;  // [2 buffers][keys, values][64][LD]
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const float *Q = (const float *)A.q, *K = (const float *)A.kv.k, *V = (const float *)A.kv.v;

    pdl_wait();
    pdl_trigger();
    constexpr bool kSpans = SCORED;
    std::conditional_t<kSpans, RowsMaskedWalk, RowsWalk> w;
    if constexpr (kSpans) {
        RowsStart *start = (RowsStart *)(((uintptr_t)(ps + R * PLD) + 15) & ~(uintptr_t)15);
        masked_layout(A, seq, wstart, start, (int *)kv, w, tid, kSimtThreads);
        const long long unit = range_units(wstart[A.nseq], A.P);
        w.begin(seq, wstart[A.nseq], A.nseq, A.geom, unit * blockIdx.x, unit * (blockIdx.x + 1), *start);
    } else {
        rows_layout(A, seq, wstart, tid, kSimtThreads);
        const long long unit = range_units(wstart[A.nseq], A.P);
        w.begin(seq, wstart, A.nseq, A.geom, unit * blockIdx.x, unit * (blockIdx.x + 1));
    }
    const long long unit = range_units(wstart[A.nseq], A.P);
    RowsPiece p;
    bool joined = false;
    while (w.next(seq, A.nseq, A.geom, p)) {
        const SeqRows sr = seq[p.s];
        const int tok0 = p.t * A.geom.PT, ntok = min(A.geom.PT, sr.n - tok0), nr = ntok * A.G;
        int L = sr.ctx + tok0 + ntok, from = 0;  // the item sees positions [from, L)
        if constexpr (kSpans) {
            from = row_from(w.mask(p.s), sr.ctx, tok0);
            L = max(L, w.mask.prefix(p.s));
        }
        __syncthreads();  // the last piece is done with every buffer
        // keys and values of block kb into buffer b; rows that no row of the item sees are zero
        auto load = [&](int kb, int b) {
            float *ks = kv + (size_t)b * 2 * kSimtBlk * LD, *vs = ks + kSimtBlk * LD;
            const int k0 = kb * kSimtBlk;
#pragma unroll 4
            for (int e = tid; e < kSimtBlk * (HDP / 4); e += kSimtThreads) {
                const int j = e / (HDP / 4), d = (e - j * (HDP / 4)) * 4;
                float *kd = ks + j * LD + d, *vd = vs + j * LD + d;
                if (k0 + j < L && (!kSpans || k0 + j >= from) && d < A.hd) {
                    const size_t at = rows_kv_offset(A, false, p.s, sr.row0, p.g, k0 + j) + d;
                    cp_async16(kd, K + at);
                    cp_async16(vd, V + (A.kv.table ? at : rows_kv_offset(A, true, p.s, sr.row0, p.g, k0 + j) + d));
                } else {
                    *(float4 *)kd = *(float4 *)vd = make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
            cp_async_commit();
        };
        if (!kSpans || p.kb1 > p.kb0) load(p.kb0, 0);
        // queries, times log2(e) / sqrt(hd)
        for (int e = tid; e < R * (HDP / 4); e += kSimtThreads) {
            const int r = e / (HDP / 4), d = (e - r * (HDP / 4)) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < nr && d < A.hd) {
                const int tok = r / A.G, h = p.g * A.G + (r - tok * A.G);
                x = *(const float4 *)(Q + (size_t)(sr.row0 + tok0 + tok) * A.q_ld + (size_t)h * A.hd + d);
            }
            const float f = simt_scale<SCORED>(A);
            *(float4 *)(qs + r * LD + d) = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
        }
        float4 o[4][C];
        float m[4], l[4];
        int low[4], seen[4];  // the rows see positions [low, seen)
        float sl[4];          // the heads' slopes, times log2(e)
#pragma unroll
        for (int i = 0; i < 4; i++) {
            m[i] = -INFINITY;
            l[i] = 0.f;
            const int r = 4 * ty + i, tok = r / A.G;
            low[i] = 0;
            sl[i] = 0.f;
            seen[i] = sr.ctx + tok0 + tok + 1;
            if constexpr (kSpans) {
                if (r < nr) {
                    row_span(A, w.mask(p.s), sr, tok0 + tok, p.g == 0 && r == tok * A.G && tx == 0 && p.begins(), low[i], seen[i]);
                    if (A.sc.slopes) sl[i] = 1.4426950408889634f * __ldg(A.sc.slopes + p.g * A.G + (r - tok * A.G));
                }
            }
#pragma unroll
            for (int c = 0; c < C; c++) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const bool some = 8 * (ty >> 1) < nr;  // the warp has rows (else it only loads and keeps step)

        for (int kb = p.kb0; kb < p.kb1; kb++) {
            const int k0 = kb * kSimtBlk, buf = (kb - p.kb0) & 1;
            const float *ks = kv + (size_t)buf * 2 * kSimtBlk * LD, *vs = ks + kSimtBlk * LD;
            cp_async_wait_upto(0);
            __syncthreads();  // block kb has landed, and everyone is done with block kb - 1
            if (kb + 1 < p.kb1) load(kb + 1, buf ^ 1);
            if (!some) continue;
            float s[4][4];
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) s[i][j] = 0.f;
#pragma unroll 4
            for (int d = 0; d < HDP; d += 4) {
                float4 a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; i++) a[i] = *(const float4 *)(qs + (4 * ty + i) * LD + d);
#pragma unroll
                for (int j = 0; j < 4; j++) b[j] = *(const float4 *)(ks + (tx + 16 * j) * LD + d);
#pragma unroll
                for (int i = 0; i < 4; i++)
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        s[i][j] = fmaf(a[i].x, b[j].x, s[i][j]);
                        s[i][j] = fmaf(a[i].y, b[j].y, s[i][j]);
                        s[i][j] = fmaf(a[i].z, b[j].z, s[i][j]);
                        s[i][j] = fmaf(a[i].w, b[j].w, s[i][j]);
                    }
            }
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int lim = seen[i] - k0, lowest = low[i] - k0;  // keys of the block that the row sees
                float mx = m[i];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    if constexpr (SCORED)
                        s[i][j] = simt_score(s[i][j], A.sc, sl[i], k0 + tx + 16 * j - (sr.ctx + tok0 + (4 * ty + i) / A.G));
                    if (tx + 16 * j >= lim || (kSpans && tx + 16 * j < lowest)) s[i][j] = -INFINITY;
                    mx = fmaxf(mx, s[i][j]);
                }
#pragma unroll
                for (int off = 8; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                const float m0 = mx == -INFINITY ? 0.f : mx;  // nothing seen yet: every weight is 2^-inf = 0
                f[i] = exp2f(m[i] - m0);
                m[i] = mx;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const float x = exp2f(s[i][j] - m0);
                    sum += x;
                    ps[(4 * ty + i) * PLD + tx + 16 * j] = x;
                }
                l[i] = l[i] * f[i] + sum;
#pragma unroll
                for (int c = 0; c < C; c++) {
                    o[i][c].x *= f[i];
                    o[i][c].y *= f[i];
                    o[i][c].z *= f[i];
                    o[i][c].w *= f[i];
                }
            }
            __syncwarp();
#pragma unroll 2
            for (int j = 0; j < kSimtBlk; j += 4) {
                float4 pv[4];
#pragma unroll
                for (int i = 0; i < 4; i++) pv[i] = *(const float4 *)(ps + (4 * ty + i) * PLD + j);
#pragma unroll
                for (int jj = 0; jj < 4; jj++)
#pragma unroll
                    for (int c = 0; c < C; c++) {
                        const float4 v = *(const float4 *)(vs + (j + jj) * LD + 4 * tx + 64 * c);
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const float a = jj == 0 ? pv[i].x : jj == 1 ? pv[i].y : jj == 2 ? pv[i].z : pv[i].w;
                            o[i][c].x = fmaf(a, v.x, o[i][c].x);
                            o[i][c].y = fmaf(a, v.y, o[i][c].y);
                            o[i][c].z = fmaf(a, v.z, o[i][c].z);
                            o[i][c].w = fmaf(a, v.w, o[i][c].w);
                        }
                    }
            }
            __syncwarp();  // the weights have been read
        }
        const bool whole = p.begins() && p.ends();
        if (!whole && p.begins()) {
            joined = true;
            if (tid == 0) write_join(A, blockIdx.x, seq, unit, &p);
        }
        float *part = slot_ptr(A, piece_slot(blockIdx.x, p));
#pragma unroll
        for (int i = 0; i < 4; i++) {
#pragma unroll
            for (int off = 8; off; off >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
            const int r = 4 * ty + i;
            if (r >= nr) continue;
            if (whole) {
                const int tok = r / A.G, h = p.g * A.G + (r - tok * A.G);
                const bool blind = kSpans && low[i] >= seen[i];  // nothing seen: zeros
                const float inv = blind ? 0.f : 1.0f / l[i];
                if (blind) {
#pragma unroll
                    for (int c = 0; c < C; c++) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
                float *dst = (float *)A.out + (size_t)(sr.row0 + tok0 + tok) * A.out_ld + (size_t)h * A.hd;
#pragma unroll
                for (int c = 0; c < C; c++)
                    if (4 * tx + 64 * c < A.hd)
                        *(float4 *)(dst + 4 * tx + 64 * c) =
                            make_float4(o[i][c].x * inv, o[i][c].y * inv, o[i][c].z * inv, o[i][c].w * inv);
            } else {
#pragma unroll
                for (int c = 0; c < C; c++)
                    if (4 * tx + 64 * c < A.hd) *(float4 *)(part + ((size_t)(tx + 16 * c) * A.slot_rows + r) * 4) = o[i][c];
                if (tx == 0) {
                    part[(size_t)A.slot_rows * A.hd + r] = piece_max(m[i], max(low[i], p.kb0 * kSimtBlk) < min(seen[i], p.kb1 * kSimtBlk));
                    part[(size_t)A.slot_rows * (A.hd + 1) + r] = l[i];
                }
            }
        }
    }
    if (!joined && tid == 0) write_join(A, blockIdx.x, seq, unit, nullptr);
}

// ---- launch

template <int HDP, bool SCORED> static cudaError_t launch_fma(const RowsArgs &a, cudaStream_t s) {
    const size_t smem = simt_smem<float, HDP, 64>(a.nseq) + (SCORED ? masked_bytes() : 0);
    const cudaError_t e = allow_smem((const void *)rows_fma_kernel<HDP, SCORED>);
    if (e != cudaSuccess) return e;
    return launch_pdl(rows_fma_kernel<HDP, SCORED>, dim3(a.P), dim3(kSimtThreads), smem, s, a);
}

template <typename T, int HDP, int R, bool SCORED> static cudaError_t launch_simt(const RowsArgs &a, cudaStream_t s) {
    const size_t smem = simt_smem<T, HDP, R>(a.nseq) + (SCORED ? masked_bytes() : 0);
    const cudaError_t e = allow_smem((const void *)rows_simt_kernel<T, HDP, R, SCORED>);
    if (e != cudaSuccess) return e;
    return launch_pdl(rows_simt_kernel<T, HDP, R, SCORED>, dim3(a.P), dim3(kSimtThreads), smem, s, a);
}

template <bool SCORED> static cudaError_t launch_cuda_cores(const RowsArgs &a, bool bf16, cudaStream_t s) {
    const bool small = a.geom.PT * a.G <= kSimtSmallTile;
    if (bf16) return small ? launch_simt<__nv_bfloat16, 256, 16, SCORED>(a, s) : launch_simt<__nv_bfloat16, 256, 32, SCORED>(a, s);
    if (a.hd <= 64) return small ? launch_simt<float, 64, 16, SCORED>(a, s) : launch_fma<64, SCORED>(a, s);
    if (a.hd <= 128) return small ? launch_simt<float, 128, 16, SCORED>(a, s) : launch_fma<128, SCORED>(a, s);
    return small ? launch_simt<float, 256, 16, SCORED>(a, s) : launch_simt<float, 256, 32, SCORED>(a, s);
}

}  // namespace slm
