// rows_attention.cu -- attention of packed rows on the CUDA cores (fp32, and bf16 heads wider
// than 128), and the kernel that joins the pieces of items that several CTAs share.
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
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

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
template <typename T, int HDP, int R> constexpr size_t simt_smem(int nseq) {
    return (size_t)(R + 2 * kSimtBlk * (kSimtAsync<T, HDP> ? 2 : 1)) * simt_ld<HDP>() * 4 + (size_t)R * (kSimtBlk + 4) * 4 +
           3 * R * 4 + (size_t)nseq * sizeof(SeqRows) + (size_t)(nseq + 1) * 8 + 16;
}

template <typename T, int HDP, int R>
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
    rows_layout(A, seq, wstart, tid, kSimtThreads);
    const long long unit = range_units(wstart[A.nseq], A.P);
    RowsWalk w;
    w.begin(seq, wstart, A.nseq, A.geom, unit * blockIdx.x, unit * (blockIdx.x + 1));
    RowsPiece p;
    bool joined = false;
    while (w.next(seq, A.nseq, A.geom, p)) {
        const SeqRows sr = seq[p.s];
        const int tok0 = p.t * A.geom.PT, ntok = min(A.geom.PT, sr.n - tok0), nr = ntok * A.G;
        const int L = sr.ctx + tok0 + ntok;  // positions the item sees
        __syncthreads();                     // the last piece is done with every buffer
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
            for (int i = 0; i < E; i++) qs[r * LD + d + i] = x[i] * A.scale_log2;
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
                if (k0 + j < L && d < A.hd) {
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
        if (ASYNC) load(p.kb0, 0);

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
                const int lim = sr.ctx + tok0 + tok + 1 - k0;  // keys of the block that the row sees
                float x[KPT], mx = mrow[r];
#pragma unroll
                for (int j = 0; j < KPT; j++) {
                    x[j] = c + j * TPR < lim ? ps[r * PLD + c + j * TPR] : -INFINITY;
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
        const bool whole = p.kb0 == 0 && p.kb1 == p.nb;
        if (!whole && p.kb0 == 0) {
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
                    const float inv = 1.0f / lrow[r];
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
                pm[tid] = piece_max(mrow[tid], sr.ctx + tok0 + tid / A.G + 1 > p.kb0 * kSimtBlk);
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
template <int HDP>
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
    rows_layout(A, seq, wstart, tid, kSimtThreads);
    const long long unit = range_units(wstart[A.nseq], A.P);
    RowsWalk w;
    w.begin(seq, wstart, A.nseq, A.geom, unit * blockIdx.x, unit * (blockIdx.x + 1));
    RowsPiece p;
    bool joined = false;
    while (w.next(seq, A.nseq, A.geom, p)) {
        const SeqRows sr = seq[p.s];
        const int tok0 = p.t * A.geom.PT, ntok = min(A.geom.PT, sr.n - tok0), nr = ntok * A.G;
        const int L = sr.ctx + tok0 + ntok;  // positions the item sees
        __syncthreads();                     // the last piece is done with every buffer
        // keys and values of block kb into buffer b; rows that no row of the item sees are zero
        auto load = [&](int kb, int b) {
            float *ks = kv + (size_t)b * 2 * kSimtBlk * LD, *vs = ks + kSimtBlk * LD;
            const int k0 = kb * kSimtBlk;
#pragma unroll 4
            for (int e = tid; e < kSimtBlk * (HDP / 4); e += kSimtThreads) {
                const int j = e / (HDP / 4), d = (e - j * (HDP / 4)) * 4;
                float *kd = ks + j * LD + d, *vd = vs + j * LD + d;
                if (k0 + j < L && d < A.hd) {
                    const size_t at = rows_kv_offset(A, false, p.s, sr.row0, p.g, k0 + j) + d;
                    cp_async16(kd, K + at);
                    cp_async16(vd, V + (A.kv.table ? at : rows_kv_offset(A, true, p.s, sr.row0, p.g, k0 + j) + d));
                } else {
                    *(float4 *)kd = *(float4 *)vd = make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
            cp_async_commit();
        };
        load(p.kb0, 0);
        // queries, times log2(e) / sqrt(hd)
        for (int e = tid; e < R * (HDP / 4); e += kSimtThreads) {
            const int r = e / (HDP / 4), d = (e - r * (HDP / 4)) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < nr && d < A.hd) {
                const int tok = r / A.G, h = p.g * A.G + (r - tok * A.G);
                x = *(const float4 *)(Q + (size_t)(sr.row0 + tok0 + tok) * A.q_ld + (size_t)h * A.hd + d);
            }
            *(float4 *)(qs + r * LD + d) = make_float4(x.x * A.scale_log2, x.y * A.scale_log2, x.z * A.scale_log2, x.w * A.scale_log2);
        }
        float4 o[4][C];
        float m[4], l[4];
        int seen[4];  // positions that the rows see
#pragma unroll
        for (int i = 0; i < 4; i++) {
            m[i] = -INFINITY;
            l[i] = 0.f;
            seen[i] = sr.ctx + tok0 + (4 * ty + i) / A.G + 1;
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
                const int lim = seen[i] - k0;  // keys of the block that the row sees
                float mx = m[i];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    if (tx + 16 * j >= lim) s[i][j] = -INFINITY;
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
        const bool whole = p.kb0 == 0 && p.kb1 == p.nb;
        if (!whole && p.kb0 == 0) {
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
                const float inv = 1.0f / l[i];
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
                    part[(size_t)A.slot_rows * A.hd + r] = piece_max(m[i], seen[i] > p.kb0 * kSimtBlk);
                    part[(size_t)A.slot_rows * (A.hd + 1) + r] = l[i];
                }
            }
        }
    }
    if (!joined && tid == 0) write_join(A, blockIdx.x, seq, unit, nullptr);
}

// ---- joining
//
// Piece i of an item has, per row, the maximum m_i, the sum l_i and the unnormalised O_i:
//     out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i,  M = max_i m_i.
// m_i = -inf stands for a row that sees none of the piece's positions, and for nothing else: only
// such a piece is left out (its O may not have been written); one whose scores are all NaN, or all
// -inf, takes part with m_i = -FLT_MAX, so that what it holds reaches the result as in one pass.
// Block x looks after the item that attention CTA x starts and another one finishes (RowsJoin);
// its pieces are slot 2x + 1 and the slots 2c of the CTAs behind x.  A slot holds O as
// [head_dim / 4][row] quads, so that the attention kernels' row-per-thread epilogue and the reads
// here are contiguous over the rows; a warp takes 32 rows and every eighth quad, and the results
// go out through shared memory as whole rows.  Pieces are added in order, so the result does not
// depend on timing.  With kJoinShared pieces or more (a long context over the whole GPU, few rows)
// the eight warps of a block share the pieces of 32 quads instead and add up in shared memory.
// Two or three dependent reads of L2 long: 2 to 3 us more for a short call (its launch overlaps the
// attention's); alone under the profiler, caches cold, 6 to 10 us, and 16 where 150 items of 250 rows
// of 128 are joined.
constexpr int kJoinShared = 12;

template <typename T> __device__ __forceinline__ void store4(T *p, float4 v);
template <> __device__ __forceinline__ void store4<float>(float *p, float4 v) { *(float4 *)p = v; }
template <> __device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16 *p, float4 v) {
    *(uint2 *)p = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

__device__ __forceinline__ void add4(float4 &a, float f, const float4 &b) {
    a.x = fmaf(f, b.x, a.x);
    a.y = fmaf(f, b.y, a.y);
    a.z = fmaf(f, b.z, a.z);
    a.w = fmaf(f, b.w, a.w);
}

template <typename T, int Q>  // Q: quads per thread, head_dim at most 32 Q
__global__ void __launch_bounds__(256) rows_join_kernel(const __grid_constant__ RowsArgs A) {
    constexpr int kRows = 32 * (32 * Q * (int)sizeof(T) + 16), kSums = 256 * 24;
    __shared__ __align__(16) uint8_t buf[kRows > kSums ? kRows : kSums];
    pdl_wait();
    pdl_trigger();
    const RowsJoin J = ((const RowsJoin *)A.ws)[blockIdx.x];
    if (J.pieces == 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = J.pieces, nr = J.tokens * A.G, cols = A.hd / 4, c0 = blockIdx.x, R = A.slot_rows;
    const size_t sf = slot_floats(R, A.hd);
    const float *slots = (const float *)(A.ws + join_bytes(A.P));
    const float *stats = slots + (size_t)R * A.hd;  // maxima, then sums, of slot 0
    auto slot = [&](int i) { return (size_t)(i == 0 ? 2 * c0 + 1 : 2 * (c0 + i)) * sf; };
    auto dest = [&](int r) {
        const int tok = r / A.G;
        return (T *)A.out + (size_t)(J.row0 + tok) * A.out_ld + (size_t)(J.head0 + r - tok * A.G) * A.hd;
    };
    if (n < kJoinShared) {
        // quads q, q + 8, ... of row r: the maximum first, then every piece's share
        auto row = [&](int r, int q0, auto &acc) {
            constexpr int N = sizeof(acc) / sizeof(float4), AT = N == 1 ? 4 : 2;  // pieces in flight
            float M = -INFINITY, l = 0.f;
            for (int i0 = 0; i0 < n; i0 += 4) {
                float mi[4];
#pragma unroll
                for (int a = 0; a < 4; a++) mi[a] = i0 + a < n ? stats[slot(i0 + a) + r] : -INFINITY;
                M = fmaxf(M, fmaxf(fmaxf(mi[0], mi[1]), fmaxf(mi[2], mi[3])));
            }
#pragma unroll
            for (int k = 0; k < N; k++) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i0 = 0; i0 < n; i0 += AT) {
                float mi[AT], li[AT];
                float4 v[AT][N];
#pragma unroll
                for (int a = 0; a < AT; a++) {
                    const float *s = slots + slot(min(i0 + a, n - 1));
                    mi[a] = i0 + a < n ? s[(size_t)R * A.hd + r] : -INFINITY;
                    li[a] = s[(size_t)R * (A.hd + 1) + r];
#pragma unroll
                    for (int k = 0; k < N; k++)
                        v[a][k] = *(const float4 *)(s + ((size_t)min(q0 + 8 * k, cols - 1) * R + r) * 4);
                }
#pragma unroll
                for (int a = 0; a < AT; a++) {
                    if (mi[a] == -INFINITY) continue;  // no piece, or the row sees none of it
                    const float f = exp2f(mi[a] - M);
                    l = fmaf(f, li[a], l);
#pragma unroll
                    for (int k = 0; k < N; k++) add4(acc[k], f, v[a][k]);
                }
            }
            const float inv = 1.0f / l;
#pragma unroll
            for (int k = 0; k < N; k++) acc[k] = make_float4(acc[k].x * inv, acc[k].y * inv, acc[k].z * inv, acc[k].w * inv);
        };
        if (nr < 32) {  // a decode step: a quad a thread, the rows side by side
            for (int e = blockIdx.y * 256 + threadIdx.x; e < nr * cols; e += gridDim.y * 256) {
                const int q = e / nr, r = e - q * nr;
                float4 one[1];
                row(r, q, one);
                store4<T>(dest(r) + 4 * q, one[0]);
            }
            return;
        }
        float4 acc[Q];
        const int pitch = A.hd * (int)sizeof(T) + 16, chunks = A.hd * (int)sizeof(T) / 16;
        for (int r0 = blockIdx.y * 32; r0 < nr; r0 += gridDim.y * 32) {
            row(min(r0 + lane, nr - 1), warp, acc);
#pragma unroll
            for (int k = 0; k < Q; k++)
                if (warp + 8 * k < cols) store4<T>((T *)(buf + lane * pitch) + 4 * (warp + 8 * k), acc[k]);
            __syncthreads();
            const int rows = min(32, nr - r0);
            for (int e = threadIdx.x; e < rows * chunks; e += 256) {
                const int rr = e / chunks, x = e - rr * chunks;
                *(uint4 *)((uint8_t *)dest(r0 + rr) + x * 16) = *(const uint4 *)(buf + rr * pitch + x * 16);
            }
            __syncthreads();
        }
        return;
    }
    float4 *ro = (float4 *)buf;                     // [8][32] sums of O
    float *rm = (float *)(ro + 256), *rl = rm + 256;  // [8][32] maxima and sums
    for (int e0 = blockIdx.y * 32; e0 < nr * cols; e0 += gridDim.y * 32) {
        const int e = min(e0 + lane, nr * cols - 1), q = e / nr, r = e - q * nr;
        float M = -INFINITY, l = 0.f;
        for (int i = warp; i < n; i += 8) M = fmaxf(M, stats[slot(i) + r]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = warp; i < n; i += 8) {
            const float mi = stats[slot(i) + r];
            if (mi == -INFINITY) continue;  // the row sees none of this piece
            const float f = exp2f(mi - M);
            l = fmaf(f, stats[slot(i) + R + r], l);
            add4(acc, f, *(const float4 *)(slots + slot(i) + ((size_t)q * R + r) * 4));
        }
        ro[warp * 32 + lane] = acc;
        rm[warp * 32 + lane] = M;
        rl[warp * 32 + lane] = l;
        __syncthreads();
        if (warp == 0) {
            M = -INFINITY;
            for (int w = 0; w < 8; w++) M = fmaxf(M, rm[w * 32 + lane]);
            l = 0.f;
            acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = 0; w < 8; w++) {
                if (rm[w * 32 + lane] == -INFINITY) continue;
                const float f = exp2f(rm[w * 32 + lane] - M);
                l = fmaf(f, rl[w * 32 + lane], l);
                add4(acc, f, ro[w * 32 + lane]);
            }
            const float inv = 1.0f / l;
            if (e0 + lane < nr * cols)
                store4<T>(dest(r) + 4 * q, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
        }
        __syncthreads();
    }
}

cudaError_t rows_join_launch(const RowsArgs &a, bool bf16, cudaStream_t s) {
    if (a.P < 2) return cudaSuccess;
    // an item's rows, 32 at a time, over up to 8 blocks
    const int gy = std::min(8, (a.slot_rows + 31) / 32 * 2);
    const dim3 grid(a.P - 1, gy);
    if (a.hd <= 64)
        return bf16 ? launch_pdl(rows_join_kernel<__nv_bfloat16, 2>, grid, dim3(256), 0, s, a)
                    : launch_pdl(rows_join_kernel<float, 2>, grid, dim3(256), 0, s, a);
    if (a.hd <= 128)
        return bf16 ? launch_pdl(rows_join_kernel<__nv_bfloat16, 4>, grid, dim3(256), 0, s, a)
                    : launch_pdl(rows_join_kernel<float, 4>, grid, dim3(256), 0, s, a);
    return bf16 ? launch_pdl(rows_join_kernel<__nv_bfloat16, 8>, grid, dim3(256), 0, s, a)
                : launch_pdl(rows_join_kernel<float, 8>, grid, dim3(256), 0, s, a);
}

// ---- launch

// 16 rows when the average sequence's rows fit them (decode steps), else 64 (32 for heads wider
// than 128, whose keys and values fill the shared memory).  The choice needs no length: any
// item of either tile is right.
int rows_simt_wide_tile(int hd) { return hd <= 128 ? 64 : 32; }
int rows_simt_tile(int rows, int nseq, int G, int hd) {
    if ((long long)rows * G <= (long long)kSimtSmallTile * nseq && G <= kSimtSmallTile) return kSimtSmallTile;
    return rows_simt_wide_tile(hd);
}

static size_t simt_bytes(int hd, int R, int nseq) {  // fp32: bf16 needs no more
    if (hd <= 64) return R == 16 ? simt_smem<float, 64, 16>(nseq) : simt_smem<float, 64, 64>(nseq);
    if (hd <= 128) return R == 16 ? simt_smem<float, 128, 16>(nseq) : simt_smem<float, 128, 64>(nseq);
    return R == 16 ? simt_smem<float, 256, 16>(nseq) : simt_smem<float, 256, 32>(nseq);
}

// CTAs of a launch: as many as the shared memory lets run at a time, at most two per SM (the
// registers of 256 threads allow no more).
int rows_simt_ctas(int sms, int hd, int R, int nseq) {
    return sms * (2 * (simt_bytes(hd, R, nseq) + 1024) <= 228 * 1024 ? 2 : 1);
}

template <int HDP> static cudaError_t launch_fma(const RowsArgs &a, cudaStream_t s) {
    const size_t smem = simt_smem<float, HDP, 64>(a.nseq);
    const cudaError_t e = allow_smem((const void *)rows_fma_kernel<HDP>);
    if (e != cudaSuccess) return e;
    return launch_pdl(rows_fma_kernel<HDP>, dim3(a.P), dim3(kSimtThreads), smem, s, a);
}

template <typename T, int HDP, int R> static cudaError_t launch_simt(const RowsArgs &a, cudaStream_t s) {
    const size_t smem = simt_smem<T, HDP, R>(a.nseq);
    const cudaError_t e = allow_smem((const void *)rows_simt_kernel<T, HDP, R>);
    if (e != cudaSuccess) return e;
    return launch_pdl(rows_simt_kernel<T, HDP, R>, dim3(a.P), dim3(kSimtThreads), smem, s, a);
}

cudaError_t rows_simt_launch(const RowsArgs &a, bool bf16, cudaStream_t s) {
    const bool small = a.geom.PT * a.G <= kSimtSmallTile;
    if (bf16) return small ? launch_simt<__nv_bfloat16, 256, 16>(a, s) : launch_simt<__nv_bfloat16, 256, 32>(a, s);
    if (a.hd <= 64) return small ? launch_simt<float, 64, 16>(a, s) : launch_fma<64>(a, s);
    if (a.hd <= 128) return small ? launch_simt<float, 128, 16>(a, s) : launch_fma<128>(a, s);
    return small ? launch_simt<float, 256, 16>(a, s) : launch_simt<float, 256, 32>(a, s);
}

}  // namespace slm
