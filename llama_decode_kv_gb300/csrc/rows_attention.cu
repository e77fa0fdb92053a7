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
// bounds prompts and large chunks; a decode step is bound by reading the cache, and takes the
// 16-row tile, where four thread groups share the keys of a block instead of multiplying
// rows that do not exist.
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

template <int HDP> constexpr int simt_ld() { return HDP + 4; }
template <int HDP, int R> constexpr size_t simt_smem(int nseq) {
    return (size_t)(R + 2 * kSimtBlk) * simt_ld<HDP>() * 4 + (size_t)R * (kSimtBlk + 4) * 4 + 3 * R * 4 +
           (size_t)nseq * sizeof(SeqRows) + (size_t)(nseq + 1) * 8 + 16;
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
    float *ks = qs + R * LD, *vs = ks + kSimtBlk * LD, *ps = vs + kSimtBlk * LD;
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

        for (int kb = p.kb0; kb < p.kb1; kb++) {
            const int k0 = kb * kSimtBlk;
            // keys and values of the block; rows that no row of the item sees are zero
            for (int e = tid; e < kSimtBlk * (HDP / E); e += kSimtThreads) {
                const int j = e / (HDP / E), d = (e - j * (HDP / E)) * E;
                float *kd = ks + j * LD + d, *vd = vs + j * LD + d;
                if (k0 + j < L && d < A.hd) {
                    widen16((const T *)A.kv.k + rows_kv_offset(A, false, p.s, sr.row0, p.g, k0 + j) + d, kd);
                    widen16((const T *)A.kv.v + rows_kv_offset(A, true, p.s, sr.row0, p.g, k0 + j) + d, vd);
                } else {
#pragma unroll
                    for (int i = 0; i < E; i++) kd[i] = vd[i] = 0.f;
                }
            }
            __syncthreads();
            // S: rows 4 ty + i, keys kq * 16 + tx (+ 16 j)
            {
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
#pragma unroll 2
            for (int j = kq * (kSimtBlk / KQ); j < (kq + 1) * (kSimtBlk / KQ); j += 4) {
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
        // the key groups' sums of O (over the key buffer: KQ R rows are exactly its length)
        if (KQ > 1) {
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
                        if (d < A.hd) *(float4 *)(part + (size_t)r * A.hd + d) = o[i][c];
                    }
                }
            if (tid < nr) {
                pm[tid] = mrow[tid];
                pm[A.slot_rows + tid] = lrow[tid];
            }
        }
    }
    if (!joined && tid == 0) write_join(A, blockIdx.x, seq, unit, nullptr);
}

// ---- joining
//
// Piece i of an item has, per row, the maximum m_i, the sum l_i and the unnormalised O_i:
//     out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i,  M = max_i m_i.
// Block x looks after the item that attention CTA x starts and another one finishes (RowsJoin);
// its pieces are slot 2x + 1 and the slots 2c of the CTAs behind x.  A thread takes four columns
// of a row and goes over the pieces in order, so the result does not depend on timing.  With
// kJoinShared pieces or more (a long context over the whole GPU, few rows) the eight warps of a
// block share the pieces of a row instead and add up in shared memory.
constexpr int kJoinShared = 12;

template <typename T> __device__ __forceinline__ void store4(T *p, float4 v, float f);
template <> __device__ __forceinline__ void store4<float>(float *p, float4 v, float f) {
    *(float4 *)p = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
}
template <> __device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16 *p, float4 v, float f) {
    *(uint2 *)p = make_uint2(pack_bf16x2(v.x * f, v.y * f), pack_bf16x2(v.z * f, v.w * f));
}

__device__ __forceinline__ void add4(float4 &a, float f, const float4 &b) {
    a.x = fmaf(f, b.x, a.x);
    a.y = fmaf(f, b.y, a.y);
    a.z = fmaf(f, b.z, a.z);
    a.w = fmaf(f, b.w, a.w);
}

template <typename T>
__global__ void __launch_bounds__(256) rows_join_kernel(const __grid_constant__ RowsArgs A) {
    pdl_wait();
    pdl_trigger();
    const RowsJoin J = ((const RowsJoin *)A.ws)[blockIdx.x];
    if (J.pieces == 0) return;
    const int n = J.pieces, nr = J.tokens * A.G, cols = A.hd / 4, c0 = blockIdx.x;
    const size_t sf = slot_floats(A.slot_rows, A.hd);
    const float *slots = (const float *)(A.ws + join_bytes(A.P));
    const float *stats = slots + (size_t)A.slot_rows * A.hd;  // maxima, then sums, of slot 0
    auto slot = [&](int i) { return (size_t)(i == 0 ? 2 * c0 + 1 : 2 * (c0 + i)) * sf; };
    auto dest = [&](int r) {
        const int tok = r / A.G;
        return (T *)A.out + (size_t)(J.row0 + tok) * A.out_ld + (size_t)(J.head0 + r - tok * A.G) * A.hd;
    };
    if (n < kJoinShared) {
        for (int e = blockIdx.y * 256 + threadIdx.x; e < nr * cols; e += gridDim.y * 256) {
            const int r = e / cols, d = (e - r * cols) * 4;
            float m[kJoinShared], M = -INFINITY, l = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kJoinShared; i++) {
                m[i] = i < n ? stats[slot(i) + r] : -INFINITY;
                M = fmaxf(M, m[i]);
            }
#pragma unroll
            for (int i = 0; i < kJoinShared; i++) {
                if (m[i] == -INFINITY) continue;  // no piece, or the row saw nothing of it: O was not written
                const float f = exp2f(m[i] - M);
                l = fmaf(f, stats[slot(i) + A.slot_rows + r], l);
                add4(acc, f, *(const float4 *)(slots + slot(i) + (size_t)r * A.hd + d));
            }
            store4<T>(dest(r) + d, acc, 1.0f / l);
        }
        return;
    }
    __shared__ __align__(16) float red[8][256];
    __shared__ float rm[8], rl[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int r = blockIdx.y; r < nr; r += gridDim.y) {
        float M = -INFINITY, l = 0.f;
        for (int i = warp + 8 * lane; i < n; i += 256) M = fmaxf(M, stats[slot(i) + r]);
#pragma unroll
        for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll 4
        for (int i = warp; i < n; i += 8) {
            const float mi = stats[slot(i) + r];
            if (mi == -INFINITY) continue;
            const float f = exp2f(mi - M);
            l = fmaf(f, stats[slot(i) + A.slot_rows + r], l);
#pragma unroll
            for (int k = 0; k < 2; k++)
                if (lane + 32 * k < cols) add4(acc[k], f, *(const float4 *)(slots + slot(i) + (size_t)r * A.hd + 4 * (lane + 32 * k)));
        }
        __syncthreads();  // the last row's sums have been read
        if (lane == 0) {
            rm[warp] = M;
            rl[warp] = l;
        }
#pragma unroll
        for (int k = 0; k < 2; k++) *(float4 *)(red[warp] + 4 * (lane + 32 * k)) = acc[k];
        __syncthreads();
        if (threadIdx.x < cols) {
            float Ma = -INFINITY, la = 0.f;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = 0; w < 8; w++) Ma = fmaxf(Ma, rm[w]);
            for (int w = 0; w < 8; w++) {
                if (rm[w] == -INFINITY) continue;
                const float f = exp2f(rm[w] - Ma);
                la = fmaf(f, rl[w], la);
                add4(a, f, *(const float4 *)(red[w] + 4 * threadIdx.x));
            }
            store4<T>(dest(r) + 4 * threadIdx.x, a, 1.0f / la);
        }
    }
}

cudaError_t rows_join_launch(const RowsArgs &a, bool bf16, cudaStream_t s) {
    if (a.P < 2) return cudaSuccess;
    // an item's rows are spread over up to 16 blocks
    const int gy = (int)std::min<long long>(16, ((long long)a.slot_rows * (a.hd / 4) + 255) / 256);
    const dim3 grid(a.P - 1, gy);
    return bf16 ? launch_pdl(rows_join_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, a)
                : launch_pdl(rows_join_kernel<float>, grid, dim3(256), 0, s, a);
}

// ---- launch

// 16 rows when the average sequence's rows fit them (decode steps), else 64 (32 for heads wider
// than 128, whose keys and values fill the shared memory).  The choice needs no length: any
// item of either tile is right.
int rows_simt_tile(int rows, int nseq, int G, int hd) {
    if ((long long)rows * G <= 16LL * nseq && G <= 16) return 16;
    return hd <= 128 ? 64 : 32;
}

static size_t simt_bytes(int hd, int R, int nseq) {
    if (hd <= 64) return R == 16 ? simt_smem<64, 16>(nseq) : simt_smem<64, 64>(nseq);
    if (hd <= 128) return R == 16 ? simt_smem<128, 16>(nseq) : simt_smem<128, 64>(nseq);
    return R == 16 ? simt_smem<256, 16>(nseq) : simt_smem<256, 32>(nseq);
}

// CTAs of a launch: as many as the shared memory lets run at a time, at most two per SM (the
// registers of 256 threads allow no more).
int rows_simt_ctas(int sms, int hd, int R, int nseq) {
    return sms * (2 * (simt_bytes(hd, R, nseq) + 1024) <= 228 * 1024 ? 2 : 1);
}

template <typename T, int HDP, int R> static cudaError_t launch_simt(const RowsArgs &a, cudaStream_t s) {
    const size_t smem = simt_smem<HDP, R>(a.nseq);
    cudaError_t e = cudaFuncSetAttribute(rows_simt_kernel<T, HDP, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(rows_simt_kernel<T, HDP, R>, dim3(a.P), dim3(kSimtThreads), smem, s, a);
}

template <typename T> static cudaError_t launch_simt_hd(const RowsArgs &a, cudaStream_t s) {
    const bool small = a.geom.PT * a.G <= 16;
    if (a.hd <= 64) return small ? launch_simt<T, 64, 16>(a, s) : launch_simt<T, 64, 64>(a, s);
    if (a.hd <= 128) return small ? launch_simt<T, 128, 16>(a, s) : launch_simt<T, 128, 64>(a, s);
    return small ? launch_simt<T, 256, 16>(a, s) : launch_simt<T, 256, 32>(a, s);
}

cudaError_t rows_simt_launch(const RowsArgs &a, bool bf16, cudaStream_t s) {
    return bf16 ? launch_simt_hd<__nv_bfloat16>(a, s) : launch_simt_hd<float>(a, s);
}

}  // namespace slm
