// rows_attention.cu -- the CUDA-core attention of packed rows (rows_attention.cuh) for plain causal
// scores, its tiles, and the kernel that joins the pieces of items that several CTAs share.
#include "rows_attention.cuh"

namespace slm {

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
            const float inv = M == -INFINITY ? 0.f : 1.0f / l;  // no piece: the row sees nothing (masked calls)
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
            const float inv = M == -INFINITY ? 0.f : 1.0f / l;
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

cudaError_t rows_simt_launch(const RowsArgs &a, bool bf16, cudaStream_t s) { return launch_cuda_cores<false>(a, bf16, s); }

}  // namespace slm
