// rows_append.cu -- append the keys and values of packed rows to a paged cache, rotating
// keys and queries by their positions on the way (slm_kv_append).
//
// Row r of sequence s stands at position p = ctx_len[s] + r - row_start[s] and goes to cache
// row p % page_size of page page_table[s][p / page_size].  The rotation takes the pairs
// (j, j + hd / 2):  y_j = x_j cos - x_{j + hd/2} sin,  y_{j + hd/2} = x_j sin + x_{j + hd/2} cos,
// with (cos, sin) from the caller's fp32 table; it is done in fp32 and rounded once, to the
// type that is stored.
//
// slm_kv_append_axes turns pair j by position positions[axis[j]][r] instead of p; the rest is the
// same kernel.
//
// Bytes bound it: every value is read once and written once, and nothing else is as large.
// A unit is VEC pairs of one head (two VEC-element loads, VEC (cos, sin), two stores), so that
// a thread's accesses are 16 bytes wide (8 for bf16 heads of 8 mod 16) and a warp's are
// contiguous.  A CTA first resolves its rows -- owner by counting the sequences that end at or
// before the row, position, page -- one warp per row, then all its threads share the units.
// 8,000 rows of 48 heads of 64, fp32 to bf16: 30.7 us = 6.0 TB/s, 88% of the copy rate, in a captured
// graph, 31.5 us through the binding; one row 2.5 us, which is the chain of lookups.  With positions of
// three axes (16 prompts of up to 1,024 rows, the same heads and types, through the binding) 30.5 us,
// 73% of the copy rate: a row's positions are one more dependent load in front of the barrier behind which
// all of its units are loaded, the values too, although their addresses do not depend on it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "device_common.cuh"
#include "rows.cuh"

namespace slm {

constexpr int kAppendThreads = 256;

template <int N> struct Floats { float v[N]; };

// N consecutive elements at p (aligned to their size), widened.
template <int N> __device__ __forceinline__ Floats<N> load_vec(const float *p) {
    Floats<N> o;
#pragma unroll
    for (int i = 0; i < N; i += 4) *(float4 *)(o.v + i) = *(const float4 *)(p + i);
    return o;
}
template <int N> __device__ __forceinline__ Floats<N> load_vec(const __nv_bfloat16 *p) {
    Floats<N> o;
    uint32_t w[N / 2];
    if (N == 8)
        *(uint4 *)w = *(const uint4 *)p;
    else
        *(uint2 *)w = *(const uint2 *)p;
#pragma unroll
    for (int i = 0; i < N / 2; i++) {
        o.v[2 * i] = bf16_lo(w[i]);
        o.v[2 * i + 1] = bf16_hi(w[i]);
    }
    return o;
}
template <int N> __device__ __forceinline__ void store_vec(float *p, const Floats<N> &a) {
#pragma unroll
    for (int i = 0; i < N; i += 4) *(float4 *)(p + i) = *(const float4 *)(a.v + i);
}
template <int N> __device__ __forceinline__ void store_vec(__nv_bfloat16 *p, const Floats<N> &a) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; i++) w[i] = pack_bf16x2(a.v[2 * i], a.v[2 * i + 1]);
    if (N == 8)
        *(uint4 *)p = *(const uint4 *)w;
    else
        *(uint2 *)p = *(const uint2 *)w;
}

struct AppendRow {
    long long cache_row;  // (page * KV) * page_size + position in the page; < 0: no row to write
    int pos;
};

// Where row r goes; one warp, the answer on lane 0.
// rope_len: positions that the rotation by p may take (no rotation by p: all).
__device__ __forceinline__ AppendRow resolve_row(const AppendArgs &A, int r, int lane, long long rope_len) {
    AppendRow o{-1, 0};
    int s = 0;  // sequences that end at or before r: the owner's number
    for (int i = lane; i < A.nseq; i += 32) s += __ldg(A.row_start + i + 1) <= r;
    s = (int)__reduce_add_sync(0xffffffffu, (unsigned)s);
    if (lane || s >= A.nseq) return o;  // s = nseq: behind the last sequence
    const int first = __ldg(A.row_start + s);
    if (r < first || r >= __ldg(A.row_start + s + 1)) return o;  // before the first sequence, or not ascending
    const int ctx = A.ctx_len ? __ldg(A.ctx_len + s) : 0;
    const long long pos = (long long)ctx + ((long long)r - first);
    if (ctx < 0 || pos >= A.cap || pos >= rope_len) {
        atomicOr(A.status, SLM_ROWS_LENGTH);
        return o;
    }
    const int page = __ldg(A.table + (size_t)s * A.table_ld + (pos >> A.page_shift));
    if (page < 0 || page >= A.n_pages) {
        atomicOr(A.status, SLM_ROWS_PAGE);
        return o;
    }
    o.pos = (int)pos;
    o.cache_row = (((long long)page * A.KV) << A.page_shift) + (pos & ((1 << A.page_shift) - 1));
    return o;
}

// The (cos, sin) of VEC pairs from pair j on, by the positions of their axes.  Sections put all of
// them on one axis as a rule, and the table row is read 16 bytes at a time as for one position.
template <int VEC>
__device__ __forceinline__ void axes_turns(const float *rope, int half, int j, const uint8_t *axis, const int *pos, float *t) {
    const int a0 = axis[j];
    bool same = a0 != 0xff;
#pragma unroll
    for (int k = 1; k < VEC; k++) same &= axis[j + k] == a0;
    if (same) {
        const float *cs = rope + ((size_t)pos[a0] * half + j) * 2;
#pragma unroll
        for (int k = 0; k < 2 * VEC; k += 4) *(float4 *)(t + k) = __ldg((const float4 *)(cs + k));
        return;
    }
#pragma unroll
    for (int k = 0; k < VEC; k++) {
        const int a = axis[j + k];
        const float2 cs = a == 0xff ? make_float2(1.f, 0.f) : __ldg((const float2 *)(rope + ((size_t)pos[a] * half + j + k) * 2));
        t[2 * k] = cs.x;
        t[2 * k + 1] = cs.y;
    }
}

__host__ __device__ inline const AppendArgs &append_args(const AppendArgs &a) { return a; }
__host__ __device__ inline const AppendArgs &append_args(const AxesArgs &a) { return a.a; }

template <typename TI, typename TC, int VEC, typename ARGS>
__global__ void __launch_bounds__(kAppendThreads) rows_append_kernel(const __grid_constant__ ARGS P, int rpc) {
    constexpr bool kAxes = sizeof(ARGS) == sizeof(AxesArgs);
    const AppendArgs &A = append_args(P);
    __shared__ AppendRow rows[8];
    __shared__ int axis_pos[kAxes ? 8 : 1][kMaxAxes];
    __shared__ uint8_t axis[kAxes ? 128 : 1];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r0 = blockIdx.x * rpc, nr = min(rpc, A.rows - r0);
    if (blockIdx.x == 0 && blockIdx.y == 0 && warp == kAppendThreads / 32 - 1) {
        bool bad = false;
        for (int i = lane; i < A.nseq; i += 32) {
            const int a = __ldg(A.row_start + i), b = __ldg(A.row_start + i + 1);
            bad |= a < 0 || b < a || b > A.rows;
        }
        if (bad) atomicOr(A.status, SLM_ROWS_LENGTH);
    }
    if (warp < nr) {
        AppendRow a = resolve_row(A, r0 + warp, lane, A.rope && !kAxes ? A.rope_len : A.cap);
        if constexpr (kAxes) {
            bool off = false;  // an axis' position outside the table: the row is left out
            const bool row = __shfl_sync(0xffffffffu, (int)(a.cache_row >= 0), 0);
            if (row && lane < P.n_axes) {
                const int x = __ldg(P.positions + lane * P.ld + r0 + warp);
                off = x < 0 || x >= A.rope_len;
                axis_pos[warp][lane] = off ? 0 : x;
            }
            if (__any_sync(0xffffffffu, off)) {
                if (lane == 0) atomicOr(A.status, SLM_ROWS_LENGTH);
                a.cache_row = -1;
            }
        }
        if (lane == 0) rows[warp] = a;
    }
    if constexpr (kAxes)
        for (int j = threadIdx.x; j < A.hd / 2; j += kAppendThreads) axis[j] = P.axis[j];
    __syncthreads();
    const int half = A.hd / 2, ph = half / VEC;        // units of a head
    const int Hq = A.q ? A.H : 0, heads = Hq + 2 * A.KV;
    const int units = heads * ph;                      // of a row
    const long long page_rows = 1LL << A.page_shift;
    for (int e = blockIdx.y * kAppendThreads + threadIdx.x; e < nr * units; e += gridDim.y * kAppendThreads) {
        const int i = e / units, u = e - i * units, h = u / ph, j = (u - h * ph) * VEC;
        const AppendRow R = rows[i];
        if (R.cache_row < 0) continue;
        const size_t r = (size_t)(r0 + i);
        const TI *src;
        TC *dst;
        if (h < Hq) {
            src = (const TI *)A.q + r * A.q_ld + (size_t)h * A.hd;
            dst = (TC *)A.q_out + r * A.q_out_ld + (size_t)h * A.hd;
        } else {
            const bool is_v = h >= Hq + A.KV;
            const int g = h - Hq - (is_v ? A.KV : 0);
            src = (const TI *)(is_v ? A.v : A.k) + r * (is_v ? A.v_ld : A.k_ld) + (size_t)g * A.hd;
            dst = (TC *)(is_v ? A.vc : A.kc) + (size_t)(R.cache_row + g * page_rows) * A.hd;
        }
        Floats<VEC> a = load_vec<VEC>(src + j), b = load_vec<VEC>(src + j + half);
        if (A.rope && h < Hq + A.KV) {
            float t[2 * VEC];
            if constexpr (kAxes) {
                axes_turns<VEC>(A.rope, half, j, axis, axis_pos[i], t);
            } else {
                const float *cs = A.rope + ((size_t)R.pos * half + j) * 2;
#pragma unroll
                for (int k = 0; k < 2 * VEC; k += 4) *(float4 *)(t + k) = __ldg((const float4 *)(cs + k));
            }
#pragma unroll
            for (int k = 0; k < VEC; k++) {
                const float x = a.v[k], y = b.v[k];
                a.v[k] = x * t[2 * k] - y * t[2 * k + 1];
                b.v[k] = x * t[2 * k + 1] + y * t[2 * k];
            }
        }
        store_vec<VEC>(dst + j, a);
        store_vec<VEC>(dst + j + half, b);
    }
}

template <typename TI, typename TC, typename ARGS>
static cudaError_t launch_append(const ARGS &p, cudaStream_t s) {
    const AppendArgs &a = append_args(p);
    const int vec = a.hd % 16 == 0 ? 8 : 4;
    const int units = ((a.q ? a.H : 0) + 2 * a.KV) * (a.hd / 2 / vec);
    // One row per CTA, its units spread over grid.y, while the rows alone do not fill the GPU;
    // then four rows per CTA, so that a CTA's chain of lookups is paid once for four rows.
    const int rpc = a.rows >= 2048 ? 4 : 1;
    const int gy = rpc > 1 ? 1 : std::min((units + kAppendThreads - 1) / kAppendThreads, 65535);
    const dim3 grid((a.rows + rpc - 1) / rpc, gy);
    return launch_pdl(vec == 8 ? rows_append_kernel<TI, TC, 8, ARGS> : rows_append_kernel<TI, TC, 4, ARGS>, grid,
                      dim3(kAppendThreads), 0, s, p, rpc);
}

template <typename ARGS>
static cudaError_t launch_typed(const ARGS &a, bool in_bf16, bool cache_bf16, cudaStream_t s) {
    if (in_bf16) return cache_bf16 ? launch_append<__nv_bfloat16, __nv_bfloat16>(a, s) : launch_append<__nv_bfloat16, float>(a, s);
    return cache_bf16 ? launch_append<float, __nv_bfloat16>(a, s) : launch_append<float, float>(a, s);
}

cudaError_t rows_append_launch(const AppendArgs &a, bool in_bf16, bool cache_bf16, cudaStream_t s) {
    return launch_typed(a, in_bf16, cache_bf16, s);
}
cudaError_t rows_append_axes_launch(const AxesArgs &a, bool in_bf16, bool cache_bf16, cudaStream_t s) {
    return launch_typed(a, in_bf16, cache_bf16, s);
}

}  // namespace slm
