// rows_step.cu -- the plan of a serving step (slm_rows_plan): row ranges, page table, slots.
//
// With n_s = max(new_len_s, 0) rows, c_s = seq_len_s and pages of P positions,
//     row_start_s = sum of n before s,   pages needed = ceil((c + n) / P) - ceil(c / P),
//     pages given back = ceil(c / P) where new_len_s < 0,
// and page j of the step (in the order of the needs' running sum) is entry F + R - 1 - j of the
// stack, F free pages before the step and R given back in it.  An entry from F on is one of those
// given back and is looked up in its sequence's table row, so nobody reads what another thread
// writes and one launch does.
//
// A sequence under a window may have lost its first pages before it ends: its table row begins with
// negative entries then, and as those stand in front of the others, a binary search of the row counts
// them.  The row's first entry, which says whether there is one to count, is read beside the lengths.
//
// Latency bounds it: the lengths, three running sums over at most 1,024 sequences (one per thread),
// then for every row a search of its sequence, its page and two stores.  Up to eight CTAs, each with
// the sums of its own, share the rows; they are a cluster, so that all have read the counters before
// one of them writes them (they may be overwritten in place).  256 sequences with a row each take 3.8 us in a
// captured graph and 9.1 through the binding (the call on the host); 96 sequences with 41,500 rows 10.1 and
// 10.3.  Where that stood at 9.8, searching four rows at a time (11.4), giving a warp adjacent rows that keep
// the last owner (10.3) and reading the written table instead of finding a page twice (10.1) did not make it
// shorter.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "device_common.cuh"
#include "rows.cuh"

namespace slm {

constexpr int kStepThreads = 1024;
static_assert(kStepThreads >= kRowsMaxSeqs, "a thread per sequence");
constexpr int kStepCtas = 8;

// What stands in shared memory: running sums before each sequence, its length, and its pages that were
// given back before it ends.
struct StepShared {
    int row[kRowsMaxSeqs + 1], need[kRowsMaxSeqs + 1], back[kRowsMaxSeqs + 1], len[kRowsMaxSeqs], gone[kRowsMaxSeqs];
    long long warp[3][32];
};

// The last s in [0, n) with a[s] <= x: the owner of x, since empty sequences share their successor's.
__device__ __forceinline__ int owner_of(const int *a, int n, int x) {
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

// Inclusive running sum over the CTA, three at a time.
__device__ __forceinline__ void scan3(long long (&v)[3], long long (*warp)[32]) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int q = 0; q < 3; q++) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, v[q], o);
            if (lane >= o) v[q] += u;
        }
        if (lane == 31) warp[q][w] = v[q];
    }
    __syncthreads();
    if (w < 3) {
        long long x = warp[w][lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += u;
        }
        warp[w][lane] = x;
    }
    __syncthreads();
    if (w > 0) {
#pragma unroll
        for (int q = 0; q < 3; q++) v[q] += warp[q][w - 1];
    }
}

// How many of a table row's n entries, of which the first is negative, are: they stand in front.
__device__ __forceinline__ int negative_entries(const int *row, int n) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (row[mid] < 0)
            lo = mid;
        else
            hi = mid;
    }
    return hi;
}

__global__ void __launch_bounds__(kStepThreads) rows_step_kernel(const __grid_constant__ StepArgs A) {
    __shared__ StepShared S;
    const int tid = threadIdx.x, cta = blockIdx.x, ctas = gridDim.x, shift = A.page_shift;
    pdl_wait();
    pdl_trigger();
    const int F = *A.free_count;
    int n = 0, c = 0, first = 0;
    bool ends = false, bad = false;
    if (tid < A.nseq) {
        first = A.page_table[(size_t)tid * A.table_ld];
        n = A.new_len[tid];
        c = A.seq_len[tid];
        ends = n < 0;
        n = max(n, 0);
        bad = c < 0 || (long long)c + n > A.cap;
    }
    const int c0 = bad ? 0 : c, n0 = bad ? 0 : n;  // inside the table, so that no sum overflows
    const int held = (int)(((long long)c0 + (1 << shift) - 1) >> shift);
    const int all = (int)(((long long)c0 + n0 + (1 << shift) - 1) >> shift);
    const int gone = ends && held > 0 && first < 0 ? negative_entries(A.page_table + (size_t)tid * A.table_ld, held) : 0;
    const int need = ends ? 0 : all - held, back = ends ? held - gone : 0;
    long long v[3] = {n0, need, back};
    scan3(v, S.warp);
    const long long rows = S.warp[0][31], T = S.warp[1][31], R = S.warp[2][31];
    if (tid < A.nseq) {
        // sums that do not fit 32 bits are of a step that is refused below
        S.row[tid] = (int)(v[0] - n0);
        S.need[tid] = (int)(v[1] - need);
        S.back[tid] = (int)(v[2] - back);
        S.len[tid] = c;
        S.gone[tid] = gone;
    }
    const bool length = __syncthreads_or(bad) || rows > A.rows;
    const bool pool = F < 0 || F > A.n_pages || (long long)F + R > A.n_pages || T > (long long)F + R;
    if (ctas > 1) {  // everyone has read the lengths and the count
        asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    }
    const bool none = length || pool;
    if (cta == 0) {
        if (tid < A.nseq) {
            A.row_start[tid + 1] = none ? 0 : (int)v[0];
            A.ctx_len[tid] = none ? c : ends ? 0 : c;
            A.seq_len_out[tid] = none ? c : ends ? 0 : c + n;
        }
        if (tid == 0) {
            A.row_start[0] = 0;
            A.free_count_out[0] = none ? F : (int)(F + R - T);
            if (none) atomicOr(A.status, (length ? SLM_ROWS_LENGTH : 0) | (pool ? SLM_ROWS_POOL : 0));
        }
    }
    const int t0 = cta * kStepThreads + tid, step = ctas * kStepThreads;
    if (none) {
        for (int r = t0; r < A.rows; r += step) {
            if (A.positions) A.positions[r] = -1;
            if (A.slots) A.slots[r] = -1;
        }
        return;
    }
    // the k-th page given back, and page j of the step
    auto given = [&](int k) {
        const int s = owner_of(S.back, A.nseq, k);
        return A.page_table[(size_t)s * A.table_ld + S.gone[s] + (k - S.back[s])];
    };
    auto taken = [&](int j) {
        const long long e = F + R - 1 - j;
        return e >= F ? given((int)(e - F)) : A.free_pages[e];
    };
    for (int k = t0; k < R; k += step) {
        const int page = given(k);
        if (page < 0 || page >= A.n_pages) atomicOr(A.status, SLM_ROWS_PAGE);
        A.free_pages[F + k] = page;
    }
    for (int j = t0; j < T; j += step) {
        const int s = owner_of(S.need, A.nseq, j), page = taken(j);
        if (page < 0 || page >= A.n_pages) atomicOr(A.status, SLM_ROWS_PAGE);
        const int b = (int)(((long long)S.len[s] + (1 << shift) - 1) >> shift) + j - S.need[s];
        A.page_table[(size_t)s * A.table_ld + b] = page;
    }
    if (!A.positions && !A.slots) return;
    for (int r = t0; r < A.rows; r += step) {
        int pos = -1;
        long long slot = -1;
        if (r < rows) {
            const int s = owner_of(S.row, A.nseq, r);
            pos = S.len[s] + r - S.row[s];
            if (A.slots) {
                const int b = pos >> shift, h = (int)(((long long)S.len[s] + (1 << shift) - 1) >> shift);
                const int page = b < h ? A.page_table[(size_t)s * A.table_ld + b] : taken(S.need[s] + b - h);
                if (page < 0 || page >= A.n_pages)
                    atomicOr(A.status, SLM_ROWS_PAGE);
                else
                    slot = ((long long)page << shift) + (pos & ((1 << shift) - 1));
            }
        }
        if (A.positions) A.positions[r] = pos;
        if (A.slots) A.slots[r] = slot;
    }
}

cudaError_t rows_step_launch(const StepArgs &a, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    // a CTA for each 2,048 rows
    const int ctas = std::min(kStepCtas, std::max(1, (a.rows + 2047) / 2048));
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kStepThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[2]{};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = ctas;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, rows_step_kernel, a);
}

}  // namespace slm
