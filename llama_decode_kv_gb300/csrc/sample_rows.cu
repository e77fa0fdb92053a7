// sample_rows.cu -- the next token of every row of logits with the row's own temperature, top-k,
// top-p and min-p (slm_sample_rows).
//
// With x_max the largest logit, token i has the weight w_i = exp((x_i - x_max) / T), kept as a whole
// number W_i of 2^-40, so that sums are exact and do not depend on their order (the exponential is
// fp32, about 2^-22 off where the weight counts).  In the order (x descending, i ascending) every cut
// keeps a prefix, so what is kept is a pair (K, I): the tokens whose ordered key is above K, and those
// with the key K up to index I.
//     top-k:  K from counts.   top-p:  K from weights, the first sum to reach p times the whole.
//     min-p:  w_i >= m.        draw:   the first i in index order with sum_{j <= i} W_j > u sum W.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "device_common.cuh"
#include "rows.cuh"

namespace slm {

constexpr int kSrThreads = 1024;
typedef unsigned long long u64;

// Monotone map of a float to an unsigned key; NaN goes where -infinity is.
__device__ __forceinline__ uint32_t sr_key(float f) {
    if (!(f >= -INFINITY)) f = -INFINITY;
    if (f == 0.f) f = 0.f;  // -0 equals 0
    const uint32_t b = __float_as_uint(f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float sr_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

template <typename T> __device__ __forceinline__ float sr_load(const T *p, int i);
template <> __device__ __forceinline__ float sr_load<float>(const float *p, int i) { return __ldg(p + i); }
template <> __device__ __forceinline__ float sr_load<uint16_t>(const uint16_t *p, int i) {
    return __uint_as_float((uint32_t)__ldg(p + i) << 16);
}

// Inclusive running sum over the CTA.
__device__ __forceinline__ u64 sr_scan(u64 v, u64 *warp) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();  // the last scan has been read
    if (lane == 31) warp[w] = v;
    __syncthreads();
    if (w == 0) {
        u64 x = warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 u = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += u;
        }
        warp[lane] = x;
    }
    __syncthreads();
    return w > 0 ? v + warp[w - 1] : v;
}

template <typename T>
__global__ void __launch_bounds__(kSrThreads) sample_rows_kernel(const __grid_constant__ SampleRowsArgs A) {
    __shared__ u64 warp[32], hist[256], found[2];
    __shared__ int index;
    const int tid = threadIdx.x, lane = tid & 31, V = A.vocab;
    pdl_wait();
    pdl_trigger();
    for (long long row = blockIdx.x; row < A.rows; row += gridDim.x) {
        const T *x = (const T *)A.logits + row * A.ld;
        const float temp = A.temperature ? __ldg(A.temperature + row) : 1.0f;
        const int k = A.top_k ? __ldg(A.top_k + row) : 0;
        const float p = A.top_p ? __ldg(A.top_p + row) : 1.0f;
        const float minp = A.min_p ? fminf(__ldg(A.min_p + row), 1.0f) : 0.0f;
        const int per = (V + kSrThreads - 1) / kSrThreads;  // contiguous indexes of a thread
        const int lo = min(V, tid * per), hi = min(V, lo + per);
        // the first of the order: key and complemented index
        u64 best = 0;
        for (int i = tid; i < V; i += kSrThreads)
            best = max(best, (u64)sr_key(sr_load(x, i)) << 32 | (0xffffffffu - (uint32_t)i));
#pragma unroll
        for (int o = 16; o; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
        __syncthreads();
        if (lane == 0) warp[tid >> 5] = best;
        __syncthreads();
        best = warp[lane];
#pragma unroll
        for (int o = 16; o; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
        const uint32_t top = (uint32_t)(best >> 32);
        const float vmax = sr_value(top);
        if (!(temp > 0.f) || vmax == -INFINITY) {
            if (tid == 0) A.next_ids[row] = vmax == -INFINITY ? 0 : (int)(0xffffffffu - (uint32_t)best);
            continue;
        }
        const float scale = 1.4426950408889634f / temp;
        auto weight = [&](uint32_t key) {
            const float d = sr_value(key) - vmax;
            return key == top ? 1.0f : d == -INFINITY ? 0.0f : exp2f(d * scale);
        };
        uint32_t K = 0;
        int I = V;  // everything
        auto kept = [&](uint32_t key, int i) { return key > K || (key == K && i <= I); };
        auto mass = [&](uint32_t key) { return (u64)(weight(key) * 1099511627776.0f + 0.5f); };
        // (K, I) cut to the shortest prefix of what is kept with a sum of at least `want`
        auto cut = [&](u64 want, auto amount) {
            uint32_t prefix = 0, mask = 0;
            u64 above = 0;
            for (int d = 24; d >= 0; d -= 8) {
                if (tid < 256) hist[tid] = 0;
                __syncthreads();
                for (int i = tid; i < V; i += kSrThreads) {
                    const uint32_t key = sr_key(sr_load(x, i));
                    if ((key & mask) == prefix && kept(key, i)) atomicAdd(&hist[key >> d & 255u], amount(key));
                }
                __syncthreads();
                if (tid == 0) {
                    int b = 255;
                    u64 a = above;
                    while (b > 0 && a + hist[b] < want) a += hist[b--];
                    found[0] = b;
                    found[1] = a;
                }
                __syncthreads();
                prefix |= (uint32_t)found[0] << d;
                mask |= 255u << d;
                above = found[1];
            }
            // the ties that are needed, in index order
            const u64 each = amount(prefix), ties = each ? (want - above + each - 1) / each : 1;
            int mine = 0;
            for (int i = lo; i < hi; i++) {
                const uint32_t key = sr_key(sr_load(x, i));
                mine += key == prefix && kept(key, i);
            }
            const u64 upto = sr_scan((u64)mine, warp);
            if (tid == 0) index = V;
            __syncthreads();
            if (upto >= ties && upto - mine < ties) {
                u64 at = upto - mine;
                for (int i = lo; i < hi; i++) {
                    const uint32_t key = sr_key(sr_load(x, i));
                    if (key == prefix && kept(key, i) && ++at == ties) {
                        index = i;
                        break;
                    }
                }
            }
            __syncthreads();
            K = prefix;
            I = index;
            __syncthreads();
        };
        if (k > 0 && k < V) cut((u64)k, [](uint32_t) { return (u64)1; });
        auto total = [&](bool least, u64 &mine) {
            mine = 0;
            for (int i = lo; i < hi; i++) {
                const uint32_t key = sr_key(sr_load(x, i));
                if (kept(key, i) && !(least && weight(key) < minp)) mine += mass(key);
            }
            const u64 s = sr_scan(mine, warp);
            __syncthreads();
            return s;
        };
        u64 mine;
        if (p < 1.0f) {
            total(false, mine);
            const u64 M = warp[31], want = (u64)ceil((double)fmaxf(p, 0.0f) * (double)M);
            cut(max(want, (u64)1), mass);
        }
        const u64 upto = total(true, mine), M = warp[31];
        float u = __ldg(A.uniforms + row);
        u = u >= 0.f ? fminf(u, 1.0f) : 0.f;
        const u64 target = min((u64)((double)u * (double)M), M - 1);
        if (upto > target && upto - mine <= target) {
            u64 at = upto - mine;
            for (int i = lo; i < hi; i++) {
                const uint32_t key = sr_key(sr_load(x, i));
                if (kept(key, i) && !(weight(key) < minp)) at += mass(key);
                if (at > target) {
                    A.next_ids[row] = i;
                    break;
                }
            }
        }
    }
}

cudaError_t sample_rows_launch(const SampleRowsArgs &a, bool bf16, cudaStream_t s) {
    const dim3 grid(a.rows < (1 << 20) ? a.rows : 1 << 20);
    return bf16 ? launch_pdl(sample_rows_kernel<uint16_t>, grid, dim3(kSrThreads), 0, s, a)
                : launch_pdl(sample_rows_kernel<float>, grid, dim3(kSrThreads), 0, s, a);
}

}  // namespace slm
