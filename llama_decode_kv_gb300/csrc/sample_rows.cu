// sample_rows.cu -- the next token of every row of logits with the row's own temperature, top-k,
// top-p and min-p (slm_sample_rows).
//
// With x_max the largest logit, token i has the weight w_i = exp((x_i - x_max) / T), kept as a whole
// number W_i of 2^-40, so that sums are exact and do not depend on their order (the exponential is
// fp32, about 2^-22 off where the weight counts).  In the order (x descending, i ascending) every cut
// keeps a prefix, so what is kept is the tokens from a threshold of that order on, given as one 64-bit
// number: the logit's ordered key above the complemented index.
//     top-k:  the k-th number.   top-p:  where the running sum of W first reaches p times the whole.
//     min-p:  w_i >= m.          draw:   the first i in index order with sum_{j <= i} W_j > u sum W.
//
// HBM bounds a batch: its logits are read once.  A row has one CTA, or a cluster of up to eight where
// there are few rows, each with a slice of the row; it reads it for the largest logit of every group
// of 16 tokens; the other steps read only groups that can matter, from the L2:
//   greedy        the first group with the largest logit;
//   top-k         256 bins of the groups' maxima give a value that at least k of them reach, and few
//                 more: the tokens that do make a list, which is sorted, cut, and
//                 sorted by index;
//   top-p alone   a histogram of the weights, 32 bins an octave, in cut whole numbers, says in which bin
//                 (or two) the sum is reached; the sum above it is then exact, the bin's tokens make a
//                 list, and a few rounds of 256 bins find the last one of them to be kept;
//   the draw      the sum of every 1,024 tokens, the segment that holds the target, its tokens.
// A top-k above 1,024 or above the number of groups, a list that overflows (thousands of equal logits next to
// the border) or an infinite logit leaves the row to the general way: a threshold by its eight bytes in turn,
// over all tokens.  The bins of a top-k are as wide as the groups' maxima are apart, so a large negative
// number in place of logits that are masked out, groups at a time, puts all others into one bin and overflows
// the list too; -infinity does not.
//
// 256 rows of 128,256 fp32 logits with every kind of cut take 90 us, of which HBM needs 19; the rest is the
// latency of a row's steps, one barrier behind the other, which three CTAs per SM hide in part (a CTA a row,
// lists ranked by comparing all pairs, 252; in slices, lists sorted, 140; loops without branches 90; the
// first kernel, the general way by one CTA a row, 3,479).  One row of 49,152 with top-p takes 21 to 24 us on
// eight SMs (61, 28 before).  256 rows of 128,256 with the same top-k: 400 83 us (bf16 74), 1,024 157, 1,025
// and 2,000, which is the general way, 893 (with top-p 1,665); one row 18 for 400, 145 for 1,025.  With half
// of the logits masked, top-k 50: 63 by -infinity, 982 by -1e9.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "device_common.cuh"
#include "rows.cuh"

namespace slm {

typedef unsigned long long u64;
constexpr int kSrThreads = 256;
constexpr int kSrResident = 3;    // CTAs per SM
constexpr int kSrList = 2048;     // tokens of a list
constexpr int kSrGroups = 16384;  // groups of a slice at most
constexpr int kSrBins = 1344;     // 42 octaves of 32 bins: weights of 2^-41 and less are 0
constexpr int kSrSegment = 1024;
constexpr int kSrCluster = 8;     // slices of a row at most

// Monotone map of a float to an unsigned key; NaN goes where -infinity is, and -0 where 0.
__device__ __forceinline__ uint32_t sr_key(float f) {
    const uint32_t b = __float_as_uint(fmaxf(f, -INFINITY) + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float sr_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// Four consecutive logits from i on; -infinity from n on.  `wide`: rows begin on boundaries of four
// elements.
__device__ __forceinline__ float4 sr_wide4(const float *x, int i) { return __ldg((const float4 *)(x + i)); }
__device__ __forceinline__ float4 sr_wide4(const uint16_t *x, int i) {
    const uint2 w = __ldg((const uint2 *)(x + i));
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}
__device__ __forceinline__ float4 sr_load4(const float *x, int i, int n, bool wide) {
    if (wide && i + 3 < n) return sr_wide4(x, i);
    float4 v;
    v.x = i < n ? __ldg(x + i) : -INFINITY;
    v.y = i + 1 < n ? __ldg(x + i + 1) : -INFINITY;
    v.z = i + 2 < n ? __ldg(x + i + 2) : -INFINITY;
    v.w = i + 3 < n ? __ldg(x + i + 3) : -INFINITY;
    return v;
}
__device__ __forceinline__ float4 sr_load4(const uint16_t *x, int i, int n, bool wide) {
    if (wide && i + 3 < n) return sr_wide4(x, i);
    auto at = [&](int j) { return j < n ? __uint_as_float((uint32_t)__ldg(x + j) << 16) : -INFINITY; };
    return make_float4(at(i), at(i + 1), at(i + 2), at(i + 3));
}
__device__ __forceinline__ float sr_load(const float *x, int i) { return __ldg(x + i); }
__device__ __forceinline__ float sr_load(const uint16_t *x, int i) { return __uint_as_float((uint32_t)__ldg(x + i) << 16); }

__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}
__device__ __forceinline__ u64 warp_total(u64 v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// What a slice's CTA shares; list and found of slice 0 are the row's in the end.
struct SrShared {
    u64 warp[kSrThreads / 32], found[2];
    u64 slices[2][kSrCluster];  // a number of every slice, two sets in turn
    int n, lo, hi;
    u64 bins[256], sums[256];
    union {
        struct {
            uint32_t hist[kSrBins], merged[kSrBins];
        };
        uint32_t queue[kSrList];     // list_bins
    };
    u64 list[kSrList], sorted[kSrList];  // places in the order
};

// Weights on their way into a sum: whole numbers of 2^-20 and of 2^-40, apart until flush(), which has to
// come before 4,096 of them are in.
struct SrSum {
    u64 sum = 0;
    uint32_t hi = 0;
    int lo = 0;
    __device__ __forceinline__ void add(float w) {
        constexpr float kMagic = 12582912.0f;  // 1.5 2^23: what is added to it is rounded to a whole number
        const float a = w * 1048576.0f, h = a + kMagic, l = fmaf(a - (h - kMagic), 1048576.0f, kMagic);
        hi += __float_as_uint(h) - 0x4b400000u;
        lo += (int)(__float_as_uint(l) - 0x4b400000u);
    }
    __device__ __forceinline__ u64 flush() {
        sum += ((u64)hi << 20) + (u64)(long long)lo;
        hi = 0;
        lo = 0;
        return sum;
    }
};

template <typename T, bool CL> struct SrRow {
    static constexpr int NT = kSrThreads;
    const T *x;
    int V, i0, i1;     // tokens of the row; the slice [i0, i1)
    int slices, rank;
    int shift;         // tokens of a group: 2^shift
    bool wide;
    uint32_t *gm;      // [groups of the slice] keys of the maxima
    u64 *seg;          // [segments of the slice] sums
    SrShared *S;
    int tid, lane, warp;
    int set;           // of S->slices
    float vmax, scale; // the largest logit, log2(e) / T
    float minp;
    int *out;

    // All threads of the row.
    __device__ __forceinline__ void sync() const {
        if (CL) {
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        } else {
            __syncthreads();
        }
    }
    // The same place in slice r's shared memory.
    template <typename P> __device__ __forceinline__ P *at_slice(P *p, int r) const {
        if (!CL) return p;
        P *q;
        asm("mapa.u64 %0, %1, %2;" : "=l"(q) : "l"(p), "r"(r));
        return q;
    }
    // Every slice's number to all slices: afterwards S->slices[returned][.] holds them.  The two sets
    // take turns, so that a set is written again only behind a barrier that its readers have reached.
    __device__ __forceinline__ int share(u64 v) {
        const int k = set;
        set ^= 1;
        if (tid < slices) at_slice(S, tid)->slices[k][rank] = v;
        sync();
        return k;
    }

    __device__ __forceinline__ float exponent(float v) const { return fmaxf((v - vmax) * scale, -200.0f); }  // log2 of the weight; NaN: nothing
    static __device__ __forceinline__ u64 whole(float w) {  // w 2^40, to the nearest
        SrSum a;
        a.add(w);
        return a.flush();
    }
    __device__ __forceinline__ int groups() const { return (i1 - i0 + (1 << shift) - 1) >> shift; }
    static __device__ __forceinline__ u64 place(uint32_t key, int i) { return (u64)key << 32 | (0xffffffffu - (uint32_t)i); }

    // Inclusive running sum over the CTA, in order of the threads, and the whole.
    __device__ __forceinline__ u64 scan(u64 v, u64 &total) const {
        v = warp_scan(v, lane);
        __syncthreads();  // the last call's sums have been read
        if (lane == 31) S->warp[warp] = v;
        __syncthreads();
        u64 before = 0;
        total = 0;
#pragma unroll 8
        for (int i = 0; i < NT / 32; i++) {
            if (i == warp) before = total;
            total += S->warp[i];
        }
        return before + v;
    }
    __device__ __forceinline__ u64 cta_total(u64 v) const {
        v = warp_total(v);
        __syncthreads();
        if (lane == 0) S->warp[warp] = v;
        __syncthreads();
        u64 t = 0;
#pragma unroll 8
        for (int i = 0; i < NT / 32; i++) t += S->warp[i];
        return t;
    }
    __device__ __forceinline__ u64 total_of(u64 v) {
        u64 t = cta_total(v);
        if (CL) {
            const int k = share(t);
            t = 0;
            for (int r = 0; r < slices; r++) t += S->slices[k][r];
        }
        return t;
    }
    // The largest of both halves of v, each for itself.
    __device__ __forceinline__ u64 both_most_of(u64 v) {
        auto both = [](u64 a, u64 b) {
            return (u64)max((uint32_t)(a >> 32), (uint32_t)(b >> 32)) << 32 | max((uint32_t)a, (uint32_t)b);
        };
        v = (u64)__reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32)) << 32 | __reduce_max_sync(0xffffffffu, (uint32_t)v);
        __syncthreads();
        if (lane == 0) S->warp[warp] = v;
        __syncthreads();
        u64 t = 0;
#pragma unroll 8
        for (int i = 0; i < NT / 32; i++) t = both(t, S->warp[i]);
        if (CL) {
            const int k = share(t);
            for (int r = 0; r < slices; r++) t = both(t, S->slices[k][r]);
        }
        return t;
    }
    __device__ __forceinline__ u64 most_of(u64 v) {
#pragma unroll
        for (int o = 16; o; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
        __syncthreads();
        if (lane == 0) S->warp[warp] = v;
        __syncthreads();
        u64 t = 0;
#pragma unroll 8
        for (int i = 0; i < NT / 32; i++) t = max(t, S->warp[i]);
        if (CL) {
            const int k = share(t);
            for (int r = 0; r < slices; r++) t = max(t, S->slices[k][r]);
        }
        return t;
    }
    // to[b] = the slices' from[b], added up: an equal part of them by each slice, for all.
    template <typename N> __device__ __forceinline__ void merge(const N *from, N *to, int n) const {
        sync();
        if (CL) {
            const int part = (n + slices - 1) / slices, b0 = rank * part;
            for (int b = b0 + tid; b < min(n, b0 + part); b += NT) {
                N v[kSrCluster], t = 0;
#pragma unroll
                for (int r = 0; r < kSrCluster; r++) v[r] = at_slice(from, min(r, slices - 1))[b];
#pragma unroll
                for (int r = 0; r < kSrCluster; r++) t += r < slices ? v[r] : 0;
#pragma unroll
                for (int r = 0; r < kSrCluster; r++)
                    if (r < slices) at_slice(to, r)[b] = t;
            }
        } else {
            for (int b = tid; b < n; b += NT) to[b] = from[b];
        }
        sync();
    }

    // f(four logits, index) of the slice's tokens of those groups that pass(maximum), 512 tokens a warp at
    // a time so that four loads are in flight; done(segment) after each segment's.  In the place of tokens
    // behind the slice's end, and of those of other groups, there is -infinity.  f's work has few
    // branches, so that the 16 tokens of a thread are worked on side by side.
    template <typename P, typename F, typename D> __device__ __forceinline__ void each(P pass, F f, D done) const {
        for (int s0 = i0 + warp * kSrSegment; s0 < i1; s0 += NT / 32 * kSrSegment) {
#pragma unroll 1
            for (int c = s0; c < min(i1, s0 + kSrSegment); c += 512) {
                bool mine[4];
                float4 v[4];
                bool any = false;
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const int i = c + 128 * q + 4 * lane;
                    mine[q] = i < i1 && pass(sr_value(gm[(i - i0) >> shift]));
                    any |= mine[q];
                }
                if (!__any_sync(0xffffffffu, any)) continue;
                if (wide && c + 512 <= i1) {
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        v[q] = mine[q] ? sr_wide4(x, c + 128 * q + 4 * lane) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; q++) v[q] = sr_load4(x, mine[q] ? c + 128 * q + 4 * lane : i1, i1, wide);
                }
#pragma unroll
                for (int q = 0; q < 4; q++) f(v[q], c + 128 * q + 4 * lane);
            }
            done((s0 - i0) / kSrSegment);
        }
    }
    __device__ __forceinline__ void append(u64 at) const {  // to the slice's list
        const int n = atomicAdd(&S->n, 1);
        if (n < kSrList) S->list[n] = at;
    }
    __device__ __forceinline__ float weight_at(u64 at) const { return fast_exp2(exponent(sr_value((uint32_t)(at >> 32)))); }
    // The slices' lists, one behind the other, to slice 0's; how many tokens they are (more than kSrList:
    // an overflow, and nothing is moved).
    __device__ __forceinline__ int gather() {
        __syncthreads();
        const int mine = S->n;
        if (!CL) return mine;
        const int k = share((u64)mine);
        int before = 0, all = 0;
        for (int r = 0; r < slices; r++) {
            if (r == rank) before = all;
            all += (int)S->slices[k][r];
        }
        if (all > kSrList) return all;
        if (rank > 0) {
            u64 *to = at_slice(S, 0)->list + before;
            for (int c = tid; c < mine; c += NT) to[c] = S->list[c];
        }
        sync();
        return all;
    }

    // Greedy: the first index with the largest logit.
    __device__ __forceinline__ void first_top() {
        const int n = groups();
        const uint32_t top = sr_key(vmax);
        u64 first = 0;  // complemented: larger is earlier
        for (int g = tid; g < n; g += NT)
            if (gm[g] == top) {
                first = 0xffffffffull - (uint32_t)g;
                break;
            }
        // the slice's first group, then its first token, then the first slice's
#pragma unroll
        for (int o = 16; o; o >>= 1) first = max(first, __shfl_xor_sync(0xffffffffu, first, o));
        __syncthreads();
        if (lane == 0) S->warp[warp] = first;
        __syncthreads();
        for (int w = 0; w < NT / 32; w++) first = max(first, S->warp[w]);
        u64 best = 0;
        if (first) {
            const int c = i0 + (int)((0xffffffffu - (uint32_t)first) << shift);
            for (int i = c + tid; i < min(i1, c + (1 << shift)); i += NT)
                if (sr_key(sr_load(x, i)) == top) best = max(best, 0xffffffffull - (uint32_t)i);
        }
        best = most_of(best);
        if (rank == 0 && tid == 0) *out = (int)(0xffffffffu - (uint32_t)best);
    }

    // 256 bins of equal width between the largest logit and the groups' smallest maximum; the bin that
    // the k-th largest of all maxima is in.
    __device__ __forceinline__ int kth_bin(int k, float low, float &width) {
        const int n = groups();
        const float range = vmax - low;
        width = range > 1e-30f ? 255.0f / range : 0.0f;
        for (int b = tid; b < 256; b += NT) S->hist[b] = 0;
        __syncthreads();
        for (int g = tid; g < n; g += NT) atomicAdd(&S->hist[bin_of_value(sr_value(gm[g]), width)], 1u);
        merge(S->hist, S->merged, 256);
        if (warp == 0) {  // lane l has bins 8 l to 8 l + 7
            int t = 0;
#pragma unroll
            for (int q = 0; q < 8; q++) t += (int)S->merged[8 * lane + q];
            int a = (int)warp_scan((u64)t, lane) - t;
            if (a < k && k <= a + t) {
                int b = 8 * lane;
                while ((a += (int)S->merged[b]) < k) b++;
                S->lo = b;
            }
        }
        __syncthreads();
        return S->lo;
    }
    __device__ __forceinline__ int bin_of_value(float v, float width) const {
        return (int)fminf((vmax - v) * width, 255.0f);
    }

    // The list of the tokens in the bins up to `last`.  Groups that hold some are put in a queue first, so
    // that the loads of all of them are in flight together.
    __device__ __forceinline__ void list_bins(float width, int last) const {
        const int n = groups();
        if (tid == 0) S->hi = 0;  // (S->lo may still be read: kth_bin)
        __syncthreads();
        for (int g = tid; g < n; g += NT) {
            const float v = sr_value(gm[g]);
            if (v > -INFINITY && bin_of_value(v, width) <= last) {
                const int at = atomicAdd(&S->hi, 1);
                if (at < kSrList) S->queue[at] = (uint32_t)g;
            }
        }
        __syncthreads();
        const int queued = S->hi;
        auto list = [&](float4 v, int i) {
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const float f = q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w;
                // tokens of -infinity have no weight and come last in the order: never listed
                if (f > -INFINITY && bin_of_value(f, width) <= last) append(place(sr_key(f), i + q));
            }
        };
        if (queued > kSrList) {
            each([&](float g) { return g > -INFINITY && bin_of_value(g, width) <= last; }, list, [](int) {});
            return;
        }
        const int quads = queued << (shift - 2);  // of four tokens
        for (int c = tid; c < quads; c += NT) {
            const int i = i0 + (int)(S->queue[c >> (shift - 2)] << shift) + 4 * (c & ((1 << (shift - 2)) - 1));
            if (i < i1) list(sr_load4(x, i, i1, wide), i);
        }
    }

    static __device__ __forceinline__ u64 target_of(float u, u64 M) {
        u = u >= 0.f ? fminf(u, 1.0f) : 0.f;
        return min((u64)((double)u * (double)M), M - 1);
    }
    static __device__ __forceinline__ u64 share_of(float p, u64 M) {  // p M, at least 1
        return max((u64)1, (u64)ceil((double)fmaxf(p, 0.0f) * (double)M));
    }

    // By slice 0: the list's tokens after top-k (k = 0: all of them), top-p and min-p; the draw.  The
    // list holds the first k tokens of the row at least.
    __device__ __forceinline__ void draw_list(int n, int k, float p, float u) const {
        sort(S->list, n);
        // every cut keeps a prefix: adjacent tokens a thread, and the sum before each
        const int per = (n + NT - 1) / NT, c0 = min(n, tid * per), c1 = min(k > 0 ? min(n, k) : n, c0 + per);
        u64 mass = 0, M;
        for (int c = c0; c < c1; c++) mass += whole(weight_at(S->list[c]));
        u64 before = scan(mass, M) - mass;
        const u64 want = p < 1.0f ? share_of(p, M) : ~0ull;
        u64 left = 0;
        for (int c = c0; c < c1; c++) {
            const float w = weight_at(S->list[c]);
            left += before < want && !(w < minp);
            before += whole(w);
        }
        const int m = (int)cta_total(left);
        for (int c = tid; c < m; c += NT) S->sorted[c] = S->list[c] << 32 | (uint32_t)c;  // complemented index first
        __syncthreads();
        sort(S->sorted, m);
        const int share = (m + NT - 1) / NT, d0 = min(m, tid * share), d1 = min(m, d0 + share);
        mass = 0;
        for (int d = d0; d < d1; d++) mass += whole(weight_at(S->list[(uint32_t)S->sorted[d]]));
        const u64 upto = scan(mass, M), target = target_of(u, M);
        if (upto > target && upto - mass <= target) {
            u64 a = upto - mass;
            for (int d = d0; d < d1; d++) {
                const u64 at = S->list[(uint32_t)S->sorted[d]];
                a += whole(weight_at(at));
                if (a > target) {
                    *out = (int)(0xffffffffu - (uint32_t)at);
                    break;
                }
            }
        }
    }
    // a[0 .. n) in order, the largest first (a bitonic network over the next power of two, at least 64;
    // the places behind n become 0).  Exchanges of up to 32 places apart stay within a warp's 64 values,
    // two a lane.
    __device__ __forceinline__ void sort(u64 *a, int n) const {
        int m = 64;
        while (m < n) m <<= 1;
        for (int c = n + tid; c < m; c += NT) a[c] = 0;
        __syncthreads();
        auto within = [&](int c, int size, u64 &x, u64 &y) {  // exchanges 32 to 1 apart of the network's `size`
#pragma unroll
            for (int stride = 32; stride > 0; stride >>= 1) {
                if (stride >= size) continue;
                if (stride == 32) {
                    const u64 hi = max(x, y), lo = min(x, y);
                    const bool down = (c & size) == 0;
                    x = down ? hi : lo;
                    y = down ? lo : hi;
                } else {
                    const u64 u = __shfl_xor_sync(0xffffffffu, x, stride), v = __shfl_xor_sync(0xffffffffu, y, stride);
                    const bool first = (lane & stride) == 0;
                    x = first == (((c + lane) & size) == 0) ? max(x, u) : min(x, u);
                    y = first == (((c + 32 + lane) & size) == 0) ? max(y, v) : min(y, v);
                }
            }
        };
        for (int c = 64 * warp; c < m; c += 64 * (NT / 32)) {
            u64 x = a[c + lane], y = a[c + 32 + lane];
#pragma unroll
            for (int size = 2; size <= 64; size <<= 1) within(c, size, x, y);
            a[c + lane] = x;
            a[c + 32 + lane] = y;
        }
        __syncthreads();
        for (int size = 128; size <= m; size <<= 1) {
            for (int stride = size >> 1; stride >= 64; stride >>= 1) {
                for (int i = tid; i < m / 2; i += NT) {
                    const int c = 2 * i - (i & (stride - 1));
                    const u64 x = a[c], y = a[c + stride];
                    if ((x < y) == ((c & size) == 0)) {
                        a[c] = y;
                        a[c + stride] = x;
                    }
                }
                __syncthreads();
            }
            for (int c = 64 * warp; c < m; c += 64 * (NT / 32)) {
                u64 x = a[c + lane], y = a[c + 32 + lane];
                within(c, size, x, y);
                a[c + lane] = x;
                a[c + 32 + lane] = y;
            }
            __syncthreads();
        }
    }

    // The draw from the tokens from `least` on, by the segments' sums.
    __device__ __forceinline__ void draw_segments(u64 least, float u) {
        const int n = (i1 - i0 + kSrSegment - 1) / kSrSegment, per = (n + NT - 1) / NT;
        const int s0 = min(n, tid * per), s1 = min(n, s0 + per);
        u64 mine = 0, M, base = 0;
        for (int s = s0; s < s1; s++) mine += seg[s];
        u64 upto = scan(mine, M);
        if (CL) {
            const int k = share(M);
            M = 0;
            for (int r = 0; r < slices; r++) {
                if (r == rank) base = M;
                M += S->slices[k][r];
            }
        }
        const u64 target = target_of(u, M);
        if (tid == 0) S->lo = -1;
        __syncthreads();
        upto += base;
        if (upto > target && upto - mine <= target) {
            u64 a = upto - mine;
            int s = s0;
            while (a + seg[s] <= target) a += seg[s++];
            S->lo = s;
            S->found[0] = a;
        }
        __syncthreads();
        if (warp > 0 || S->lo < 0) return;
        u64 a = S->found[0];
        const int c0 = i0 + S->lo * kSrSegment;
        for (int c = c0; c < min(i1, c0 + kSrSegment); c += 128) {
            const int i = c + 4 * lane;
            const float4 v = sr_load4(x, i, i1, wide);
            const float f[4] = {v.x, v.y, v.z, v.w};
            u64 w[4], sum = 0;
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const float r = fast_exp2(exponent(f[q]));
                w[q] = i + q < i1 && place(sr_key(f[q]), i + q) >= least && !(r < minp) ? whole(r) : 0;
                sum += w[q];
            }
            const u64 to = a + warp_scan(sum, lane);
            const bool here = to > target && to - sum <= target;
            if (here) {
                u64 b = to - sum;
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    if (b <= target && b + w[q] > target) *out = i + q;
                    b += w[q];
                }
            }
            if (__any_sync(0xffffffffu, here)) break;
            a = __shfl_sync(0xffffffffu, to, 31);
        }
    }

    // Sums of the segments, min-p applied.
    __device__ __forceinline__ void sum_segments() const {
        SrSum sum;
        each([&](float m) {
                 const float e = exponent(m);
                 return e > -42.0f && !(fast_exp2(e) < minp);
             },
             [&](float4 v, int) {
#pragma unroll
                 for (int q = 0; q < 4; q++) {
                     const float w = fast_exp2(exponent(q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w));
                     sum.add(w < minp ? 0.0f : w);
                 }
             },
             [&](int s) {
                 const u64 t = warp_total(sum.flush());
                 if (lane == 0) seg[s] = t;
                 sum.sum = 0;
             });
        __syncthreads();
    }

    // The bin of a weight's exponent: the nearest whole number to -32 e.
    static __device__ __forceinline__ int bin_of(float e) {
        return (int)(__float_as_uint(fmaf(e, -32.0f, 12582912.0f)) - 0x4b400000u);
    }

    // The place in the order of the last token of the shortest prefix that reaches p of the whole mass,
    // and the sums of the segments over that prefix (min-p applied to them).  false: the list overflowed.
    __device__ __forceinline__ bool nucleus(float p, u64 &least) {
        // bits of a weight in the histogram: 13, less where a bin of the whole vocabulary could overflow
        int bits = 13;
        for (int v = V; v > (1 << 18); v >>= 1) bits--;
        for (int b = tid; b < kSrBins; b += NT) S->hist[b] = 0;
        if (tid == 0) S->n = 0;
        __syncthreads();
        SrSum mass;
        each([&](float m) { return exponent(m) > -42.0f; },
             [&](float4 v, int) {
                 int b[4];
                 uint32_t t[4];
                 bool some[4];
#pragma unroll
                 for (int q = 0; q < 4; q++) {
                     const float e = exponent(q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w), w = fast_exp2(e);
                     some[q] = e > -41.0f;
                     mass.add(some[q] ? w : 0.0f);
                     b[q] = bin_of(e);  // w 2^floor(b / 32) is between 2^-1.01 and 2^0.02
                     t[q] = __float2uint_rz(__uint_as_float(__float_as_uint(w) + ((uint32_t)(bits + (b[q] >> 5)) << 23)));
                 }
#pragma unroll
                 for (int q = 0; q < 4; q++)
                     if (some[q]) atomicAdd(&S->hist[b[q]], t[q]);
                 mass.flush();
             },
             [](int) {});
        merge(S->hist, S->merged, kSrBins);
        const u64 M = total_of(mass.sum), want = share_of(p, M);
        // Cutting took less than 2^(2 - bits) of every weight, and the whole numbers of 2^-40 have half of
        // one a token besides.  Adjacent bins a thread: the first of all that may reach the share, and the
        // first that must.
        if (tid == 0) S->lo = S->hi = kSrBins - 1;
        constexpr int B = (kSrBins + NT - 1) / NT;
        u64 a[B], t = 0, all;
#pragma unroll
        for (int q = 0; q < B; q++) {
            const int b = B * tid + q, sh = 40 - bits - (b >> 5);
            const u64 h = b < kSrBins ? S->merged[b] : 0;
            a[q] = sh >= 0 ? h << sh : h >> -sh;
            t += a[q];
        }
        u64 c = scan(t, all) - t;
        bool may = false, must = false;
#pragma unroll
        for (int q = 0; q < B; q++) {
            c += a[q];
            if (!may && c + (c >> (bits - 2)) + (u64)V >= want) {
                atomicMin(&S->lo, B * tid + q);
                may = true;
            }
            if (!must && c >= want + (u64)V) {
                atomicMin(&S->hi, B * tid + q);
                must = true;
            }
        }
        __syncthreads();
        const int b1 = S->lo, b2 = S->hi;
        u64 above = 0;
        SrSum sum, cut_off;  // what min-p leaves, and takes, above the list
        each([&](float m) { return exponent(m) > -42.0f && bin_of(exponent(m)) <= b2; },
             [&](float4 v, int i) {
                 bool in_list[4], any = false;
#pragma unroll
                 for (int q = 0; q < 4; q++) {
                     const float e = exponent(q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w), w = fast_exp2(e);
                     const int b = bin_of(e);
                     const bool up = b < b1;
                     sum.add(up && !(w < minp) ? w : 0.0f);
                     if (minp > 0.0f) cut_off.add(up && w < minp ? w : 0.0f);
                     any |= in_list[q] = !up && b <= b2 && e > -41.0f;
                 }
                 if (any) {
#pragma unroll
                     for (int q = 0; q < 4; q++)
                         if (in_list[q]) append(place(sr_key(q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w), i + q));
                 }
             },
             [&](int s) {
                 const u64 mine = sum.flush();
                 above += mine + cut_off.flush();
                 cut_off.sum = 0;
                 const u64 t = warp_total(mine);
                 if (lane == 0) seg[s] = t;
                 sum.sum = 0;
             });
        above = total_of(above);
        const int n = gather();
        if (n > kSrList) return false;
        if (rank == 0) last_of_list(n, want - above);
        sync();
        least = S->found[1];
        return true;
    }

    // By slice 0: the list's tokens up to the one that reaches `rest`, which all slices are told, added to
    // their segments.  Rounds of 256 bins of their keys, each within the bin that the last one found,
    // until few tokens are left in it.
    __device__ __forceinline__ void last_of_list(int n, u64 rest) {
        uint32_t from = 0xffffffffu, to = 0;
        for (int c = tid; c < n; c += NT) {
            const uint32_t key = (uint32_t)(S->list[c] >> 32);
            from = min(from, key);
            to = max(to, key);
        }
        from = __reduce_min_sync(0xffffffffu, from);
        to = __reduce_max_sync(0xffffffffu, to);
        __syncthreads();
        if (lane == 0) S->warp[warp] = (u64)from << 32 | to;
        __syncthreads();
        for (int w = 0; w < NT / 32; w++) {
            from = min(from, (uint32_t)(S->warp[w] >> 32));
            to = max(to, (uint32_t)S->warp[w]);
        }
        int left = n;
        while (left > 64 && from < to) {
            const int sh = max(0, 24 - __clz(to - from));
            for (int b = tid; b < 256; b += NT) {
                S->bins[b] = 0;
                S->hist[b] = 0;
            }
            __syncthreads();
            for (int c = tid; c < n; c += NT) {
                const uint32_t key = (uint32_t)(S->list[c] >> 32);
                if (key < from || key > to) continue;
                atomicAdd(&S->bins[(key - from) >> sh], whole(fast_exp2(exponent(sr_value(key)))));
                atomicAdd(&S->hist[(key - from) >> sh], 1u);
            }
            __syncthreads();
            if (warp == 0) top_bin(S->bins, rest);
            __syncthreads();
            rest -= S->found[0];
            left = (int)S->hist[S->lo];
            from += (uint32_t)S->lo << sh;
            to = min(to, from + ((1u << sh) - 1));
            __syncthreads();
        }
        // the last one: the tokens before it within [from, to] do not reach `rest`, with it they do
        if (tid == 0) S->n = 0;
        __syncthreads();
        for (int c = tid; c < n; c += NT) {
            const uint32_t key = (uint32_t)(S->list[c] >> 32);
            if (key >= from && key <= to) S->sorted[atomicAdd(&S->n, 1)] = S->list[c];
        }
        __syncthreads();
        left = S->n;
        for (int c = tid; c < left; c += NT) {
            const u64 at = S->sorted[c];
            u64 before = 0;
            for (int j = 0; j < left; j++) {
                const u64 o = S->sorted[j];
                if (o > at) before += whole(weight_at(o));
            }
            if (before < rest && before + whole(weight_at(at)) >= rest)
                for (int r = 0; r < slices; r++) at_slice(S, r)->found[1] = at;
        }
        __syncthreads();
        const u64 least = S->found[1];
        const int len = i1 - i0;  // of slice 0, so of all but the last
        for (int c = tid; c < n; c += NT) {
            const u64 at = S->list[c];
            const float w = weight_at(at);
            if (at < least || w < minp) continue;
            const int i = (int)(0xffffffffu - (uint32_t)at), r = CL ? i / len : 0;
            atomicAdd(&at_slice(seg, r)[(i - r * len) / kSrSegment], whole(w));
        }
    }

    // By one warp: the first bin from the top at which the sum of a[0 .. 255] reaches `want` (S->lo), and
    // the sum above it (S->found[0]).
    __device__ __forceinline__ void top_bin(const u64 *a, u64 want) const {
        u64 t = 0;
#pragma unroll
        for (int q = 0; q < 8; q++) t += a[255 - 8 * lane - q];
        const u64 upto = warp_scan(t, lane);
        if (upto >= want && upto - t < want) {
            u64 c = upto - t;
            int b = 255 - 8 * lane;
            while (c + a[b] < want) c += a[b--];
            S->lo = b;
            S->found[0] = c;
        }
    }

    // The general way: weights of keys, with every infinity in its place.
    __device__ __forceinline__ float any_weight(float v) const {
        const float d = fmaxf(v, -INFINITY) - vmax;
        return fmaxf(v, -INFINITY) == vmax ? 1.0f : d == -INFINITY ? 0.0f : fast_exp2(d * scale);
    }
    // `least` moved up to the shortest prefix of what it keeps with a sum of at least `want` of
    // amount(logit), a byte at a time.
    template <typename A> __device__ __forceinline__ void cut(u64 &least, u64 want, A amount) const {
        u64 prefix = 0, mask = 0;
        for (int d = 56; d >= 0; d -= 8) {
            for (int b = tid; b < 256; b += NT) S->bins[b] = 0;
            __syncthreads();
            for (int i = i0 + tid; i < i1; i += NT) {
                const float v = sr_load(x, i);
                const u64 at = place(sr_key(v), i);
                if ((at & mask) == prefix && at >= least) atomicAdd(&S->bins[at >> d & 255u], amount(v));
            }
            merge(S->bins, S->sums, 256);
            if (warp == 0) top_bin(S->sums, want);
            __syncthreads();
            prefix |= (u64)S->lo << d;
            mask |= (u64)255 << d;
            want -= S->found[0];
            __syncthreads();
        }
        least = prefix;
    }
    __device__ __forceinline__ void general(int k, float p, float u) {
        u64 least = 0;
        if (k > 0) cut(least, (u64)k, [](float) { return (u64)1; });
        if (p < 1.0f) {
            u64 mass = 0;
            for (int i = i0 + tid; i < i1; i += NT) {
                const float v = sr_load(x, i);
                if (place(sr_key(v), i) >= least) mass += whole(any_weight(v));
            }
            const u64 M = total_of(mass);
            cut(least, share_of(p, M), [&](float v) { return whole(any_weight(v)); });
        }
        // The draw, token by token: a thread's are adjacent.
        const int per = (i1 - i0 + NT - 1) / NT, lo = min(i1, i0 + tid * per), hi = min(i1, lo + per);
        auto weight = [&](int i) {
            const float v = sr_load(x, i), w = any_weight(v);
            return place(sr_key(v), i) >= least && !(w < minp) ? whole(w) : 0;
        };
        u64 mine = 0, M, base = 0;
        for (int i = lo; i < hi; i++) mine += weight(i);
        u64 upto = scan(mine, M);
        if (CL) {
            const int q = share(M);
            M = 0;
            for (int r = 0; r < slices; r++) {
                if (r == rank) base = M;
                M += S->slices[q][r];
            }
        }
        upto += base;
        const u64 target = target_of(u, M);
        if (upto > target && upto - mine <= target) {
            u64 a = upto - mine;
            for (int i = lo; i < hi; i++) {
                a += weight(i);
                if (a > target) {
                    *out = i;
                    break;
                }
            }
        }
    }
};

// Apart from the kernel, whose registers its loops would take.
template <typename R> __device__ __noinline__ void sample_general(R row, int k, float p, float u) { row.general(k, p, u); }

template <typename T, bool CL>
__global__ void __launch_bounds__(kSrThreads, kSrResident) sample_rows_kernel(const __grid_constant__ SampleRowsArgs A, int slices, int shift) {
    constexpr int NT = kSrThreads;
    extern __shared__ __align__(16) uint8_t smem[];
    SrRow<T, CL> R;
    R.V = A.vocab;
    R.slices = CL ? slices : 1;
    R.rank = CL ? blockIdx.x % slices : 0;
    // slices are whole segments, the last ones may be shorter or empty
    const int len = (A.vocab + R.slices * kSrSegment - 1) / (R.slices * kSrSegment) * kSrSegment;
    R.i0 = min(A.vocab, R.rank * len);
    R.i1 = min(A.vocab, R.i0 + len);
    R.shift = shift;
    R.S = (SrShared *)smem;
    R.seg = (u64 *)(R.S + 1);
    R.gm = (uint32_t *)(R.seg + len / kSrSegment);
    R.tid = threadIdx.x;
    R.lane = R.tid & 31;
    R.warp = R.tid >> 5;
    R.set = 0;
    R.wide = ((uintptr_t)A.logits | (uintptr_t)(A.ld * (long long)sizeof(T))) % (4 * sizeof(T)) == 0;
    SrShared *S = R.S;
    const int V = A.vocab, tid = R.tid, lane = R.lane;
    pdl_wait();
    pdl_trigger();
    const int step = gridDim.x / R.slices;
    for (long long row = blockIdx.x / R.slices; row < A.rows; row += step) {
        R.x = (const T *)A.logits + row * A.ld;
        R.out = A.next_ids + row;
        const float temp = A.temperature ? __ldg(A.temperature + row) : 1.0f;
        int k = A.top_k ? __ldg(A.top_k + row) : 0;
        k = k > 0 && k < V ? k : 0;
        const float p = A.top_p ? __ldg(A.top_p + row) : 1.0f, u = __ldg(A.uniforms + row);
        const float m = A.min_p ? __ldg(A.min_p + row) : 0.0f;
        R.minp = m > 0.f ? fminf(m, 1.0f) : 0.0f;
        R.sync();  // the last row is done with the shared memory
        if (shift > 4) {
            for (int g = tid; g < R.groups(); g += NT) R.gm[g] = 0;
            __syncthreads();
        }
        // the largest logit of every 16 tokens (four lanes), four loads in flight
        float most = -INFINITY;
        uint32_t least = 0xffffffffu;  // key of the smallest maximum that is a number
        for (int c = R.i0 + R.warp * 512; c < R.i1; c += NT / 32 * 512) {
            float4 v[4];
            if (R.wide && c + 512 <= R.i1) {
#pragma unroll
                for (int q = 0; q < 4; q++) v[q] = sr_wide4(R.x, c + 128 * q + 4 * lane);
            } else {
#pragma unroll
                for (int q = 0; q < 4; q++) v[q] = sr_load4(R.x, c + 128 * q + 4 * lane, R.i1, R.wide);
            }
#pragma unroll
            for (int q = 0; q < 4; q++) {
                float g = fmaxf(fmaxf(v[q].x, v[q].y), fmaxf(v[q].z, v[q].w));
                g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 1));
                g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 2));
                most = fmaxf(most, g);
                if (g > -INFINITY) least = min(least, sr_key(g));
                const int i = c + 128 * q + 4 * lane;
                if ((lane & 3) == 0 && i < R.i1) {
                    if (shift == 4)
                        R.gm[(i - R.i0) >> 4] = sr_key(g);
                    else
                        atomicMax(&R.gm[(i - R.i0) >> shift], sr_key(g));
                }
            }
        }
        if (tid == 0) S->n = 0;
        const u64 ends = R.both_most_of((u64)sr_key(most) << 32 | (0xffffffffu - least));
        R.vmax = sr_value((uint32_t)(ends >> 32));
        const float low = sr_value(0xffffffffu - (uint32_t)ends);
        if (R.vmax == -INFINITY) {
            if (R.rank == 0 && tid == 0) *R.out = 0;
            continue;
        }
        if (!(temp > 0.f) || k == 1) {
            R.first_top();
            continue;
        }
        R.scale = fminf(1.4426950408889634f / temp, FLT_MAX);
        if (R.vmax < INFINITY) {
            if (V <= kSrList / 2 || (k > 0 && k <= min((V + (1 << shift) - 1) >> shift, kSrList / 2))) {
                float width = 0.0f;
                const int last = V <= kSrList / 2 ? 255 : R.kth_bin(k, low, width);
                R.list_bins(width, last);
                const int n = R.gather();
                if (n <= kSrList) {
                    if (R.rank == 0) R.draw_list(n, k, p, u);
                    continue;
                }
            } else if (k == 0 && p < 1.0f) {
                u64 least;
                if (R.nucleus(p, least)) {
                    R.draw_segments(least, u);
                    continue;
                }
            } else if (k == 0) {
                R.sum_segments();
                R.draw_segments(0, u);
                continue;
            }
        }
        sample_general(R, k, p, u);
        R.set = 0;
    }
    R.sync();  // nobody leaves while another slice may still look into its shared memory
}

template <typename T, bool CL> static cudaError_t launch_sample(const SampleRowsArgs &a, int slices, cudaStream_t s) {
    const int len = (a.vocab + slices * kSrSegment - 1) / (slices * kSrSegment) * kSrSegment;
    int shift = 4;
    while (((len - 1) >> shift) + 1 > kSrGroups) shift++;
    const size_t smem = sizeof(SrShared) + (size_t)(len / kSrSegment) * 8 + (size_t)(((len - 1) >> shift) + 1) * 4;
    const cudaError_t e = allow_smem((const void *)sample_rows_kernel<T, CL>);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(std::min(a.rows, 1 << 20) * slices);
    cfg.blockDim = dim3(kSrThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2]{};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = slices;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = CL ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, sample_rows_kernel<T, CL>, a, slices, shift);
}

cudaError_t sample_rows_launch(const SampleRowsArgs &a, bool bf16, int sms, cudaStream_t s) {
    // Slices of 16,384 tokens and more: what an SM has to do is then cut finely enough to be even, and rows
    // that wait for memory run beside rows that do not.  Of 4,096 and more while there is room for all rows.
    int slices = 1;
    while (slices < kSrCluster &&
           (a.vocab / (2 * slices) >= 16384 ||
            (a.vocab / (2 * slices) >= 4096 && (long long)a.rows * 2 * slices <= kSrResident * sms)))
        slices *= 2;
    if (slices > 1) return bf16 ? launch_sample<uint16_t, true>(a, slices, s) : launch_sample<float, true>(a, slices, s);
    return bf16 ? launch_sample<uint16_t, false>(a, 1, s) : launch_sample<float, false>(a, 1, s);
}

}  // namespace slm
