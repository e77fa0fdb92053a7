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
// HBM bounds a batch: its logits are read once.  A CTA has a row, and reads it for the largest logit of
// every group of 16 tokens; the other steps read only groups that can matter, from the L2:
//   greedy        the first group with the largest logit;
//   top-k         groups whose maximum is among the k largest (at least k tokens are no smaller than the
//                 k-th largest maximum, and hardly more): their tokens make a list, and each token of it
//                 finds its rank and the sum before it by looking at the others;
//   top-p alone   a histogram of the weights, 8 bins an octave, in cut whole numbers, says in which bin
//                 (or two) the sum is reached; the sum above it is then exact, the bin's tokens make a
//                 list, and a few rounds of 256 bins find the last one of them to be kept;
//   the draw      the sum of every 1,024 tokens, the segment that holds the target, its tokens.
// A list that overflows (a top-k of a good part of the vocabulary, thousands of equal logits next to the
// border) leaves the row to the general way: a threshold by its four bytes in turn, over all tokens.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "device_common.cuh"
#include "rows.cuh"

namespace slm {

typedef unsigned long long u64;
constexpr int kSrList = 2048;    // tokens of a list
constexpr int kSrGroups = 16384; // groups of a row at most
constexpr int kSrBins = 352;     // 44 octaves of 8 bins: weights of 2^-41 and less are 0
constexpr int kSrSegment = 1024;

// Monotone map of a float to an unsigned key; NaN goes where -infinity is, and -0 where 0.
__device__ __forceinline__ uint32_t sr_key(float f) {
    const uint32_t b = __float_as_uint(fmaxf(f, -INFINITY) + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float sr_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// Four consecutive logits from i on; -infinity behind the row.  `wide`: rows begin on boundaries of four
// elements.
__device__ __forceinline__ float4 sr_load4(const float *x, int i, int V, bool wide) {
    if (wide && i + 3 < V) return __ldg((const float4 *)(x + i));
    float4 v;
    v.x = i < V ? __ldg(x + i) : -INFINITY;
    v.y = i + 1 < V ? __ldg(x + i + 1) : -INFINITY;
    v.z = i + 2 < V ? __ldg(x + i + 2) : -INFINITY;
    v.w = i + 3 < V ? __ldg(x + i + 3) : -INFINITY;
    return v;
}
__device__ __forceinline__ float4 sr_load4(const uint16_t *x, int i, int V, bool wide) {
    if (wide && i + 3 < V) {
        const uint2 w = __ldg((const uint2 *)(x + i));
        return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
    }
    auto at = [&](int j) { return j < V ? __uint_as_float((uint32_t)__ldg(x + j) << 16) : -INFINITY; };
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

struct SrToken {
    u64 at, w;  // place in the order; weight
};

// What a row's CTA shares.
struct SrShared {
    u64 warp[32], bins[256], found[2];
    uint32_t hist[kSrBins];
    int n, id, lo, hi;
    uint32_t kmin, kmax;
    SrToken list[kSrList];
};

template <typename T, int NT> struct SrRow {
    const T *x;
    int V, shift;      // tokens of a group: 2^shift
    bool wide;
    uint32_t *gm;      // [groups] keys of the maxima
    u64 *seg;          // [segments] sums
    SrShared *S;
    int tid, lane, warp;
    uint32_t top;      // key of the largest logit
    float vmax, scale; // it, and log2(e) / T
    float minp;

    __device__ __forceinline__ float exponent(uint32_t key) const {  // log2 of the weight
        const float d = sr_value(key) - vmax;
        return key == top ? 0.0f : d == -INFINITY ? -INFINITY : d * scale;
    }
    static __device__ __forceinline__ u64 whole(float w) { return (u64)__float2ull_rn(w * 1099511627776.0f); }
    __device__ __forceinline__ int groups() const { return (V + (1 << shift) - 1) >> shift; }
    static __device__ __forceinline__ u64 place(uint32_t key, int i) { return (u64)key << 32 | (0xffffffffu - (uint32_t)i); }

    // Inclusive running sum over the CTA, in order of the threads; the whole sum in warp[NT / 32 - 1].
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
    __device__ __forceinline__ u64 total_of(u64 v) const {
        v = warp_total(v);
        __syncthreads();
        if (lane == 0) S->warp[warp] = v;
        __syncthreads();
        u64 t = 0;
#pragma unroll 8
        for (int i = 0; i < NT / 32; i++) t += S->warp[i];
        return t;
    }

    // f(key, index) of the tokens of those groups that pass(maximum's key), 128 tokens a warp at a time;
    // done() after each segment's, if any.
    template <typename P, typename F, typename D> __device__ __forceinline__ void each(P pass, F f, D done) const {
        for (int s0 = warp * kSrSegment; s0 < V; s0 += NT / 32 * kSrSegment) {
#pragma unroll 2
            for (int c = s0; c < min(V, s0 + kSrSegment); c += 128) {
                const int i = c + 4 * lane;
                const bool mine = i < V && pass(gm[i >> shift]);
                if (!__any_sync(0xffffffffu, mine)) continue;
                if (mine) {
                    const float4 v = sr_load4(x, i, V, wide);
                    f(sr_key(v.x), i);
                    f(sr_key(v.y), i + 1);
                    f(sr_key(v.z), i + 2);
                    f(sr_key(v.w), i + 3);
                }
            }
            done(s0 / kSrSegment);
        }
    }
    __device__ __forceinline__ void append(u64 at, u64 w) const {
        const int n = atomicAdd(&S->n, 1);
        if (n < kSrList) S->list[n] = SrToken{at, w};
    }

    // The first index with the key `top`.
    __device__ __forceinline__ int first_top() const {
        if (tid == 0) S->id = V;
        __syncthreads();
        const int n = groups();
        int g = 0x7fffffff;
        for (int i = tid; i < n; i += NT)
            if (gm[i] == top) {
                g = i;
                break;
            }
        g = (int)__reduce_min_sync(0xffffffffu, (unsigned)g);
        if (lane == 0 && g < n) atomicMin(&S->id, g);
        __syncthreads();
        g = S->id;
        __syncthreads();
        if (tid == 0) S->id = V;
        __syncthreads();
        for (int i = (g << shift) + tid; i < min(V, (g + 1) << shift); i += NT)
            if (sr_key(sr_load(x, i)) == top) atomicMin(&S->id, i);
        __syncthreads();
        return S->id;
    }

    // A key that at least k of the groups' maxima reach, and not many more.
    __device__ __forceinline__ uint32_t kth_maximum(int k) const {
        const int n = groups();
        uint32_t prefix = 0, mask = 0;
        int above = 0;
        for (int d = 24; d >= 0; d -= 8) {
            for (int b = tid; b < 256; b += NT) S->hist[b] = 0;
            __syncthreads();
            for (int i = tid; i < n; i += NT)
                if ((gm[i] & mask) == prefix) atomicAdd(&S->hist[gm[i] >> d & 255u], 1u);
            __syncthreads();
            if (warp == 0) {  // lane l has bins 255 - 8 l down to 248 - 8 l
                int t = 0;
#pragma unroll
                for (int q = 0; q < 8; q++) t += (int)S->hist[255 - 8 * lane - q];
                const int upto = (int)warp_scan((u64)t, lane);
                int a = above + upto - t;
                if (a < k && k <= a + t) {
                    int q = 0;
                    while (q < 7 && a + (int)S->hist[255 - 8 * lane - q] < k) a += (int)S->hist[255 - 8 * lane - q++];
                    S->lo = 255 - 8 * lane - q;
                    S->hi = a;
                }
            }
            __syncthreads();
            prefix |= (uint32_t)S->lo << d;
            mask |= 255u << d;
            above = S->hi;
            const int reach = above + (int)S->hist[S->lo];
            __syncthreads();
            if (reach <= k + k / 8 + 16) break;
        }
        return prefix;
    }

    // The list's tokens after top-k (k = 0: all of them), top-p and min-p; the draw.  The list holds the
    // first k tokens of the row at least.
    __device__ __forceinline__ int draw_list(int n, int k, float p, float u) const {
        constexpr int E = kSrList / NT;
        u64 before[E], w[E], at[E], mass = 0;
        bool in[E];
#pragma unroll
        for (int e = 0; e < E; e++) {
            const int c = tid + e * NT;
            in[e] = false;
            if (c < n) {
                at[e] = S->list[c].at;
                w[e] = S->list[c].w;
                before[e] = 0;
                int rank = 0;
#pragma unroll 4
                for (int j = 0; j < n; j++)
                    if (S->list[j].at > at[e]) {
                        rank++;
                        before[e] += S->list[j].w;
                    }
                in[e] = k == 0 || rank < k;
                if (in[e]) mass += w[e];
            }
        }
        u64 M = total_of(mass);
        const u64 want = p < 1.0f ? max((u64)1, (u64)ceil((double)fmaxf(p, 0.0f) * (double)M)) : ~0ull;
        mass = 0;
#pragma unroll
        for (int e = 0; e < E; e++) {
            const int c = tid + e * NT;
            if (c >= n) continue;
            const uint32_t key = (uint32_t)(at[e] >> 32);
            in[e] = in[e] && before[e] < want && !(exp2f(exponent(key)) < minp);
            if (!in[e]) S->list[c].w = w[e] = 0;
            mass += w[e];
        }
        M = total_of(mass);  // (its barriers order the list too)
        const u64 target = target_of(u, M);
#pragma unroll
        for (int e = 0; e < E; e++) {
            const int c = tid + e * NT;
            if (c >= n || w[e] == 0) continue;
            const uint32_t idx = (uint32_t)at[e];  // complemented: larger is earlier
            u64 upto = 0;
#pragma unroll 4
            for (int j = 0; j < n; j++)
                if ((uint32_t)S->list[j].at >= idx) upto += S->list[j].w;
            if (upto > target && upto - w[e] <= target) S->id = (int)(0xffffffffu - idx);
        }
        __syncthreads();
        return S->id;
    }

    static __device__ __forceinline__ u64 target_of(float u, u64 M) {
        u = u >= 0.f ? fminf(u, 1.0f) : 0.f;
        return min((u64)((double)u * (double)M), M - 1);
    }

    // The draw from the tokens from `least` on, by the segments' sums.
    __device__ __forceinline__ int draw_segments(u64 least, float u) const {
        const int n = (V + kSrSegment - 1) / kSrSegment, per = (n + NT - 1) / NT;
        const int s0 = min(n, tid * per), s1 = min(n, s0 + per);
        u64 mine = 0, M;
        for (int s = s0; s < s1; s++) mine += seg[s];
        const u64 upto = scan(mine, M);
        const u64 target = target_of(u, M);
        if (upto > target && upto - mine <= target) {
            u64 a = upto - mine;
            int s = s0;
            while (a + seg[s] <= target) a += seg[s++];
            S->lo = s;
            S->found[0] = a;
        }
        __syncthreads();
        if (warp == 0) {
            u64 a = S->found[0];
            const int c0 = S->lo * kSrSegment;
            for (int c = c0; c < min(V, c0 + kSrSegment); c += 128) {
                const int i = c + 4 * lane;
                const float4 v = sr_load4(x, i, V, wide);
                const float f[4] = {v.x, v.y, v.z, v.w};
                u64 w[4], sum = 0;
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const uint32_t key = sr_key(f[q]);
                    const float r = exp2f(exponent(key));
                    w[q] = i + q < V && place(key, i + q) >= least && !(r < minp) ? whole(r) : 0;
                    sum += w[q];
                }
                const u64 upto = a + warp_scan(sum, lane);
                const bool here = upto > target && upto - sum <= target;
                if (here) {
                    u64 b = upto - sum;
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        if (b <= target && b + w[q] > target) S->id = i + q;
                        b += w[q];
                    }
                }
                if (__any_sync(0xffffffffu, here)) break;
                a = __shfl_sync(0xffffffffu, upto, 31);
            }
        }
        __syncthreads();
        return S->id;
    }

    // Sums of the segments over tokens from `least` on.
    __device__ __forceinline__ void sum_segments(u64 least) const {
        u64 sum = 0;
        each([&](uint32_t m) {
                 const float r = exp2f(exponent(m));
                 return (u64)m >= least >> 32 && !(r < minp) && r > 0.f;
             },
             [&](uint32_t key, int i) {
                 const float r = exp2f(exponent(key));
                 if (i < V && place(key, i) >= least && !(r < minp)) sum += whole(r);
             },
             [&](int s) {
                 sum = warp_total(sum);
                 if (lane == 0) seg[s] = sum;
                 sum = 0;
             });
        __syncthreads();
    }

    __device__ __forceinline__ int bin_of(float e) const { return (int)fminf(e * -8.0f, (float)(kSrBins - 1)); }

    // The place in the order of the last token of the shortest prefix that reaches p of the whole mass,
    // and the sums of the segments over that prefix (min-p applied to them).  false: a list overflowed.
    __device__ __forceinline__ bool nucleus(float p, u64 &least) const {
        // bits of a weight in the histogram: 13, less where the vocabulary could overflow 32
        int bits = 13;
        for (int v = V; v > (1 << 18); v >>= 1) bits--;
        for (int b = tid; b < kSrBins; b += NT) S->hist[b] = 0;
        if (tid == 0) S->n = 0;
        __syncthreads();
        u64 mass = 0;
        each([&](uint32_t m) { return exponent(m) > -42.0f; },
             [&](uint32_t key, int) {
                 const float e = exponent(key);
                 const u64 w = whole(exp2f(e));
                 if (w == 0) return;
                 mass += w;
                 const int b = bin_of(e), cut = 40 - bits - (b >> 3);
                 atomicAdd(&S->hist[b], (uint32_t)(cut >= 0 ? w >> cut : w << -cut));
             },
             [](int) {});
        const u64 M = total_of(mass);
        const u64 want = max((u64)1, (u64)ceil((double)fmaxf(p, 0.0f) * (double)M));
        if (warp == 0) {  // 11 bins a lane; a cut weight is at most 2^(2 - bits) below the weight
            constexpr int B = kSrBins / 32;
            u64 a[B], t = 0;
#pragma unroll
            for (int q = 0; q < B; q++) {
                const int b = B * lane + q, cut = 40 - bits - (b >> 3);
                a[q] = cut >= 0 ? (u64)S->hist[b] << cut : (u64)S->hist[b] >> -cut;
                t += a[q];
            }
            u64 c = warp_scan(t, lane) - t;
            int b1 = kSrBins, b2 = kSrBins;
#pragma unroll
            for (int q = 0; q < B; q++) {
                c += a[q];
                if (b1 == kSrBins && c + (c >> (bits - 2)) + 1 >= want) b1 = B * lane + q;
                if (b2 == kSrBins && c >= want) b2 = B * lane + q;
            }
            b1 = (int)__reduce_min_sync(0xffffffffu, (unsigned)b1);
            b2 = (int)__reduce_min_sync(0xffffffffu, (unsigned)b2);
            if (lane == 0) {
                S->lo = min(b1, kSrBins - 1);
                S->hi = min(b2, kSrBins - 1);
                S->kmin = 0xffffffffu;
                S->kmax = 0;
            }
        }
        __syncthreads();
        const int b1 = S->lo, b2 = S->hi;
        u64 above = 0, sum = 0;
        each([&](uint32_t m) { return exponent(m) > -42.0f && bin_of(exponent(m)) <= b2; },
             [&](uint32_t key, int i) {
                 const float e = exponent(key), r = exp2f(e);
                 const u64 w = whole(r);
                 if (w == 0) return;
                 const int b = bin_of(e);
                 if (b < b1) {
                     above += w;
                     if (!(r < minp)) sum += w;
                 } else if (b <= b2) {
                     append(place(key, i), w);
                 }
             },
             [&](int s) {
                 sum = warp_total(sum);
                 if (lane == 0) seg[s] = sum;
                 sum = 0;
             });
        above = total_of(above);
        const int n = S->n;
        if (n > kSrList) return false;
        // The tokens of the list up to the one that reaches `rest`: rounds of 256 bins of their keys, each
        // within the bin that the last one found, until few tokens are left in it.
        u64 rest = want - above;
        uint32_t from = 0xffffffffu, to = 0;
        for (int c = tid; c < n; c += NT) {
            const uint32_t key = (uint32_t)(S->list[c].at >> 32);
            from = min(from, key);
            to = max(to, key);
        }
        from = __reduce_min_sync(0xffffffffu, from);
        to = __reduce_max_sync(0xffffffffu, to);
        if (lane == 0) {
            atomicMin(&S->kmin, from);
            atomicMax(&S->kmax, to);
        }
        __syncthreads();
        from = S->kmin;
        to = S->kmax;
        int left = n;
        while (left > 64 && from < to) {
            const int sh = max(0, 24 - __clz(to - from));
            for (int b = tid; b < 256; b += NT) {
                S->bins[b] = 0;
                S->hist[b] = 0;
            }
            __syncthreads();
            for (int c = tid; c < n; c += NT) {
                const uint32_t key = (uint32_t)(S->list[c].at >> 32);
                if (key < from || key > to) continue;
                atomicAdd(&S->bins[(key - from) >> sh], S->list[c].w);
                atomicAdd(&S->hist[(key - from) >> sh], 1u);
            }
            __syncthreads();
            if (warp == 0) {
                u64 t = 0;
#pragma unroll
                for (int q = 0; q < 8; q++) t += S->bins[255 - 8 * lane - q];
                const u64 upto = warp_scan(t, lane);
                if (upto >= rest && upto - t < rest) {
                    u64 a = upto - t;
                    int b = 255 - 8 * lane;
                    while (a + S->bins[b] < rest) a += S->bins[b--];
                    S->lo = b;
                    S->found[0] = a;
                }
            }
            __syncthreads();
            rest -= S->found[0];
            left = (int)S->hist[S->lo];
            from += (uint32_t)S->lo << sh;
            to = min(to, from + ((1u << sh) - 1));
            __syncthreads();
        }
        // the last one: the tokens before it within [from, to] do not reach `rest`, with it they do
        for (int c = tid; c < n; c += NT) {
            const u64 at = S->list[c].at;
            const uint32_t key = (uint32_t)(at >> 32);
            if (key < from || key > to) continue;
            u64 before = 0;
            for (int j = 0; j < n; j++) {
                const u64 o = S->list[j].at;
                if (o > at && (uint32_t)(o >> 32) <= to) before += S->list[j].w;
            }
            if (before < rest && before + S->list[c].w >= rest) S->found[1] = at;
        }
        __syncthreads();
        least = S->found[1];
        for (int c = tid; c < n; c += NT) {
            const u64 at = S->list[c].at;
            if (at < least || exp2f(exponent((uint32_t)(at >> 32))) < minp) continue;
            atomicAdd(&seg[(0xffffffffu - (uint32_t)at) / kSrSegment], S->list[c].w);
        }
        __syncthreads();
        return true;
    }

    // The general cut: `least` moved up to the shortest prefix of what it keeps with a sum of at least
    // `want` of amount(key); every token is looked at, a byte of the key and then of the index at a time.
    template <typename A> __device__ __forceinline__ void cut(u64 &least, u64 want, A amount) const {
        u64 prefix = 0, mask = 0;
        for (int d = 56; d >= 0; d -= 8) {
            for (int b = tid; b < 256; b += NT) S->bins[b] = 0;
            __syncthreads();
            for (int i = tid; i < V; i += NT) {
                const uint32_t key = sr_key(sr_load(x, i));
                const u64 at = place(key, i);
                if ((at & mask) == prefix && at >= least) atomicAdd(&S->bins[at >> d & 255u], amount(key));
            }
            __syncthreads();
            if (warp == 0) {
                u64 t = 0;
#pragma unroll
                for (int q = 0; q < 8; q++) t += S->bins[255 - 8 * lane - q];
                const u64 upto = warp_scan(t, lane);
                if (upto >= want && upto - t < want) {
                    u64 a = upto - t;
                    int b = 255 - 8 * lane;
                    while (a + S->bins[b] < want) a += S->bins[b--];
                    S->lo = b;
                    S->found[0] = a;
                }
            }
            __syncthreads();
            prefix |= (u64)S->lo << d;
            mask |= (u64)255 << d;
            want -= S->found[0];
            __syncthreads();
        }
        least = prefix;
    }
};

template <typename T, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) sample_rows_kernel(const __grid_constant__ SampleRowsArgs A, int shift) {
    extern __shared__ __align__(16) uint8_t smem[];
    SrRow<T, NT> R;
    R.V = A.vocab;
    R.shift = shift;
    R.S = (SrShared *)smem;
    R.seg = (u64 *)(R.S + 1);
    R.gm = (uint32_t *)(R.seg + (A.vocab + kSrSegment - 1) / kSrSegment);
    R.tid = threadIdx.x;
    R.lane = R.tid & 31;
    R.warp = R.tid >> 5;
    R.wide = ((uintptr_t)A.logits | (uintptr_t)(A.ld * (long long)sizeof(T))) % (4 * sizeof(T)) == 0;
    SrShared *S = R.S;
    const int V = A.vocab, tid = R.tid, lane = R.lane;
    pdl_wait();
    pdl_trigger();
    for (long long row = blockIdx.x; row < A.rows; row += gridDim.x) {
        const T *x = R.x = (const T *)A.logits + row * A.ld;
        const float temp = A.temperature ? __ldg(A.temperature + row) : 1.0f;
        int k = A.top_k ? __ldg(A.top_k + row) : 0;
        k = k > 0 && k < V ? k : 0;
        const float p = A.top_p ? __ldg(A.top_p + row) : 1.0f, u = __ldg(A.uniforms + row);
        const float m = A.min_p ? __ldg(A.min_p + row) : 0.0f;
        R.minp = m > 0.f ? fminf(m, 1.0f) : 0.0f;
        __syncthreads();  // the last row is done with the shared memory
        if (shift > 4) {
            for (int g = tid; g < R.groups(); g += NT) R.gm[g] = 0;
            __syncthreads();
        }
        // the largest logit of every 16 tokens (four lanes), four loads in flight
        float most = -INFINITY;
        for (int c = R.warp * 512; c < V; c += NT / 32 * 512) {
            float4 v[4];
#pragma unroll
            for (int q = 0; q < 4; q++) v[q] = sr_load4(x, c + 128 * q + 4 * lane, V, R.wide);
#pragma unroll
            for (int q = 0; q < 4; q++) {
                float m = fmaxf(fmaxf(v[q].x, v[q].y), fmaxf(v[q].z, v[q].w));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                most = fmaxf(most, m);
                const int i = c + 128 * q + 4 * lane;
                if ((lane & 3) == 0 && i < V) {
                    if (shift == 4)
                        R.gm[i >> 4] = sr_key(m);
                    else
                        atomicMax(&R.gm[i >> shift], sr_key(m));
                }
            }
        }
        const uint32_t mine = __reduce_max_sync(0xffffffffu, sr_key(most));
        if (lane == 0) S->warp[R.warp] = mine;
        if (tid == 0) S->n = 0;
        __syncthreads();
        uint32_t top = 0;
#pragma unroll 8
        for (int w = 0; w < NT / 32; w++) top = max(top, (uint32_t)S->warp[w]);
        R.top = top;
        R.vmax = sr_value(top);
        int id = 0;
        if (R.vmax == -INFINITY) {
            id = 0;
        } else if (!(temp > 0.f) || k == 1) {
            id = R.first_top();
        } else {
            R.scale = 1.4426950408889634f / temp;
            bool done = false;
            if (V <= kSrList / 2 || (k > 0 && k <= min(R.groups(), kSrList / 2))) {
                const uint32_t least = V <= kSrList / 2 ? 0u : R.kth_maximum(k);
                R.each([&](uint32_t m) { return m >= least; },
                       [&](uint32_t key, int i) {
                           if (i < V && key >= least) R.append(R.place(key, i), R.whole(exp2f(R.exponent(key))));
                       },
                       [](int) {});
                __syncthreads();
                done = S->n <= kSrList;
                if (done) id = R.draw_list(S->n, k, p, u);
            } else if (k == 0 && p < 1.0f) {
                u64 least;
                done = R.nucleus(p, least);
                if (done) id = R.draw_segments(least, u);
            }
            if (!done) {
                u64 least = 0;
                if (k > 0) R.cut(least, (u64)k, [](uint32_t) { return (u64)1; });
                if (p < 1.0f) {
                    u64 mass = 0;
                    for (int i = tid; i < V; i += NT) {
                        const uint32_t key = sr_key(sr_load(x, i));
                        if (R.place(key, i) >= least) mass += R.whole(exp2f(R.exponent(key)));
                    }
                    const u64 M = R.total_of(mass);
                    R.cut(least, max((u64)1, (u64)ceil((double)fmaxf(p, 0.0f) * (double)M)),
                          [&](uint32_t key) { return R.whole(exp2f(R.exponent(key))); });
                }
                R.sum_segments(least);
                id = R.draw_segments(least, u);
            }
        }
        if (tid == 0) A.next_ids[row] = id;
    }
}

template <typename T, int NT> static cudaError_t launch_sample(const SampleRowsArgs &a, cudaStream_t s) {
    int shift = 4;
    while (((a.vocab - 1) >> shift) + 1 > kSrGroups) shift++;
    const size_t smem = sizeof(SrShared) + (size_t)((a.vocab + kSrSegment - 1) / kSrSegment) * 8 +
                        (size_t)(((a.vocab - 1) >> shift) + 1) * 4;
    const cudaError_t e = allow_smem((const void *)sample_rows_kernel<T, NT>);
    if (e != cudaSuccess) return e;
    return launch_pdl(sample_rows_kernel<T, NT>, dim3(std::min(a.rows, 1 << 20)), dim3(NT), smem, s, a, shift);
}

cudaError_t sample_rows_launch(const SampleRowsArgs &a, bool bf16, cudaStream_t s) {
    return bf16 ? launch_sample<uint16_t, 512>(a, s) : launch_sample<float, 512>(a, s);
}

}  // namespace slm
