// rows_plan.h -- how the attention of packed rows is cut into work (host and device, no
// CUDA calls, so that the host tests walk the same code).
//
// Sequence s of a batch has n new rows (tokens) after ctx cached positions.  Its work for
// one kv head is cut into items of up to PT tokens (all G query heads of the group
// together); an item walks the blocks of BLK positions [0, ctx + its last token], so item t
// has nb(t) = ceil((ctx + min((t + 1) PT, n)) / BLK) blocks and counts nb(t) + cost units
// (the units on top stand for its queries and its epilogue).  All items of a batch,
// in the order (sequence, kv head, item), form one line of `total` units, which is cut into
// ranges of ceil(total / P) units, one per CTA: every CTA gets the same work whatever the
// lengths are, and an item that a cut divides is joined afterwards from the partial states of
// its pieces.  Where every item is short (split = 0), a CTA takes the items that begin in its
// range whole, and nothing has to be joined.
//
// With masks (MaskedWalk) an item walks only the blocks [b0, b1) that some token of it sees (item_span),
// and counts those; the units of a sequence are added up item by item (masked_layout in rows.cuh), as no
// formula holds for documents.
#pragma once

#include <math.h>
#include <stdint.h>

#ifdef __CUDACC__
#define SLM_HD __host__ __device__ __forceinline__
#else
#define SLM_HD inline
#endif

namespace slm {

constexpr int kRowsMaxSeqs = 1024;  // sequences per call (their lengths sit in shared memory)
constexpr int kRowsMaxRows = 1 << 30;  // packed rows per call
constexpr int kRowsMaxHeads = 65536;  // a row's units are counted in 32 bits
constexpr int kRowsMaxGroup = 64;   // query heads per kv head

// A sequence's rows after its lengths were checked: first packed row, rows, cached positions.
struct SeqRows {
    int row0, n, ctx;
};

// Check one sequence against the packed buffer (rows) and what the cache can hold (cap
// positions; the lengths are device data, so nothing was checked before).  false: a length
// was out of bounds and has been cut to fit.
SLM_HD bool seq_rows(int begin, int end, int ctx, int rows, long long cap, SeqRows &o) {
    bool ok = true;
    int a = begin, b = end;
    if (a < 0 || a > rows) {
        a = a < 0 ? 0 : rows;
        ok = false;
    }
    if (b < a || b > rows) {
        b = b < a ? a : rows;
        ok = false;
    }
    int n = b - a;
    if (n > 0 && (ctx < 0 || (long long)ctx + n > cap)) {
        ok = false;
        ctx = 0;
        if (n > cap) n = (int)cap;
    }
    o.row0 = a;
    o.n = n;
    o.ctx = n > 0 ? ctx : 0;
    return ok;
}

// Quotient of values that nearly always fit 32 bits (a 64-bit division is a long routine).
SLM_HD unsigned long long udiv(unsigned long long a, unsigned long long b) {
    return ((a | b) >> 32) == 0 ? (unsigned)a / (unsigned)b : a / b;
}

// sum over i in [0, n) of floor((a i + b) / m), by exchanging the roles of a and m (the
// lattice points under a line, counted by rows and by columns in turn).
SLM_HD unsigned long long floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
    unsigned long long s = 0;
    while (n > 0) {
        s += (unsigned long long)(a / m) * ((unsigned long long)n * (n - 1) / 2);
        a %= m;
        s += (unsigned long long)n * (b / m);
        b %= m;
        const unsigned long long top = (unsigned long long)a * n + b, q = udiv(top, m);
        if (q == 0) break;
        n = (unsigned)q;
        b = (unsigned)(top - q * m);
        const unsigned t = m;
        m = a;
        a = t;
    }
    return s;
}

struct RowsGeom {
    int KV;      // kv heads
    int PT;      // tokens per item
    int shift;   // log2 of the positions per block (BLK)
    int split;   // 1: ranges cut through items; 0: items stay whole
    int cost;    // units of an item besides its blocks
};

SLM_HD int item_count(const RowsGeom &g, int n) { return (n + g.PT - 1) / g.PT; }

// Whether `left` tokens of G heads are at most `rows` rows (all of a sequence's may be more than 2^31, so
// the tokens are cut first).
SLM_HD bool fits_rows(int left, int G, int rows) { return (left <= rows ? left : rows + 1) * G <= rows; }

SLM_HD int item_blocks(const RowsGeom &g, int ctx, int n, int t) {
    const int left = n - t * g.PT, end = left < g.PT ? n : n - left + g.PT;
    return (int)(((unsigned)ctx + (unsigned)end + (1u << g.shift) - 1) >> g.shift);
}

// Units of the items [0, t) of one kv head of a sequence.
SLM_HD long long head_units(const RowsGeom &g, int ctx, int n, int t) {
    if (t <= 0) return 0;
    const int T = item_count(g, n), full = t < T ? t : T - 1;
    long long s = full > 0 ? (long long)floor_sum((unsigned)full, 1u << g.shift, (unsigned)g.PT,
                                                  (unsigned)ctx + g.PT + (1u << g.shift) - 1)
                           : 0;
    if (t >= T) s += item_blocks(g, ctx, n, T - 1);
    return s + (long long)g.cost * (t < T ? t : T);
}

// Units of a range.
SLM_HD long long range_units(long long total, int P) {
    return total > 0 ? (long long)udiv((unsigned long long)total + P - 1, (unsigned long long)P) : 1;
}

// One piece of one item: blocks [kb0, kb1) of its [b0, b0 + nb).
struct RowsPiece {
    int s, g, t, nb, kb0, kb1;
    long long base;  // the item's first unit
    int b0;          // 0 but for masked items

    SLM_HD bool begins() const { return kb0 == b0; }
    SLM_HD bool ends() const { return kb1 == b0 + nb; }
};

// Walks the pieces of the units [from, to).  seq: the checked sequences; wstart[s]: units of
// the sequences before s (wstart[nseq] = total).
struct RowsWalk {
    long long x, end, base;
    int s, g, t, nb;

    SLM_HD void open(const SeqRows *seq, const RowsGeom &G) { nb = item_blocks(G, seq[s].ctx, seq[s].n, t); }

    // On to the item after this one; false behind the last.
    SLM_HD bool advance(const SeqRows *seq, int nseq, const RowsGeom &G) {
        base += G.cost + nb;
        t++;
        if ((long long)t * G.PT >= seq[s].n) {
            t = 0;
            if (++g == G.KV) {
                g = 0;
                s++;
                while (s < nseq && seq[s].n == 0) s++;
            }
        }
        if (s >= nseq) return false;
        open(seq, G);
        return true;
    }

    SLM_HD void begin(const SeqRows *seq, const long long *wstart, int nseq, const RowsGeom &G, long long from,
                      long long to) {
        const long long total = wstart[nseq];
        x = from;
        end = to < total ? to : total;
        if (x >= end) return;
        int lo = 0, hi = nseq - 1;  // the last s with wstart[s] <= x (empty sequences have no units)
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (wstart[mid] <= x)
                lo = mid;
            else
                hi = mid - 1;
        }
        s = lo;
        const unsigned long long per = udiv(wstart[s + 1] - wstart[s], G.KV);
        unsigned long long rem = x - wstart[s];
        g = (int)udiv(rem, per);
        rem -= (unsigned long long)g * per;
        // The last item with head_units(t) <= rem.  About t^2 PT / (2 BLK) + t b units stand before item
        // t, b being the first item's; from that guess it is a step or two.
        const int ctx = seq[s].ctx, n = seq[s].n, T = item_count(G, n);
        unsigned long long at = 0;  // head_units(t)
        t = 0;
        if (T > 1) {
            const float blk = (float)(1 << G.shift), qa = 0.5f * (float)G.PT / blk;
            const float qb = G.cost + 0.5f + ((float)ctx + 0.5f * (float)G.PT) / blk;
            const float guess = 2.0f * (float)rem / (qb + sqrtf(qb * qb + 4.0f * qa * (float)rem));
            t = guess < (float)(T - 1) ? (int)guess : T - 1;
            at = (unsigned long long)head_units(G, ctx, n, t);
            while (at > rem) at -= G.cost + item_blocks(G, ctx, n, --t);
            while (t < T - 1) {
                const unsigned long long after = at + G.cost + item_blocks(G, ctx, n, t);
                if (after > rem) break;
                at = after;
                t++;
            }
        }
        base = wstart[s] + (long long)(g * per + at);
        open(seq, G);
        if (!G.split && base < x) {  // the item belongs to the range that it begins in
            if (!advance(seq, nseq, G)) end = x;
            x = base;
        }
    }

    // The next piece with at least one block; false at the end of the range.
    SLM_HD bool next(const SeqRows *seq, int nseq, const RowsGeom &G, RowsPiece &p) {
        while (x < end) {
            const long long first = base + G.cost, stop = first + nb;
            const long long hi = end < stop && G.split ? end : stop;
            p.s = s;
            p.g = g;
            p.t = t;
            p.nb = nb;
            p.base = base;
            p.b0 = 0;
            p.kb0 = x > first ? (int)(x - first) : 0;
            p.kb1 = hi > first ? (int)(hi - first) : 0;
            x = hi;
            if (x >= stop && !advance(seq, nseq, G)) end = x;
            if (p.kb1 > p.kb0) return true;
        }
        return false;
    }
};

// A CTA has at most two pieces that are not whole items: one that starts inside an item
// (its first) and one that starts an item and does not finish it (its last).
SLM_HD int piece_slot(int cta, const RowsPiece &p) { return 2 * cta + (p.begins() ? 1 : 0); }

// ---- items whose rows do not see all positions up to their own
//
// Row i of a sequence, at position p = ctx + i, sees [lo, hi): lo = max(first, p + 1 - window, 0),
// hi = max(p + 1, prefix).  first does not descend within a sequence, so an item's span begins at
// its first row's lo and ends at its last row's hi, and has blocks [b0, b0 + nb) of its own (none
// where the span is empty: such an item still counts its `cost` units, and writes its rows).  There
// is no closed form for their sum: the units of all items are added up one by one (masked_layout in rows.cuh).

// The mask of one sequence: its first packed row's entry of `first` (null: none), its prefix cut to
// [0, ctx + n], the window (0: none).
struct RowsMask {
    const int *first;
    int prefix, window;
};

SLM_HD int row_from(const RowsMask &m, int ctx, int i) {
    int lo = m.first ? m.first[i] : 0;
    lo = lo > 0 ? lo : 0;
    const int w = m.window ? ctx + i + 1 - m.window : 0;
    return lo > w ? lo : w;
}
SLM_HD int row_to(const RowsMask &m, int ctx, int i) { return ctx + i + 1 > m.prefix ? ctx + i + 1 : m.prefix; }

struct RowsSpan {
    int lo, hi, b0, nb;
};
SLM_HD RowsSpan item_span(const RowsGeom &g, const SeqRows &r, const RowsMask &m, int t) {
    const int i0 = t * g.PT, i1 = r.n - i0 < g.PT ? r.n : i0 + g.PT;
    RowsSpan s{row_from(m, r.ctx, i0), row_to(m, r.ctx, i1 - 1), 0, 0};
    if (s.lo < s.hi) {
        s.b0 = s.lo >> g.shift;
        s.nb = (int)(((unsigned)s.hi + (1u << g.shift) - 1) >> g.shift) - s.b0;
    }
    return s;
}

// Positions that an item can see at most, of sequences of at most `longest` positions in a call of `rows`
// rows.  Behind a window an item's span begins at most window - 1 positions before its first row and ends
// with its last row, or with the prefix, which ends with the sequence's last row at the latest.
SLM_HD long long most_seen(long long longest, int window, bool prefixes, int PT, int rows) {
    const long long most = (long long)window + (prefixes ? rows : PT);
    return window && most < longest ? most : longest;
}

// The item that holds a unit of the line.
struct RowsStart {
    int s, g, t;
    long long base;
};

// RowsWalk over masked items.  mask(s): the mask of sequence s.
template <typename MASK> struct MaskedWalk {
    long long x, end, base;
    int s, g, t;
    RowsSpan span;
    MASK mask;

    SLM_HD void open(const SeqRows *seq, const RowsGeom &G) { span = item_span(G, seq[s], mask(s), t); }

    SLM_HD bool advance(const SeqRows *seq, int nseq, const RowsGeom &G) {
        base += G.cost + span.nb;
        t++;
        if ((long long)t * G.PT >= seq[s].n) {
            t = 0;
            if (++g == G.KV) {
                g = 0;
                s++;
                while (s < nseq && seq[s].n == 0) s++;
            }
        }
        if (s >= nseq) return false;
        open(seq, G);
        return true;
    }

    // at: the item that holds unit `from` (not looked at where the range is empty).
    SLM_HD void begin(const SeqRows *seq, long long total, int nseq, const RowsGeom &G, long long from, long long to,
                      const RowsStart &at) {
        x = from;
        end = to < total ? to : total;
        if (x >= end) return;
        s = at.s;
        g = at.g;
        t = at.t;
        base = at.base;
        open(seq, G);
        if (!G.split && base < x) {  // the item belongs to the range that it begins in
            if (!advance(seq, nseq, G)) end = x;
            x = base;
        }
    }

    // The next piece: at least one block, or the whole of an item without any.
    SLM_HD bool next(const SeqRows *seq, int nseq, const RowsGeom &G, RowsPiece &p) {
        while (x < end) {
            const long long first = base + G.cost, stop = first + span.nb;
            const long long hi = end < stop && G.split ? end : stop;
            const bool empty = span.nb == 0 && x == base;
            p.s = s;
            p.g = g;
            p.t = t;
            p.nb = span.nb;
            p.base = base;
            p.b0 = span.b0;
            p.kb0 = span.b0 + (x > first ? (int)(x - first) : 0);
            p.kb1 = span.b0 + (hi > first ? (int)(hi - first) : 0);
            x = hi;
            if (x >= stop && !advance(seq, nseq, G)) end = x;
            if (p.kb1 > p.kb0 || empty) return true;
        }
        return false;
    }
};
}  // namespace slm
