// Host test of the work split of masked items (rows_plan.h), built and run by
// tests/test_rows_masked.py with the system C++ compiler: over random batches and masks, the spans
// of rows and items agree with their definition, every block of every item is walked exactly once
// (an item without blocks is handed out once), each partial-state slot is used at most once, and
// the pieces of a divided item are found again from the record that its first piece leaves.
// Prints "ok" or the first failure and exits nonzero.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <tuple>
#include <vector>

#include "rows_plan.h"

using namespace slm;

static int fails = 0;
#define CHECK(cond, ...)                                   \
    do {                                                   \
        if (!(cond)) {                                     \
            std::printf("FAIL line %d: ", __LINE__);       \
            std::printf(__VA_ARGS__);                      \
            std::printf("\n");                             \
            if (++fails > 5) std::exit(1);                 \
        }                                                  \
    } while (0)

static std::mt19937 rng(11);
static int pick(int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); }

struct Masks {
    const SeqRows *seq;
    const int *prefix, *first;
    int window;
    RowsMask operator()(int s) const { return RowsMask{first ? first + seq[s].row0 : nullptr, prefix[s], window}; }
};

static void test_walk(int nseq, int maxn, int maxctx) {
    const int G = pick(1, 8), tile = pick(0, 1) ? 256 : pick(0, 1) ? 64 : 16;
    const RowsGeom g{pick(1, 8), tile / G > 0 ? tile / G : 1, pick(6, 7), pick(0, 2) > 0, pick(1, 3)};
    const int P = pick(0, 3) ? pick(1, 400) : pick(1, 5);
    const int window = pick(0, 2) ? 0 : pick(0, 1) ? pick(1, 40) : pick(1, 2000);
    const bool docs = pick(0, 1), prefixes = pick(0, 2) == 0;
    std::vector<SeqRows> seq(nseq);
    std::vector<int> prefix(nseq, 0), first;
    int row = 0;
    for (int s = 0; s < nseq; s++) {
        seq[s] = {row, pick(0, 3) ? pick(0, maxn) : 0, pick(0, maxctx)};
        if (!seq[s].n) seq[s].ctx = 0;
        row += seq[s].n;
        if (prefixes) prefix[s] = pick(0, seq[s].ctx + seq[s].n);
        int at = pick(0, 3) ? 0 : pick(-5, seq[s].ctx);
        for (int i = 0; i < seq[s].n; i++) {  // documents, and stretches of rows that see nothing
            if (!pick(0, 30)) at = std::max(at, seq[s].ctx + i + pick(0, 3) / 3 * pick(1, 200));
            first.push_back(at);
        }
    }
    const Masks masks{seq.data(), prefix.data(), docs ? first.data() : nullptr, window};
    std::vector<long long> wstart(nseq + 1, 0);
    long long items = 0;
    for (int s = 0; s < nseq; s++) {
        const RowsMask m = masks(s);
        long long units = 0;
        for (int t = 0; t < (seq[s].n ? item_count(g, seq[s].n) : 0); t++) {
            const RowsSpan span = item_span(g, seq[s], m, t);
            int lo = 1 << 30, hi = 0;
            for (int i = t * g.PT; i < std::min(seq[s].n, (t + 1) * g.PT); i++) {
                const int p = seq[s].ctx + i;
                const int a = std::max({0, docs ? first[seq[s].row0 + i] : 0, window ? p + 1 - window : 0});
                const int b = std::max(p + 1, prefix[s]);
                CHECK(row_from(m, seq[s].ctx, i) == a && row_to(m, seq[s].ctx, i) == b, "row %d", i);
                if (a < b) {
                    lo = std::min(lo, a);
                    hi = std::max(hi, b);
                }
            }
            if (lo < hi) {
                CHECK(span.lo <= lo && span.hi >= hi, "span of the item");
                CHECK(span.b0 << g.shift <= lo && (span.b0 + span.nb) << g.shift >= hi, "blocks of the item");
                CHECK((span.b0 + span.nb - 1) << g.shift < span.hi && (span.b0 + 1) << g.shift > span.lo, "no block too many");
            }
            CHECK(span.nb >= 0 && (span.lo < span.hi || span.nb == 0), "blocks of an empty item");
            units += g.cost + span.nb;
            items += g.KV;
        }
        wstart[s + 1] = wstart[s] + units * g.KV;
    }
    const long long total = wstart[nseq], unit = range_units(total, P);
    std::map<std::tuple<int, int, int>, int> done;
    std::map<int, std::tuple<int, int, int>> slots;
    std::map<std::tuple<int, int, int>, std::vector<int>> of;
    std::map<int, RowsPiece> joins;
    for (int c = 0; c < P; c++) {
        RowsStart at{0, 0, 0, 0};
        const long long from = unit * c;
        for (int s = 0; s < nseq && from < total; s++) {  // the item that holds unit `from`
            if (!(wstart[s] <= from && from < wstart[s + 1])) continue;
            long long base = wstart[s];
            for (int h = 0; h < g.KV; h++)
                for (int t = 0; t < item_count(g, seq[s].n); t++) {
                    const int u = g.cost + item_span(g, seq[s], masks(s), t).nb;
                    if (base <= from && from < base + u) at = RowsStart{s, h, t, base};
                    base += u;
                }
        }
        MaskedWalk<Masks> w;
        w.mask = masks;
        w.begin(seq.data(), total, nseq, g, from, unit * (c + 1), at);
        RowsPiece p;
        while (w.next(seq.data(), nseq, g, p)) {
            const auto item = std::make_tuple(p.s, p.g, p.t);
            CHECK(p.s >= 0 && p.s < nseq && p.g >= 0 && p.g < g.KV && p.t >= 0 && p.t < item_count(g, seq[p.s].n), "item bounds");
            const RowsSpan span = item_span(g, seq[p.s], masks(p.s), p.t);
            CHECK(p.nb == span.nb && p.b0 == span.b0, "blocks of the item");
            if (span.nb == 0) {
                CHECK(!done.count(item) && p.kb0 == 0 && p.kb1 == 0 && p.begins() && p.ends(), "an empty item, once");
                done[item] = 0;
                continue;
            }
            CHECK(p.kb0 == p.b0 + done[item] && p.kb1 > p.kb0 && p.kb1 <= p.b0 + p.nb, "blocks in order, once");
            CHECK(p.base >= 0 && p.base + g.cost + p.nb <= total, "item within the line");
            CHECK(p.begins() == (done[item] == 0), "begins");
            done[item] = p.kb1 - p.b0;
            CHECK(p.ends() == (done[item] == p.nb), "ends");
            if (p.begins() && p.ends()) continue;
            CHECK(g.split, "a whole item was divided");
            const int slot = piece_slot(c, p);
            CHECK(slot >= 0 && slot < 2 * P && !slots.count(slot), "slot %d used twice", slot);
            slots[slot] = item;
            of[item].push_back(slot);
            if (p.begins()) {
                CHECK(!joins.count(c), "one open item per CTA");
                CHECK(c < P - 1, "the last CTA leaves nothing open");
                joins[c] = p;
            }
        }
    }
    CHECK((long long)done.size() == items, "%zu items of %lld", done.size(), items);
    for (auto &d : done) {
        const int s = std::get<0>(d.first), t = std::get<2>(d.first);
        CHECK(d.second == item_span(g, seq[s], masks(s), t).nb, "item finished");
    }
    size_t found = 0;
    for (auto &j : joins) {
        const RowsPiece &p = j.second;
        const int c0 = j.first, c1 = (int)((p.base + g.cost + p.nb - 1) / unit);
        std::vector<int> want{2 * c0 + 1};
        for (int c = c0 + 1; c <= c1; c++) want.push_back(2 * c);
        CHECK(of[std::make_tuple(p.s, p.g, p.t)] == want, "pieces of a divided item");
        found++;
    }
    CHECK(found == of.size(), "every divided item has a record");
}

int main() {
    for (int i = 0; i < 300; i++) test_walk(pick(1, 6), 700, 3000);
    for (int i = 0; i < 100; i++) test_walk(pick(1, 64), 1, 4000);
    for (int i = 0; i < 100; i++) test_walk(pick(1, 3), 2, 100);
    for (int i = 0; i < 20; i++) test_walk(1, 1, 200000);
    for (int i = 0; i < 20; i++) test_walk(pick(1, 3), 5000, i % 2 ? 0 : 300000);
    // positions next to 2^31: no overflow
    const RowsGeom g{1, 64, 7, 1, 2};
    const SeqRows far{0, 100, 0x7fffff00 - 100};
    const RowsMask m{nullptr, 0, 0x7fffffff}, none{nullptr, 0x7fffff00, 1};
    CHECK(item_span(g, far, m, 1).lo == 0 && item_span(g, far, m, 1).hi == 0x7fffff00, "a window of 2^31 - 1");
    CHECK(item_span(g, far, none, 0).lo == 0x7fffff00 - 100 && item_span(g, far, none, 0).nb == 1, "a window of 1");
    if (fails) return 1;
    std::printf("ok\n");
    return 0;
}
