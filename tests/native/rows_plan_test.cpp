// Host test of the packed rows' work split (rows_plan.h), built and run by
// tests/test_rows_plan.py with the system C++ compiler: over random batches, every block of
// every item is walked exactly once, each partial-state slot is used at most once, and the
// pieces of a divided item are found again from the record that its first piece leaves.
// Prints "ok" or the first failure and exits nonzero.
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

static std::mt19937 rng(7);
static int pick(int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); }

static void test_sums() {
    for (int i = 0; i < 2000; i++) {
        const unsigned n = pick(0, 200), m = 1u << pick(0, 8), a = pick(1, 300), b = pick(0, 100000);
        unsigned long long want = 0;
        for (unsigned k = 0; k < n; k++) want += ((unsigned long long)a * k + b) / m;
        CHECK(floor_sum(n, m, a, b) == want, "floor_sum(%u, %u, %u, %u)", n, m, a, b);
    }
    for (int i = 0; i < 500; i++) {
        const RowsGeom g{pick(1, 4), pick(1, 128), pick(6, 7), 1, pick(1, 3)};
        const int n = pick(1, 3000), ctx = pick(0, 5000);
        long long sum = 0;
        for (int t = 0; t <= item_count(g, n); t++) {
            CHECK(head_units(g, ctx, n, t) == sum, "head_units ctx %d n %d t %d", ctx, n, t);
            if (t < item_count(g, n)) sum += item_blocks(g, ctx, n, t) + g.cost;
        }
    }
    for (int i = 0; i < 500; i++) {
        const RowsGeom g{1, pick(1, 128), pick(6, 7), 1, pick(1, 3)};
        const int n = pick(1, 3000), ctx = pick(0, 5000), t = pick(0, item_count(g, n) - 1);
        const int last = (t + 1) * g.PT < n ? (t + 1) * g.PT : n;
        CHECK(item_blocks(g, ctx, n, t) == (ctx + last + (1 << g.shift) - 1) / (1 << g.shift), "item_blocks");
    }
    // a sequence of two billion positions: no overflow
    const RowsGeom g{1, 1, 6, 1, 1};
    CHECK(head_units(g, 2000000000, 1000, 1000) > 1000LL * (2000000000LL / 64), "long context");
}

static void test_lengths() {
    SeqRows r;
    CHECK(seq_rows(3, 10, 5, 20, 100, r) && r.row0 == 3 && r.n == 7 && r.ctx == 5, "plain");
    CHECK(seq_rows(3, 3, -9, 20, 100, r) && r.n == 0, "no rows: the context is not looked at");
    CHECK(!seq_rows(-5, 10, 0, 20, 100, r) && r.row0 == 0 && r.n == 10, "begins before the buffer");
    CHECK(!seq_rows(5, 30, 0, 20, 100, r) && r.row0 == 5 && r.n == 15, "ends behind the buffer");
    CHECK(!seq_rows(40, 50, 0, 20, 100, r) && r.n == 0, "wholly behind the buffer");
    CHECK(!seq_rows(10, 3, 0, 20, 100, r) && r.n == 0, "descends");
    CHECK(!seq_rows(0, 5, -1, 20, 100, r) && r.ctx == 0, "negative context");
    CHECK(!seq_rows(0, 5, 96, 20, 100, r) && r.ctx == 0, "past the page table");
    CHECK(seq_rows(0, 5, 95, 20, 100, r) && r.ctx == 95, "last position of the page table");
    CHECK(!seq_rows(0, 5, 2147483647, 20, 100, r) && r.ctx == 0, "context of 2^31 - 1");
    CHECK(!seq_rows(0, 18, 0, 20, 16, r) && r.n == 16, "more rows than the table holds");
    CHECK(!seq_rows(-2147483647 - 1, 2147483647, 2147483647, 20, 16, r) && r.row0 == 0 && r.n == 16, "extremes");
}

static void test_walk(int nseq, int maxn, int maxctx) {
    const int G = pick(1, 8), tile = pick(0, 1) ? 256 : pick(0, 1) ? 64 : 16;
    const RowsGeom g{pick(1, 8), tile / G > 0 ? tile / G : 1, pick(6, 7), pick(0, 2) > 0, pick(1, 3)};
    const int P = pick(0, 3) ? pick(1, 400) : pick(1, 5);
    std::vector<SeqRows> seq(nseq);
    std::vector<long long> wstart(nseq + 1, 0);
    int row = 0;
    for (int s = 0; s < nseq; s++) {
        seq[s] = {row, pick(0, 3) ? pick(0, maxn) : 0, pick(0, maxctx)};
        if (!seq[s].n) seq[s].ctx = 0;
        row += seq[s].n;
        wstart[s + 1] = wstart[s] + (seq[s].n ? head_units(g, seq[s].ctx, seq[s].n, item_count(g, seq[s].n)) * g.KV : 0);
    }
    const long long total = wstart[nseq];
    std::map<std::tuple<int, int, int>, int> done;            // (s, g, t) -> blocks walked so far
    std::map<int, std::tuple<int, int, int>> slots;           // slot -> item
    std::map<std::tuple<int, int, int>, std::vector<int>> of; // item -> its slots in order
    std::map<int, RowsPiece> joins;                           // CTA -> the item it starts
    const long long unit = range_units(total, P);
    CHECK(unit * P >= total && (unit == 1 || (unit - 1) * P < total), "range of %lld for %lld over %d", unit, total, P);
    for (int c = 0; c < P; c++) {
        RowsWalk w;
        w.begin(seq.data(), wstart.data(), nseq, g, unit * c, unit * (c + 1));
        RowsPiece p;
        while (w.next(seq.data(), nseq, g, p)) {
            const auto item = std::make_tuple(p.s, p.g, p.t);
            CHECK(p.s >= 0 && p.s < nseq && p.g >= 0 && p.g < g.KV && p.t >= 0 && p.t < item_count(g, seq[p.s].n), "item bounds");
            CHECK(p.nb == item_blocks(g, seq[p.s].ctx, seq[p.s].n, p.t), "blocks of the item");
            CHECK(p.kb0 == done[item] && p.kb1 > p.kb0 && p.kb1 <= p.nb, "blocks in order, once");
            CHECK(p.base >= 0 && p.base + g.cost + p.nb <= total, "item within the line");
            done[item] = p.kb1;
            if (p.kb0 == 0 && p.kb1 == p.nb) continue;
            CHECK(g.split, "a whole item was divided");
            const int slot = piece_slot(c, p);
            CHECK(slot >= 0 && slot < 2 * P && !slots.count(slot), "slot %d used twice", slot);
            slots[slot] = item;
            of[item].push_back(slot);
            if (p.kb0 == 0) {
                CHECK(!joins.count(c), "one open item per CTA");
                CHECK(c < P - 1, "the last CTA leaves nothing open");
                joins[c] = p;
            }
        }
    }
    long long items = 0;
    for (int s = 0; s < nseq; s++) items += seq[s].n ? (long long)g.KV * item_count(g, seq[s].n) : 0;
    CHECK((long long)done.size() == items, "%zu items of %lld", done.size(), items);
    for (auto &d : done) CHECK(d.second == item_blocks(g, seq[std::get<0>(d.first)].ctx, seq[std::get<0>(d.first)].n, std::get<2>(d.first)), "item finished");
    // every divided item is found again from its first piece's record
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
    test_sums();
    test_lengths();
    for (int i = 0; i < 300; i++) test_walk(pick(1, 6), 700, 3000);
    for (int i = 0; i < 100; i++) test_walk(pick(1, 64), 1, 4000);
    for (int i = 0; i < 100; i++) test_walk(pick(1, 3), 2, 100);
    for (int i = 0; i < 20; i++) test_walk(1, 1, 200000);
    for (int i = 0; i < 20; i++) test_walk(pick(1, 3), 20000, i % 2 ? 0 : 300000);
    test_walk(1024, 3, 50);
    if (fails) return 1;
    std::printf("ok\n");
    return 0;
}
