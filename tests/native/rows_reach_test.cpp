// Host test of most_seen (rows_plan.h), built and run by tests/test_rows_reach.py: over random batches,
// windows, documents and prefixes no item sees more positions than it says, and some see nearly as many.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "rows_plan.h"

using namespace slm;

static std::mt19937 rng(7);
static int pick(int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); }

int main() {
    int close[2] = {0, 0};
    for (int round = 0; round < 4000; round++) {
        const int nseq = pick(1, 6), window = pick(0, 4) ? pick(1, pick(0, 1) ? 30 : 1500) : 0;
        const bool prefixes = pick(0, 1), docs = pick(0, 2) == 0;
        const RowsGeom g{1, pick(0, 1) ? 256 / pick(1, 8) : pick(1, 16), 7, 1, 1};
        std::vector<SeqRows> seq(nseq);
        std::vector<int> prefix(nseq, 0), first;
        int rows = 0;
        long long longest = 0;
        for (int s = 0; s < nseq; s++) {
            seq[s] = {rows, pick(0, 3) ? pick(1, pick(0, 1) ? 4 : 1200) : 1, pick(0, 3000)};
            rows += seq[s].n;
            longest = std::max(longest, (long long)seq[s].ctx + seq[s].n);
            if (prefixes) prefix[s] = pick(0, 2) ? pick(0, seq[s].ctx + seq[s].n) : seq[s].ctx + seq[s].n;
            int at = 0;
            for (int i = 0; i < seq[s].n; i++) {
                if (!pick(0, 60)) at = seq[s].ctx + i;
                first.push_back(at);
            }
        }
        const long long most = most_seen(longest, window, prefixes, g.PT, rows);
        for (int s = 0; s < nseq; s++) {
            const RowsMask m{docs ? first.data() + seq[s].row0 : nullptr, prefix[s], window};
            for (int t = 0; t < item_count(g, seq[s].n); t++) {
                const RowsSpan p = item_span(g, seq[s], m, t);
                if (p.hi - p.lo > most) {
                    std::printf("FAIL: %d positions, %lld said (window %d, prefix %d, %d rows after %d)\n", p.hi - p.lo, most, window,
                                prefix[s], seq[s].n, seq[s].ctx);
                    return 1;
                }
                close[prefixes] += window && most < longest && p.hi - p.lo + 4 >= most;
            }
        }
    }
    if (close[0] < 100 || close[1] < 100) {
        std::printf("FAIL: far from what items see (%d, %d)\n", close[0], close[1]);
        return 1;
    }
    std::puts("ok");
}
