// Host test of fits_rows (rows_plan.h), built and run by tests/test_rows_few.py: for every group size
// and token counts up to the most that a call takes, it agrees with the product in 64 bits.
#include <cstdio>
#include <initializer_list>

#include "rows_plan.h"

using namespace slm;

int main() {
    for (int G = 1; G <= kRowsMaxGroup; G++)
        for (int rows : {32, 128})
            for (int shift = 0; shift <= 30; shift++)
                for (int d = -70; d <= 70; d++) {
                    const long long left = (1LL << shift) + d;
                    if (left < 1 || left > kRowsMaxRows) continue;
                    if (fits_rows((int)left, G, rows) != (left * G <= rows)) {
                        std::printf("FAIL: %lld tokens of %d heads in %d rows\n", left, G, rows);
                        return 1;
                    }
                }
    std::puts("ok");
}
