// rows_scored_tc_straight_64.cu -- scored rows on the tensor cores, heads of up to 64, long items.
#include "rows_scored_tc.cuh"

namespace slm {

cudaError_t rows_tc_scored_straight_64(const RowsArgs &a, cudaStream_t s) { return scored<64, kStraight>(a, s); }

}  // namespace slm
