// rows_scored_tc_64.cu -- scored rows on the tensor cores, heads of up to 64.
#include "rows_scored_tc.cuh"

namespace slm {

cudaError_t rows_tc_scored_64(const RowsArgs &a, cudaStream_t s) { return scored<64, 0>(a, s); }

}  // namespace slm
