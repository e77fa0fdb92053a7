// rows_scored_tc_128.cu -- scored rows on the tensor cores, heads of 72 to 128.
#include "rows_scored_tc.cuh"

namespace slm {

cudaError_t rows_tc_scored_128(const RowsArgs &a, cudaStream_t s) { return scored<128, 0>(a, s); }

}  // namespace slm
