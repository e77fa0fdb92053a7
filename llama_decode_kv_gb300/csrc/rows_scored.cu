// rows_scored.cu -- the CUDA-core attention of packed rows (rows_attention.cuh) for scored rows.
#include "rows_attention.cuh"

namespace slm {

cudaError_t rows_simt_scored_launch(const RowsArgs &a, bool bf16, cudaStream_t s) { return launch_cuda_cores<true>(a, bf16, s); }

}  // namespace slm
