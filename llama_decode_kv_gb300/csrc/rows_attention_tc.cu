// rows_attention_tc.cu -- the tensor-core attention of packed rows (rows_attention_tc.cuh) for plain
// causal scores.
#include "rows_attention_tc.cuh"

namespace slm {

cudaError_t rows_tc_launch(const RowsArgs &a, cudaStream_t s) {
    RowsTcArgs t = tc_args(a, false);
    const bool paged = a.kv.table != nullptr;
    if (a.hd <= 64) return paged ? launch_tc<64, true, 0>(t, s) : launch_tc<64, false, 0>(t, s);
    return paged ? launch_tc<128, true, 0>(t, s) : launch_tc<128, false, 0>(t, s);
}

}  // namespace slm
