// rows_scored_tc_64.cu -- the tensor-core attention of packed rows (rows_attention_tc.cuh) for scored
// rows with heads of up to 64.
#include "rows_attention_tc.cuh"

namespace slm {

template <bool PAGED> static cudaError_t launch(RowsTcArgs &t, cudaStream_t s) {
    const bool cap = t.a.sc.cap_log2 > 0.f;
    if (t.a.sc.slopes) return cap ? launch_tc<64, PAGED, kMasked | kCapped | kBiased>(t, s) : launch_tc<64, PAGED, kMasked | kBiased>(t, s);
    return cap ? launch_tc<64, PAGED, kMasked | kCapped>(t, s) : launch_tc<64, PAGED, kMasked>(t, s);
}

cudaError_t rows_tc_scored_launch_64(const RowsArgs &a, cudaStream_t s) {
    RowsTcArgs t = tc_args(a, true);
    return a.kv.table ? launch<true>(t, s) : launch<false>(t, s);
}

}  // namespace slm
