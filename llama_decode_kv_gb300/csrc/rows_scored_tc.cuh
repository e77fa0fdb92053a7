// rows_scored_tc.cuh -- one translation unit's share of the tensor-core attention of scored rows
// (rows_attention_tc.cuh).
#pragma once

#include "rows_attention_tc.cuh"

namespace slm {

template <int HDP, bool PAGED, int MORE> static cudaError_t launch_scored(RowsTcArgs &t, cudaStream_t s) {
    constexpr int M = kMasked | MORE;
    const bool cap = t.a.sc.cap_log2 > 0.f;
    if (t.a.sc.slopes)
        return cap ? launch_tc<HDP, PAGED, M | kCapped | kBiased>(t, s) : launch_tc<HDP, PAGED, M | kBiased>(t, s);
    return cap ? launch_tc<HDP, PAGED, M | kCapped>(t, s) : launch_tc<HDP, PAGED, M>(t, s);
}

template <int HDP, int MORE> static cudaError_t scored(const RowsArgs &a, cudaStream_t s) {
    RowsTcArgs t = tc_args(a, true);
    return a.kv.table ? launch_scored<HDP, true, MORE>(t, s) : launch_scored<HDP, false, MORE>(t, s);
}

}  // namespace slm
