// prefix_tc.h -- host entry points of the tensor-core prefix kernels.
#pragma once

#include "prefix_common.cuh"

namespace zp {

constexpr int kPtRows = 256;  // query rows of an item

// The pieces of every item of a bf16 cache (d 64 or 128; h_q/h_kv 1, 2, 4 or 8).
zp_status prefix_part_tc(const PfxArgs &a, int d, cudaStream_t st);
// The window score of the prefix tokens from a.stats.
zp_status prefix_score_tc(const PfxArgs &a, int d, cudaStream_t st);

}  // namespace zp
