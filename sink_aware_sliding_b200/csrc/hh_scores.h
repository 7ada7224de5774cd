// Launch interface of the prompt-score kernel.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "swa_internal.h"

namespace swa {

struct HhScoresArgs {
  PrefillArgs pa;     // geometry: n_seq sequences of length L, heads, window (<= L), sinks, scale
  const float* lse;   // [n_seq, Hq, L]
  float* score;       // [n_seq, Hkv, L]
  int n_obs;          // queries that observe: the last ones
  int n_units;        // key tiles of all (sequence, KV head)
};
cudaError_t launch_hh_scores(const HhScoresArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, int d, int grid,
                             cudaStream_t stream);

}  // namespace swa
