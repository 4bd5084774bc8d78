// token_ops.h -- launchers of the passes in front of block-sparse attention:
// rotation table, per-head norm + rotation + block means, block selection.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/dt.h"

namespace dt {

constexpr int kMaxPairs = 128;              // rotated pairs of a row (rot <= 256)

struct RopeTableArgs {
  const int32_t* pos;
  float* table;
  int S, pairs;
  uint64_t turns[kMaxPairs];                // turns per unit of position, base^(-2j/dim) / (2 pi), as a 64-bit fraction
  uint8_t axis[kMaxPairs];
};
int launch_rope_table(const RopeTableArgs& a, cudaStream_t stream);

struct NormRopeArgs {
  const void *q, *k, *v;
  void *Q, *K, *V;
  const float *wq, *wk, *table;
  float *q_mean, *k_mean;
  dt_norm_rope_params p;
  int wt, groups;                           // warps per head and tile, CTAs per tile (set by the launcher, like inv_d)
  float inv_d;
};
int launch_qk_norm_rope(NormRopeArgs a, int sms, cudaStream_t stream);

int launch_block_select(const dt_select_params& p, const float* q_mean, const float* k_mean, int32_t* idx,
                        int32_t* count, cudaStream_t stream);

}  // namespace dt
