// rope.h -- the rotary positions' parameters and launch call.
#pragma once

#include "attn.h"

namespace qgemv {

// An entry of a plan: {turns low, turns high, axis, 0}.
struct RopeParams {
  qgemv_kv_cache cache;  // pages NULL: rows only
  RowsIn q, k, v;
  RowsOut out;
  int out_dtype, q_heads;
  const int64_t* slots;
  const int32_t* positions;
  int n_axes, pairs, neighbours;
  const uint4* plan;
  int64_t n_tokens;
};

cudaError_t launch_rope(const RopeParams& p, int dtype, int head_dim, cudaStream_t s);

}  // namespace qgemv
