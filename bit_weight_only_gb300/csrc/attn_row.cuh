// attn_row.cuh -- attention of one query row by one warp, on the CUDA cores:
// an online softmax over 32 keys at a time (each lane one key's score, then
// every lane its d/32 columns of the weighted sum).
#pragma once

#include "kv_layout.cuh"

namespace qgemv {

// score(j) and value(j, d) of visible keys only; see(j): whether key j counts.
template <int D, class See, class Score, class Value>
__device__ __forceinline__ void attend_row(int64_t n, See see, Score score, Value value, float (&acc)[D / 32], float& m,
                                           float& l) {
  const int lane = threadIdx.x & 31;
  m = -INFINITY;
  l = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
  for (int64_t j0 = 0; j0 < n; j0 += 32) {
    const bool on = j0 + lane < n && see(j0 + lane);
    const float s = on ? score(j0 + lane) : -INFINITY;
    float top = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float mn = fmaxf(m, top);
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float p = on ? exp2f(s - ref) : 0.f;
    const float f = exp2f(m - ref);
    float sum = p;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * f + sum;
    m = mn;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] *= f;
    unsigned live = __ballot_sync(0xffffffffu, on);
    while (live) {
      const int k = __ffs(live) - 1;
      live &= live - 1;
      const float pk = __shfl_sync(0xffffffffu, p, k);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) acc[i] = fmaf(pk, value(j0 + k, 32 * i + lane), acc[i]);
    }
  }
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// out and lse of a finished row (scores in units of log 2).
template <int D, typename T>
__device__ __forceinline__ void store_row(T* out, float* lse, const float (&acc)[D / 32], float m, float l) {
  const int lane = threadIdx.x & 31;
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) out[32 * i + lane] = from_f32<T>(acc[i] * inv);
  if (lse && lane == 0) *lse = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace qgemv
