// attn_prompt.cu -- causal attention over packed prompts with grouped heads
// (qgemv_attn_prompt): one warp per (query, head) row.
#include "attn_row.cuh"

namespace qgemv {
namespace {

constexpr int kThreads = 128;

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) prompt_row_kernel(const PromptParams p) {
  __shared__ float qs[kThreads / 32][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + warp;
  const int64_t token = row / p.q_heads;
  if (token >= p.n_q) return;
  const int head = static_cast<int>(row - token * p.q_heads);
  const int kvh = head / (p.q_heads / p.kv_heads);
  int seq = 0;
  while (seq < p.n_seqs && p.cu_q[seq + 1] <= token) ++seq;
  if (seq >= p.n_seqs || p.cu_q[seq] > token) return;
  const int64_t i = token - p.cu_q[seq];
  const int64_t k0 = max(0, p.cu_k[seq]), k1 = min(static_cast<int64_t>(p.cu_k[seq + 1]), p.n_k);
  const int64_t n = max(static_cast<int64_t>(0), min(k1 - k0, i + 1 + (k1 - k0) - (p.cu_q[seq + 1] - p.cu_q[seq])));
  const T* q = static_cast<const T*>(p.q.ptr) + token * p.q.token_stride + head * p.q.head_stride;
  const T* kb = static_cast<const T*>(p.k.ptr) + k0 * p.k.token_stride + kvh * p.k.head_stride;
  const T* vb = static_cast<const T*>(p.v.ptr) + k0 * p.v.token_stride + kvh * p.v.head_stride;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) qs[warp][32 * e + lane] = to_f32<T>(q[32 * e + lane]);
  __syncwarp();
  float acc[D / 32], m, l;
  attend_row<D>(
      n, [&](int64_t) { return true; },
      [&](int64_t j) {
        const T* k = kb + j * p.k.token_stride;
        float s = 0.f;
        for (int d = 0; d < D; ++d) s = fmaf(qs[warp][d], to_f32<T>(k[d]), s);
        return s * p.scale * kLog2e;
      },
      [&](int64_t j, int d) { return to_f32<T>(vb[j * p.v.token_stride + d]); }, acc, m, l);
  store_row<D>(static_cast<T*>(p.out.ptr) + token * p.out.token_stride + head * p.out.head_stride,
               p.lse ? p.lse + token * p.q_heads + head : nullptr, acc, m, l);
}

}  // namespace

cudaError_t launch_attn_prompt(const PromptParams& p, cudaStream_t s) {
  const int64_t rows = p.n_q * p.q_heads;
  const unsigned grid = static_cast<unsigned>((rows + kThreads / 32 - 1) / (kThreads / 32));
  if (p.dtype == QGEMV_DT_F16) {
    if (p.head_dim == 64) prompt_row_kernel<64, __half><<<grid, kThreads, 0, s>>>(p);
    else prompt_row_kernel<128, __half><<<grid, kThreads, 0, s>>>(p);
  } else {
    if (p.head_dim == 64) prompt_row_kernel<64, __nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
    else prompt_row_kernel<128, __nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace qgemv
