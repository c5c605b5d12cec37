// attn_tree.cu -- attention of drafted tokens over the paged key/value cache
// (qgemv_attn_tree): one warp per (token, head) row.
#include "attn_row.cuh"

namespace qgemv {

int64_t tree_ws_bytes(int64_t, int, int) { return 0; }

namespace {

constexpr int kThreads = 128;

template <int FMT, int D>
__global__ void __launch_bounds__(kThreads) tree_row_kernel(const TreeParams p) {
  __shared__ float qs[kThreads / 32][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + warp;
  const int64_t token = row / p.q_heads;
  if (token >= p.n_q) return;
  const int head = static_cast<int>(row - token * p.q_heads);
  const int kvh = head / (p.q_heads / p.cache.kv_heads);
  int seq = 0;
  while (seq < p.n_seqs && p.cu_q[seq + 1] <= token) ++seq;
  if (seq >= p.n_seqs || p.cu_q[seq] > token) return;
  const int i = static_cast<int>(token - p.cu_q[seq]);
  const int T = min(p.cu_q[seq + 1] - p.cu_q[seq], kMaxDrafts);
  if (i >= T) return;
  const int ctx = max(0, p.ctx_lens[seq]);
  const uint64_t mask = p.masks ? p.masks[token] : (i == 63 ? ~0ull : (1ull << (i + 1)) - 1);
  const __half* q = static_cast<const __half*>(p.q.ptr) + token * p.q.token_stride + head * p.q.head_stride;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) qs[warp][32 * e + lane] = __half2float(q[32 * e + lane]);
  __syncwarp();
  auto block = [&](int64_t j) -> const uint8_t* {
    const int64_t pi = j / p.cache.page_tokens;
    if (pi >= p.table_stride) return nullptr;
    const int64_t page = p.table[seq * p.table_stride + pi];
    if (page < 0 || page >= p.cache.n_pages) return nullptr;
    return kv_block<FMT, D>(p.cache, page, kvh, static_cast<int>(j % p.cache.page_tokens) / kKvBlockTokens);
  };
  float acc[D / 32], m, l;
  attend_row<D>(
      static_cast<int64_t>(ctx) + T,
      [&](int64_t j) { return (j < ctx || ((mask >> (j - ctx)) & 1)) && block(j) != nullptr; },
      [&](int64_t j) {
        const uint8_t* b = block(j);
        float s = 0.f;
        for (int d = 0; d < D; ++d) s = fmaf(qs[warp][d], kv_value<FMT, D>(b, false, j % kKvBlockTokens, d), s);
        return s * p.scale * kLog2e;
      },
      [&](int64_t j, int d) { return kv_value<FMT, D>(block(j), true, j % kKvBlockTokens, d); }, acc, m, l);
  store_row<D>(static_cast<__half*>(p.out.ptr) + token * p.out.token_stride + head * p.out.head_stride,
               p.lse ? p.lse + token * p.q_heads + head : nullptr, acc, m, l);
}

}  // namespace

cudaError_t launch_attn_tree(const TreeParams& p, cudaStream_t s) {
  const int64_t rows = p.n_q * p.q_heads;
  const unsigned grid = static_cast<unsigned>((rows + kThreads / 32 - 1) / (kThreads / 32));
  auto by_dim = [&](auto fmt) {
    constexpr int F = decltype(fmt)::value;
    if (p.cache.head_dim == 64) tree_row_kernel<F, 64><<<grid, kThreads, 0, s>>>(p);
    else tree_row_kernel<F, 128><<<grid, kThreads, 0, s>>>(p);
  };
  switch (p.cache.format) {
    case QGEMV_KV_F16: by_dim(std::integral_constant<int, QGEMV_KV_F16>()); break;
    case QGEMV_KV_INT8: by_dim(std::integral_constant<int, QGEMV_KV_INT8>()); break;
    default: by_dim(std::integral_constant<int, QGEMV_KV_Q4_0>());
  }
  return cudaGetLastError();
}

}  // namespace qgemv
