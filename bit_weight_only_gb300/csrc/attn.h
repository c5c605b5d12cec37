// attn.h -- the key/value cache and attention operators: the parameter
// structures that attn_api.cu hands to the kernels, and the launch calls.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "qgemv.h"

namespace qgemv {

// Tokens of a cache block: the unit of the page layout (kv_layout.cuh).
constexpr int kKvBlockTokens = 16;
// Most drafted tokens of a sequence in one attention call: a mask word.
constexpr int kMaxDrafts = 64;

// Rows of heads: element strides between tokens and between heads; the
// head_dim values of a row are contiguous.
struct RowsIn {
  const void* ptr;
  int64_t token_stride, head_stride;
};
struct RowsOut {
  void* ptr;
  int64_t token_stride, head_stride;
};

struct KvWriteParams {
  qgemv_kv_cache cache;
  RowsIn k, v;
  const int64_t* slots;
  int64_t n_tokens;
};

struct KvReadParams {
  qgemv_kv_cache cache;
  const int32_t* table;
  int64_t table_stride, n_seqs;
  const int32_t* starts;
  const int32_t* cu;
  int64_t n_tokens;
  RowsOut k, v;
};

struct TreeParams {
  qgemv_kv_cache cache;
  const int32_t* table;
  int64_t table_stride;
  // rows of the table of a sequence: 1, or one for each key/value head
  int table_heads;
  int n_seqs;
  const int32_t* ctx_lens;
  RowsIn q;
  int q_heads;
  const int32_t* cu_q;
  int64_t n_q;
  const uint64_t* masks;
  int max_ctx, max_new;
  float scale;
  RowsOut out;
  float* lse;
  uint8_t* ws;
};

struct PromptParams {
  int dtype, head_dim, q_heads, kv_heads;
  RowsIn q, k, v;
  int n_seqs;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int64_t n_q, n_k;
  float scale;
  RowsOut out;
  float* lse;
  uint8_t* ws;
};

cudaError_t launch_kv_write(const KvWriteParams& p, int dtype, cudaStream_t s);
cudaError_t launch_kv_read(const KvReadParams& p, int dtype, cudaStream_t s);
cudaError_t launch_attn_tree(const TreeParams& p, cudaStream_t s);
cudaError_t launch_attn_prompt(const PromptParams& p, cudaStream_t s);

// Workspace of the attention calls: a header -- the error word, and the prompt
// kernel's counters (next piece, blocks that are done), 0 between calls -- then
// the slots of whichever kernel runs, which need no setting up.
constexpr int64_t kWsHeaderBytes = 256;
int64_t tree_ws_bytes(int head_dim);
int64_t prompt_ws_bytes(int head_dim);

}  // namespace qgemv
