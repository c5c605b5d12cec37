// select.h -- key summaries of pages and the selection of pages by them:
// parameters and launch calls.
#pragma once

#include "attn.h"

namespace qgemv {

// A summary: for each page and head, 2 head_dim INT8 codes (largest values,
// then smallest) and an fp32 scale.
struct SummaryParams {
  qgemv_kv_cache cache;
  const int32_t* pages;
  int64_t n;
  int8_t* codes;
  float* scales;
};

struct SelectParams {
  qgemv_kv_cache cache;  // pages are not read
  const int8_t* codes;
  const float* scales;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* ctx_lens;
  RowsIn q;
  int q_heads;
  const int32_t* cu_q;
  int64_t n_q;
  int n_seqs, n_select, tail, width;  // entries of the tail and of a row of out
  int32_t* out;
  int32_t* out_lens;
};

// Pages of a sequence, at most: the scores lie in a block's shared memory.
int64_t select_most_pages();
cudaError_t launch_summary(const SummaryParams& p, cudaStream_t s);
cudaError_t launch_select(const SelectParams& p, cudaStream_t s);

}  // namespace qgemv
