// pages.h -- bookkeeping and copying of cache pages: parameters and launch
// calls.
#pragma once

#include "attn.h"

namespace qgemv {

// Sequences of a bookkeeping call, at most (their needs are summed in shared
// memory).
constexpr int kMaxPoolSeqs = 4096;
// Pages of a tile of the compacting scan.
constexpr int kPoolTile = 4096;

struct PoolParams {
  int32_t* refs;
  int64_t n_pages;
  int page_tokens;
  int32_t* table;
  int64_t table_stride, n_seqs;
  const int32_t* from;  // reserve: have; fork: lens; release: keep (may be NULL)
  const int32_t* to;    // reserve: need; release: lens
  int32_t* state;       // pages that were missing; arrivals, 0 between calls
  // fork
  const int32_t* old_table;
  int64_t old_stride, n_old;
  const int32_t* parents;
  int32_t* src;
  int32_t* dst;
  int32_t* tokens;
  int64_t n_moves;
  // compact: counts of the tiles, then a number for each page
  int32_t* scratch;
};

cudaError_t launch_pool_reserve(const PoolParams& p, cudaStream_t s);
cudaError_t launch_pool_fork(const PoolParams& p, cudaStream_t s);
cudaError_t launch_pool_release(const PoolParams& p, cudaStream_t s);
cudaError_t launch_pool_compact(const PoolParams& p, cudaStream_t s);

struct CopyPagesParams {
  uint8_t* pages;
  int64_t n_pages, page_bytes;
  int heads, blocks, block_bytes;  // a page: heads x blocks of 16 tokens
  const int32_t* src;
  const int32_t* dst;
  const int32_t* tokens;
  int64_t n;
};
cudaError_t launch_copy_pages(const CopyPagesParams& p, cudaStream_t s);

}  // namespace qgemv
