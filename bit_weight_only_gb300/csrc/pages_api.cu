// pages_api.cu -- the C ABI of the page pool and of page copies
// (include/qgemv.h): argument checks on the host, then the launches.
#include "api_checks.h"
#include "pages.h"

#include <initializer_list>

namespace {

using namespace qgemv;

constexpr int64_t kMaxEntries = int64_t(1) << 20;  // of a row of a table, in a pool's call

bool aligned4(std::initializer_list<const void*> ps) {
  uintptr_t a = 0;
  for (const void* p : ps) a |= reinterpret_cast<uintptr_t>(p);
  return (a & 3) == 0;
}

int check_pool(const int32_t* refs, int64_t n_pages, int page_tokens, int64_t table_stride, int64_t n_seqs) {
  if (!refs) return fail(QGEMV_ERR_ARG, "refs is NULL");
  if (n_pages < 1 || n_pages >= (int64_t(1) << 31)) return fail(QGEMV_ERR_ARG, "n_pages outside [1, 2^31)");
  if (page_tokens < 16 || page_tokens > 256 || (page_tokens & (page_tokens - 1)))
    return fail(QGEMV_ERR_ARG, "page_tokens=%d: 16, 32, 64, 128 or 256", page_tokens);
  if (n_seqs < 0 || n_seqs > kMaxPoolSeqs) return fail(QGEMV_ERR_ARG, "rows outside [0, %d]", kMaxPoolSeqs);
  if (table_stride < 0 || table_stride > kMaxEntries) return fail(QGEMV_ERR_ARG, "table_stride outside [0, 2^20]");
  if (reinterpret_cast<uintptr_t>(refs) & 3) return fail(QGEMV_ERR_ALIGN, "refs must be 4-byte aligned");
  return QGEMV_OK;
}

PoolParams pool(int32_t* refs, int64_t n_pages, int page_tokens, int32_t* table, int64_t table_stride, int64_t n_seqs) {
  PoolParams p = {};
  p.refs = refs;
  p.n_pages = n_pages;
  p.page_tokens = page_tokens;
  p.table = table;
  p.table_stride = p.old_stride = table_stride;
  p.n_seqs = n_seqs;
  return p;
}

}  // namespace

extern "C" {

int qgemv_pool_reserve(int32_t* refs, int64_t n_pages, int page_tokens, int32_t* table, int64_t table_stride, int64_t n_seqs,
                       const int32_t* have, const int32_t* need, int32_t* state, void* stream) {
  QG_TRY(check_pool(refs, n_pages, page_tokens, table_stride, n_seqs));
  if (n_seqs == 0 || table_stride == 0) return report_error(QGEMV_OK, "");
  if (!table || !have || !need || !state) return fail(QGEMV_ERR_ARG, "table, have, need or state is NULL");
  if (!aligned4({table, have, need, state})) return fail(QGEMV_ERR_ALIGN, "arrays must be 4-byte aligned");
  PoolParams p = pool(refs, n_pages, page_tokens, table, table_stride, n_seqs);
  p.from = have;
  p.to = need;
  p.state = state;
  return done(launch_pool_reserve(p, static_cast<cudaStream_t>(stream)), "launching the reservation");
}

int qgemv_pool_fork(int32_t* refs, int64_t n_pages, int page_tokens, const int32_t* table, int64_t table_stride, int64_t n_rows,
                    const int32_t* parents, int64_t n_new, const int32_t* lens, int32_t* new_table, int32_t* src, int32_t* dst,
                    int32_t* tokens, int32_t* state, void* stream) {
  QG_TRY(check_pool(refs, n_pages, page_tokens, table_stride, n_rows));
  QG_TRY(check_pool(refs, n_pages, page_tokens, table_stride, n_new));
  if (n_rows == 0 && n_new == 0) return report_error(QGEMV_OK, "");
  if (n_rows > 0 && ((!table && table_stride > 0) || !lens)) return fail(QGEMV_ERR_ARG, "table or lens is NULL");
  if (n_new > 0 && (!parents || (!new_table && table_stride > 0) || !src || !dst || !tokens))
    return fail(QGEMV_ERR_ARG, "parents, new_table, src, dst or tokens is NULL");
  if (!state) return fail(QGEMV_ERR_ARG, "state is NULL");
  if (!aligned4({table, parents, lens, new_table, src, dst, tokens, state})) return fail(QGEMV_ERR_ALIGN, "arrays must be 4-byte aligned");
  if (new_table && new_table < table + n_rows * table_stride && table < new_table + n_new * table_stride)
    return fail(QGEMV_ERR_ARG, "the new table overlaps the old one");
  PoolParams p = pool(refs, n_pages, page_tokens, new_table, table_stride, n_new);
  p.old_table = table;
  p.n_old = n_rows;
  p.parents = parents;
  p.from = lens;
  p.src = src;
  p.dst = dst;
  p.tokens = tokens;
  p.state = state;
  return done(launch_pool_fork(p, static_cast<cudaStream_t>(stream)), "launching the fork");
}

int qgemv_pool_release(int32_t* refs, int64_t n_pages, int page_tokens, int32_t* table, int64_t table_stride, int64_t n_seqs,
                       const int32_t* lens, const int32_t* keep, void* stream) {
  QG_TRY(check_pool(refs, n_pages, page_tokens, table_stride, n_seqs));
  if (n_seqs == 0 || table_stride == 0) return report_error(QGEMV_OK, "");
  if (!table || !lens) return fail(QGEMV_ERR_ARG, "table or lens is NULL");
  if (!aligned4({table, lens, keep})) return fail(QGEMV_ERR_ALIGN, "arrays must be 4-byte aligned");
  PoolParams p = pool(refs, n_pages, page_tokens, table, table_stride, n_seqs);
  p.from = keep;
  p.to = lens;
  return done(launch_pool_release(p, static_cast<cudaStream_t>(stream)), "launching the release");
}

int64_t qgemv_pool_ws_bytes(int64_t n_pages) {
  return n_pages < 1 || n_pages >= (int64_t(1) << 31) ? 0 : 4 * ((n_pages + kPoolTile - 1) / kPoolTile + n_pages);
}

int qgemv_pool_compact(int32_t* refs, int64_t n_pages, const int32_t* table, int64_t table_stride, int64_t n_seqs,
                       int32_t* new_table, int32_t* src, int32_t* dst, int64_t n_moves, void* ws, int64_t ws_bytes, void* stream) {
  QG_TRY(check_pool(refs, n_pages, 16, table_stride, n_seqs));
  if (n_moves < n_pages / 2) return fail(QGEMV_ERR_ARG, "n_moves=%lld: room for n_pages / 2 moves is needed", (long long)n_moves);
  if (n_moves > n_pages) return fail(QGEMV_ERR_ARG, "n_moves=%lld is more than there are pages", (long long)n_moves);
  if (n_seqs > 0 && table_stride > 0 && (!table || !new_table)) return fail(QGEMV_ERR_ARG, "table or new_table is NULL");
  if (!ws || (n_moves > 0 && (!src || !dst))) return fail(QGEMV_ERR_ARG, "src, dst or the workspace is NULL");
  if (!aligned4({table, new_table, src, dst, ws})) return fail(QGEMV_ERR_ALIGN, "arrays must be 4-byte aligned");
  if (ws_bytes < qgemv_pool_ws_bytes(n_pages))
    return fail(QGEMV_ERR_ARG, "the workspace has %lld bytes, %lld are needed", (long long)ws_bytes, (long long)qgemv_pool_ws_bytes(n_pages));
  if (new_table != table && new_table && new_table < table + n_seqs * table_stride && table < new_table + n_seqs * table_stride)
    return fail(QGEMV_ERR_ARG, "the new table overlaps the old one in part");
  PoolParams p = pool(refs, n_pages, 16, new_table, table_stride, n_seqs);
  p.old_table = table;
  p.src = src;
  p.dst = dst;
  p.n_moves = n_moves;
  p.scratch = static_cast<int32_t*>(ws);
  return done(launch_pool_compact(p, static_cast<cudaStream_t>(stream)), "launching the compaction");
}

int qgemv_kv_copy_pages(const qgemv_kv_cache* cache, const int32_t* src, const int32_t* dst, const int32_t* tokens, int64_t n,
                        void* stream) {
  QG_TRY(check_cache(cache));
  if (n < 0 || n >= (int64_t(1) << 31)) return fail(QGEMV_ERR_ARG, "n outside [0, 2^31)");
  if (n == 0) return report_error(QGEMV_OK, "");
  if (!src || !dst) return fail(QGEMV_ERR_ARG, "src or dst is NULL");
  if (!aligned4({src, dst, tokens})) return fail(QGEMV_ERR_ALIGN, "arrays must be 4-byte aligned");
  CopyPagesParams p = {};
  p.pages = static_cast<uint8_t*>(cache->pages);
  p.n_pages = cache->n_pages;
  p.heads = cache->kv_heads;
  p.blocks = cache->page_tokens / kKvBlockTokens;
  const int row = cache->format == QGEMV_KV_F16 ? 2 * cache->head_dim
                  : cache->format == QGEMV_KV_INT8 ? cache->head_dim + 4 : cache->head_dim / 32 * 18;
  p.block_bytes = kKvBlockTokens * 2 * row;
  p.page_bytes = static_cast<int64_t>(p.heads) * p.blocks * p.block_bytes;
  p.src = src;
  p.dst = dst;
  p.tokens = tokens;
  p.n = n;
  return done(launch_copy_pages(p, static_cast<cudaStream_t>(stream)), "launching the page copies");
}

}  // extern "C"
