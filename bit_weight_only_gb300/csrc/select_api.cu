// select_api.cu -- the C ABI of key summaries and of the selection of pages
// (include/qgemv.h): argument checks on the host, then the launches.
#include "api_checks.h"
#include "select.h"

namespace {

using namespace qgemv;

// Pages from the last whole one on that hold a context's end and its drafted tokens.
int tail_pages(int page_tokens) { return (2 * page_tokens + kMaxDrafts - 2) / page_tokens; }

int check_summary(const void* codes, const void* scales) {
  if (!codes || !scales) return fail(QGEMV_ERR_ARG, "the summary's codes or scales are NULL");
  if (reinterpret_cast<uintptr_t>(codes) & 15) return fail(QGEMV_ERR_ALIGN, "the summary's codes must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(scales) & 3) return fail(QGEMV_ERR_ALIGN, "the summary's scales must be 4-byte aligned");
  return QGEMV_OK;
}

}  // namespace

extern "C" {

int qgemv_kv_summarize(const qgemv_kv_cache* cache, const int32_t* pages, int64_t n, int8_t* codes, float* scales, void* stream) {
  QG_TRY(check_cache(cache));
  if (n < 0 || n >= (int64_t(1) << 31)) return fail(QGEMV_ERR_ARG, "n outside [0, 2^31)");
  QG_TRY(check_summary(codes, scales));
  if (n == 0) return report_error(QGEMV_OK, "");
  if (!pages) return fail(QGEMV_ERR_ARG, "pages is NULL");
  if (reinterpret_cast<uintptr_t>(pages) & 3) return fail(QGEMV_ERR_ALIGN, "pages must be 4-byte aligned");
  SummaryParams p = {*cache, pages, n, codes, scales};
  return done(launch_summary(p, static_cast<cudaStream_t>(stream)), "launching the summaries");
}

int64_t qgemv_kv_select_width(int page_tokens, int64_t n_select) {
  if (page_tokens < 16 || page_tokens > 256 || (page_tokens & (page_tokens - 1)) || n_select < 0 || n_select > (1 << 20)) return 0;
  return n_select + tail_pages(page_tokens);
}

int qgemv_kv_select(const qgemv_kv_cache* cache, const int8_t* codes, const float* scales, const int32_t* table,
                    int64_t table_stride, int64_t n_seqs, const int32_t* ctx_lens, const void* q, int64_t q_token_stride,
                    int64_t q_head_stride, int q_heads, const int32_t* cu_q, int64_t n_q, int64_t n_select, int32_t* pages,
                    int32_t* lens, void* stream) {
  QG_TRY(check_cache(cache));
  QG_TRY(check_summary(codes, scales));
  if (q_heads <= 0 || q_heads > 1024 || q_heads % cache->kv_heads)
    return fail(QGEMV_ERR_ARG, "q_heads=%d must be a positive multiple of kv_heads=%d, at most 1024", q_heads, cache->kv_heads);
  if (n_seqs < 0 || n_seqs > (1 << 20) || n_q < 0 || n_q > kMaxTokens || n_select < 0 || n_select > (1 << 20))
    return fail(QGEMV_ERR_ARG, "n_seqs or n_select outside [0, 2^20], or n_q outside [0, 2^30]");
  if (table_stride < 0 || table_stride > select_most_pages())
    return fail(QGEMV_ERR_ARG, "table_stride=%lld: at most %lld pages of a sequence", (long long)table_stride, (long long)select_most_pages());
  if (n_seqs == 0) return report_error(QGEMV_OK, "");
  if ((!table && table_stride > 0) || !ctx_lens || !cu_q || !pages || !lens)
    return fail(QGEMV_ERR_ARG, "table, ctx_lens, cu_q, pages or lens is NULL");
  if ((reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(ctx_lens) | reinterpret_cast<uintptr_t>(cu_q) |
       reinterpret_cast<uintptr_t>(pages) | reinterpret_cast<uintptr_t>(lens)) & 3)
    return fail(QGEMV_ERR_ALIGN, "index arrays must be 4-byte aligned");
  if (n_q > 0) QG_TRY(check_rows("q", q, q_token_stride, q_head_stride, 2, q_heads, cache->head_dim, n_q, false));
  SelectParams p = {};
  p.cache = *cache;
  p.codes = codes;
  p.scales = scales;
  p.table = table;
  p.table_stride = table_stride;
  p.ctx_lens = ctx_lens;
  p.q = {q, q_token_stride, q_head_stride};
  p.q_heads = q_heads;
  p.cu_q = cu_q;
  p.n_q = n_q;
  p.n_seqs = static_cast<int>(n_seqs);
  p.n_select = static_cast<int>(n_select);
  p.tail = tail_pages(cache->page_tokens);
  p.width = static_cast<int>(qgemv_kv_select_width(cache->page_tokens, n_select));
  p.out = pages;
  p.out_lens = lens;
  return done(launch_select(p, static_cast<cudaStream_t>(stream)), "launching the selection");
}

}  // extern "C"
