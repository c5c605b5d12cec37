// api_checks.h -- checks of arguments that the cache's and the attention's C
// calls share.  No exception crosses the ABI.
#pragma once

#include <cstdarg>
#include <cstdio>

#include "attn.h"
#include "formats.h"

namespace qgemv {

inline int fail(int code, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return report_error(code, msg);
}

inline int done(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return report_error(QGEMV_OK, "");
  return fail(QGEMV_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

inline bool cache_sizes_ok(int format, int64_t n_pages, int page_tokens, int kv_heads, int head_dim) {
  return format >= QGEMV_KV_F16 && format <= QGEMV_KV_Q4_0 && n_pages > 0 && n_pages < (int64_t(1) << 31) &&
         page_tokens >= 16 && page_tokens <= 256 && (page_tokens & (page_tokens - 1)) == 0 && kv_heads > 0 &&
         kv_heads <= 1024 && (head_dim == 64 || head_dim == 128);
}

inline int check_cache(const qgemv_kv_cache* c) {
  if (!c || !c->pages) return fail(QGEMV_ERR_ARG, "the cache or its pages are NULL");
  if (!cache_sizes_ok(c->format, c->n_pages, c->page_tokens, c->kv_heads, c->head_dim))
    return fail(QGEMV_ERR_ARG, "invalid cache: format %d, %lld pages of %d tokens, %d heads of %d", c->format,
                (long long)c->n_pages, c->page_tokens, c->kv_heads, c->head_dim);
  if (reinterpret_cast<uintptr_t>(c->pages) & 127) return fail(QGEMV_ERR_ALIGN, "the cache must be 128-byte aligned");
  return QGEMV_OK;
}

inline int dtype_size(int dtype) {
  return dtype == QGEMV_DT_F32 ? 4 : dtype == QGEMV_DT_F16 || dtype == QGEMV_DT_BF16 ? 2 : 0;
}

// Whether two of the rows (token i, head h) at i * ts + h * hs, of d elements
// each, share one.
inline bool rows_overlap(int64_t n, int heads, int64_t ts, int64_t hs, int d) {
  if ((n > 1 && ts < d) || (heads > 1 && hs < d)) return true;
  if (n <= 1 || heads <= 1 || ts >= (heads - 1) * hs + d || (hs - d) / ts >= n - 1) return false;
  for (int h = 1; h < heads; ++h) {  // the tokens just below and above h heads further
    const int64_t below = h * hs / ts, past = h * hs - below * ts;
    if ((below < n && past < d) || (below + 1 < n && ts - past < d)) return true;
  }
  return false;
}

// A row argument: not NULL, aligned, strides not negative nor (outputs, `n` of
// them) such that rows overlap.
inline int check_rows(const char* name, const void* ptr, int64_t ts, int64_t hs, int size, int heads, int head_dim, int64_t n,
               bool out) {
  if (!ptr) return fail(QGEMV_ERR_ARG, "%s is NULL", name);
  const int64_t lim = int64_t(1) << 38;
  if (ts < 0 || hs < 0 || ts > lim || hs > lim) return fail(QGEMV_ERR_ARG, "%s: strides outside [0, 2^38]", name);
  if (out && rows_overlap(n, heads, ts, hs, head_dim))
    return fail(QGEMV_ERR_ARG, "%s: output rows overlap (strides %lld, %lld)", name, (long long)ts, (long long)hs);
  if ((reinterpret_cast<uintptr_t>(ptr) & 15) || (ts * size & 15) || (hs * size & 15))
    return fail(QGEMV_ERR_ALIGN, "%s and its strides must be 16-byte aligned", name);
  return QGEMV_OK;
}

#define QG_TRY(expr)                  \
  do {                                \
    const int rc_ = (expr);           \
    if (rc_ != QGEMV_OK) return rc_;  \
  } while (0)

constexpr int64_t kMaxTokens = int64_t(1) << 30;

}  // namespace qgemv
