// attn_api.cu -- the C ABI of the key/value cache and the attention calls
// (include/qgemv.h): argument checks on the host, then the launches.  No
// exception crosses the ABI and no call allocates.
#include <cstdarg>
#include <cstdio>

#include "attn.h"
#include "formats.h"

namespace {

int fail(int code, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return qgemv::report_error(code, msg);
}

int done(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return qgemv::report_error(QGEMV_OK, "");
  return fail(QGEMV_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

bool cache_sizes_ok(int format, int64_t n_pages, int page_tokens, int kv_heads, int head_dim) {
  return format >= QGEMV_KV_F16 && format <= QGEMV_KV_Q4_0 && n_pages > 0 && n_pages < (int64_t(1) << 31) &&
         page_tokens >= 16 && page_tokens <= 256 && (page_tokens & (page_tokens - 1)) == 0 && kv_heads > 0 &&
         kv_heads <= 1024 && (head_dim == 64 || head_dim == 128);
}

int check_cache(const qgemv_kv_cache* c) {
  if (!c || !c->pages) return fail(QGEMV_ERR_ARG, "the cache or its pages are NULL");
  if (!cache_sizes_ok(c->format, c->n_pages, c->page_tokens, c->kv_heads, c->head_dim))
    return fail(QGEMV_ERR_ARG, "invalid cache: format %d, %lld pages of %d tokens, %d heads of %d", c->format,
                (long long)c->n_pages, c->page_tokens, c->kv_heads, c->head_dim);
  if (reinterpret_cast<uintptr_t>(c->pages) & 127) return fail(QGEMV_ERR_ALIGN, "the cache must be 128-byte aligned");
  return QGEMV_OK;
}

int dtype_size(int dtype) {
  return dtype == QGEMV_DT_F32 ? 4 : dtype == QGEMV_DT_F16 || dtype == QGEMV_DT_BF16 ? 2 : 0;
}

// Whether two of the rows (token i, head h) at i * ts + h * hs, of d elements
// each, share one.
bool rows_overlap(int64_t n, int heads, int64_t ts, int64_t hs, int d) {
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
int check_rows(const char* name, const void* ptr, int64_t ts, int64_t hs, int size, int heads, int head_dim, int64_t n,
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

int check_ws(void* ws, int64_t ws_bytes, int64_t n_seqs, int q_heads, int head_dim) {
  if (!ws) return fail(QGEMV_ERR_ARG, "the workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) & 255) return fail(QGEMV_ERR_ALIGN, "the workspace must be 256-byte aligned");
  const int64_t need = qgemv_attn_ws_bytes(n_seqs, q_heads, head_dim);
  if (ws_bytes < need)
    return fail(QGEMV_ERR_ARG, "the workspace has %lld bytes, %lld are needed", (long long)ws_bytes, (long long)need);
  return QGEMV_OK;
}

#define QG_TRY(expr)                  \
  do {                                \
    const int rc_ = (expr);           \
    if (rc_ != QGEMV_OK) return rc_;  \
  } while (0)

constexpr int64_t kMaxTokens = int64_t(1) << 30;

}  // namespace

extern "C" {

int64_t qgemv_kv_bytes(int format, int64_t n_pages, int page_tokens, int kv_heads, int head_dim) {
  if (!cache_sizes_ok(format, n_pages, page_tokens, kv_heads, head_dim)) return 0;
  const int64_t row = format == QGEMV_KV_F16 ? 2 * head_dim : format == QGEMV_KV_INT8 ? head_dim + 4 : head_dim / 32 * 18;
  return n_pages * page_tokens * kv_heads * 2 * row;
}

int qgemv_kv_write(const qgemv_kv_cache* cache, int dtype, const void* k, int64_t k_token_stride,
                   int64_t k_head_stride, const void* v, int64_t v_token_stride, int64_t v_head_stride,
                   const int64_t* slots, int64_t n_tokens, void* stream) {
  QG_TRY(check_cache(cache));
  const int size = dtype_size(dtype);
  if (size == 0) return fail(QGEMV_ERR_ARG, "unknown dtype %d", dtype);
  if (n_tokens < 0 || n_tokens > kMaxTokens) return fail(QGEMV_ERR_ARG, "n_tokens outside [0, 2^30]");
  if (n_tokens == 0) return qgemv::report_error(QGEMV_OK, "");
  QG_TRY(check_rows("k", k, k_token_stride, k_head_stride, size, cache->kv_heads, cache->head_dim, n_tokens, false));
  QG_TRY(check_rows("v", v, v_token_stride, v_head_stride, size, cache->kv_heads, cache->head_dim, n_tokens, false));
  if (!slots) return fail(QGEMV_ERR_ARG, "slots is NULL");
  if (reinterpret_cast<uintptr_t>(slots) & 7) return fail(QGEMV_ERR_ALIGN, "slots must be 8-byte aligned");
  qgemv::KvWriteParams p = {*cache, {k, k_token_stride, k_head_stride}, {v, v_token_stride, v_head_stride}, slots, n_tokens};
  return done(qgemv::launch_kv_write(p, dtype, static_cast<cudaStream_t>(stream)), "launching the cache write");
}

int qgemv_kv_read(const qgemv_kv_cache* cache, const int32_t* table, int64_t table_stride, int64_t n_seqs,
                  const int32_t* starts, const int32_t* cu, int64_t n_tokens, int dtype, void* k,
                  int64_t k_token_stride, int64_t k_head_stride, void* v, int64_t v_token_stride,
                  int64_t v_head_stride, void* stream) {
  QG_TRY(check_cache(cache));
  const int size = dtype_size(dtype);
  if (size == 0) return fail(QGEMV_ERR_ARG, "unknown dtype %d", dtype);
  if (n_tokens < 0 || n_tokens > kMaxTokens) return fail(QGEMV_ERR_ARG, "n_tokens outside [0, 2^30]");
  if (n_seqs < 0 || n_seqs > kMaxTokens || table_stride < 0) return fail(QGEMV_ERR_ARG, "n_seqs or table_stride is invalid");
  if (n_tokens == 0 || n_seqs == 0) return qgemv::report_error(QGEMV_OK, "");
  if ((!table && table_stride > 0) || !cu) return fail(QGEMV_ERR_ARG, "table or cu is NULL");
  if (((reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(cu) | reinterpret_cast<uintptr_t>(starts)) & 3))
    return fail(QGEMV_ERR_ALIGN, "table, starts and cu must be 4-byte aligned");
  QG_TRY(check_rows("k", k, k_token_stride, k_head_stride, size, cache->kv_heads, cache->head_dim, n_tokens, true));
  QG_TRY(check_rows("v", v, v_token_stride, v_head_stride, size, cache->kv_heads, cache->head_dim, n_tokens, true));
  qgemv::KvReadParams p = {*cache, table, table_stride, n_seqs, starts, cu, n_tokens,
                           {k, k_token_stride, k_head_stride}, {v, v_token_stride, v_head_stride}};
  return done(qgemv::launch_kv_read(p, dtype, static_cast<cudaStream_t>(stream)), "launching the cache read");
}

int64_t qgemv_attn_ws_bytes(int64_t n_seqs, int q_heads, int head_dim) {
  if (n_seqs < 0 || n_seqs > kMaxTokens || q_heads <= 0 || q_heads > 1024 || (head_dim != 64 && head_dim != 128)) return 0;
  const int64_t tree = qgemv::tree_ws_bytes(head_dim), prompt = qgemv::prompt_ws_bytes(head_dim);
  return qgemv::kWsHeaderBytes + (tree > prompt ? tree : prompt);
}

int qgemv_attn_ws_init(void* ws, int64_t ws_bytes, void* stream) {
  if (!ws || ws_bytes < qgemv::kWsHeaderBytes) return fail(QGEMV_ERR_ARG, "the workspace is NULL or too small");
  return done(cudaMemsetAsync(ws, 0, static_cast<size_t>(qgemv::kWsHeaderBytes), static_cast<cudaStream_t>(stream)),
              "clearing the workspace");
}

int qgemv_attn_status(void* ws) {
  if (!ws) return fail(QGEMV_ERR_ARG, "the workspace is NULL");
  int err = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(&err, ws, sizeof(int), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && err) e = cudaMemset(ws, 0, sizeof(int));
  if (e != cudaSuccess) return done(e, "reading the attention status");
  if (err) return fail(QGEMV_ERR_TIMEOUT, "an attention kernel gave up a bounded wait (code %d)", err);
  return qgemv::report_error(QGEMV_OK, "");
}

int qgemv_attn_tree(const qgemv_kv_cache* cache, const int32_t* table, int64_t table_stride, int64_t n_seqs,
                    const int32_t* ctx_lens, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                    int q_heads, const int32_t* cu_q, int64_t n_q, const uint64_t* masks, int64_t max_ctx,
                    int64_t max_new, float scale, void* out, int64_t out_token_stride, int64_t out_head_stride,
                    float* lse, void* ws, int64_t ws_bytes, void* stream) {
  QG_TRY(check_cache(cache));
  if (q_heads <= 0 || q_heads > 1024 || q_heads % cache->kv_heads)
    return fail(QGEMV_ERR_ARG, "q_heads=%d must be a positive multiple of kv_heads=%d, at most 1024", q_heads, cache->kv_heads);
  if (n_seqs < 0 || n_seqs > (1 << 20) || n_q < 0 || n_q > kMaxTokens || table_stride < 0 || max_ctx < 0 || max_new < 0)
    return fail(QGEMV_ERR_ARG, "n_seqs outside [0, 2^20], n_q outside [0, 2^30], or a negative size");
  if (n_q == 0 || n_seqs == 0) return qgemv::report_error(QGEMV_OK, "");
  if ((!table && table_stride > 0) || !ctx_lens || !cu_q) return fail(QGEMV_ERR_ARG, "table, ctx_lens or cu_q is NULL");
  if (((reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(ctx_lens) | reinterpret_cast<uintptr_t>(cu_q) |
        reinterpret_cast<uintptr_t>(lse)) & 3) || (reinterpret_cast<uintptr_t>(masks) & 7))
    return fail(QGEMV_ERR_ALIGN, "index arrays and lse must be aligned to their elements");
  QG_TRY(check_rows("q", q, q_token_stride, q_head_stride, 2, q_heads, cache->head_dim, n_q, false));
  QG_TRY(check_rows("out", out, out_token_stride, out_head_stride, 2, q_heads, cache->head_dim, n_q, true));
  QG_TRY(check_ws(ws, ws_bytes, n_seqs, q_heads, cache->head_dim));
  const int64_t lim = int64_t(1) << 30;
  qgemv::TreeParams p = {*cache, table, table_stride, static_cast<int>(n_seqs), ctx_lens,
                         {q, q_token_stride, q_head_stride}, q_heads, cu_q, n_q, masks,
                         static_cast<int>(max_ctx < lim ? max_ctx : lim), static_cast<int>(max_new < lim ? max_new : lim),
                         scale, {out, out_token_stride, out_head_stride}, lse, static_cast<uint8_t*>(ws)};
  return done(qgemv::launch_attn_tree(p, static_cast<cudaStream_t>(stream)), "launching the attention");
}

int qgemv_attn_prompt(int dtype, int head_dim, int q_heads, int kv_heads, const void* q, int64_t q_token_stride,
                      int64_t q_head_stride, const void* k, int64_t k_token_stride, int64_t k_head_stride,
                      const void* v, int64_t v_token_stride, int64_t v_head_stride, int64_t n_seqs,
                      const int32_t* cu_q, const int32_t* cu_k, int64_t n_q, int64_t n_k, int64_t max_q,
                      float scale, void* out, int64_t out_token_stride, int64_t out_head_stride, float* lse,
                      void* ws, int64_t ws_bytes, void* stream) {
  if (dtype != QGEMV_DT_F16 && dtype != QGEMV_DT_BF16)
    return fail(QGEMV_ERR_ARG, "dtype %d: prompts are fp16 or bf16", dtype);
  if (head_dim != 64 && head_dim != 128) return fail(QGEMV_ERR_ARG, "head_dim=%d must be 64 or 128", head_dim);
  if (kv_heads <= 0 || q_heads <= 0 || q_heads > 1024 || q_heads % kv_heads)
    return fail(QGEMV_ERR_ARG, "q_heads=%d must be a positive multiple of kv_heads=%d, at most 1024", q_heads, kv_heads);
  if (n_seqs < 0 || n_seqs > (1 << 20) || n_q < 0 || n_q > kMaxTokens || n_k < 0 || n_k > kMaxTokens || max_q < 0)
    return fail(QGEMV_ERR_ARG, "n_seqs outside [0, 2^20], or a token count outside [0, 2^30]");
  if (n_q == 0 || n_seqs == 0 || max_q == 0) return qgemv::report_error(QGEMV_OK, "");
  if (q_heads / kv_heads > 128)
    return fail(QGEMV_ERR_ARG, "%d query heads of a key/value head: at most 128", q_heads / kv_heads);
  if (n_q * (q_heads / 128.0) + static_cast<double>(n_seqs) * kv_heads > 2e9)
    return fail(QGEMV_ERR_ARG, "too many rows for one call: %lld tokens of %d heads", (long long)n_q, q_heads);
  if (!cu_q || !cu_k) return fail(QGEMV_ERR_ARG, "cu_q or cu_k is NULL");
  if ((reinterpret_cast<uintptr_t>(cu_q) | reinterpret_cast<uintptr_t>(cu_k) | reinterpret_cast<uintptr_t>(lse)) & 3)
    return fail(QGEMV_ERR_ALIGN, "index arrays and lse must be 4-byte aligned");
  QG_TRY(check_rows("q", q, q_token_stride, q_head_stride, 2, q_heads, head_dim, n_q, false));
  if (n_k > 0) {
    QG_TRY(check_rows("k", k, k_token_stride, k_head_stride, 2, kv_heads, head_dim, n_k, false));
    QG_TRY(check_rows("v", v, v_token_stride, v_head_stride, 2, kv_heads, head_dim, n_k, false));
    if ((n_q > 1 && q_token_stride == 0) || (q_heads > 1 && q_head_stride == 0) ||
        (n_k > 1 && (k_token_stride == 0 || v_token_stride == 0)) || (kv_heads > 1 && (k_head_stride == 0 || v_head_stride == 0)))
      return fail(QGEMV_ERR_ARG, "q, k and v of a prompt have no strides of zero");
  }
  QG_TRY(check_rows("out", out, out_token_stride, out_head_stride, 2, q_heads, head_dim, n_q, true));
  QG_TRY(check_ws(ws, ws_bytes, n_seqs, q_heads, head_dim));
  qgemv::PromptParams p = {dtype, head_dim, q_heads, kv_heads,
                           {q, q_token_stride, q_head_stride}, {k, k_token_stride, k_head_stride},
                           {v, v_token_stride, v_head_stride}, static_cast<int>(n_seqs), cu_q, cu_k, n_q, n_k, scale,
                           {out, out_token_stride, out_head_stride}, lse, static_cast<uint8_t*>(ws)};
  return done(qgemv::launch_attn_prompt(p, static_cast<cudaStream_t>(stream)), "launching the prompt attention");
}

}  // extern "C"
