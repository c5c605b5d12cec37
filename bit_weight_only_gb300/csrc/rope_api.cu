// rope_api.cu -- the C ABI of the rotary positions (include/qgemv.h):
// argument checks on the host, then the launches.
#include <cmath>

#include "api_checks.h"
#include "rope.h"

namespace {

using namespace qgemv;

constexpr double kMaxFreq = 1024;

// round(2^64 f / 2 pi) mod 2^64, to less than 1: f = m 2^e with a whole m of at
// most 53 bits, and 2^128 / 2 pi from the digits of pi.
uint64_t turns_of(double f) {
  constexpr uint64_t kHi = 0x28be60db9391054aull, kLo = 0x7f09d5f47d4d3770ull;
  int e = 0;
  const double m = std::frexp(std::fabs(f), &e) * 0x1p53;  // f = m 2^(e - 53)
  const unsigned __int128 w = static_cast<uint64_t>(m);
  const unsigned __int128 p = w * kHi + ((w * kLo) >> 64);  // m 2^64 / 2 pi
  const int shift = 53 - e;                                  // at least 42
  const uint64_t t = shift >= 120 ? 0 : static_cast<uint64_t>((p + (static_cast<unsigned __int128>(1) << (shift - 1))) >> shift);
  return f < 0 ? 0 - t : t;
}

int check_plan(const void* plan, int pairs, int pairing, int n_axes, const int32_t* positions, int head_dim, int64_t n_tokens) {
  if (head_dim != 64 && head_dim != 128) return fail(QGEMV_ERR_ARG, "head_dim=%d must be 64 or 128", head_dim);
  if (pairs < 1 || pairs > head_dim / 2) return fail(QGEMV_ERR_ARG, "%d pairs of a head of %d", pairs, head_dim);
  if (pairing != QGEMV_ROPE_HALVES && pairing != QGEMV_ROPE_NEIGHBOURS) return fail(QGEMV_ERR_ARG, "unknown pairing %d", pairing);
  if (n_axes < 1 || n_axes > 4) return fail(QGEMV_ERR_ARG, "n_axes=%d outside [1, 4]", n_axes);
  if (n_tokens < 0 || n_tokens > kMaxTokens) return fail(QGEMV_ERR_ARG, "n_tokens outside [0, 2^30]");
  if (n_tokens == 0) return QGEMV_OK;
  if (!plan || !positions) return fail(QGEMV_ERR_ARG, "the plan or the positions are NULL");
  if (reinterpret_cast<uintptr_t>(plan) & 15) return fail(QGEMV_ERR_ALIGN, "the plan must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(positions) & 3) return fail(QGEMV_ERR_ALIGN, "positions must be 4-byte aligned");
  return QGEMV_OK;
}

}  // namespace

extern "C" {

int64_t qgemv_rope_plan_bytes(int pairs) { return pairs < 1 || pairs > 64 ? 0 : 16 * static_cast<int64_t>(pairs); }

int qgemv_rope_plan(const double* freqs, const int32_t* axes, int pairs, void* plan) {
  if (pairs < 1 || pairs > 64) return fail(QGEMV_ERR_ARG, "pairs=%d outside [1, 64]", pairs);
  if (!freqs || !axes || !plan) return fail(QGEMV_ERR_ARG, "freqs, axes or plan is NULL");
  if (reinterpret_cast<uintptr_t>(plan) & 7) return fail(QGEMV_ERR_ALIGN, "the plan must be 8-byte aligned");
  for (int j = 0; j < pairs; ++j) {
    if (!(std::fabs(freqs[j]) <= kMaxFreq)) return fail(QGEMV_ERR_ARG, "frequency %d is %g, outside [-1024, 1024]", j, freqs[j]);
    if (axes[j] < 0 || axes[j] > 3) return fail(QGEMV_ERR_ARG, "axis %d of pair %d outside [0, 3]", (int)axes[j], j);
  }
  uint64_t* out = static_cast<uint64_t*>(plan);
  for (int j = 0; j < pairs; ++j) {
    out[2 * j] = turns_of(freqs[j]);
    out[2 * j + 1] = static_cast<uint64_t>(axes[j]);
  }
  return report_error(QGEMV_OK, "");
}

int qgemv_rope_rows(const void* plan, int pairs, int pairing, int n_axes, const int32_t* positions, int dtype, int heads,
                    int head_dim, const void* x, int64_t x_token_stride, int64_t x_head_stride, int64_t n_tokens,
                    int out_dtype, void* out, int64_t out_token_stride, int64_t out_head_stride, void* stream) {
  QG_TRY(check_plan(plan, pairs, pairing, n_axes, positions, head_dim, n_tokens));
  const int size = dtype_size(dtype), out_size = dtype_size(out_dtype);
  if (size == 0 || out_size == 0) return fail(QGEMV_ERR_ARG, "unknown dtype %d or %d", dtype, out_dtype);
  if (heads < 1 || heads > 1024) return fail(QGEMV_ERR_ARG, "heads=%d outside [1, 1024]", heads);
  if (n_tokens == 0) return report_error(QGEMV_OK, "");
  QG_TRY(check_rows("x", x, x_token_stride, x_head_stride, size, heads, head_dim, n_tokens, false));
  QG_TRY(check_rows("out", out, out_token_stride, out_head_stride, out_size, heads, head_dim, n_tokens, true));
  RopeParams p = {};
  p.q = {x, x_token_stride, x_head_stride};
  p.out = {out, out_token_stride, out_head_stride};
  p.out_dtype = out_dtype;
  p.q_heads = heads;
  p.positions = positions;
  p.n_axes = n_axes;
  p.pairs = pairs;
  p.neighbours = pairing == QGEMV_ROPE_NEIGHBOURS;
  p.plan = static_cast<const uint4*>(plan);
  p.n_tokens = n_tokens;
  return done(launch_rope(p, dtype, head_dim, static_cast<cudaStream_t>(stream)), "launching the rotation");
}

int qgemv_kv_write_rotated(const qgemv_kv_cache* cache, const void* plan, int pairs, int pairing, int n_axes,
                           const int32_t* positions, int dtype, const void* q, int64_t q_token_stride,
                           int64_t q_head_stride, int q_heads, const void* k, int64_t k_token_stride,
                           int64_t k_head_stride, const void* v, int64_t v_token_stride, int64_t v_head_stride,
                           const int64_t* slots, int64_t n_tokens, int out_dtype, void* q_out,
                           int64_t out_token_stride, int64_t out_head_stride, void* stream) {
  QG_TRY(check_cache(cache));
  QG_TRY(check_plan(plan, pairs, pairing, n_axes, positions, cache->head_dim, n_tokens));
  const int size = dtype_size(dtype), out_size = dtype_size(out_dtype);
  if (size == 0 || out_size == 0) return fail(QGEMV_ERR_ARG, "unknown dtype %d or %d", dtype, out_dtype);
  if (q_heads < 1 || q_heads > 1024) return fail(QGEMV_ERR_ARG, "q_heads=%d outside [1, 1024]", q_heads);
  if (n_tokens == 0) return report_error(QGEMV_OK, "");
  const int d = cache->head_dim;
  QG_TRY(check_rows("q", q, q_token_stride, q_head_stride, size, q_heads, d, n_tokens, false));
  QG_TRY(check_rows("k", k, k_token_stride, k_head_stride, size, cache->kv_heads, d, n_tokens, false));
  QG_TRY(check_rows("v", v, v_token_stride, v_head_stride, size, cache->kv_heads, d, n_tokens, false));
  QG_TRY(check_rows("q_out", q_out, out_token_stride, out_head_stride, out_size, q_heads, d, n_tokens, true));
  if (!slots) return fail(QGEMV_ERR_ARG, "slots is NULL");
  if (reinterpret_cast<uintptr_t>(slots) & 7) return fail(QGEMV_ERR_ALIGN, "slots must be 8-byte aligned");
  RopeParams p = {*cache, {q, q_token_stride, q_head_stride}, {k, k_token_stride, k_head_stride},
                  {v, v_token_stride, v_head_stride}, {q_out, out_token_stride, out_head_stride}, out_dtype, q_heads, slots,
                  positions, n_axes, pairs, pairing == QGEMV_ROPE_NEIGHBOURS, static_cast<const uint4*>(plan), n_tokens};
  return done(launch_rope(p, dtype, d, static_cast<cudaStream_t>(stream)), "launching the rotated cache write");
}

}  // extern "C"
