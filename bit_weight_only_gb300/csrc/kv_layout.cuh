// kv_layout.cuh -- the page layout of the key/value cache and its codes.
//
// A page holds page_tokens tokens of every key/value head; head h of page p
// is one run of page_tokens / 16 blocks of 16 tokens.  A block is contiguous
//
//     [K codes 16 x RB] [V codes 16 x RB] [K scales] [V scales]
//
// (RB bytes per token: fp16 2d, INT8 d, Q4_0 d / 2), so that any range of
// blocks of a page is one bulk copy, and a warp of the attention kernel takes
// a block.  Inside the code regions the bytes lie so that the attention's
// matrix operands are read from shared memory by the widest loads without
// bank conflicts (lane = 4g + t; one MMA step takes 4 values of k from each
// of the four t and a row from each of the eight g):
//   * fp16, K and V: chunks of 64 values, each 16 rows of 128 bytes in the
//     128-byte swizzle (16-byte unit u of token r at u ^ (r & 7)): what the
//     tensor cores read, as a descriptor operand or by ldmatrix.
//   * K: lane (g, t) reads token g.  INT8: 16-byte units t (values 64h + 16t
//     ..), codes + 128; Q4_0: one cell of d/32 words, word i the 8 values 32i
//     + 8t .., in nibble order 0 2 4 6 1 3 5 7 (so that masking a word yields
//     neighbouring pairs).  Rows of 128 bytes swap their 64-byte halves for
//     odd tokens.
//   * V: lane (g, t) reads tokens 2t, 2t + 1, 2t + 8, 2t + 9 at column cell
//     g.  INT8: values (d/8) g ..; Q4_0: one halfword of each group i, the
//     values 32i + 4g ...  Byte bits 5, 6 of a region are xored with the
//     token's bits 1, 2.
// Scales: INT8 fp32 [16]; Q4_0 fp16 [16][d/32].
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn.h"

namespace qgemv {

template <int FMT, int D>
struct KvLayout {
  static_assert(D == 64 || D == 128, "head_dim");
  static constexpr int kRow = FMT == QGEMV_KV_F16 ? 2 * D : FMT == QGEMV_KV_INT8 ? D : D / 2;
  static constexpr int kScaleRow = FMT == QGEMV_KV_F16 ? 0 : FMT == QGEMV_KV_INT8 ? 4 : D / 16;
  static constexpr int kV = kKvBlockTokens * kRow;
  static constexpr int kKs = 2 * kV;
  static constexpr int kVs = kKs + kKvBlockTokens * kScaleRow;
  static constexpr int kBlock = kVs + kKvBlockTokens * kScaleRow;
  static_assert(kBlock % 128 == 0 && kV % 128 == 0, "blocks and regions start on bank lines");

  // Byte c of a token's row, K and V.
  __host__ __device__ static constexpr int f16_off(int tok, int c) {
    return (c >> 7) * 2048 + tok * 128 + ((c & 127) ^ ((tok & 7) << 4));
  }
  __host__ __device__ static constexpr int k_off(int tok, int c) {
    if (FMT == QGEMV_KV_F16) return f16_off(tok, c);
    return kRow >= 128 ? (tok * kRow + c) ^ ((tok & 1) << 6) : tok * kRow + c;
  }
  __host__ __device__ static constexpr int v_off(int tok, int c) {
    if (FMT == QGEMV_KV_F16) return kV + f16_off(tok, c);
    return kV + ((tok * kRow + c) ^ (((tok >> 1) & 3) << 5));
  }
};

inline int64_t kv_block_bytes(int format, int head_dim) {
  const int row = format == QGEMV_KV_F16 ? 2 * head_dim : format == QGEMV_KV_INT8 ? head_dim + 4 : head_dim / 32 * 18;
  return int64_t(kKvBlockTokens) * 2 * row;
}

// a / b of values that nearly always fit 32 bits
__device__ __forceinline__ int64_t div_small(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// Start of the block of (page, head, block in page).
template <int FMT, int D>
__device__ __forceinline__ uint8_t* kv_block(const qgemv_kv_cache& c, int64_t page, int head, int blk) {
  const int per = c.page_tokens / kKvBlockTokens;
  return static_cast<uint8_t*>(c.pages) + ((page * c.kv_heads + head) * per + blk) * KvLayout<FMT, D>::kBlock;
}

}  // namespace qgemv
