// rope.cu -- rotary positions of up to four axes: rows of heads rotated, and
// rotated keys written into the key/value cache beside their values
// (qgemv_rope_rows, qgemv_kv_write_rotated).
//
// Pair j of a head vector turns by position[axis(j)] * freq(j).  The angle is
// a 64-bit fixed-point number of turns: turns(j) = round(2^64 freq(j) / 2 pi),
// and position * turns(j) mod 2^64 is the angle without its whole turns, off by
// at most |position| 2^-65 -- nothing is lost at far positions, and no 64-bit
// floating point, which this GPU has little of, is needed.  Its upper 32 bits
// become a float of at most 1 and sincospif's argument.
//
// Bytes bound it, as the cache write (kv_cache.cu), whose layout it takes: a
// lane for eight neighbouring values, a warp for eight rows of one token, so
// that the angles are worked out once for eight rows.  The other value of a
// pair comes by a shuffle where the pairs are a multiple of eight (any head
// whose halves are rotated whole), else through shared memory.
#include <type_traits>

#include "kv_codes.cuh"
#include "rope.h"

namespace qgemv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarpRows = 8;

// FMT 0: rows only, no cache.
template <int FMT, int D, typename T>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  constexpr int kLanes = D / 8, kAt = 32 / kLanes;  // kAt rows at a time
  constexpr int kPasses = kWarpRows / kAt;
  __shared__ float s_row[kThreads / 32][kAt][D];
  const unsigned full = 0xffffffffu;
  const int lane = threadIdx.x & 31, H = FMT ? p.cache.kv_heads : 0;
  const int q_warps = (p.q_heads + kWarpRows - 1) / kWarpRows, per = q_warps + (2 * H + kWarpRows - 1) / kWarpRows;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const int64_t token = div_small(w, per);
  if (token >= p.n_tokens) return;
  const int part = static_cast<int>(w - token * per);
  const bool is_q = part < q_warps;
  const int rows = is_q ? p.q_heads : 2 * H;  // cache rows: 2 * head + (V ? 1 : 0)
  const int row0 = (is_q ? part : part - q_warps) * kWarpRows;
  const int d0 = (lane % kLanes) * 8;

  uint8_t* b0 = nullptr;
  int at = 0;
  int64_t step = 0;
  if constexpr (FMT != 0) {
    if (!is_q) {
      const int64_t slot = __ldg(p.slots + token);
      if (slot < 0 || slot >= p.cache.n_pages * p.cache.page_tokens) return;
      at = static_cast<int>(slot) & (p.cache.page_tokens - 1);
      b0 = kv_block<FMT, D>(p.cache, slot >> (31 - __clz(p.cache.page_tokens)), 0, at / kKvBlockTokens);
      step = static_cast<int64_t>(p.cache.page_tokens / kKvBlockTokens) * KvLayout<FMT, D>::kBlock;
    }
  }
  Raw<T> raw[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int row = min(row0 + i * kAt + lane / kLanes, rows - 1);
    const RowsIn& in = is_q ? p.q : row & 1 ? p.v : p.k;
    raw[i].load_own(static_cast<const T*>(in.ptr) + token * in.token_stride + (is_q ? row : row >> 1) * in.head_stride + d0);
  }

  // ---- the angles of this lane's values
  const int n = p.pairs;
  int pos[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) pos[a] = a < p.n_axes ? __ldg(p.positions + token * p.n_axes + a) : 0;
  auto angle = [&](int j, float& c, float& s) {
    const uint4 e = __ldg(p.plan + j);
    const int x = e.z == 0 ? pos[0] : e.z == 1 ? pos[1] : e.z == 2 ? pos[2] : pos[3];
    const uint64_t turns = static_cast<uint64_t>(e.y) << 32 | e.x;
    const uint64_t t = turns * static_cast<uint64_t>(static_cast<int64_t>(x));
    sincospif(static_cast<float>(static_cast<int32_t>(t >> 32)) * 0x1p-31f, &s, &c);
  };
  float c[8], s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int i = d0 + e;
    c[e] = 1.f, s[e] = 0.f;
    if (p.neighbours) {
      if (e & 1) c[e] = c[e - 1], s[e] = -s[e - 1];
      else if (i < 2 * n) angle(i >> 1, c[e], s[e]), s[e] = -s[e];
    } else if (i < 2 * n) {
      angle(i < n ? i : i - n, c[e], s[e]);
      if (i < n) s[e] = -s[e];
    }
  }

#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int row = row0 + i * kAt + lane / kLanes;
    float x[8], y[8];
    raw[i].values(x);
    if (p.neighbours) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
    } else if ((n & 7) == 0) {
      const int other = d0 < n ? lane + n / 8 : d0 < 2 * n ? lane - n / 8 : lane;
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(full, x[e], other);
    } else {
      float* mine = s_row[threadIdx.x >> 5][lane / kLanes];
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 8; ++e) mine[d0 + e] = x[e];
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = d0 + e < 2 * n ? mine[d0 + e < n ? d0 + e + n : d0 + e - n] : 0.f;
    }
    const bool turn = is_q || !(row & 1);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (turn && d0 + e < 2 * n) x[e] = fmaf(x[e], c[e], y[e] * s[e]);
    if (is_q) {
      if (row < rows) {
        const int64_t to = token * p.out.token_stride + row * p.out.head_stride + d0;
        if (p.out_dtype == QGEMV_DT_F16) store_values(static_cast<__half*>(p.out.ptr) + to, x);
        else if (p.out_dtype == QGEMV_DT_BF16) store_values(static_cast<__nv_bfloat16*>(p.out.ptr) + to, x);
        else store_values(static_cast<float*>(p.out.ptr) + to, x);
      }
    } else if constexpr (FMT != 0) {
      encode<FMT, D>(b0 + (row >> 1) * step, row & 1, at % kKvBlockTokens, d0, x, row < rows);
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int dtype, int head_dim, cudaStream_t s) {
  const int H = p.cache.pages ? p.cache.kv_heads : 0;
  const int64_t warps = p.n_tokens * ((p.q_heads + kWarpRows - 1) / kWarpRows + (2 * H + kWarpRows - 1) / kWarpRows);
  const int64_t grid = (warps + kThreads / 32 - 1) / (kThreads / 32);
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  auto go = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(grid), kThreads, 0, s>>>(p);
    return cudaGetLastError();
  };
  auto by_type = [&](auto fmt, auto d) {
    constexpr int F = decltype(fmt)::value, D = decltype(d)::value;
    switch (dtype) {
      case QGEMV_DT_F32: return go(rope_kernel<F, D, float>);
      case QGEMV_DT_F16: return go(rope_kernel<F, D, __half>);
      default: return go(rope_kernel<F, D, __nv_bfloat16>);
    }
  };
  auto by_dim = [&](auto fmt) {
    return head_dim == 64 ? by_type(fmt, std::integral_constant<int, 64>()) : by_type(fmt, std::integral_constant<int, 128>());
  };
  if (!p.cache.pages) return by_dim(std::integral_constant<int, 0>());
  switch (p.cache.format) {
    case QGEMV_KV_F16: return by_dim(std::integral_constant<int, QGEMV_KV_F16>());
    case QGEMV_KV_INT8: return by_dim(std::integral_constant<int, QGEMV_KV_INT8>());
    default: return by_dim(std::integral_constant<int, QGEMV_KV_Q4_0>());
  }
}

}  // namespace qgemv
