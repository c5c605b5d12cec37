// kv_cache.cu -- writing rows into the quantised key/value cache and reading
// them back (qgemv_kv_write, qgemv_kv_read).
//
// Memory-bound in bytes, but the codes cost instructions enough to matter
// (issue slots 65-80% busy at half of the bandwidth in the first form): a lane
// takes eight neighbouring values, so that a row's reductions, scale and
// address are shared by few lanes, d / 8; quantisers work without divisions or
// conversions per value.  A warp takes eight (head, K or V) rows of one token
// and has all of their loads in flight together.  20463 tokens of 32 heads of
// 128, fp32 rows into an INT8 cache and back as fp16: 219 us, 0.92 of the copy
// bandwidth; a chunk into an fp16 cache and all of it back: 0.98.
#include <type_traits>

#include "kv_codes.cuh"

namespace qgemv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarpRows = 8;

// The warp's (token, first of kWarpRows rows); rows are 2 * head + (V ? 1 : 0).
struct WarpRows {
  int64_t token;
  int row0;
};
__device__ __forceinline__ WarpRows warp_rows(int H) {
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const int per = (2 * H + kWarpRows - 1) / kWarpRows;
  WarpRows r;
  r.token = div_small(w, per);
  r.row0 = static_cast<int>(w - r.token * per) * kWarpRows;
  return r;
}

// Start of the block of (page, head 0, block in page); a head further is
// `step` bytes.
template <int FMT, int D>
__device__ __forceinline__ uint8_t* block_of_token(const qgemv_kv_cache& c, int64_t page, int at, int& step) {
  step = (c.page_tokens / kKvBlockTokens) * KvLayout<FMT, D>::kBlock;
  return kv_block<FMT, D>(c, page, 0, at / kKvBlockTokens);
}

template <int FMT, int D, typename T>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const KvWriteParams p) {
  constexpr int kLanes = D / 8, kAt = 32 / kLanes;  // kAt rows at a time
  const int lane = threadIdx.x & 31, H = p.cache.kv_heads;
  const WarpRows wr = warp_rows(H);
  if (wr.token >= p.n_tokens) return;
  const int64_t slot = __ldg(p.slots + wr.token);
  if (slot < 0 || slot >= p.cache.n_pages * p.cache.page_tokens) return;
  const int shift = 31 - __clz(p.cache.page_tokens);
  const int at = static_cast<int>(slot) & (p.cache.page_tokens - 1);
  const int d0 = (lane % kLanes) * 8;
  int step;
  uint8_t* b0 = block_of_token<FMT, D>(p.cache, slot >> shift, at, step);
  Raw<T> raw[kWarpRows / kAt];
#pragma unroll
  for (int i = 0; i < kWarpRows / kAt; ++i) {
    const int row = min(wr.row0 + i * kAt + lane / kLanes, 2 * H - 1);
    const RowsIn& in = row & 1 ? p.v : p.k;
    raw[i].load(static_cast<const T*>(in.ptr) + wr.token * in.token_stride + (row >> 1) * in.head_stride + d0);
  }
#pragma unroll
  for (int i = 0; i < kWarpRows / kAt; ++i) {
    const int row = wr.row0 + i * kAt + lane / kLanes;
    float x[8];
    raw[i].values(x);
    encode<FMT, D>(b0 + static_cast<int64_t>(row >> 1) * step, row & 1, at % kKvBlockTokens, d0, x, row < 2 * H);
  }
}

template <int FMT, int D, typename T>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvReadParams p) {
  constexpr int kLanes = D / 8, kAt = 32 / kLanes;
  const int lane = threadIdx.x & 31, H = p.cache.kv_heads;
  const WarpRows wr = warp_rows(H);
  if (wr.token >= p.n_tokens) return;
  // the sequence of this token: the first with cu[seq + 1] > token
  int64_t lo = 0, hi = p.n_seqs;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (__ldg(p.cu + mid + 1) <= wr.token) lo = mid + 1;
    else hi = mid;
  }
  if (lo >= p.n_seqs) return;
  const int64_t first = __ldg(p.cu + lo);
  if (first > wr.token) return;
  const int64_t pos = wr.token - first + (p.starts ? __ldg(p.starts + lo) : 0);
  const int shift = 31 - __clz(p.cache.page_tokens);
  int64_t page = -1;
  if (pos >= 0 && (pos >> shift) < p.table_stride) page = __ldg(p.table + lo * p.table_stride + (pos >> shift));
  const bool there = page >= 0 && page < p.cache.n_pages;
  const int at = static_cast<int>(pos) & (p.cache.page_tokens - 1);
  const int d0 = (lane % kLanes) * 8;
  Eight<FMT, D> e[kWarpRows / kAt];
  if (there) {
    int step;
    const uint8_t* b0 = block_of_token<FMT, D>(p.cache, page, at, step);
#pragma unroll
    for (int i = 0; i < kWarpRows / kAt; ++i) {
      const int row = min(wr.row0 + i * kAt + lane / kLanes, 2 * H - 1);
      e[i].load(b0 + static_cast<int64_t>(row >> 1) * step, row & 1, at % kKvBlockTokens, d0);
    }
  }
#pragma unroll
  for (int i = 0; i < kWarpRows / kAt; ++i) {
    const int row = wr.row0 + i * kAt + lane / kLanes;
    if (row >= 2 * H) continue;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (there) e[i].values(x);
    const RowsOut& o = row & 1 ? p.v : p.k;
    store_values<T>(static_cast<T*>(o.ptr) + wr.token * o.token_stride + (row >> 1) * o.head_stride + d0, x);
  }
}

template <int F, int D, typename T>
struct WriteK {
  static auto fn() { return kv_write_kernel<F, D, T>; }
};
template <int F, int D, typename T>
struct ReadK {
  static auto fn() { return kv_read_kernel<F, D, T>; }
};

template <template <int, int, typename> class K, typename P>
cudaError_t dispatch(const P& p, int dtype, int64_t n_tokens, cudaStream_t s) {
  const int64_t warps = n_tokens * ((2 * p.cache.kv_heads + kWarpRows - 1) / kWarpRows);
  const int64_t grid = (warps + kThreads / 32 - 1) / (kThreads / 32);
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  auto go = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(grid), kThreads, 0, s>>>(p);
    return cudaGetLastError();
  };
  auto by_type = [&](auto fmt, auto d) {
    constexpr int F = decltype(fmt)::value, D = decltype(d)::value;
    switch (dtype) {
      case QGEMV_DT_F32: return go(K<F, D, float>::fn());
      case QGEMV_DT_F16: return go(K<F, D, __half>::fn());
      default: return go(K<F, D, __nv_bfloat16>::fn());
    }
  };
  auto by_dim = [&](auto fmt) {
    return p.cache.head_dim == 64 ? by_type(fmt, std::integral_constant<int, 64>())
                                  : by_type(fmt, std::integral_constant<int, 128>());
  };
  switch (p.cache.format) {
    case QGEMV_KV_F16: return by_dim(std::integral_constant<int, QGEMV_KV_F16>());
    case QGEMV_KV_INT8: return by_dim(std::integral_constant<int, QGEMV_KV_INT8>());
    default: return by_dim(std::integral_constant<int, QGEMV_KV_Q4_0>());
  }
}

}  // namespace

cudaError_t launch_kv_write(const KvWriteParams& p, int dtype, cudaStream_t s) {
  return dispatch<WriteK>(p, dtype, p.n_tokens, s);
}
cudaError_t launch_kv_read(const KvReadParams& p, int dtype, cudaStream_t s) {
  return dispatch<ReadK>(p, dtype, p.n_tokens, s);
}

}  // namespace qgemv
