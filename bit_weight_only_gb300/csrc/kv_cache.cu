// kv_cache.cu -- writing rows into the quantised key/value cache and reading
// them back (qgemv_kv_write, qgemv_kv_read).
//
// One warp per (token, head, K or V) row of d values; lane l holds the values
// l, l + 32, ..  Memory-bound: a row is read once and its codes written once.
#include "kv_layout.cuh"

namespace qgemv {
namespace {

constexpr int kThreads = 256;

// Largest |x| of the warp's 32 values, its sign kept, the first one on ties.
__device__ __forceinline__ float signed_peak(float x) {
  float best = x;
  int at = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float ob = __shfl_xor_sync(0xffffffffu, best, o);
    const int oa = __shfl_xor_sync(0xffffffffu, at, o);
    const float fa = fabsf(best), fb = fabsf(ob);
    if (fb > fa || (fb == fa && oa < at)) {
      best = ob;
      at = oa;
    }
  }
  return best;
}

template <int FMT, int D, typename T>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const KvWriteParams p) {
  using L = KvLayout<FMT, D>;
  const int lane = threadIdx.x & 31;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const int H = p.cache.kv_heads;
  const int64_t token = row / (2 * H);
  if (token >= p.n_tokens) return;
  const int rest = static_cast<int>(row - token * 2 * H);
  const int head = rest >> 1;
  const bool v = rest & 1;
  const int64_t slot = p.slots[token];
  if (slot < 0 || slot >= p.cache.n_pages * p.cache.page_tokens) return;
  const int64_t page = slot / p.cache.page_tokens;
  const int at = static_cast<int>(slot - page * p.cache.page_tokens);
  uint8_t* b = kv_block<FMT, D>(p.cache, page, head, at / kKvBlockTokens);
  const int tok = at % kKvBlockTokens;
  const RowsIn& in = v ? p.v : p.k;
  const T* src = static_cast<const T*>(in.ptr) + token * in.token_stride + head * in.head_stride;
  float x[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) x[i] = to_f32<T>(src[32 * i + lane]);
  if constexpr (FMT == QGEMV_KV_F16) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int c = 2 * (32 * i + lane);
      *reinterpret_cast<__half*>(b + (v ? L::v_off(tok, c) : L::k_off(tok, c))) = __float2half_rn(x[i]);
    }
  } else if constexpr (FMT == QGEMV_KV_INT8) {
    float m = 0.f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      m = fmaxf(m, fabsf(x[i]));
      nan |= x[i] != x[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (__any_sync(0xffffffffu, nan) || m == INFINITY) m = __int_as_float(0x7fffffff);
    const float a = __fdiv_rn(m, 127.f);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      int q = 0;
      if (a > 0.f) q = max(-127, min(127, __float2int_rn(__fdiv_rn(x[i], a))));
      const int c = 32 * i + lane;
      b[v ? L::v_off(tok, c) : L::k_off(tok, c)] = static_cast<uint8_t>(q + 128);
    }
    if (lane == 0) reinterpret_cast<float*>(b + (v ? L::kVs : L::kKs))[tok] = a;
  } else {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const bool bad = __any_sync(0xffffffffu, !(fabsf(x[i]) < INFINITY));
      float d = __fdiv_rn(signed_peak(x[i]), -8.f);
      if (bad) d = __int_as_float(0x7fffffff);
      int q = 8;
      if (!bad && d != 0.f) q = static_cast<int>(fminf(fmaxf(roundf(__fdiv_rn(x[i], d)) + 8.f, 0.f), 15.f));
      // a lane's nibble and its partner's share a byte
      const int e = lane;
      if (v) {
        const int hi = __shfl_down_sync(0xffffffffu, q, 1);
        if (!(e & 1)) b[L::v_off(tok, (e >> 2) * (D / 16) + 2 * i + ((e & 3) >> 1))] = static_cast<uint8_t>(q | hi << 4);
      } else {
        const int hi = __shfl_down_sync(0xffffffffu, q, 2);
        const int j = ((e & 7) >> 1) + 4 * (e & 1);
        if (!(j & 1)) b[L::k_off(tok, (e >> 3) * (D / 8) + 4 * i + (j >> 1))] = static_cast<uint8_t>(q | hi << 4);
      }
      if (lane == 0) reinterpret_cast<__half*>(b + (v ? L::kVs : L::kKs))[tok * (D / 32) + i] = __float2half_rn(d);
    }
  }
}

template <int FMT, int D, typename T>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvReadParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const int H = p.cache.kv_heads;
  const int64_t token = row / (2 * H);
  if (token >= p.n_tokens) return;
  const int rest = static_cast<int>(row - token * 2 * H);
  const int head = rest >> 1;
  const bool v = rest & 1;
  // the sequence of this row: the last one with cu[seq] <= token
  int64_t lo = 0, hi = p.n_seqs;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (p.cu[mid + 1] <= token) lo = mid + 1;
    else hi = mid;
  }
  const RowsOut& o = v ? p.v : p.k;
  T* dst = static_cast<T*>(o.ptr) + token * o.token_stride + head * o.head_stride;
  if (lo >= p.n_seqs || p.cu[lo] > token) return;
  const int64_t pos = token - p.cu[lo] + (p.starts ? p.starts[lo] : 0);
  const int64_t pi = pos >= 0 ? pos / p.cache.page_tokens : -1;
  int64_t page = -1;
  if (pi >= 0 && pi < p.table_stride) page = p.table[lo * p.table_stride + pi];
  if (page < 0 || page >= p.cache.n_pages) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) dst[32 * i + lane] = from_f32<T>(0.f);
    return;
  }
  const int at = static_cast<int>(pos - pi * p.cache.page_tokens);
  const uint8_t* b = kv_block<FMT, D>(p.cache, page, head, at / kKvBlockTokens);
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
    dst[32 * i + lane] = from_f32<T>(kv_value<FMT, D>(b, v, at % kKvBlockTokens, 32 * i + lane));
}

template <template <int, int, typename> class K, typename P>
cudaError_t dispatch(const P& p, int dtype, int64_t n_tokens, cudaStream_t s) {
  const int64_t rows = n_tokens * 2 * p.cache.kv_heads;
  const unsigned grid = static_cast<unsigned>((rows + kThreads / 32 - 1) / (kThreads / 32));
  auto go = [&](auto kernel) {
    kernel<<<grid, kThreads, 0, s>>>(p);
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

template <int F, int D, typename T>
struct WriteK {
  static auto fn() { return kv_write_kernel<F, D, T>; }
};
template <int F, int D, typename T>
struct ReadK {
  static auto fn() { return kv_read_kernel<F, D, T>; }
};

}  // namespace

cudaError_t launch_kv_write(const KvWriteParams& p, int dtype, cudaStream_t s) {
  return dispatch<WriteK>(p, dtype, p.n_tokens, s);
}
cudaError_t launch_kv_read(const KvReadParams& p, int dtype, cudaStream_t s) {
  return dispatch<ReadK>(p, dtype, p.n_tokens, s);
}

}  // namespace qgemv
