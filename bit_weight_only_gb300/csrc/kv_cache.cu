// kv_cache.cu -- writing rows into the quantised key/value cache and reading
// them back (qgemv_kv_write, qgemv_kv_read).
//
// Memory-bound: rows are read once and codes written once.  A warp takes
// eight (head, K or V) rows of one token, so that the slot, the sequence and
// the divisions are worked out once for them, and has all of their loads in
// flight together.
//
// Write: a lane holds 16 bytes of the input, V = 4 or 8 neighbouring values;
// d / V lanes make a row.  A Q4_0 group is 8 or 4 lanes.
// Read: a lane takes 8 neighbouring values.
#include <type_traits>

#include "kv_layout.cuh"

namespace qgemv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarpRows = 8;

template <typename T>
__device__ __forceinline__ void load_values(const T* src, float (&x)[16 / sizeof(T)]) {
  const uint4 w = __ldg(reinterpret_cast<const uint4*>(src));
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<T, float>::value) {
      x[i] = __uint_as_float(u[i]);
    } else if constexpr (std::is_same<T, __half>::value) {
      x[2 * i] = __half2float(__ushort_as_half(static_cast<unsigned short>(u[i] & 0xffffu)));
      x[2 * i + 1] = __half2float(__ushort_as_half(static_cast<unsigned short>(u[i] >> 16)));
    } else {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ uint32_t half_bits(float lo, float hi) {
  return __half_as_ushort(__float2half_rn(lo)) | static_cast<uint32_t>(__half_as_ushort(__float2half_rn(hi))) << 16;
}

// round(fl32(x / a)) by a product with 1 / a: that is off by a few units in the
// last place, so only a result close to a tie can round otherwise, and those
// are worked out by the division (as are NaN).  |x / a| is at most 128.
template <bool HALF_AWAY>
__device__ __forceinline__ float round_quotient(float x, float a, float inv) {
  constexpr float kShift = 12582912.f;  // 1.5 * 2^23
  const float r = x * inv, q = (r + kShift) - kShift;
  if (fabsf(r - q) < 0.4999f) return q;
  const float e = __fdiv_rn(x, a);
  return HALF_AWAY ? roundf(e) : rintf(e);
}

// The codes of lane values x[V] (values d0 .. of a row) into token tok of
// block b.  Lanes of a row call it together.
template <int FMT, int D, int V>
__device__ __forceinline__ void encode(uint8_t* b, bool v, int tok, int d0, const float (&x)[V], bool on) {
  using L = KvLayout<FMT, D>;
  const unsigned full = 0xffffffffu;
  if constexpr (FMT == QGEMV_KV_F16) {
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = half_bits(x[2 * i], x[2 * i + 1]);
    if (!on) return;
    uint8_t* at = b + (v ? L::v_off(tok, 2 * d0) : L::k_off(tok, 2 * d0));
    if constexpr (V == 8) *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
  } else if constexpr (FMT == QGEMV_KV_INT8) {
    float m = 0.f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      m = fmaxf(m, fabsf(x[i]));
      bad |= !(fabsf(x[i]) < INFINITY);
    }
    if (bad) m = INFINITY;
#pragma unroll
    for (int o = 1; o < D / V; o <<= 1) m = fmaxf(m, __shfl_xor_sync(full, m, o));
    const float a = m == INFINITY ? __int_as_float(0x7fffffff) : __fdiv_rn(m, 127.f);
    uint32_t w[V / 4];
    const float inv = 1.f / a;
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float q = 0.f;
        if (a > 0.f) q = fminf(fmaxf(round_quotient<false>(x[4 * j + i], a, inv), -127.f), 127.f);
        c[i] = __float_as_uint(q + 8388736.f);  // 2^23 + 128: the code + 128 in the low byte
      }
      w[j] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    }
    if (!on) return;
    uint8_t* at = b + (v ? L::v_off(tok, d0) : L::k_off(tok, d0));
    if constexpr (V == 8) *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(at) = w[0];
    if (d0 == 0) reinterpret_cast<float*>(b + (v ? L::kVs : L::kKs))[tok] = a;
  } else {
    // the value of largest magnitude of the group, the first one on ties
    float peak = x[0];
    int where = d0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      bad |= !(fabsf(x[i]) < INFINITY);
      if (fabsf(x[i]) > fabsf(peak)) peak = x[i], where = d0 + i;
    }
    if (bad) peak = INFINITY;
#pragma unroll
    for (int o = 1; o < 32 / V; o <<= 1) {
      const float op = __shfl_xor_sync(full, peak, o);
      const int ow = __shfl_xor_sync(full, where, o);
      if (fabsf(op) > fabsf(peak) || (fabsf(op) == fabsf(peak) && ow < where)) peak = op, where = ow;
    }
    bad = fabsf(peak) == INFINITY;
    const float a = bad ? __int_as_float(0x7fffffff) : __fdiv_rn(peak, -8.f);
    uint32_t q[V];
    const float inv = 1.f / a;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float c = 8.f;
      if (!bad && a != 0.f) c = fminf(fmaxf(round_quotient<true>(x[i], a, inv) + 8.f, 0.f), 15.f);
      q[i] = __float_as_uint(c + 8388608.f) & 15u;
    }
    const int grp = d0 >> 5, e = d0 & 31;
    // K: word (group, e / 8), values 0 2 4 6 1 3 5 7 from the low nibble.  The
    // shuffle stands outside of the branch: a warp can hold rows of both kinds.
    uint32_t w;
    if constexpr (V == 8) {
      w = q[0] | q[2] << 4 | q[4] << 8 | q[6] << 12 | q[1] << 16 | q[3] << 20 | q[5] << 24 | q[7] << 28;
    } else {
      w = q[0] | q[2] << 4 | q[1] << 16 | q[3] << 20;
      w |= __shfl_down_sync(full, w, 1) << 8;  // values 4 .. 7
    }
    if (on && v) {  // V: halfword (group, e / 4), four neighbouring values
#pragma unroll
      for (int j = 0; j < V / 4; ++j)
        *reinterpret_cast<uint16_t*>(b + L::v_off(tok, ((e >> 2) + j) * (D / 16) + 2 * grp)) =
            static_cast<uint16_t>(q[4 * j] | q[4 * j + 1] << 4 | q[4 * j + 2] << 8 | q[4 * j + 3] << 12);
    } else if (on && (e & 7) == 0) {
      *reinterpret_cast<uint32_t*>(b + L::k_off(tok, (e >> 3) * (D / 8) + 4 * grp)) = w;
    }
    if (on && e == 0) reinterpret_cast<__half*>(b + (v ? L::kVs : L::kKs))[tok * (D / 32) + grp] = __float2half_rn(a);
  }
}

// The warp's (token, first of kWarpRows rows); rows are 2 * head + (V ? 1 : 0).
struct WarpRows {
  int64_t token;
  int row0;
};
__device__ __forceinline__ WarpRows warp_rows(int H) {
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const int per = (2 * H + kWarpRows - 1) / kWarpRows;
  WarpRows r;
  r.token = w / per;
  r.row0 = static_cast<int>(w - r.token * per) * kWarpRows;
  return r;
}

template <int FMT, int D, typename T>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const KvWriteParams p) {
  constexpr int V = 16 / sizeof(T), kLanes = D / V, kAt = 32 / kLanes;  // kAt rows at a time
  const int lane = threadIdx.x & 31, H = p.cache.kv_heads;
  const WarpRows wr = warp_rows(H);
  if (wr.token >= p.n_tokens) return;
  const int64_t slot = __ldg(p.slots + wr.token);
  if (slot < 0 || slot >= p.cache.n_pages * p.cache.page_tokens) return;
  const int shift = 31 - __clz(p.cache.page_tokens);
  const int64_t page = slot >> shift;
  const int at = static_cast<int>(slot) & (p.cache.page_tokens - 1);
  const int d0 = (lane % kLanes) * V;
  float x[kWarpRows / kAt][V];
#pragma unroll
  for (int i = 0; i < kWarpRows / kAt; ++i) {
    const int row = min(wr.row0 + i * kAt + lane / kLanes, 2 * H - 1);
    const RowsIn& in = row & 1 ? p.v : p.k;
    load_values<T>(static_cast<const T*>(in.ptr) + wr.token * in.token_stride + (row >> 1) * in.head_stride + d0, x[i]);
  }
#pragma unroll
  for (int i = 0; i < kWarpRows / kAt; ++i) {
    const int row = wr.row0 + i * kAt + lane / kLanes;
    uint8_t* b = kv_block<FMT, D>(p.cache, page, min(row, 2 * H - 1) >> 1, at / kKvBlockTokens);
    encode<FMT, D, V>(b, row & 1, at % kKvBlockTokens, d0, x[i], row < 2 * H);
  }
}

// Eight values of a row, from d0: their codes, read ahead of their use.
template <int FMT, int D>
struct Eight {
  uint4 w;
  float s;
  __device__ void load(const uint8_t* b, bool v, int tok, int d0) {
    using L = KvLayout<FMT, D>;
    if constexpr (FMT == QGEMV_KV_F16) {
      w = __ldg(reinterpret_cast<const uint4*>(b + (v ? L::v_off(tok, 2 * d0) : L::k_off(tok, 2 * d0))));
    } else if constexpr (FMT == QGEMV_KV_INT8) {
      const uint2 c = __ldg(reinterpret_cast<const uint2*>(b + (v ? L::v_off(tok, d0) : L::k_off(tok, d0))));
      w.x = c.x, w.y = c.y;
      s = __ldg(reinterpret_cast<const float*>(b + (v ? L::kVs : L::kKs)) + tok);
    } else {
      const int grp = d0 >> 5, e = d0 & 31;
      if (v) {
        w.x = __ldg(reinterpret_cast<const unsigned short*>(b + L::v_off(tok, (e >> 2) * (D / 16) + 2 * grp)));
        w.x |= static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(b + L::v_off(tok, ((e >> 2) + 1) * (D / 16) + 2 * grp)))) << 16;
      } else {
        const uint32_t k = __ldg(reinterpret_cast<const unsigned*>(b + L::k_off(tok, (e >> 3) * (D / 8) + 4 * grp)));
        // nibble order 0 2 4 6 1 3 5 7 to 0 .. 7
        uint32_t lo = k & 0xffffu, hi = k >> 16;
        auto spread = [](uint32_t x) {
          x = (x | x << 8) & 0x00ff00ffu;
          return (x | x << 4) & 0x0f0f0f0fu;
        };
        w.x = spread(lo) | spread(hi) << 4;
      }
      s = __half2float(__ushort_as_half(__ldg(reinterpret_cast<const unsigned short*>(b + (v ? L::kVs : L::kKs)) + tok * (D / 32) + grp)));
    }
  }
  __device__ void values(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (FMT == QGEMV_KV_F16) {
        const uint32_t u = (&w.x)[i >> 1];
        x[i] = __half2float(__ushort_as_half(static_cast<unsigned short>(i & 1 ? u >> 16 : u & 0xffffu)));
      } else if constexpr (FMT == QGEMV_KV_INT8) {
        x[i] = static_cast<float>(static_cast<int>(((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 255u) - 128) * s;
      } else {
        x[i] = static_cast<float>(static_cast<int>((w.x >> (4 * i)) & 15u) - 8) * s;
      }
    }
  }
};

template <typename T>
__device__ __forceinline__ void store_values(T* dst, const float (&x)[8]) {
  if constexpr (std::is_same<T, float>::value) {
    reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        w[i] = half_bits(x[2 * i], x[2 * i + 1]);
      } else {
        w[i] = __bfloat16_as_ushort(__float2bfloat16_rn(x[2 * i])) |
               static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(x[2 * i + 1]))) << 16;
      }
    }
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
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
#pragma unroll
    for (int i = 0; i < kWarpRows / kAt; ++i) {
      const int row = min(wr.row0 + i * kAt + lane / kLanes, 2 * H - 1);
      e[i].load(kv_block<FMT, D>(p.cache, page, row >> 1, at / kKvBlockTokens), row & 1, at % kKvBlockTokens, d0);
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
