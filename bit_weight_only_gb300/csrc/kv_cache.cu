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

#include "tc_common.cuh"
#include "kv_layout.cuh"

namespace qgemv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarpRows = 8;

// Eight values as they lie in memory, and in fp32.
template <typename T>
struct Raw {
  uint4 w[sizeof(T) / 2];
  __device__ void load(const T* src) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
  }
  __device__ void values(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (std::is_same<T, float>::value) {
        x[i] = __uint_as_float((&w[i >> 2].x)[i & 3]);
      } else {
        const uint32_t u = (&w[0].x)[i >> 1];
        if constexpr (std::is_same<T, __half>::value)
          x[i] = __half2float(__ushort_as_half(static_cast<unsigned short>(i & 1 ? u >> 16 : u & 0xffffu)));
        else
          x[i] = __uint_as_float(i & 1 ? u & 0xffff0000u : u << 16);
      }
    }
  }
};

// round(fl32(x / a)) of eight values, by products with about 1 / a: those are
// off by some units in the last place of at most 128, below 1e-4, so that only
// a result within 1e-4 of a tie could round otherwise; then (and where NaN or
// a = 0 come up) all eight are worked out by the division.  q in the low byte of
// each word, as a signed number.
template <bool HALF_AWAY>
__device__ __forceinline__ void round_quotients(const float (&x)[8], float a, uint32_t (&q)[8]) {
  constexpr float kShift = 12582912.f;  // 1.5 * 2^23
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(a));
  const uint64_t inv2 = pack2(inv, inv), up = pack2(kShift, kShift), down = pack2(-kShift, -kShift), less = pack2(-1.f, -1.f);
  float worst = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint64_t r = mul2(pack2(x[i], x[i + 1]), inv2), t = add2(r, up);
    float y, z;
    unpack2(t, y, z);
    q[i] = __float_as_uint(y), q[i + 1] = __float_as_uint(z);
    unpack2(fma2(add2(t, down), less, r), y, z);
    worst = fmaxf(worst, fmaxf(fabsf(y), fabsf(z)));
  }
  // (where a result is NaN, 1 / a is infinite or NaN: x / a is at most 127)
  const bool sure = worst < 0.4999f && fabsf(inv) < INFINITY;
  if (!sure) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float e = __fdiv_rn(x[i], a);
      // (a subnormal a is coarse: the quotient can pass 127)
      const float c = fminf(fmaxf(HALF_AWAY ? roundf(e) : rintf(e), -127.f), 127.f);
      q[i] = a != 0.f && e == e ? static_cast<uint32_t>(static_cast<int>(c)) : 0u;
    }
  }
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
constexpr uint32_t kInfBits = 0x7f800000u;

// The codes of a lane's values x (d0 .. of a row) into token tok of block b.
// The lanes of a warp call it together; a row is D / 8 of them.
template <int FMT, int D>
__device__ __forceinline__ void encode(uint8_t* b, bool v, int tok, int d0, const float (&x)[8], bool on) {
  using L = KvLayout<FMT, D>;
  const unsigned full = 0xffffffffu;
  if constexpr (FMT == QGEMV_KV_F16) {
    if (on)
      *reinterpret_cast<uint4*>(b + (v ? L::v_off(tok, 2 * d0) : L::k_off(tok, 2 * d0))) =
          make_uint4(half_pair(x[0], x[1]), half_pair(x[2], x[3]), half_pair(x[4], x[5]), half_pair(x[6], x[7]));
  } else if constexpr (FMT == QGEMV_KV_INT8) {
    // magnitudes compare as integers, infinities and NaN above all numbers
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(x[i]));
#pragma unroll
    for (int o = 1; o < D / 8; o <<= 1) m = max(m, __shfl_xor_sync(full, m, o));
    const bool bad = m >= kInfBits;
    const float a = bad ? __int_as_float(0x7fffffff) : __fdiv_rn(__uint_as_float(m), 127.f);
    uint32_t q[8];
    round_quotients<false>(x, a, q);  // at most 127: no clamp
    // code + 128 in a byte
    const uint32_t lo = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410) ^ 0x80808080u;
    const uint32_t hi = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410) ^ 0x80808080u;
    if (!on) return;
    *reinterpret_cast<uint2*>(b + (v ? L::v_off(tok, d0) : L::k_off(tok, d0))) = make_uint2(lo, hi);
    if (d0 == 0) reinterpret_cast<float*>(b + (v ? L::kVs : L::kKs))[tok] = a;
  } else {
    // the value of largest magnitude of the group's 32, the first one on ties
    float peak = x[0];
    int where = d0;
#pragma unroll
    for (int i = 1; i < 8; ++i)
      if (abs_bits(x[i]) > abs_bits(peak)) peak = x[i], where = d0 + i;
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      const float op = __shfl_xor_sync(full, peak, o);
      const int ow = __shfl_xor_sync(full, where, o);
      if (abs_bits(op) > abs_bits(peak) || (abs_bits(op) == abs_bits(peak) && ow < where)) peak = op, where = ow;
    }
    // a from 65520 on is past fp16: its group, too, is kept as NaN (an infinite
    // scale would make infinities of some codes, and hide the row's other groups
    // from the attention)
    const bool bad = abs_bits(peak) >= __float_as_uint(8.f * 65520.f);
    const float a = bad ? __int_as_float(0x7fffffff) : __fdiv_rn(peak, -8.f);
    uint32_t q[8];
    round_quotients<true>(x, a, q);
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // -8 .. 8 to 0 .. 15
      const int c = (static_cast<int>(q[i] << 24) >> 24) + 8;
      q[i] = static_cast<uint32_t>(min(max(c, 0), 15));
    }
    if (!on) return;
    const int grp = d0 >> 5, e = d0 & 31;
    if (v) {  // halfword (group, e / 4): four neighbouring values
#pragma unroll
      for (int j = 0; j < 2; ++j)
        *reinterpret_cast<uint16_t*>(b + L::v_off(tok, ((e >> 2) + j) * (D / 16) + 2 * grp)) =
            static_cast<uint16_t>(q[4 * j] | q[4 * j + 1] << 4 | q[4 * j + 2] << 8 | q[4 * j + 3] << 12);
    } else {  // word (group, e / 8): values 0 2 4 6 1 3 5 7 from the low nibble
      *reinterpret_cast<uint32_t*>(b + L::k_off(tok, (e >> 3) * (D / 8) + 4 * grp)) =
          q[0] | q[2] << 4 | q[4] << 8 | q[6] << 12 | q[1] << 16 | q[3] << 20 | q[5] << 24 | q[7] << 28;
    }
    if (e == 0) reinterpret_cast<__half*>(b + (v ? L::kVs : L::kKs))[tok * (D / 32) + grp] = __float2half_rn(a);
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
    if constexpr (FMT != QGEMV_KV_F16) {
      // 2^23 + code + offset as a pattern, no conversion
      const float off = FMT == QGEMV_KV_INT8 ? -8388736.f : -8388616.f;
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        auto bits = [&](int e) {
          return __uint_as_float(FMT == QGEMV_KV_INT8 ? __byte_perm(e < 4 ? w.x : w.y, 0x4B000000u, 0x7540 + (e & 3))
                                                      : ((w.x >> (4 * e)) & 15u) | 0x4B000000u);
        };
        unpack2(mul2(add2(pack2(bits(i), bits(i + 1)), pack2(off, off)), pack2(s, s)), x[i], x[i + 1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t u = (&w.x)[i >> 1];
        x[i] = __half2float(__ushort_as_half(static_cast<unsigned short>(i & 1 ? u >> 16 : u & 0xffffu)));
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
        w[i] = half_pair(x[2 * i], x[2 * i + 1]);
      } else {
        w[i] = cvt_pair<true>(x[2 * i], x[2 * i + 1]);
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
