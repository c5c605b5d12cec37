// rope.cu -- rotary positions of up to four axes: rows of heads rotated, and
// rotated keys written into the key/value cache beside their values
// (qgemv_rope_rows, qgemv_kv_write_rotated).
//
// Pair j of a head vector turns by position[axis(j)] * freq(j).  The angle is
// a 64-bit fixed-point number of turns: turns(j) = round(2^64 freq(j) / 2 pi),
// and position * turns(j) mod 2^64 is the angle without its whole turns, off by
// at most |position| 2^-65 -- nothing is lost at far positions, and no 64-bit
// floating point, which this GPU has little of, is needed.  As a signed number it
// is rounded once, to a float of at most 1 (half turns), sincospif's argument: small
// angles keep their 24 bits, and -position gives the opposite angle exactly.
//
// Bytes bound it, as the cache write (kv_cache.cu), whose layout it takes: a
// lane for eight neighbouring values, a warp for eight rows of one token, all of
// them queries, keys or values.  A block works out the angles of its four warps'
// tokens once, while their rows are on their way, and keeps cosines and sines in
// shared memory; with an angle for each lane's values in every warp the
// instructions were the bound (27003 tokens of 32 + 32 + 32 heads, bf16 into an
// fp16 cache, and the cache read again: 408 us; so 284, of which the rotation is
// 168, 7.9 TB/s with what L2 keeps).  Blocks of four warps wait for one another
// less than those of eight (10% longer) and of sixteen (16%).  fp32 rows take more
// registers and instructions a byte (2674 tokens of 80 heads into INT8: 29 us, 5.5
// TB/s; with loads of 32 bytes no faster, nor with half the rows for a warp).  A
// single token is one launch's latency, 3 us.
#include <type_traits>

#include "kv_codes.cuh"
#include "rope.h"

namespace qgemv {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;  // and tokens of a block, at most
constexpr int kWarpRows = 8;

// Warps of a token's queries, keys or values.
__host__ __device__ __forceinline__ int row_warps(int heads) { return (heads + kWarpRows - 1) / kWarpRows; }

// Four floats of shared memory, read where it is written.
__device__ __forceinline__ void lds_here(const float4* p, float* x) {
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "r"(smem_u32(p)));
}

enum { kNone, kWhole, kAny, kNext };

// FMT 0: rows only, no cache.  Blocks on an SM as measured (fp32: 30.1 us for the
// tokens above with seven, 28.6 with eight, 34.2 with nine; 16 bits into fp16: 171
// with nine, 168 with ten, 181 with eleven).  Their 64 and 48 registers hold a warp's
// rows, but not all that the ways below and the quantisers want; at d = 128 a thread
// stores and loads of what is spilled (bytes, over all of the kernel's code): 16 bits
// into INT8 148 and 596, Q4_0 128 and 532, fp16 108 and 248, rows alone 96 and 168;
// fp32 100 and 312, 104 and 320, 104 and 196, 48 and 60.  For 16 bits into INT8 and
// Q4_0 nine blocks would be 2% better (27003 tokens of 96 heads in bf16, pairs in
// halves, with eight, nine and ten: fp16 204, 196, 194 us; INT8 328, 322, 329; Q4_0
// 521, 501, 513).
template <int FMT, int D, typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 8 : 10) rope_kernel(const RopeParams p) {
  constexpr int kLanes = D / 8, kAt = 32 / kLanes;  // kAt rows at a time
  constexpr int kPasses = kWarpRows / kAt;
  // Cosines and sines of a token's D / 2 pairs, as quads of pairs 4 i .. 4 i + 3:
  // the even quads first, so that neighbouring lanes, two quads each, read
  // neighbouring ones.
  __shared__ float4 s_cos[kWarps][D / 8], s_sin[2][kWarps][D / 8];  // (sines, and their opposites)
  __shared__ float s_row[kWarps][kAt][D];
  const unsigned full = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = p.pairs;
  const int H = FMT ? p.cache.kv_heads : 0, q_warps = row_warps(p.q_heads), k_warps = row_warps(H), per = q_warps + 2 * k_warps;
  // the block's warps are w0 .. of all, the first of them warp `r0` of token t0
  const int64_t w0 = static_cast<int64_t>(blockIdx.x) * kWarps, t0 = div_small(w0, per);
  const unsigned r0 = static_cast<unsigned>(w0 - t0 * per), mine = (r0 + warp) / static_cast<unsigned>(per);
  const int64_t token = t0 + mine;
  const int part = static_cast<int>(r0 + warp - mine * per), kind = part < q_warps ? 0 : part < q_warps + k_warps ? 1 : 2;  // q, k, v
  const int heads = kind == 0 ? p.q_heads : H;
  const int row0 = (kind == 0 ? part : kind == 1 ? part - q_warps : part - q_warps - k_warps) * kWarpRows;
  const int d0 = (lane % kLanes) * 8;
  bool on = token < p.n_tokens;

  int64_t slot = 0;
  if (FMT != 0 && on && kind != 0) slot = __ldg(p.slots + token);
  Raw<T> raw[kPasses];  // (also of a token without a slot: its rows need not wait)
  if (on) {
    const RowsIn& in = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
    const T* src = static_cast<const T*>(in.ptr) + token * in.token_stride + d0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) raw[i].load_own(src + min(row0 + i * kAt + lane / kLanes, heads - 1) * in.head_stride);
  }

  // ---- the angles of the block's tokens
  const int tokens = static_cast<int>(min(static_cast<int64_t>((r0 + kWarps - 1) / static_cast<unsigned>(per)), p.n_tokens - 1 - t0)) + 1;
  for (int i = threadIdx.x; i < tokens * (D / 2); i += kThreads) {
    const int t = i / (D / 2), j = i % (D / 2);
    float c = 1.f, s = 0.f;
    if (j < n) {
      const uint4 e = __ldg(p.plan + j);
      int x = 0;
#pragma unroll
      for (int a = 0; a < 4; ++a) {  // all of them, with nothing to wait for
        const int at = a < p.n_axes ? __ldg(p.positions + (t0 + t) * p.n_axes + a) : 0;
        if (e.z == a) x = at;
      }
      const uint64_t turns = static_cast<uint64_t>(e.y) << 32 | e.x;
      const uint64_t turn = turns * static_cast<uint64_t>(static_cast<int64_t>(x));
      sincospif(__ll2float_rn(static_cast<int64_t>(turn)) * 0x1p-63f, &s, &c);
    }
    const int quad = ((j >> 2) & 1) * (D / 16) + (j >> 3);
    reinterpret_cast<float*>(&s_cos[t][quad])[j & 3] = c;
    reinterpret_cast<float*>(&s_sin[0][t][quad])[j & 3] = s;
    reinterpret_cast<float*>(&s_sin[1][t][quad])[j & 3] = -s;
  }
  __syncthreads();
  uint8_t* b0 = nullptr;
  int at = 0;
  int64_t step = 0;
  if constexpr (FMT != 0) {
    on = on && slot >= 0 && slot < p.cache.n_pages * p.cache.page_tokens;
    if (on && kind != 0) {
      at = static_cast<int>(slot) & (p.cache.page_tokens - 1);
      b0 = kv_block<FMT, D>(p.cache, slot >> (31 - __clz(p.cache.page_tokens)), 0, at / kKvBlockTokens);
      step = static_cast<int64_t>(p.cache.page_tokens / kKvBlockTokens) * KvLayout<FMT, D>::kBlock;
    }
  }
  if (!on) return;

  // ---- the rows, by the way in which a value meets the other one of its pair
  auto rows = [&](auto how) {
    constexpr int kHow = decltype(how)::value;  // kWhole, kAny, kNext: halves; neighbours; kNone: values
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int row = row0 + i * kAt + lane / kLanes;
      if (row0 + i * kAt >= heads) break;  // (the warp's)
      float x[8];
      raw[i].values(x);
      if constexpr (kHow != kNone) {
        float y[8];
        if constexpr (kHow == kNext) {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
        } else if constexpr (kHow == kWhole) {
          const int other = d0 < n ? lane + n / 8 : d0 < 2 * n ? lane - n / 8 : lane;
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(full, x[e], other);
        } else {
          float* here = s_row[warp][lane / kLanes];
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e) here[d0 + e] = x[e];
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = d0 + e < 2 * n ? here[d0 + e < n ? d0 + e + n : d0 + e - n] : 0.f;
        }
        // x = x c + y s, with -s for the first of a pair: read for each pass (held for
        // all of them they would take a quarter of the registers)
        auto turn = [&](int e, float c0, float c1, float s0, float s1, float& u, float& v) {
          unpack2(fma2(pack2(x[e], x[e + 1]), pack2(c0, c1), mul2(pack2(y[e], y[e + 1]), pack2(s0, s1))), u, v);
        };
        if constexpr (kHow == kNext) {
          float c[4], s[4];
          const int q = d0 / 8, at = (q & 1) * (D / 16) + (q >> 1);
          lds_here(&s_cos[mine][at], c);
          lds_here(&s_sin[0][mine][at], s);
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            float u, v;
            turn(e, c[e / 2], c[e / 2], -s[e / 2], s[e / 2], u, v);
            if (d0 + e < 2 * n) x[e] = u, x[e + 1] = v;
          }
        } else if constexpr (kHow == kWhole) {
          if (d0 < 2 * n) {  // a lane's eight values are turned or not together
            const int j0 = d0 < n ? d0 : d0 - n, at = j0 >> 3;
            float c[8], s[8];
            lds_here(&s_cos[mine][at], c);
            lds_here(&s_cos[mine][D / 16 + at], c + 4);
            lds_here(&s_sin[d0 < n][mine][at], s);
            lds_here(&s_sin[d0 < n][mine][D / 16 + at], s + 4);
#pragma unroll
            for (int e = 0; e < 8; e += 2) turn(e, c[e], c[e + 1], s[e], s[e + 1], x[e], x[e + 1]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            float c[2], s[2], u, v;
#pragma unroll
            for (int o = 0; o < 2; ++o) {
              const int i = d0 + e + o, j = i < n ? i : i < 2 * n ? i - n : 0, q = ((j >> 2) & 1) * (D / 16) + (j >> 3);
              c[o] = reinterpret_cast<const float*>(&s_cos[mine][q])[j & 3];
              s[o] = reinterpret_cast<const float*>(&s_sin[i < n][mine][q])[j & 3];
            }
            turn(e, c[0], c[1], s[0], s[1], u, v);
            if (d0 + e < 2 * n) x[e] = u;
            if (d0 + e + 1 < 2 * n) x[e + 1] = v;
          }
        }
      }
      if (kind == 0) {
        if (row < heads) {
          const int64_t to = token * p.out.token_stride + row * p.out.head_stride + d0;
          if (p.out_dtype == QGEMV_DT_F16) store_values(static_cast<__half*>(p.out.ptr) + to, x);
          else if (p.out_dtype == QGEMV_DT_BF16) store_values(static_cast<__nv_bfloat16*>(p.out.ptr) + to, x);
          else store_values(static_cast<float*>(p.out.ptr) + to, x);
        }
      } else if constexpr (FMT != 0) {
        encode<FMT, D>(b0 + row * step, kind == 2, at % kKvBlockTokens, d0, x, row < heads);
      }
    }
  };
  if (kind == 2) rows(std::integral_constant<int, kNone>());
  else if (p.neighbours) rows(std::integral_constant<int, kNext>());
  // The other value of a pair comes by a shuffle where the pairs are a multiple of
  // eight, else through shared memory, whose banks the stores and the single reads of
  // cosines meet in (4096 tokens of 32 fp16 heads of 128: 64 pairs 12.4 us, 60 pairs
  // 37.1; of 64: 32 pairs 8.5, 28 pairs 20.2).
  else if ((n & 7) == 0) rows(std::integral_constant<int, kWhole>());
  else rows(std::integral_constant<int, kAny>());
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int dtype, int head_dim, cudaStream_t s) {
  const int H = p.cache.pages ? p.cache.kv_heads : 0;
  const int64_t warps = p.n_tokens * (row_warps(p.q_heads) + 2 * row_warps(H));
  const int64_t grid = (warps + kWarps - 1) / kWarps;
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
