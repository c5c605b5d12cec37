// beam.cu -- the selection of beam search (qgemv_beam_select): of a sequence's
// candidates (beam b, token t) the `width` of largest
//
//   score[b] + x[b][t] - log sum_u exp x[b][u].
//
// One pass over the logits, which are its bytes' floor.  A block takes a part
// of a row in tiles of 4096 values: each thread keeps a running maximum and sum
// of exponentials, and whatever passes the part's threshold goes to a list in
// shared memory.  Of one row the order of the candidates is that of its logits
// (ties: the lower token first), so a candidate is a 64-bit key, value above
// inverted token, and no two are equal.  The threshold is the list's
// `width`-th key, taken anew when the list has grown a little; for the first
// tile, a value that each warp has width / 8 threads at.  The block meets once
// in four tiles.  Where their candidates overflow the list (values that rise
// along the row) they are taken again tile by tile, behind the `width`-th
// largest of the threads' maxima, which at most `width` threads' values
// pass.  The last block of a sequence to end merges the parts' sorted lists, with
// the beams' scores in 64 bits: fp32 would make ties of scores that differ.
// (Which block that is changes nothing of the result.)
//
// Sums of exponentials are fp32, 17 additions a tile in a thread; the log sum,
// whose whole powers of two are taken apart, and the scores are 64-bit.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "beam.h"
#include "per_device.h"
#include "tc_common.cuh"

namespace qgemv {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 16;                       // values of a thread in a tile
constexpr int kTile = kThreads * kPer;         // values of a tile
constexpr int kListMax = 2048;                 // keys of the list
constexpr int kSpare = 32;                     // of them beyond `width` before it is cut
constexpr int kGroup = 4;                      // tiles between the block's meetings
static_assert(kMaxWidth * kPer <= kListMax / 2, "a tile's candidates fit beside half a list");

// Order of floats as unsigned numbers, +0 and -0 as one; 0 is below all.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
// Larger values first, then lower tokens; 0 for what is no candidate.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t token) {
  return x > -INFINITY ? static_cast<uint64_t>(ordered(x)) << 32 | (0xffffffffu - token) : 0;
}

// 16-byte loads of a row that may start anywhere: the row's values are those of
// 16-byte units from the unit that holds the first one.
template <typename T>
struct RowUnits {
  static constexpr int kVec = 16 / sizeof(T);
  const T* base;  // unit 0 (its first values may lie before the row)
  int64_t lead, end;  // the row is values [lead, end) from base
  __device__ RowUnits(const T* row, int64_t n) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(row);
    lead = static_cast<int64_t>((a & 15) / sizeof(T));
    base = row - lead;
    end = lead + n;
  }
  // unit u as it lies in memory; what is outside the row is -infinity
  __device__ uint4 load(int64_t u) const {
    const int64_t i0 = u * kVec;
    if (i0 >= lead && i0 + kVec <= end) return __ldg(reinterpret_cast<const uint4*>(base) + u);
    uint32_t w[4] = {0, 0, 0, 0};
    constexpr uint32_t kNone = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00u : 0xff80u;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      uint32_t v = kNone;
      if (i0 + i >= lead && i0 + i < end) {
        if constexpr (sizeof(T) == 4) v = reinterpret_cast<const uint32_t*>(base)[i0 + i];
        else v = reinterpret_cast<const unsigned short*>(base)[i0 + i];
      }
      if constexpr (sizeof(T) == 4) w[i] = v;
      else w[i >> 1] |= v << (16 * (i & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ static void values(const uint4& w, float* x) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      if constexpr (std::is_same<T, float>::value) {
        x[i] = __uint_as_float((&w.x)[i]);
      } else {
        const uint32_t h = (&w.x)[i >> 1];
        if constexpr (std::is_same<T, __half>::value)
          x[i] = __half2float(__ushort_as_half(static_cast<unsigned short>(i & 1 ? h >> 16 : h & 0xffffu)));
        else
          x[i] = __uint_as_float(i & 1 ? h & 0xffff0000u : h << 16);
      }
    }
  }
};

struct Lists {
  uint64_t list[kListMax];
  uint64_t sorted[kThreads];  // the warps' maxima, each warp's in order
  uint64_t threshold;
  int fill;
  int added[3];               // keys that a group of tiles added; two groups on, 0 again
  float warp_low[kThreads / 32];
};

// The k-th largest (k <= 256) of the threads' keys, which differ or are 0; to
// all threads.  Each warp sorts its own, then a key's rank is found by binary
// searches in the others'.
__device__ uint64_t kth_of_threads(uint64_t key, int k, Lists& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned full = 0xffffffffu;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
    for (int o = size >> 1; o > 0; o >>= 1) {
      const uint64_t other = __shfl_xor_sync(full, key, o);
      const bool descending = (lane & size) == 0 || size == 32, low = (lane & o) == 0;
      if ((key < other) == (descending == low)) key = other;
    }
  }
  s.sorted[threadIdx.x] = key;
  if (threadIdx.x == 0) s.threshold = 0;
  __syncthreads();
  int rank = lane;  // of equal keys (0 only) any order does
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == warp) continue;
    int n = 0;  // keys of warp w above this one
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (s.sorted[w * 32 + n + o - 1] > key) n += o;
    if (n == 31 && s.sorted[w * 32 + 31] > key) n = 32;
    rank += n;
  }
  if (rank == k - 1 && key) s.threshold = key;
  __syncthreads();
  return s.threshold;
}

// Leaves the `width` largest of the list's n keys in it, in order, and returns
// the last of them as the threshold (0 while there are fewer); n becomes their
// number.
__device__ uint64_t cut_list(int width, int& n, Lists& s) {
  __syncthreads();
  if (n > 2 * kThreads) {  // first by the threads' maxima: at most `width` threads' keys stay
    uint64_t top = 0;
    for (int i = threadIdx.x; i < n; i += kThreads) top = max(top, s.list[i]);
    const uint64_t th = kth_of_threads(top, width, s);
    uint64_t mine[kListMax / kThreads];
#pragma unroll
    for (int j = 0; j < kListMax / kThreads; ++j) {
      const int i = threadIdx.x + j * kThreads;
      mine[j] = i < n ? s.list[i] : 0;
    }
    if (threadIdx.x == 0) s.fill = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kListMax / kThreads; ++j)
      if (mine[j] >= th && mine[j]) s.list[atomicAdd(&s.fill, 1)] = mine[j];
    __syncthreads();
    n = s.fill;
  }
  static_assert(kMaxWidth * (kListMax / kThreads) <= 2 * kThreads, "what stays is two keys a thread");
  uint64_t mine[2];
  int rank[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = threadIdx.x + j * kThreads;
    mine[j] = i < n ? s.list[i] : 0;
    if (i - static_cast<int>(threadIdx.x & 31) >= n) continue;  // (the warp's)
    for (int o = 0; o < n; ++o) rank[j] += s.list[o] > mine[j];
  }
  if (threadIdx.x == 0) s.threshold = 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (mine[j] && rank[j] < width) {
      s.list[rank[j]] = mine[j];
      if (rank[j] == width - 1) s.threshold = mine[j];
    }
  }
  n = min(n, width);
  __syncthreads();
  return s.threshold;
}

__device__ __forceinline__ uint64_t ordered64(double x) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ double from_ordered64(uint64_t o) {
  return __longlong_as_double(static_cast<long long>(o >> 63 ? o & ~(1ull << 63) : ~o));
}

constexpr int kMergeKeys = 2048;  // scores kept in shared memory
constexpr int kMaxLists = kMaxBeams * kMaxParts;

struct Merge {
  double base[kMaxBeams];  // what a beam's candidates start from
  uint64_t score[kMergeKeys];
  uint32_t token[kMergeKeys];
  unsigned char at[kMaxLists];
};

// A list is a part of a beam's row: list i is part i % parts of beam i / parts,
// so that of equal scores the one from the lower list goes first.
__device__ __forceinline__ void merge_beams(const BeamParams& p, int64_t seq, Merge& s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned full = 0xffffffffu;
  const int lists = p.beams * p.parts, first = min(p.width, kMergeKeys / lists);  // scores of a list that are kept
  const unsigned long long* keys = p.keys + seq * lists * p.width;
  for (int i = tid; i < lists; i += kThreads) s.at[i] = 0;
  // this thread's first keys, on their way while the log sums are worked out
  constexpr int kAhead = 2;
  unsigned long long ahead[kAhead];
  auto key_at = [&](int i) {
    const int list = i / first;
    return __ldcg(keys + static_cast<int64_t>(list) * p.width + i - list * first);
  };
#pragma unroll
  for (int j = 0; j < kAhead; ++j) ahead[j] = tid + j * kThreads < lists * first ? key_at(tid + j * kThreads) : 0;
  for (int b = warp; b < p.beams; b += kThreads / 32) {
    const int64_t row = seq * p.beams + b;
    const float2 ml = lane < p.parts ? __ldcg(p.sums + row * p.parts + lane) : make_float2(-INFINITY, 0.f);
    const float score = __ldg(p.scores + row);
    float top = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(full, top, o));
    float l = ml.x == -INFINITY && ml.y == 0.f ? 0.f : ml.y * ex2((ml.x - top) * kLog2e);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(full, l, o);
    // log l = e log 2 + log m, 1 <= m < 2: the fp32 logarithm is small
    const bool fine = l >= 0.5f && l < INFINITY && fabsf(top) < INFINITY && fabsf(score) < INFINITY;
    const int e = static_cast<int>(__float_as_uint(l) >> 23) - 127;
    const float m = __uint_as_float((__float_as_uint(l) & 0x007fffffu) | 0x3f800000u);
    if (lane == 0)
      s.base[b] = fine ? static_cast<double>(score) - static_cast<double>(top) - e * 0.69314718055994530942 - static_cast<double>(logf(m))
                       : -INFINITY;
  }
  __syncthreads();
  auto score_of = [&](int list, uint64_t key) -> uint64_t {
    const double base = s.base[list / p.parts];
    return key && base > -INFINITY ? ordered64(base + static_cast<double>(from_ordered(static_cast<uint32_t>(key >> 32)))) : 0;
  };
  auto keep = [&](int i, uint64_t key) {
    s.score[i] = score_of(i / first, key);
    s.token[i] = 0xffffffffu - static_cast<uint32_t>(key);
  };
#pragma unroll
  for (int j = 0; j < kAhead; ++j)
    if (tid + j * kThreads < lists * first) keep(tid + j * kThreads, ahead[j]);
  for (int i = tid + kAhead * kThreads; i < lists * first; i += kThreads) keep(i, key_at(i));
  __syncthreads();
  if (warp != 0) return;
  // rounds: each lane has the best of its lists (score, list, token)
  uint64_t best = 0;
  uint32_t token = 0;
  int mine = 0;
  auto look = [&] {
    best = 0;
    mine = 0x7fffffff;
    for (int i = lane; i < lists; i += 32) {
      const int at = s.at[i];
      if (at >= p.width) continue;
      uint64_t sc;
      uint32_t tk;
      if (at < first) {
        sc = s.score[i * first + at], tk = s.token[i * first + at];
      } else {
        const uint64_t key = __ldcg(keys + static_cast<int64_t>(i) * p.width + at);
        sc = score_of(i, key), tk = 0xffffffffu - static_cast<uint32_t>(key);
      }
      if (sc > best) best = sc, mine = i, token = tk;
    }
  };
  look();
  for (int i = 0; i < p.width; ++i) {
    const uint32_t hi = static_cast<uint32_t>(best >> 32), top = __reduce_max_sync(full, hi);
    const uint32_t lo = hi == top ? static_cast<uint32_t>(best) : 0, low = __reduce_max_sync(full, lo);
    const bool have = hi == top && static_cast<uint32_t>(best) == low;
    const int list = __reduce_min_sync(full, have ? mine : 0x7fffffff);
    const int64_t to = seq * p.width + i;
    if (top == 0) {  // (a score's pattern has high bits) no candidate is left
      if (lane == 0) p.out_scores[to] = -INFINITY, p.out_beams[to] = -1, p.out_tokens[to] = -1;
    } else if (have && mine == list) {
      p.out_scores[to] = static_cast<float>(from_ordered64(best));
      p.out_beams[to] = list / p.parts;
      p.out_tokens[to] = static_cast<int32_t>(token);
      ++s.at[list];
      look();
    }
    __syncwarp();
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) beam_kernel(const BeamParams p) {
  __shared__ union Shared {
    Lists lists;
    Merge merge;
    __device__ Shared() {}
  } shared;
  __shared__ float2 s_sum[kThreads / 32];
  __shared__ bool s_last;
  Lists& s = shared.lists;
  using Units = RowUnits<T>;
  constexpr int kVec = Units::kVec, kUnits = kPer / kVec;
  const int64_t row = blockIdx.x / p.parts;
  const int part = static_cast<int>(blockIdx.x - row * p.parts);
  const Units units(static_cast<const T*>(p.logits) + row * p.row_stride, p.vocab);
  const int64_t first = static_cast<int64_t>(part) * p.tiles * kTile, last = min(units.end, first + static_cast<int64_t>(p.tiles) * kTile);
  if (threadIdx.x < 3) s.added[threadIdx.x] = 0;
  __syncthreads();

  float m = -INFINITY, l = 0.f;
  int n = 0;               // keys of the list
  uint64_t threshold = 0;  // keys above it are candidates (what equals it is in the list)
  float low = -INFINITY;   // their values are not below it
  uint4 ahead[kUnits];
  auto fetch = [&](int64_t at, uint4* w) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i) w[i] = units.load(at / kVec + i * kThreads + threadIdx.x);
  };
  auto token = [&](int64_t at, int i) {
    return static_cast<uint32_t>(at + (static_cast<int64_t>(i / kVec) * kThreads + threadIdx.x) * kVec + i % kVec - units.lead);
  };
  auto top_of = [](const float (&x)[kPer]) {
    float top = fmaxf(x[0], x[1]);
#pragma unroll
    for (int i = 2; i < kPer; i += 2) top = fmaxf(top, fmaxf(x[i], x[i + 1]));
    return top;
  };
  // adds a tile's candidates to the list, its places counted by `count` from n0 on
  auto add = [&](int64_t at, const float (&x)[kPer], int n0, int* count) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (!(x[i] >= low)) continue;
      const uint64_t k = key_of(x[i], token(at, i));
      if (k > threshold) {
        const int to = n0 + atomicAdd(count, 1);
        if (to < kListMax) s.list[to] = k;
      }
    }
  };
  if (first < last) fetch(first, ahead);
  int turn = 0;
  for (int64_t g0 = first; g0 < last; g0 += kGroup * kTile) {
    int* count = s.added + turn;
    turn = turn == 2 ? 0 : turn + 1;
    if (threadIdx.x == 0) s.added[turn] = 0;  // (read last before the group before)
    const int64_t g1 = min(last, g0 + kGroup * kTile);
    for (int64_t at = g0; at < g1; at += kTile) {
      float x[kPer];
#pragma unroll
      for (int i = 0; i < kUnits; ++i) Units::values(ahead[i], x + i * kVec);
      if (at + kTile < last) fetch(at + kTile, ahead);
      const float top = top_of(x), mn = fmaxf(m, top), ref = mn == -INFINITY ? 0.f : mn;
      const uint64_t less = pack2(-ref, -ref), scale = pack2(kLog2e, kLog2e);
      uint64_t sum = pack2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kPer; i += 2) {
        float u, v;
        unpack2(mul2(add2(pack2(x[i], x[i + 1]), less), scale), u, v);
        sum = add2(sum, pack2(ex2(u), ex2(v)));
      }
      float even, odd;
      unpack2(sum, even, odd);
      l = l * ex2((m - ref) * kLog2e) + (even + odd);
      m = mn;
      if (at == first) {
        // the (width / 8)-th largest of each warp's threads: `width` values at
        // least are not below the smallest of those
        const int k = (p.width + kThreads / 32 - 1) / (kThreads / 32), lane = threadIdx.x & 31;
        const uint32_t mine = top > -INFINITY ? ordered(top) : 0;
        int above = 0;
#pragma unroll
        for (int o = 0; o < 32; ++o) {
          const uint32_t other = __shfl_sync(0xffffffffu, mine, o);
          above += other > mine || (other == mine && o < lane);
        }
        if (above == k - 1) s.warp_low[threadIdx.x >> 5] = mine ? top : -INFINITY;
        __syncthreads();
        low = s.warp_low[0];
#pragma unroll
        for (int w = 1; w < kThreads / 32; ++w) low = fminf(low, s.warp_low[w]);
      }
      if (top >= low) add(at, x, n, count);
    }
    __syncthreads();
    const int all = n + *count;
    if (all <= kListMax) {
      n = all;
      // a tight threshold keeps the candidates few, and a short list is cut quickly
      if (n > p.width + kSpare) threshold = max(threshold, cut_list(p.width, n, s));
    } else {
      // too many: this group again, tile by tile
      if (n > kListMax / 2) threshold = max(threshold, cut_list(p.width, n, s));
      for (int64_t at = g0; at < g1; at += kTile) {
        uint4 w[kUnits];
        float x[kPer];
        fetch(at, w);
#pragma unroll
        for (int i = 0; i < kUnits; ++i) Units::values(w[i], x + i * kVec);
        uint64_t best = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) best = max(best, key_of(x[i], token(at, i)));
        // at least `width` of the tile reach it, of at most `width` threads
        const uint64_t th = kth_of_threads(best, p.width, s);
        if (th > threshold) threshold = th - 1;
        low = threshold ? from_ordered(static_cast<uint32_t>(threshold >> 32)) : -INFINITY;
        if (threadIdx.x == 0) s.fill = 0;
        __syncthreads();
        add(at, x, n, &s.fill);
        __syncthreads();
        n += s.fill;
        threshold = max(threshold, cut_list(p.width, n, s));
      }
    }
    if (threshold) low = from_ordered(static_cast<uint32_t>(threshold >> 32));
  }
  cut_list(p.width, n, s);
  unsigned long long* keys = p.keys + (row * p.parts + part) * p.width;
  for (int i = threadIdx.x; i < p.width; i += kThreads) keys[i] = i < n ? s.list[i] : 0;

  // the sums of the threads
  auto join = [](float& m, float& l, float om, float ol) {
    const float mn = fmaxf(m, om), ref = mn == -INFINITY ? 0.f : mn;
    l = l * ex2((m - ref) * kLog2e) + ol * ex2((om - ref) * kLog2e);
    m = mn;
  };
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float om = __shfl_xor_sync(0xffffffffu, m, o), ol = __shfl_xor_sync(0xffffffffu, l, o);
    join(m, l, om, ol);
  }
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = make_float2(m, l);
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kThreads / 32; ++w) join(m, l, s_sum[w].x, s_sum[w].y);
    p.sums[row * p.parts + part] = make_float2(m, l);
  }
  // ---- the sequence's last block; the count is 0 again behind it
  __threadfence();
  __syncthreads();
  const int64_t seq = row / p.beams;
  if (threadIdx.x == 0) {
    const unsigned blocks = static_cast<unsigned>(p.beams * p.parts);
    s_last = atomicInc(p.arrived + seq, blocks - 1) == blocks - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  merge_beams(p, seq, shared.merge);
}

}  // namespace

// Parts of a row: enough blocks to fill the GPU, of a tile at least.
int beam_parts(int64_t rows, int64_t vocab, int sms) {
  const int64_t tiles = (vocab + 7 + kTile - 1) / kTile;  // (a row that starts inside a 16-byte unit is up to 7 longer)
  const int64_t want = (4 * static_cast<int64_t>(sms) + rows - 1) / rows;
  int64_t parts = want < tiles ? want : tiles;
  if (parts > kMaxParts) parts = kMaxParts;
  const int64_t per = (tiles + parts - 1) / parts;
  return static_cast<int>((tiles + per - 1) / per);
}

cudaError_t launch_beam(const BeamParams& given, int dtype, cudaStream_t s) {
  int dev = 0, sms = 0;
  const cudaError_t found = current_device(&dev, &sms);
  if (found != cudaSuccess) return found;
  BeamParams p = given;
  const int64_t rows = p.n_seqs * p.beams;
  p.parts = beam_parts(rows, p.vocab, sms);
  p.tiles = static_cast<int>(((p.vocab + 7 + kTile - 1) / kTile + p.parts - 1) / p.parts);
  p.sums = reinterpret_cast<float2*>(p.keys + rows * p.parts * p.width);
  const int64_t grid = rows * p.parts;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  auto go = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(grid), kThreads, 0, s>>>(p);
    return cudaGetLastError();
  };
  switch (dtype) {
    case QGEMV_DT_F32: return go(beam_kernel<float>);
    case QGEMV_DT_F16: return go(beam_kernel<__half>);
    default: return go(beam_kernel<__nv_bfloat16>);
  }
}

}  // namespace qgemv
