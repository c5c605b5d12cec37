// beam.cu -- the selection of beam search (qgemv_beam_select): of a sequence's
// candidates (beam b, token t) the `width` of largest
//
//   score[b] + x[b][t] - log sum_u exp x[b][u].
//
// One pass over the logits, which are its bytes' floor, leaves two numbers of
// each chunk of 512: its largest value m and the sum of exp(x - m).  A warp for a
// chunk, with nothing to wait for but its loads: it takes many warps to have
// enough bytes on their way (512 rows of 128000 tokens in fp32: 65 us with lists of
// candidates kept during the pass, 96 with warps that take several chunks; 38 so,
// 6.9 TB/s; in bf16 27, 4.9 TB/s, with as many warps, exponentials and
// instructions).  Then, by a block for each sequence, the beams' log sums and
// each chunk's best score are known; the `width`-th largest of its threads' best
// chunks bounds the result from below, so that only the chunks that reach it,
// little more than `width`, are read again, the best ones first, and their values
// ranked: latencies of 10 us, whatever the logits are.  (Fewer chunks with good
// values than `width`, as in a first step of one beam, make a second, closer bound
// of their lanes' best values: 4 beams of 32000 tokens, 64 kept, one beam alive: 24
// us, against 180 with the chunks one after the other.)
//
// Sums of exponentials are fp32, and no longer chains of roundings for longer rows
// (2^26 tokens in chunks that are alike: off by 2^-20.5, by 2^-14.6 if a lane's
// chunks were added up one after the other):
// a chunk's is six additions deep in a lane and five between the lanes, a beam's of
// its chunks four, a sum whose rounding errors are added up beside it, and five.
// The log sum, whose whole powers of two are taken apart, and the scores are
// 64-bit: fp32 would make ties of scores that differ.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "beam.h"
#include "kv_layout.cuh"
#include "per_device.h"
#include "tc_common.cuh"

namespace qgemv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = kBeamChunk / 32;  // values of a lane
constexpr int kWindow = 2048;          // chunks that are looked at together
constexpr int kPicked = 512;           // chunks that are read again, at a time
constexpr int kCands = 1024;           // candidates, at a time
constexpr int kFewCands = 256;         // candidates that are soon put in order
static_assert(kMaxWidth + kBeamChunk <= kCands && kWindow % kPicked == 0, "a chunk's values fit beside those that stay");

// Order of floats as unsigned numbers, +0 and -0 as one; 0 is below all.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint64_t ordered64(double x) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ double from_ordered64(uint64_t o) {
  return __longlong_as_double(static_cast<long long>(o >> 63 ? o & ~(1ull << 63) : ~o));
}

// A row's chunks of kBeamChunk tokens from its first one on, wherever the row
// starts: which lane has which tokens, and so the order of all sums, does not
// depend on where the row lies (equal rows have equal sums).  Rows that start
// inside a lane's unit are read by words (64 x 8 of 128001 tokens in bf16 38.7 us,
// of 128000 36.5; fp32 50.9 and 48.0; by two whole units each, whose words are
// shifted, bf16 42.4; with the words exchanged between lanes 46).
template <typename T>
struct RowUnits {
  using Unit = typename std::conditional<sizeof(T) == 4, uint4, uint2>::type;
  static constexpr int kVec = sizeof(Unit) / sizeof(T), kUnits = kPer / kVec, kWords = sizeof(Unit) / 4;
  const T* row;
  int n;
  __device__ RowUnits(const T* first, int vocab) : row(first), n(vocab) {}
  // whether a row of 16-bit values starts inside a word
  __device__ bool odd() const { return sizeof(T) == 2 && (reinterpret_cast<uintptr_t>(row) & 2); }
  __device__ bool aligned() const { return (reinterpret_cast<uintptr_t>(row) & (sizeof(Unit) - 1)) == 0; }
  // whether what `load` reads of a chunk lies in the row whole (odd ones: half a word
  // more at each end)
  __device__ bool inside(int chunk) const { return (chunk + 1) * kBeamChunk + odd() <= n && chunk >= odd(); }
  // a lane's values of such a chunk: by units, or by words, of which an odd row takes a
  // half each
  __device__ void load(int chunk, float (&x)[kPer]) const {
    uint32_t w[kUnits][kWords];
    const int lane = threadIdx.x & 31;
    if (aligned()) {
      const Unit* from = reinterpret_cast<const Unit*>(row) + chunk * (kBeamChunk / kVec) + lane;
#pragma unroll
      for (int i = 0; i < kUnits; ++i) *reinterpret_cast<Unit*>(w[i]) = __ldg(from + 32 * i);
    } else {
      const uint32_t* from = reinterpret_cast<const uint32_t*>(row - odd()) + (chunk * (kBeamChunk / kVec) + lane) * kWords;
      uint32_t last[kUnits] = {};
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
#pragma unroll
        for (int k = 0; k < kWords; ++k) w[i][k] = __ldg(from + 32 * kWords * i + k);
        if (odd()) last[i] = __ldg(from + 32 * kWords * i + kWords);
      }
      if (odd()) {
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
#pragma unroll
          for (int k = 0; k < kWords; ++k) w[i][k] = __funnelshift_r(w[i][k], k + 1 < kWords ? w[i][(k + 1) % kWords] : last[i], 16);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if constexpr (std::is_same<T, float>::value) {
        x[i] = __uint_as_float(w[i / kVec][i % kVec]);
      } else {
        const uint32_t h = w[i / kVec][i % kVec >> 1];
        if constexpr (std::is_same<T, __half>::value)
          x[i] = __half2float(__ushort_as_half(static_cast<unsigned short>(i & 1 ? h >> 16 : h & 0xffffu)));
        else
          x[i] = __uint_as_float(i & 1 ? h & 0xffff0000u : h << 16);
      }
    }
  }
  // a lane's values of another; what is outside the row is -infinity
  __device__ void edge(int chunk, float (&x)[kPer]) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int at = place(chunk, i);
      x[i] = at < n ? static_cast<float>(row[at]) : -INFINITY;
    }
  }
  __device__ void get(int chunk, float (&x)[kPer]) const {
    if (inside(chunk)) load(chunk, x);
    else edge(chunk, x);
  }
  // the token of a lane's value i of a chunk
  __device__ static int place(int chunk, int i) {
    return chunk * kBeamChunk + ((i / kVec) * 32 + static_cast<int>(threadIdx.x & 31)) * kVec + i % kVec;
  }
};

__device__ __forceinline__ float largest(const float (&x)[kPer]) {
  float top = fmaxf(x[0], x[1]);
#pragma unroll
  for (int i = 2; i < kPer; i += 2) top = fmaxf(top, fmaxf(x[i], x[i + 1]));
  return top;
}

struct Candidate {
  uint64_t score, place;  // ordered64, and (beam, token): the lower place goes first
};
__device__ __forceinline__ bool better(uint64_t score, uint64_t place, uint64_t o_score, uint64_t o_place) {
  return score > o_score || (score == o_score && place < o_place);
}

struct Shared {
  double base[kMaxBeams];  // what a beam's candidates start from, or -infinity
  Candidate cand[kCands];
  float about[kWindow];    // the chunks' best scores in fp32, of the first window
  uint32_t bound[2 * kWarps];
  int reach[2 * kWarps];
  uint32_t turned[kWarps * 33];
  float picked_score[kPicked];
  int picked[kPicked], order[kPicked];
  uint32_t far;
  int n_picked, n_cand;
};

// A value that k of the threads' keys at least reach, and few more; 0 where fewer
// than k are above 0.  Of the two keys of each warp about the (k / kWarps)-th
// largest, the largest one that k reach; the keys of neighbouring threads, which
// are chunks of one beam, go to different warps first, so that it is a good one
// where one beam has all of the best chunks.
__device__ __forceinline__ uint32_t reached_by(uint32_t key, int k, Shared& s) {
  const unsigned full = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  static_assert(kWarps == 16, "two bounds of a warp are a lane's each");
  if (threadIdx.x < 2 * kWarps) s.reach[threadIdx.x] = 0;
  s.turned[warp * 33 + lane] = key;
  __syncthreads();
  key = s.turned[lane / 2 * 33 + (lane & 1) * 16 + warp];
  uint32_t left = key, top = 0;
#pragma unroll 1
  for (int j = (k + kWarps - 1) / kWarps; j >= 0; --j) {
    top = __reduce_max_sync(full, left);
    if (j < 2 && lane == 0) s.bound[2 * warp + j] = top;
    if (lane == __ffs(__ballot_sync(full, left == top)) - 1) left = 0;
  }
  __syncthreads();
  const uint32_t bound = s.bound[lane];
  int reach = 0;  // keys of this warp that reach the lane's bound
#pragma unroll 4
  for (int o = 0; o < 32; ++o) reach += __shfl_sync(full, key, o) >= bound;
  atomicAdd(&s.reach[lane], reach);
  __syncthreads();
  return __reduce_max_sync(full, s.reach[lane] >= k ? bound : 0);
}

// Leaves the `width` best of the n candidates, in order; returns their number.
__device__ __forceinline__ int cut(int width, int n, Shared& s) {
  __syncthreads();
  constexpr int kMine = kCands / kThreads;
  Candidate mine[kMine];
  int rank[kMine];
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int i = threadIdx.x + j * kThreads;
    rank[j] = width;
    if (i >= n) continue;
    mine[j] = s.cand[i];
    int above = 0;
#pragma unroll 4
    for (int o = 0; o < n; ++o) {
      const Candidate c = s.cand[o];
      above += better(c.score, c.place, mine[j].score, mine[j].place);
    }
    rank[j] = above;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kMine; ++j)
    if (rank[j] < width) s.cand[rank[j]] = mine[j];
  __syncthreads();
  return min(n, width);
}

// A sequence's candidates, by the block, from its chunks' sums.
template <typename T>
__device__ __forceinline__ void choose(const BeamParams& p, int64_t seq) {
  extern __shared__ __align__(16) uint8_t s_all[];
  Shared& s = *reinterpret_cast<Shared*>(s_all);
  using Units = RowUnits<T>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, C = p.n_chunks, n_all = p.beams * C;
  const unsigned full = 0xffffffffu;
  const float2* chunks = p.chunks + seq * n_all;
  // ---- the beams' log sums
  for (int b = warp; b < p.beams; b += kWarps) {
    const float score = __ldg(p.scores + seq * p.beams + b);
    // the largest chunk, then the sum relative to it: 16 chunks of a lane by a tree,
    // these sums one after the other with what each addition rounds off, and the lanes
    constexpr int kAt = 16;  // (one round of reads for up to 262144 tokens; 2 x 8 of 256000: 14.5 us, 15.5 with 8)
    float2 first[kAt];
    auto fetch = [&](int c0, float2 (&ml)[kAt]) {
#pragma unroll
      for (int k = 0; k < kAt; ++k) {
        const int c = c0 + 32 * k + lane;
        ml[k] = c < C ? __ldcg(chunks + b * C + c) : make_float2(-INFINITY, 0.f);
      }
    };
    fetch(0, first);
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < kAt; ++k) top = fmaxf(top, first[k].x);
#pragma unroll 4
    for (int c = 32 * kAt + lane; c < C; c += 32) top = fmaxf(top, __ldcg(&chunks[b * C + c].x));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(full, top, o));
    const float ref = top == -INFINITY ? 0.f : top;
    auto sum = [&](const float2 (&ml)[kAt]) {
      float e[kAt];
#pragma unroll
      for (int k = 0; k < kAt; ++k) e[k] = ml[k].y * ex2((ml[k].x - ref) * kLog2e);
#pragma unroll
      for (int step = 1; step < kAt; step *= 2)
#pragma unroll
        for (int k = 0; k < kAt; k += 2 * step) e[k] += e[k + step];
      return e[0];
    };
    float l = sum(first), off = 0.f;
#pragma unroll 1
    for (int c0 = 32 * kAt; c0 < C; c0 += 32 * kAt) {
      float2 ml[kAt];
      fetch(c0, ml);
      const float add = sum(ml), both = __fadd_rn(l, add), back = __fsub_rn(both, l);
      off += __fadd_rn(__fsub_rn(l, __fsub_rn(both, back)), __fsub_rn(add, back));  // l + add - both, exactly
      l = both;
    }
    l += off;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(full, l, o);
    // log l = e log 2 + log f, 1 <= f < 2: the fp32 logarithm is small
    const bool fine = l >= 0.5f && l < INFINITY && fabsf(top) < INFINITY && fabsf(score) < INFINITY;
    const int e = static_cast<int>(__float_as_uint(l) >> 23) - 127;
    const float f = __uint_as_float((__float_as_uint(l) & 0x007fffffu) | 0x3f800000u);
    if (lane == 0)
      s.base[b] = fine ? static_cast<double>(score) - static_cast<double>(top) - e * 0.69314718055994530942 - static_cast<double>(logf(f))
                       : -INFINITY;
  }
  if (tid == 0) s.n_cand = 0, s.far = 0;
  __syncthreads();
  // ---- the chunks' best scores, in fp32: off by less than 2^-23 of the largest
  // base and the score itself
  auto score_of = [&](int b, float x) { return ordered64(s.base[b] + static_cast<double>(x)); };
  auto about_of = [](double base, float x) {  // -infinity: no candidate
    return base > -INFINITY && x > -INFINITY ? fminf(fmaxf(static_cast<float>(base) + x, -FLT_MAX), FLT_MAX) : -INFINITY;
  };
  auto about = [&](int i) {
    return about_of(s.base[i / C], __ldcg(&chunks[i].x));
  };
  if (tid < p.beams && s.base[tid] > -INFINITY) atomicMax(&s.far, __float_as_uint(fabsf(static_cast<float>(s.base[tid]))));
  float best = -INFINITY;
#pragma unroll 4
  for (int i = tid; i < n_all; i += kThreads) {
    const float mine = about(i);
    if (i < kWindow) s.about[i] = mine;
    best = fmaxf(best, mine);
  }
  const uint32_t bound = reached_by(best > -INFINITY ? ordered(best) : 0, p.width, s);
  const float far = __uint_as_float(s.far);
  auto less = [&](float x) { return x - 0x1p-20f * (far + fabsf(x)); };  // surely below what `x` stands for
  // Chunks that have candidates are not below `from`; once there are `width`
  // candidates (`filled`), others are not worse than (low, place).
  float from = bound ? less(from_ordered(bound)) : -INFINITY;
  uint64_t low = 0, place = 0;
  bool filled = false;
  int n = 0;
  // whether no value of chunk i, which reaches `from`, is a candidate
  auto worse = [&](int i) {
    const int b = i / C, c = i - b * C;
    const uint64_t at = static_cast<uint64_t>(b) << 32 | static_cast<uint32_t>(c * kBeamChunk);  // its first token
    return filled && better(low, place, score_of(b, __ldcg(&chunks[i].x)), at);
  };
  int step = kWindow;
#pragma unroll 1
  for (int i0 = 0; i0 < n_all; i0 += step) {
    // ---- of `step` chunks those that reach it, the best first
    __syncthreads();
    if (tid == 0) s.n_picked = 0;
    __syncthreads();
#pragma unroll 1
    for (int i = i0 + tid; i < min(i0 + step, n_all); i += kThreads) {
      const float mine = i < kWindow ? s.about[i] : about(i);
      if (mine >= from && mine > -INFINITY && !worse(i)) {
        const int to = atomicAdd(&s.n_picked, 1);
        if (to < kPicked) s.picked_score[to] = mine, s.picked[to] = i;
      }
    }
    __syncthreads();
    const int n_picked = s.n_picked;
    if (n_picked > kPicked) {  // (many equal ones) fewer at a time
      i0 -= kPicked;
      step = kPicked;
      continue;
    }
    if (tid < n_picked) {
      static_assert(kPicked <= kThreads, "a thread for each");
      const float mine = s.picked_score[tid];
      const int at = s.picked[tid];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < n_picked; ++j) rank += s.picked_score[j] > mine || (s.picked_score[j] == mine && s.picked[j] < at);
      s.order[rank] = tid;
    }
    __syncthreads();
    // ---- the r-th chunk of them, by a warp: its values that may be candidates
    float x[kPer], least;  // values below that are worse
    int b, c;
    auto look = [&](int r) {
      const int i = s.picked[s.order[r]];
      b = i / C, c = i - b * C;
      Units(static_cast<const T*>(p.logits) + (seq * p.beams + b) * p.row_stride, static_cast<int>(p.vocab)).get(c, x);
      least = less(from - static_cast<float>(s.base[b]));
      if (!(least > -INFINITY && least < INFINITY)) least = -FLT_MAX;  // (also where fp32 ends)
    };
    // to the candidates with their places and, for the time being, values; returns
    // whether there was room
    auto add = [&] {
      uint32_t on = 0;
#pragma unroll
      for (int k = 0; k < kPer; ++k) on |= (x[k] >= least ? 1u : 0u) << k;
      const int mine = __popc(on);
      if (!__any_sync(full, mine > 0)) return true;
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(full, upto, o);
        if (lane >= o) upto += y;
      }
      int first = 0;
      if (lane == 31) first = atomicAdd(&s.n_cand, upto);
      first = __shfl_sync(full, first, 31);
      if (first + __shfl_sync(full, upto, 31) > kCands) return false;
      Candidate* to = s.cand + first + upto - mine;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (!(on >> k & 1)) continue;
        to->place = static_cast<uint64_t>(b) << 32 | static_cast<uint32_t>(Units::place(c, k));
        to->score = __float_as_uint(x[k]);
        ++to;
      }
      return true;
    };
    auto score = [&](int n1) {  // of the candidates from n on
      for (int j = n + tid; j < n1; j += kThreads)
        s.cand[j].score = score_of(static_cast<int>(s.cand[j].place >> 32), __uint_as_float(static_cast<uint32_t>(s.cand[j].score)));
      n = n1;
    };
    auto shorten = [&] {
      n = cut(p.width, n, s);
      if (tid == 0) s.n_cand = n;
      if (n == p.width) {
        low = s.cand[n - 1].score, place = s.cand[n - 1].place;
        from = less(static_cast<float>(from_ordered64(low)));
        filled = true;
      }
      __syncthreads();
    };
    // Few: the warps go through them on their own.  Many, or with many candidates
    // (fewer chunks than `width` have the best ones): again, from a closer bound, of
    // the lanes' best ones.  If it does not help (values that are alike): the best
    // chunks one at a time, one, two, four and so on, until few are left that may
    // have candidates.
    int left = n_picked, alone = 1;
    bool close = false;
#pragma unroll 1
    while (left > 0) {
      if (left <= 8 * kWarps || close) {
#pragma unroll 1
        for (int r = warp; r < left; r += kWarps) {
          look(r);
          if (!add()) break;
        }
        __syncthreads();
        const int n1 = s.n_cand;
        __syncthreads();
        if (n1 <= (close ? kCands : kFewCands)) {
          score(n1);
          if (n > p.width && i0 + step < n_all) shorten();
          break;
        }
        if (tid == 0) s.n_cand = n;
      }
      int batch = 0;
      if (!close) {
        close = true;
        float mine = -INFINITY;
#pragma unroll 1
        for (int r = warp; r < left; r += kWarps) {
          look(r);
          mine = fmaxf(mine, about_of(s.base[b], largest(x)));
        }
        const uint32_t bound = reached_by(mine > -INFINITY ? ordered(mine) : 0, p.width, s);
        if (bound) from = fmaxf(from, less(from_ordered(bound)));
      } else {
        batch = min(alone, left);
        alone *= 2;
#pragma unroll 1
        for (int r = 0; r < batch; ++r) {
          __syncthreads();
          if (warp == 0) {
            look(r);
            add();
          }
          __syncthreads();
          score(s.n_cand);
          if (n > p.width) shorten();
        }
      }
      // the others that are not worse, in their order
      __syncthreads();
      int at = -1;
      if (tid >= batch && tid < left) {
        at = s.order[tid];
        if (s.picked_score[at] < from || worse(s.picked[at])) at = -1;
      }
      const unsigned on = __ballot_sync(full, at >= 0);
      if (lane == 0) s.reach[warp] = __popc(on);
      __syncthreads();
      const int of_warp = lane < kWarps ? s.reach[lane] : 0, before = __reduce_add_sync(full, lane < warp ? of_warp : 0);
      if (at >= 0) s.order[before + __popc(on & ((1u << lane) - 1))] = at;
      left = __reduce_add_sync(full, of_warp);
      __syncthreads();
    }
  }
  n = cut(p.width, n, s);
  for (int i = tid; i < p.width; i += kThreads) {
    const int64_t to = seq * p.width + i;
    p.out_scores[to] = i < n ? static_cast<float>(from_ordered64(s.cand[i].score)) : -INFINITY;
    p.out_beams[to] = i < n ? static_cast<int32_t>(s.cand[i].place >> 32) : -1;
    p.out_tokens[to] = i < n ? static_cast<int32_t>(s.cand[i].place) : -1;
  }
}

// A chunk's largest value and sum, by a warp.
template <typename T>
__device__ __forceinline__ void sum_up(const BeamParams& p, int64_t chunk) {
  using Units = RowUnits<T>;
  const int64_t row = div_small(chunk, p.n_chunks);
  const int c = static_cast<int>(chunk - row * p.n_chunks);
  float x[kPer];
  Units(static_cast<const T*>(p.logits) + row * p.row_stride, static_cast<int>(p.vocab)).get(c, x);
  const float m = from_ordered(__reduce_max_sync(0xffffffffu, ordered(largest(x)))), ref = m == -INFINITY ? 0.f : m;
  uint64_t sum[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
#pragma unroll
  for (int k = 0; k < kPer; k += 2) {
    float u, v;
    unpack2(mul2(add2(pack2(x[k], x[k + 1]), pack2(-ref, -ref)), pack2(kLog2e, kLog2e)), u, v);
    sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], pack2(ex2(u), ex2(v)));
  }
  float l, odd;
  unpack2(add2(sum[0], sum[1]), l, odd);
  l += odd;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if ((threadIdx.x & 31) == 0) p.chunks[chunk] = make_float2(m, l);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 3) beam_sums_kernel(const BeamParams p) {
  const int64_t chunk = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (chunk < p.n_seqs * p.beams * p.n_chunks) sum_up<T>(p, chunk);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) beam_choice_kernel(const BeamParams p) {
  wait_for_last_kernel();
  choose<T>(p, blockIdx.x);
}

// Both: a sequence's chunks are those of `blocks` blocks.
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) beam_kernel(const BeamParams p, int blocks) {
  __shared__ bool s_last;
  const int per_seq = p.beams * p.n_chunks;
  const int64_t seq = blockIdx.x / blocks;
  const int i = (blockIdx.x - static_cast<int>(seq) * blocks) * kWarps + (threadIdx.x >> 5);
  if (i < per_seq) sum_up<T>(p, seq * per_seq + i);
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicInc(p.arrived + seq, static_cast<unsigned>(blocks) - 1) == static_cast<unsigned>(blocks) - 1;  // 0 again behind it
    __threadfence();
  }
  __syncthreads();
  if (s_last) choose<T>(p, seq);
}

template <typename T>
cudaError_t launch(const BeamParams& p, int dev, int sms, cudaStream_t s) {
  constexpr int kBytes = static_cast<int>(sizeof(Shared));
  const int64_t per_seq = static_cast<int64_t>(p.beams) * p.n_chunks, blocks = (per_seq + kWarps - 1) / kWarps;
  // Few chunks are summed up all at once, and the block that has a sequence's last
  // one goes on with the choice: a launch fewer (2 x 8 beams of 128000 tokens, fp16,
  // 250 blocks: a call 13.8 us, 16.7 with two kernels, which take 9.6 on the device
  // against 10.4).  More: the choice is a kernel of its own, and its registers and
  // shared memory do not hold up the sums (4 x 8, 500 blocks: 10.4 us on the device,
  // 12.5 in one kernel; 64 x 8: bf16 36.7 against 77.9, fp32 48.6 against 80.7).
  if (blocks * p.n_seqs <= 2 * static_cast<int64_t>(sms)) {
    static std::atomic<uint64_t> set;
    const cudaError_t e = allow_shared_memory(set, dev, beam_kernel<T>, kBytes);
    if (e != cudaSuccess) return e;
    beam_kernel<T><<<static_cast<unsigned>(blocks * p.n_seqs), kThreads, kBytes, s>>>(p, static_cast<int>(blocks));
    return cudaGetLastError();
  }
  static std::atomic<uint64_t> set;
  cudaError_t e = allow_shared_memory(set, dev, beam_choice_kernel<T>, kBytes);
  if (e != cudaSuccess) return e;
  const int64_t grid = (per_seq * p.n_seqs + kWarps - 1) / kWarps;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  beam_sums_kernel<T><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(p);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_after(beam_choice_kernel<T>, static_cast<unsigned>(p.n_seqs), p, s, kThreads, kBytes);
}

}  // namespace

cudaError_t launch_beam(const BeamParams& p, int dtype, cudaStream_t s) {
  int dev = 0, sms = 0;
  const cudaError_t found = current_device(&dev, &sms);
  if (found != cudaSuccess) return found;
  switch (dtype) {
    case QGEMV_DT_F32: return launch<float>(p, dev, sms, s);
    case QGEMV_DT_F16: return launch<__half>(p, dev, sms, s);
    default: return launch<__nv_bfloat16>(p, dev, sms, s);
  }
}

}  // namespace qgemv
