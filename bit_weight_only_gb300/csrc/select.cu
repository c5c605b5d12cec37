// select.cu -- key summaries of cache pages, and the choice of the pages that
// a sequence's new tokens attend (qgemv_kv_summarize, qgemv_kv_select).
//
// With a page's largest and smallest key values per channel, hi and lo, no key
// of it has a larger product with a query q than sum_d max(q_d hi_d, q_d lo_d).
// Summed over the queries that share the key/value head this is one product of
// 2 d values, sum_d (sum max(q_d, 0)) hi_d + (sum min(q_d, 0)) lo_d, whatever
// their number is.  Both sides are rounded to INT8 codes, so that the sum is a
// whole number, exact in any order; the score is it times the page's scale, one
// fp32 product.  So the choice is a matter of the inputs alone, ties included.
//
// Bytes of the summaries (2 d + 4 for a page and head) bound a long context, a
// chain of latencies a short one.  A cluster of up to eight blocks takes a head
// of a sequence: each scores a run of pages and writes the scores into the
// first block's shared memory, which then finds the n_select-th of them by a
// histogram over their range (and another over its bin, until the bin is taken
// whole) and writes the pages in order.  One launch, nothing kept in global
// memory, and two barriers of the cluster: the first block has started before
// others write to it (they arrive on entry and wait when their first score is due),
// and has all of the scores before it goes on.  One token over 8187 pages of 8 heads
// 12.4 us, over 1000 pages 9.0.  (With the scores left in their blocks' shared
// memory and histograms read across, nine synchronisations: 24 us.)
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "kv_codes.cuh"
#include "per_device.h"
#include "select.h"

namespace cg = cooperative_groups;

namespace qgemv {
namespace {

// The INT8 code of a value with the scale max / 127 of a whole vector (an IEEE
// division: codes are decided in fp32); 0 where the scale is 0 or NaN.
__device__ __forceinline__ int8_t code_of(float x, float a) {
  const float q = fminf(fmaxf(rintf(__fdiv_rn(x, a)), -127.f), 127.f);
  return static_cast<int8_t>(a > 0.f ? static_cast<int>(q) : 0);
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

constexpr int kSummaryThreads = 128;

// W warps, one or the block's four, for a head of a page, each for a run of its
// tokens.  Keys with an infinity or NaN leave codes of 0 and a scale of NaN: such
// a page comes before all others.
template <int FMT, int D, int W>
__global__ void __launch_bounds__(kSummaryThreads, W > 1 ? 1 : 8) summary_kernel(const SummaryParams p) {
  constexpr int kLanes = D / 8, kAt = 32 / kLanes;  // kAt tokens at a time
  constexpr int kLoads = kKvBlockTokens / kAt;       // of a block of tokens
  __shared__ float s_edge[2][W][D];
  __shared__ int s_bad[W];
  const unsigned full = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % W, H = p.cache.kv_heads;
  const int64_t item = (static_cast<int64_t>(blockIdx.x) * (kSummaryThreads / 32) + warp) / W, i = div_small(item, H);
  if (i >= p.n) return;  // (W > 1: the block's)
  const int head = static_cast<int>(item - i * H);
  const int64_t page = __ldg(p.pages + i);
  if (page < 0 || page >= p.cache.n_pages) return;
  const int d0 = (lane % kLanes) * 8, run = p.cache.page_tokens / W, t1 = (part + 1) * run;
  // NaN stays in the largest and smallest values, infinities show in them
  float hi[8], lo[8];
  // use(values) of this lane's eight of each token of the run, a block of tokens (or
  // the run's part of one) at a time, all of it on its way together
  auto every = [&](auto use) {
    const int here = min(run, kKvBlockTokens);
    for (int t0 = part * run; t0 < t1; t0 += kKvBlockTokens) {
      const uint8_t* b = kv_block<FMT, D>(p.cache, page, head, t0 / kKvBlockTokens);
      const int t = t0 % kKvBlockTokens + lane / kLanes;
      Eight<FMT, D> x[kLoads];
      if (here == kKvBlockTokens) {
#pragma unroll
        for (int k = 0; k < kLoads; ++k) x[k].load(b, false, t + k * kAt, d0);
#pragma unroll
        for (int k = 0; k < kLoads; ++k) use(x[k]);
      } else {
        for (int k = 0; k * kAt < here; k += 2) {  // four or eight tokens
          x[0].load(b, false, t + k * kAt, d0);
          x[1].load(b, false, t + min(k + 1, here / kAt - 1) * kAt, d0);  // (a token twice changes nothing)
          use(x[0]);
          use(x[1]);
        }
      }
    }
  };
  if constexpr (FMT == QGEMV_KV_F16) {
    __half2 h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = __half2half2(__ushort_as_half(0xfc00)), l[e] = __half2half2(__ushort_as_half(0x7c00));
    every([&](const Eight<FMT, D>& x) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __half2 v = *reinterpret_cast<const __half2*>(&(&x.w.x)[e]);
        h[e] = __hmax2_nan(h[e], v), l[e] = __hmin2_nan(l[e], v);
      }
    });
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 a = __half22float2(h[e]), b = __half22float2(l[e]);
      hi[2 * e] = a.x, hi[2 * e + 1] = a.y, lo[2 * e] = b.x, lo[2 * e + 1] = b.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) hi[e] = -INFINITY, lo[e] = INFINITY;
    every([&](const Eight<FMT, D>& x) {
      float v[8];
      x.values(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) hi[e] = max_nan(hi[e], v[e]), lo[e] = min_nan(lo[e], v[e]);
    });
  }
  bool bad = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1) {
      hi[e] = max_nan(hi[e], __shfl_xor_sync(full, hi[e], o));
      lo[e] = min_nan(lo[e], __shfl_xor_sync(full, lo[e], o));
    }
    bad |= !(fabsf(hi[e]) < INFINITY) || !(fabsf(lo[e]) < INFINITY);
  }
  bad = __any_sync(full, bad);
  // lanes of a token have eight channels each: those of the first hi, of the second lo
  const bool low = lane / kLanes == 1;
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = low ? lo[e] : hi[e];
  if constexpr (W > 1) {
    if (lane < 2 * kLanes) {
#pragma unroll
      for (int e = 0; e < 8; ++e) s_edge[low][part][d0 + e] = x[e];
    }
    if (lane == 0) s_bad[part] = bad;
    __syncthreads();
    if (part != 0) return;
#pragma unroll
    for (int w = 1; w < W; ++w) {
      bad |= s_bad[w] != 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y = s_edge[low][w][d0 + e];
        x[e] = low ? fminf(x[e], y) : fmaxf(x[e], y);
      }
    }
  }
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, lane < 2 * kLanes ? fabsf(x[e]) : 0.f);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(full, m, o));
  const float a = bad ? __int_as_float(0x7fffffff) : __fdiv_rn(m, 127.f);
  const int64_t row = page * H + head;
  if (lane < 2 * kLanes) {
    uint32_t q[8];
    round_quotients<false>(x, a, q);  // 0 where a is 0 or NaN
    *reinterpret_cast<uint2*>(p.codes + row * 2 * D + low * D + d0) =
        make_uint2(__byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410),
                   __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410));
  }
  if (lane == 0) p.scales[row] = a;
}

// Another block's shared memory may be touched once that block has started: all
// arrive first, and wait before they touch it.  (Orders no memory.)
__device__ __forceinline__ void cluster_started() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_for_cluster() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kKeys = 16;  // keys of a thread at a time
constexpr int kMaxCluster = 8;
constexpr int kMaxKeys = 48 * 1024;  // pages of a sequence

// Order of scores as unsigned numbers above 0 (no page); NaN before all.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) select_kernel(const SelectParams p) {
  constexpr int kLanes = 4;                    // lanes of a page
  constexpr int kUnits = 2 * D / 16 / kLanes;  // 16-byte units of a lane
  constexpr int kParts = kThreads / D;
  __shared__ __align__(16) int s_hist[kBins];
  __shared__ long long s_sum[kParts][2][D];
  __shared__ __align__(16) int8_t s_q[2 * D];
  __shared__ uint32_t s_lo[kWarps], s_hi[kWarps];
  __shared__ int s_n[kWarps], s_eq[kWarps];
  __shared__ int s_digit, s_rest, s_count;
  extern __shared__ uint32_t s_key[];  // the first block's: of every page
  cluster_started();
  cg::cluster_group cluster = cg::this_cluster();
  const unsigned full = 0xffffffffu;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = static_cast<int>(cluster.num_blocks()), me = static_cast<int>(cluster.block_rank());
  const int item = blockIdx.x / C, H = p.cache.kv_heads;
  const int seq = item / H, head = item - seq * H, G = p.q_heads / H;
  const int shift = 31 - __clz(p.cache.page_tokens);
  const int ctx = max(0, __ldg(p.ctx_lens + seq));
  int64_t q0 = __ldg(p.cu_q + seq);
  int64_t T = static_cast<int64_t>(__ldg(p.cu_q + seq + 1)) - q0;
  if (q0 < 0) T = 0;
  T = max(static_cast<int64_t>(0), min(T, min(static_cast<int64_t>(kMaxDrafts), p.n_q - q0)));
  const int64_t whole = ctx >> shift;                              // pages that end before the context does
  const int pages = static_cast<int>(min(whole, p.table_stride));  // of them in the table
  const int32_t* table = p.table + static_cast<int64_t>(seq) * p.table_stride;
  // this block's pages [i0, i1)
  const int per = (pages + C - 1) / C, i0 = min(me * per, pages), i1 = min(i0 + per, pages);
  auto page_at = [&](int i) {
    const int page = i < i1 ? __ldg(table + i) : -1;
    return page < p.cache.n_pages ? page : -1;
  };
  // 32 pages of a warp: lane l has the number and scale of page l, and of page 8 g
  // + l / 4 the units l % 4, l % 4 + 4, ..
  struct Pages {
    int page;
    float scale;
    int4 c[4][kUnits];
  } now;
  auto fetch = [&](int page, Pages& x) {
    x.page = page;
    x.scale = page >= 0 ? __ldg(p.scales + static_cast<int64_t>(page) * H + head) : 0.f;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int pg = __shfl_sync(full, page, 8 * g + lane / kLanes);
      const int4* from = reinterpret_cast<const int4*>(p.codes + (static_cast<int64_t>(pg) * H + head) * 2 * D) + lane % kLanes;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) x.c[g][u] = pg >= 0 ? __ldg(from + u * kLanes) : make_int4(0, 0, 0, 0);
    }
  };
  // the first ones are on their way while the queries' codes are worked out
  const int first = i0 + tid;
  fetch(page_at(first), now);
  int ahead = page_at(first + kThreads);

  // ---- the queries' codes
  bool bad = false;
  {
    // exact sums: an fp16 value is a whole number of 2^-24
    const int d = tid % D;
    long long up = 0, down = 0;
    const int rows = static_cast<int>(T) * G;
    for (int r = tid / D; r < rows; r += kParts) {
      const int t = r / G, h = head * G + r - t * G;
      const float x = __half2float(static_cast<const __half*>(p.q.ptr)[(q0 + t) * p.q.token_stride + h * p.q.head_stride + d]);
      bad |= !(fabsf(x) < INFINITY);
      const long long n = static_cast<long long>(x * 16777216.f);
      if (n > 0) up += n;
      else down += n;
    }
    s_sum[tid / D][0][d] = up;
    s_sum[tid / D][1][d] = down;
  }
  bad = __syncthreads_or(bad);
  float wq = 0.f;
  if (tid < 2 * D && !bad) {
    long long n = 0;
#pragma unroll
    for (int k = 0; k < kParts; ++k) n += (&s_sum[k][0][0])[tid];
    wq = __ll2float_rn(n) * 0x1p-24f;
  }
  const uint32_t top = __reduce_max_sync(full, __float_as_uint(fabsf(wq)));
  if (lane == 0) s_hi[warp] = top;
  __syncthreads();
  if (tid < 2 * D) {
    const uint32_t m = __reduce_max_sync(full, lane < 2 * D / 32 ? s_hi[lane] : 0);
    s_q[tid] = code_of(wq, __fdiv_rn(__uint_as_float(m), 127.f));
  }
  __syncthreads();

  // ---- scores
  wait_for_cluster();
  uint32_t* keys = cluster.map_shared_rank(s_key, 0);
  int4 qc[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) qc[u] = reinterpret_cast<const int4*>(s_q)[u * kLanes + lane % kLanes];
  for (int k = first; k - lane < i1; k += kThreads) {
    int dot = 0;  // of this lane's page
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      int sum = 0;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        sum = __dp4a(now.c[g][u].x, qc[u].x, sum);
        sum = __dp4a(now.c[g][u].y, qc[u].y, sum);
        sum = __dp4a(now.c[g][u].z, qc[u].z, sum);
        sum = __dp4a(now.c[g][u].w, qc[u].w, sum);
      }
      sum += __shfl_xor_sync(full, sum, 1);
      sum += __shfl_xor_sync(full, sum, 2);
      const int got = __shfl_sync(full, sum, (lane & 7) * kLanes);
      if (lane / 8 == g) dot = got;
    }
    if (k < i1) keys[k] = now.page >= 0 ? score_key(__fmul_rn(static_cast<float>(dot), now.scale)) : 0;
    if (k - lane + kThreads < i1) {
      fetch(ahead, now);
      ahead = page_at(k + 2 * kThreads);
    }
  }
  cluster.sync();
  if (me != 0) return;

  // ---- the first block: candidates, and the range of their keys
  auto every = [&](auto use) {  // use(key) of this thread's keys; 0 for those behind the end
    for (int k0 = tid; k0 - tid < pages; k0 += kKeys * kThreads) {
      uint32_t key[kKeys];
#pragma unroll
      for (int j = 0; j < kKeys; ++j) key[j] = k0 + j * kThreads < pages ? s_key[k0 + j * kThreads] : 0;
#pragma unroll
      for (int j = 0; j < kKeys; ++j) use(key[j]);
    }
  };
  uint32_t lo = 0xffffffffu, hi = 0;
  int n = 0;
  every([&](uint32_t key) {
    if (key) lo = min(lo, key), hi = max(hi, key), ++n;
  });
  lo = __reduce_min_sync(full, lo), hi = __reduce_max_sync(full, hi), n = __reduce_add_sync(full, n);
  if (lane == 0) s_lo[warp] = lo, s_hi[warp] = hi, s_n[warp] = n;
  __syncthreads();
  lo = __reduce_min_sync(full, s_lo[lane % kWarps]), hi = __reduce_max_sync(full, s_hi[lane % kWarps]);
  const int all = __reduce_add_sync(full, lane < kWarps ? s_n[lane] : 0), want = min(all, p.n_select);

  // ---- what is taken: keys above `limit`, and `at_limit` of those at it
  uint32_t limit = 0;
  int at_limit = 0;
  if (want == 0) {
    limit = 0xffffffffu;
  } else if (all > want) {
    uint32_t base = lo;        // the range [base, base + (kBins << low)) holds the want-th
    int low = max(0, 32 - __clz(hi - lo) - 11), rest = want;
    uint32_t span = hi - lo;   // the last key of the range, from base
    for (;;) {
      for (int b = tid; b < kBins; b += kThreads) s_hist[b] = 0;
      __syncthreads();
      every([&](uint32_t key) {
        const uint32_t from = key - base;
        if (key >= base && from <= span && key) atomicAdd(&s_hist[from >> low], 1);
      });
      __syncthreads();
      // a thread for four neighbouring bins, the highest first
      const int b0 = kBins - 4 - 4 * tid;
      const int4 h = *reinterpret_cast<const int4*>(s_hist + b0);
      const int sum = h.x + h.y + h.z + h.w;
      int upto = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(full, upto, o);
        if (lane >= o) upto += y;
      }
      if (lane == 31) s_eq[warp] = upto;
      __syncthreads();
      upto += __reduce_add_sync(full, lane < warp ? s_eq[lane] : 0);
      const int above = upto - sum;  // keys in higher bins
      if (above < rest && upto >= rest) {
        int b = b0 + 3, left = rest - above, count = h.w;
        if (left > h.w) {
          left -= h.w, b = b0 + 2, count = h.z;
          if (left > h.z) {
            left -= h.z, b = b0 + 1, count = h.y;
            if (left > h.y) left -= h.y, b = b0, count = h.x;
          }
        }
        s_digit = b, s_rest = left, s_count = count;
      }
      __syncthreads();
      base += static_cast<uint32_t>(s_digit) << low;
      rest = s_rest;
      if (rest == s_count) {  // the bin is taken whole
        limit = base - 1;
        break;
      }
      if (low == 0) {
        limit = base, at_limit = rest;
        break;
      }
      span = (1u << low) - 1;
      low = max(0, low - 11);
    }
  }

  // ---- the pages, in order: a warp for a run of keys
  constexpr int kAt = kKeys;
  const int run = (pages + kThreads - 1) / kThreads * 32, r0 = warp * run + lane, r1 = min(warp * run + run, pages);
  int above = 0, equal = 0;
  for (int k0 = r0; k0 - lane < r1; k0 += kAt * 32) {
#pragma unroll
    for (int j = 0; j < kAt; ++j) {
      const int k = k0 + 32 * j;
      const uint32_t key = k < r1 ? s_key[k] : 0;
      above += key > limit;
      equal += k < r1 && key == limit;
    }
  }
  above = __reduce_add_sync(full, above), equal = __reduce_add_sync(full, equal);
  __syncthreads();
  if (lane == 0) s_n[warp] = above, s_eq[warp] = equal;
  __syncthreads();
  // keys at the limit that lower warps have, and pages that they write
  int before = __reduce_add_sync(full, lane < warp ? s_eq[lane] : 0);
  int to = __reduce_add_sync(full, lane < warp ? s_n[lane] : 0) + min(before, at_limit);
  int32_t* out = p.out + static_cast<int64_t>(item) * p.width;
  const unsigned lower = (1u << lane) - 1;
  if (above + equal > 0) {
    for (int k0 = r0; k0 - lane < r1; k0 += kAt * 32) {
      uint32_t key[kAt];
      int32_t page[kAt];
#pragma unroll
      for (int j = 0; j < kAt; ++j) {
        const int k = k0 + 32 * j;
        key[j] = k < r1 ? s_key[k] : 0;
        page[j] = k < r1 && key[j] >= limit ? __ldg(table + k) : -1;
      }
#pragma unroll
      for (int j = 0; j < kAt; ++j) {
        const bool in = k0 + 32 * j < r1;
        const unsigned eqs = __ballot_sync(full, in && key[j] == limit);
        const bool take = in && (key[j] > limit || (key[j] == limit && before + __popc(eqs & lower) < at_limit));
        const unsigned takes = __ballot_sync(full, take);
        const int at = to + __popc(takes & lower);
        if (take && at < want) out[at] = page[j];
        to += __popc(takes);
        before += __popc(eqs);
      }
    }
  }
  // ---- the tail: the pages from the last whole one on
  for (int c = want + tid; c < p.width; c += kThreads) {
    const int64_t e = whole + c - want;
    out[c] = c < want + p.tail && e < p.table_stride ? __ldg(table + e) : -1;
  }
  if (head == 0 && tid == 0) p.out_lens[seq] = (want << shift) + (ctx & (p.cache.page_tokens - 1));
}

template <typename K>
cudaError_t launch_cluster(K* kernel, int cluster, unsigned grid, int smem, const SelectParams& p, cudaStream_t s) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(cluster);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D>
cudaError_t launch_select_of(const SelectParams& p, int cluster, int dev, int smem, cudaStream_t s) {
  static std::atomic<uint64_t> set;
  const cudaError_t e = allow_shared_memory(set, dev, select_kernel<D>, kMaxKeys * 4);
  if (e != cudaSuccess) return e;
  return launch_cluster(select_kernel<D>, cluster, static_cast<unsigned>(p.n_seqs * p.cache.kv_heads * cluster), smem, p, s);
}

}  // namespace

int64_t select_most_pages() { return kMaxKeys; }

cudaError_t launch_summary(const SummaryParams& p, cudaStream_t s) {
  int dev = 0, sms = 0;
  const cudaError_t found = current_device(&dev, &sms);
  if (found != cudaSuccess) return found;
  const int64_t items = p.n * p.cache.kv_heads;
  // Few heads of pages: a block each, for its latency (12 pages of 64 tokens, 8
  // heads, Q4_0: 3.6 us, 6.1 with a warp each).  Many: a warp each (250 pages of 16
  // tokens, 32 heads, fp16: 13.8 us, 22.7 with a block each).
  const bool few = items <= 4 * static_cast<int64_t>(sms);
  const int64_t grid = few ? items : (items + kSummaryThreads / 32 - 1) / (kSummaryThreads / 32);
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  auto go = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(grid), kSummaryThreads, 0, s>>>(p);
    return cudaGetLastError();
  };
  auto by_dim = [&](auto fmt) {
    constexpr int F = decltype(fmt)::value;
    if (few) return p.cache.head_dim == 64 ? go(summary_kernel<F, 64, 4>) : go(summary_kernel<F, 128, 4>);
    return p.cache.head_dim == 64 ? go(summary_kernel<F, 64, 1>) : go(summary_kernel<F, 128, 1>);
  };
  switch (p.cache.format) {
    case QGEMV_KV_F16: return by_dim(std::integral_constant<int, QGEMV_KV_F16>());
    case QGEMV_KV_INT8: return by_dim(std::integral_constant<int, QGEMV_KV_INT8>());
    default: return by_dim(std::integral_constant<int, QGEMV_KV_Q4_0>());
  }
}

cudaError_t launch_select(const SelectParams& p, cudaStream_t s) {
  int dev = 0, sms = 0;
  const cudaError_t found = current_device(&dev, &sms);
  if (found != cudaSuccess) return found;
  // Blocks of a cluster: while each has 256 pages at least, and there is an SM for
  // each (us with 1, 2, 4 and 8 of them; 8 heads of one sequence of 512 pages: 10.1,
  // 9.0, 9.0, 8.9; of 8187: 30.8, 20.6, 15.4, 12.4; 32 heads of 1000: 11.8, 10.2,
  // 9.2, 14.3; 12 sequences of 8 heads of 900: 12.7, 18.4, 20.3, 32.2).  The host knows
  // the table's width and not the contexts' lengths: a table wider than its contexts
  // takes the blocks and the shared memory of its width.
  const int64_t heads = static_cast<int64_t>(p.n_seqs) * p.cache.kv_heads;
  int cluster = 1;
  while (cluster < kMaxCluster && p.table_stride > 256 * cluster && heads * cluster * 2 <= sms) cluster *= 2;
  if (heads * cluster > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const int smem = static_cast<int>(std::max<int64_t>(4 * p.table_stride, 16));
  return p.cache.head_dim == 64 ? launch_select_of<64>(p, cluster, dev, smem, s) : launch_select_of<128>(p, cluster, dev, smem, s);
}

}  // namespace qgemv
