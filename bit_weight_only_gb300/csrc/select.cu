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
// of a sequence: each scores a run of pages into its shared memory, the
// blocks' histograms of the scores' bits, read from one another's shared
// memory, give the n_select-th score, and every block writes its own pages in
// order.  One launch, nothing kept in global memory.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "kv_codes.cuh"
#include "per_device.h"
#include "select.h"

namespace cg = cooperative_groups;

namespace qgemv {
namespace {

// The INT8 codes of eight values with the scale max / 127 of a whole vector
// (IEEE divisions: the codes are decided in fp32).
__device__ __forceinline__ uint2 codes_of(const float (&x)[8], float a) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = fminf(fmaxf(rintf(__fdiv_rn(x[i], a)), -127.f), 127.f);
    const int c = a > 0.f ? static_cast<int>(q) : 0;
    w[i >> 2] |= (static_cast<uint32_t>(c) & 0xffu) << (8 * (i & 3));
  }
  return make_uint2(w[0], w[1]);
}

constexpr int kSummaryThreads = 256;

// A warp for a head of a page.  Keys with an infinity or NaN leave codes of 0
// and a scale of NaN: such a page comes before all others.
template <int FMT, int D>
__global__ void __launch_bounds__(kSummaryThreads) summary_kernel(const SummaryParams p) {
  constexpr int kLanes = D / 8, kAt = 32 / kLanes;  // kAt tokens at a time
  constexpr int kAhead = 4;
  const unsigned full = 0xffffffffu;
  const int lane = threadIdx.x & 31, H = p.cache.kv_heads;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * kSummaryThreads + threadIdx.x) >> 5;
  const int64_t i = div_small(w, H);
  if (i >= p.n) return;
  const int head = static_cast<int>(w - i * H);
  const int64_t page = __ldg(p.pages + i);
  if (page < 0 || page >= p.cache.n_pages) return;
  const int d0 = (lane % kLanes) * 8;
  float hi[8], lo[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) hi[e] = -INFINITY, lo[e] = INFINITY;
  bool bad = false;
  for (int t0 = 0; t0 < p.cache.page_tokens; t0 += kAt * kAhead) {
    Eight<FMT, D> x[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int t = t0 + k * kAt + lane / kLanes;
      x[k].load(kv_block<FMT, D>(p.cache, page, head, t / kKvBlockTokens), false, t % kKvBlockTokens, d0);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      float v[8];
      x[k].values(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        bad |= !(fabsf(v[e]) < INFINITY);
        hi[e] = fmaxf(hi[e], v[e]);
        lo[e] = fminf(lo[e], v[e]);
      }
    }
  }
#pragma unroll
  for (int o = kLanes; o < 32; o <<= 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      hi[e] = fmaxf(hi[e], __shfl_xor_sync(full, hi[e], o));
      lo[e] = fminf(lo[e], __shfl_xor_sync(full, lo[e], o));
    }
  }
  bad = __any_sync(full, bad);
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fmaxf(fabsf(hi[e]), fabsf(lo[e])));
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(full, m, o));
  const float a = bad ? __int_as_float(0x7fffffff) : __fdiv_rn(m, 127.f);
  const int64_t row = page * H + head;
  // the lanes of the first token write hi, those of the next one lo
  const int part = lane / kLanes;
  if (part < 2) {
    const uint2 c = bad ? make_uint2(0, 0) : part == 0 ? codes_of(hi, a) : codes_of(lo, a);
    *reinterpret_cast<uint2*>(p.codes + row * 2 * D + part * D + d0) = c;
  }
  if (lane == 0) p.scales[row] = a;
}

constexpr int kThreads = 512;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kMaxKeys = 48 * 1024;  // scores of a block

// Order of scores as unsigned numbers above 0 (no page); NaN before all.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct __align__(16) SelectShared {
  int hist[kBins];
  int warp[kThreads / 32];
  int counts[4];  // of this block: candidates; above the limit, at it
  int digit, rest;
  uint32_t amax;
  int bad;
};

template <int D>
__global__ void __launch_bounds__(kThreads) select_kernel(const SelectParams p) {
  constexpr int kLanes = 4;                    // lanes of a page
  constexpr int kUnits = 2 * D / 16 / kLanes;  // 16-byte units of a lane
  __shared__ SelectShared s;
  __shared__ long long s_sum[2][D];
  __shared__ __align__(16) int8_t s_q[2 * D];
  extern __shared__ uint32_t s_key[];
  cg::cluster_group cluster = cg::this_cluster();
  const unsigned full = 0xffffffffu;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = static_cast<int>(cluster.num_blocks()), me = static_cast<int>(cluster.block_rank());
  const int item = blockIdx.x / C, H = p.cache.kv_heads;
  const int seq = item / H, head = item - seq * H, G = p.q_heads / H;
  const int shift = 31 - __clz(p.cache.page_tokens);
  const int ctx = max(0, __ldg(p.ctx_lens + seq));
  const int64_t whole = ctx >> shift;                              // pages that end before the context does
  const int pages = static_cast<int>(min(whole, p.table_stride));  // of them in the table
  const int32_t* table = p.table + static_cast<int64_t>(seq) * p.table_stride;

  // ---- the queries' codes
  int64_t q0 = __ldg(p.cu_q + seq);
  int64_t T = static_cast<int64_t>(__ldg(p.cu_q + seq + 1)) - q0;
  if (q0 < 0) T = 0;
  T = max(static_cast<int64_t>(0), min(T, min(static_cast<int64_t>(kMaxDrafts), p.n_q - q0)));
  if (tid < 2 * D) (&s_sum[0][0])[tid] = 0;
  if (tid == 0) s.amax = 0, s.bad = 0;
  __syncthreads();
  {
    // exact sums: an fp16 value is a whole number of 2^-24
    const int d = tid % D;
    long long up = 0, down = 0;
    bool bad = false;
    const int rows = static_cast<int>(T) * G;
    for (int r = tid / D; r < rows; r += kThreads / D) {
      const int t = r / G, h = head * G + r - t * G;
      const float x = __half2float(static_cast<const __half*>(p.q.ptr)[(q0 + t) * p.q.token_stride + h * p.q.head_stride + d]);
      bad |= !(fabsf(x) < INFINITY);
      const long long n = static_cast<long long>(x * 16777216.f);
      if (n > 0) up += n;
      else down += n;
    }
    if (up) atomicAdd(reinterpret_cast<unsigned long long*>(&s_sum[0][d]), static_cast<unsigned long long>(up));
    if (down) atomicAdd(reinterpret_cast<unsigned long long*>(&s_sum[1][d]), static_cast<unsigned long long>(down));
    if (bad) s.bad = 1;
  }
  __syncthreads();
  float wq = 0.f;
  if (tid < 2 * D) {
    wq = s.bad ? 0.f : __ll2float_rn((&s_sum[0][0])[tid]) * 0x1p-24f;
    atomicMax(&s.amax, __float_as_uint(fabsf(wq)));
  }
  __syncthreads();
  if (tid < 2 * D) {
    const float a = __fdiv_rn(__uint_as_float(s.amax), 127.f);
    const float c = fminf(fmaxf(rintf(__fdiv_rn(wq, a)), -127.f), 127.f);
    s_q[tid] = static_cast<int8_t>(a > 0.f ? static_cast<int>(c) : 0);
  }
  __syncthreads();

  // ---- scores of this block's pages [i0, i1)
  const int per = (pages + C - 1) / C, i0 = min(me * per, pages), i1 = min(i0 + per, pages), n = i1 - i0;
  int4 qc[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) qc[u] = reinterpret_cast<const int4*>(s_q)[u * kLanes + lane % kLanes];
  int mine = 0;
  for (int k0 = warp * 32; k0 < n; k0 += kThreads) {  // 32 pages of a warp
    const int k = k0 + lane;
    int page = k < n ? __ldg(table + i0 + k) : -1;
    if (page >= p.cache.n_pages) page = -1;
    float scale = page >= 0 ? __ldg(p.scales + static_cast<int64_t>(page) * H + head) : 0.f;
    int dot = 0;  // of this lane's page
#pragma unroll
    for (int g = 0; g < 4; ++g) {  // eight pages at a time
      const int pg = __shfl_sync(full, page, 8 * g + lane / kLanes);
      int4 c[kUnits];
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
        c[u] = pg >= 0 ? __ldg(reinterpret_cast<const int4*>(p.codes + (static_cast<int64_t>(pg) * H + head) * 2 * D) + u * kLanes + lane % kLanes)
                       : make_int4(0, 0, 0, 0);
      int sum = 0;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        sum = __dp4a(c[u].x, qc[u].x, sum);
        sum = __dp4a(c[u].y, qc[u].y, sum);
        sum = __dp4a(c[u].z, qc[u].z, sum);
        sum = __dp4a(c[u].w, qc[u].w, sum);
      }
      sum += __shfl_xor_sync(full, sum, 1);
      sum += __shfl_xor_sync(full, sum, 2);
      const int got = __shfl_sync(full, sum, (lane & 7) * kLanes);
      if (lane / 8 == g) dot = got;
    }
    if (k < n) s_key[k] = page >= 0 ? score_key(__fmul_rn(static_cast<float>(dot), scale)) : 0;
    mine += k < n && page >= 0;
  }
  auto block_total = [&](int x) {  // to all threads
    x = __reduce_add_sync(full, x);
    __syncthreads();
    if (lane == 0) s.warp[warp] = x;
    __syncthreads();
    int t = lane < kThreads / 32 ? s.warp[lane] : 0;
    return __reduce_add_sync(full, t);
  };
  const int cand = block_total(mine);
  if (tid == 0) s.counts[0] = cand;
  cluster.sync();
  int all = 0;
  for (int r = 0; r < C; ++r) all += cluster.map_shared_rank(s.counts, r)[0];

  // ---- the limit: the n_select-th key, by 11, 11 and 10 bits from the top
  const int want = min(all, p.n_select);
  const bool choose = all > p.n_select;
  uint32_t limit = 0xffffffffu;  // (nothing is above it: for n_select = 0)
  int at_limit = 0;              // how many of those at it are taken
  if (choose && want > 0) {
    int rest = want;  // to take among the keys that agree with `limit` so far
    uint32_t seen = 0;
    for (int step = 0; step < 3; ++step) {
      const int low = step == 0 ? 21 : step == 1 ? 10 : 0, bits = step == 2 ? 10 : 11;
      const uint32_t mask = (1u << bits) - 1;
      cluster.sync();  // the others have read the last histogram
      for (int b = tid; b < kBins; b += kThreads) s.hist[b] = 0;
      __syncthreads();
      for (int k0 = warp * 32; k0 < n; k0 += kThreads) {
        const int k = k0 + lane;
        const uint32_t key = k < n ? s_key[k] : 0;
        const bool in = key && (step == 0 || (key >> (low + bits)) == (seen >> (low + bits)));
        const int bin = in ? static_cast<int>((key >> low) & mask) : -1;
        const unsigned same = __match_any_sync(full, bin);
        if (in && lane == __ffs(same) - 1) atomicAdd(&s.hist[bin], __popc(same));
      }
      cluster.sync();
      // a thread for four neighbouring bins, the highest first
      const int b0 = kBins - 4 - 4 * tid;
      int4 h = make_int4(0, 0, 0, 0);
      for (int r = 0; r < C; ++r) {
        const int4 o = *reinterpret_cast<const int4*>(cluster.map_shared_rank(s.hist, r) + b0);
        h.x += o.x, h.y += o.y, h.z += o.z, h.w += o.w;
      }
      const int sum = h.x + h.y + h.z + h.w;
      int upto = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(full, upto, o);
        if (lane >= o) upto += y;
      }
      __syncthreads();
      if (lane == 31) s.warp[warp] = upto;
      __syncthreads();
      for (int w = 0; w < warp; ++w) upto += s.warp[w];
      const int above = upto - sum;  // keys in higher bins
      if (above < rest && upto >= rest) {
        int b = b0 + 3, left = rest - above;
        if (left > h.w) {
          left -= h.w, b = b0 + 2;
          if (left > h.z) {
            left -= h.z, b = b0 + 1;
            if (left > h.y) left -= h.y, b = b0;
          }
        }
        s.digit = b, s.rest = left;
      }
      __syncthreads();
      seen |= static_cast<uint32_t>(s.digit) << low;
      rest = s.rest;
    }
    limit = seen;
    at_limit = rest;
  }

  // ---- the pages, in order: those above the limit, and the first at it
  int above = 0, equal = 0;
  for (int k = tid; k < n; k += kThreads) {
    const uint32_t key = s_key[k];
    above += choose ? key > limit : key != 0;
    equal += choose && key == limit;
  }
  above = block_total(above);
  equal = block_total(equal);
  if (tid == 0) s.counts[1] = above, s.counts[2] = equal;
  cluster.sync();
  int to = 0, before = 0;  // pages that lower blocks write; keys at the limit in them
  for (int r = 0; r < me; ++r) {
    const int* c = cluster.map_shared_rank(s.counts, r);
    to += c[1] + max(0, min(c[2], at_limit - before));
    before += c[2];
  }
  int32_t* out = p.out + static_cast<int64_t>(item) * p.width;
  for (int k0 = 0; k0 < n; k0 += kThreads) {
    const int k = k0 + tid;
    const uint32_t key = k < n ? s_key[k] : 0;
    const bool eq = choose && key == limit && key != 0;
    // the order among the keys at the limit, then among those taken
    const unsigned eqs = __ballot_sync(full, eq);
    __syncthreads();
    if (lane == 0) s.warp[warp] = __popc(eqs);
    __syncthreads();
    int eq_at = before + __popc(eqs & ((1u << lane) - 1)), eq_all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) eq_at += s.warp[w];
      eq_all += s.warp[w];
    }
    const bool take = choose ? key > limit || (eq && eq_at < at_limit) : key != 0;
    const unsigned takes = __ballot_sync(full, take);
    __syncthreads();
    if (lane == 0) s.warp[warp] = __popc(takes);
    __syncthreads();
    int at = to + __popc(takes & ((1u << lane) - 1)), all_taken = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) at += s.warp[w];
      all_taken += s.warp[w];
    }
    if (take && at < want) out[at] = __ldg(table + i0 + k);
    to += all_taken;
    before += eq_all;
  }
  // ---- the tail: the pages from the last whole one on
  if (me == 0) {
    for (int c = want + tid; c < p.width; c += kThreads) {
      const int64_t e = whole + c - want;
      out[c] = c < want + p.tail && e < p.table_stride ? __ldg(table + e) : -1;
    }
    if (head == 0 && tid == 0) p.out_lens[seq] = (want << shift) + (ctx & (p.cache.page_tokens - 1));
  }
  cluster.sync();  // shared memory is read by the others
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

int64_t select_most_pages() { return static_cast<int64_t>(kMaxCluster) * kMaxKeys; }

cudaError_t launch_summary(const SummaryParams& p, cudaStream_t s) {
  const int64_t grid = (p.n * p.cache.kv_heads + kSummaryThreads / 32 - 1) / (kSummaryThreads / 32);
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  auto go = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(grid), kSummaryThreads, 0, s>>>(p);
    return cudaGetLastError();
  };
  auto by_dim = [&](auto fmt) {
    constexpr int F = decltype(fmt)::value;
    return p.cache.head_dim == 64 ? go(summary_kernel<F, 64>) : go(summary_kernel<F, 128>);
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
  // Blocks of a cluster: while each has 256 pages at least, and the blocks are
  // no more than the SMs twice over; as many as the scores' room takes.
  const int64_t heads = static_cast<int64_t>(p.n_seqs) * p.cache.kv_heads;
  int cluster = 1;
  while (cluster < kMaxCluster && p.table_stride > 256 * cluster && heads * cluster * 2 <= 2 * sms) cluster *= 2;
  while (cluster < kMaxCluster && p.table_stride > static_cast<int64_t>(cluster) * kMaxKeys) cluster *= 2;
  if (heads * cluster > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const int64_t keys = (p.table_stride + cluster - 1) / cluster;
  const int smem = static_cast<int>(std::max<int64_t>(4 * keys, 16));
  return p.cache.head_dim == 64 ? launch_select_of<64>(p, cluster, dev, smem, s) : launch_select_of<128>(p, cluster, dev, smem, s);
}

}  // namespace qgemv
