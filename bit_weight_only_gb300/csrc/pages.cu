// pages.cu -- pages of a cache given out, shared, returned, packed and copied
// (qgemv_pool_*, qgemv_kv_copy_pages).
//
// A pool is a count of rows for each page (0: free).  All of it is whole
// numbers: counts change by atomic additions, whose order does not matter, and
// free pages are given out lowest first in the rows' order, so a call's results
// depend on its inputs alone.  Nothing returns to the host.
//
// Bookkeeping reads tables and counts of a few hundred kB at most: a chain of
// latencies, of a launch and a scan, bounds it.  Free pages are found by one
// block in steps of 16384 counts, as many as are needed, the lowest first; the
// compacting scan, which needs all counts, is spread over blocks of 4096 each,
// whose sums every block adds up for itself (of few pages, a cluster does all of
// it).  Copies are bytes: a block takes
// 32 kB of a page with all of its loads in flight.
#include <cooperative_groups.h>

#include "pages.h"
#include "per_device.h"
#include "kv_layout.cuh"
#include "tc_common.cuh"

namespace cg = cooperative_groups;

namespace qgemv {
namespace {

constexpr int kGive = 1024;     // threads of the block that gives pages out
constexpr int kGivePer = 16;    // counts of a thread in a step
constexpr int kRowThreads = 256;

// Inclusive sum over the block's threads; `total` to all of them.
template <int THREADS>
__device__ int block_sum(int x, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = lane < THREADS / 32 ? s_warp[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  const int before = warp > 0 ? s_warp[warp - 1] : 0;
  total = s_warp[THREADS / 32 - 1];
  __syncthreads();
  return before + x;
}

// kPer neighbouring counts from refs[at]; past the end 1 (in use).
template <int kPer>
struct Counts {
  int v[kPer];
  __device__ void load(const int32_t* refs, int64_t n_pages, int64_t at) {
    if (at + kPer <= n_pages && (reinterpret_cast<uintptr_t>(refs) & 15) == 0) {
#pragma unroll
      for (int i = 0; i < kPer; i += 4) *reinterpret_cast<int4*>(v + i) = __ldcg(reinterpret_cast<const int4*>(refs + at + i));
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = at + i < n_pages ? __ldcg(refs + at + i) : 1;
    }
  }
};

// The lowest free pages, `want` of them where there are as many: give(rank,
// page), each by some thread of the block; `c` has the first step's counts.
// Returns how many there were.
template <int THREADS, typename F>
__device__ int free_pages(const int32_t* refs, int64_t n_pages, int want, Counts<kGivePer>& c, int* s_warp, F give) {
  int got = 0;
  for (int64_t p0 = 0; p0 < n_pages && got < want; p0 += THREADS * kGivePer) {
    const int64_t mine = p0 + static_cast<int64_t>(threadIdx.x) * kGivePer;
    if (p0 > 0) c.load(refs, n_pages, mine);
    int n = 0, total;
#pragma unroll
    for (int i = 0; i < kGivePer; ++i) n += c.v[i] <= 0;
    int rank = got + block_sum<THREADS>(n, s_warp, total) - n;
#pragma unroll
    for (int i = 0; i < kGivePer; ++i) {
      if (c.v[i] <= 0) {
        if (rank < want) give(rank, static_cast<int32_t>(mine + i));
        ++rank;
      }
    }
    got += total;
  }
  return min(got, want);
}

__device__ __forceinline__ int64_t pages_for(int64_t tokens, int page) { return tokens <= 0 ? 0 : (tokens + page - 1) / page; }

// ---- reserve: one block
__global__ void __launch_bounds__(kGive) reserve_kernel(const PoolParams p) {
  __shared__ int s_warp[32];
  extern __shared__ int s_upto[];  // pages that the sequences up to and with this one need
  const int n = static_cast<int>(p.n_seqs);
  Counts<kGivePer> counts;
  counts.load(p.refs, p.n_pages, static_cast<int64_t>(threadIdx.x) * kGivePer);
  auto range = [&](int b, int64_t& e0, int64_t& e1) {
    e0 = pages_for(p.from[b], p.page_tokens);
    e1 = min(pages_for(p.to[b], p.page_tokens), p.table_stride);
    if (e1 < e0) e1 = e0;
  };
  int64_t want = 0;
  for (int b0 = 0; b0 < n; b0 += kGive) {
    const int b = b0 + threadIdx.x;
    int64_t e0 = 0, e1 = 0;
    if (b < n) range(b, e0, e1);
    int total;
    const int mine = block_sum<kGive>(static_cast<int>(e1 - e0), s_warp, total);  // (a row has at most 2^20 entries)
    if (b < n) s_upto[b] = static_cast<int>(min(want + mine, static_cast<int64_t>(0x7fffffff)));
    want += total;
  }
  want = min(want, static_cast<int64_t>(0x7fffffff));
  __syncthreads();
  auto place = [&](int rank) -> int32_t* {  // the entry that gets the page of this rank
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_upto[mid] <= rank) lo = mid + 1;
      else hi = mid;
    }
    return p.table + lo * p.table_stride + pages_for(p.from[lo], p.page_tokens) + rank - (lo > 0 ? s_upto[lo - 1] : 0);
  };
  const int got = free_pages<kGive>(p.refs, p.n_pages, static_cast<int>(want), counts, s_warp, [&](int rank, int32_t page) {
    *place(rank) = page;
    p.refs[page] = 1;
  });
  for (int64_t r = got + static_cast<int64_t>(threadIdx.x); r < want; r += kGive) *place(static_cast<int>(r)) = -1;
  if (threadIdx.x == 0 && got < want) p.state[0] += static_cast<int>(want - got);
}

// ---- fork: a block for each old row (its pages' counts, its children's
// copies) and each new one (its entries); the last one to end gives the copies
// their pages.
constexpr int kForkThreads = 512;

__global__ void __launch_bounds__(kForkThreads) fork_kernel(const PoolParams p) {
  __shared__ int s_warp[32];
  __shared__ int s_kids, s_first;
  __shared__ bool s_last;
  extern __shared__ int2 s_rows[];  // (row, entry) of the rows that get a copy
  if (blockIdx.x < p.n_old) {
    const int64_t b = blockIdx.x;
    const int32_t* row = p.old_table + b * p.old_stride;
    // on their way while the children are counted
    const int len = max(p.from[b], 0), rest = len % p.page_tokens;
    const int32_t ahead = threadIdx.x < p.old_stride ? row[threadIdx.x] : -1;
    if (threadIdx.x == 0) s_kids = 0, s_first = 0x7fffffff;
    __syncthreads();
    for (int64_t r = threadIdx.x; r < p.n_seqs; r += kForkThreads)
      if (p.parents[r] == b) atomicAdd(&s_kids, 1), atomicMin(&s_first, static_cast<int>(r));
    __syncthreads();
    const int kids = s_kids;
    const int64_t used = pages_for(len, p.page_tokens), here = min(used, p.old_stride);
    for (int64_t e = threadIdx.x; e < here; e += kForkThreads) {
      const int32_t page = e < kForkThreads ? ahead : row[e];
      // the page that is filled in part stays with the first child alone
      const int change = (rest && e == used - 1 ? min(kids, 1) : kids) - 1;
      if (page >= 0 && page < p.n_pages && change) atomicAdd(p.refs + page, change);
    }
    const int32_t last = rest && used <= p.old_stride ? row[used - 1] : -1;
    const bool copies = last >= 0 && last < p.n_pages;
    for (int64_t r = threadIdx.x; r < p.n_seqs; r += kForkThreads) {
      if (p.parents[r] != b) continue;
      const bool copy = copies && r != s_first;
      p.src[r] = copy ? last : -1;
      p.dst[r] = copy ? static_cast<int32_t>(used - 1) : -1;  // its entry, for the block that gives the page
      p.tokens[r] = copy ? rest : 0;
    }
  } else {
    const int64_t r = blockIdx.x - p.n_old;
    const int64_t b = p.parents[r];
    const bool there = b >= 0 && b < p.n_old;
    if (!there && threadIdx.x == 0) p.src[r] = p.dst[r] = -1, p.tokens[r] = 0;
    const int64_t used = there ? min(pages_for(p.from[b], p.page_tokens), p.old_stride) : 0;
    for (int64_t e = threadIdx.x; e < p.table_stride; e += kForkThreads)
      p.table[r * p.table_stride + e] = e < used ? p.old_table[b * p.old_stride + e] : -1;
  }
  // ---- the last block; the count of arrivals is 0 again behind it
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicInc(reinterpret_cast<unsigned*>(p.state) + 1, gridDim.x - 1) == gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (!s_last) return;
  Counts<kGivePer> counts;
  counts.load(p.refs, p.n_pages, static_cast<int64_t>(threadIdx.x) * kGivePer);
  int want = 0;
  for (int64_t r0 = 0; r0 < p.n_seqs; r0 += kForkThreads) {
    const int64_t r = r0 + threadIdx.x;
    const int entry = r < p.n_seqs ? __ldcg(p.dst + r) : -1;
    int total;
    const int at = want + block_sum<kForkThreads>(entry >= 0, s_warp, total) - 1;
    if (entry >= 0) s_rows[at] = make_int2(static_cast<int>(r), entry);
    want += total;
  }
  __syncthreads();
  auto give = [&](int rank, int32_t page) {
    const int2 r = s_rows[rank];
    p.dst[r.x] = page;
    p.table[r.x * p.table_stride + r.y] = page;
    if (page >= 0) p.refs[page] = 1;
  };
  const int got = free_pages<kForkThreads>(p.refs, p.n_pages, want, counts, s_warp, give);
  for (int i = got + threadIdx.x; i < want; i += kForkThreads) give(i, -1);
  if (threadIdx.x == 0 && got < want) p.state[0] += want - got;
}

// ---- release: a block for each row
__global__ void __launch_bounds__(kRowThreads) release_kernel(const PoolParams p) {
  const int64_t b = blockIdx.x;
  const int64_t e0 = p.from ? pages_for(p.from[b], p.page_tokens) : 0;
  const int64_t e1 = min(pages_for(p.to[b], p.page_tokens), p.table_stride);
  for (int64_t e = e0 + threadIdx.x; e < e1; e += kRowThreads) {
    int32_t& page = p.table[b * p.table_stride + e];
    if (page >= 0 && page < p.n_pages) atomicSub(p.refs + page, 1);
    page = -1;
  }
}

// ---- compact
__device__ __forceinline__ int64_t pool_tiles(int64_t n_pages) { return (n_pages + kPoolTile - 1) / kPoolTile; }

constexpr int kTilePer = kPoolTile / kRowThreads;  // counts of a thread
constexpr int kFewTiles = 4, kFewBlocks = 8;
constexpr int64_t kFewEntries = 1 << 15;

// The moves: with U pages in use, the j-th one from number U on goes to the
// j-th free one below.  map[page] = j for a page that moves, else -1.  `used`: U;
// `upto`: pages in use before this thread's first one, page0, of which `on` has a
// bit each; `below`: pages in use below number U.
__device__ __forceinline__ void write_moves(const PoolParams& p, int64_t page0, uint32_t on, int upto, int used, int below) {
  int32_t* map = p.scratch + pool_tiles(p.n_pages);
#pragma unroll
  for (int i = 0; i < kTilePer; ++i) {
    const int64_t page = page0 + i;
    if (page >= p.n_pages) break;
    const bool here = on >> i & 1, moves = here && page >= used;
    const int64_t j = moves ? upto - below : page - upto;
    upto += here;
    map[page] = moves ? static_cast<int32_t>(j) : -1;
    if (j >= p.n_moves) continue;
    if (moves) p.src[j] = static_cast<int32_t>(page);
    else if (!here && page < used) p.dst[j] = static_cast<int32_t>(page);
  }
  // behind the moves: as many as there are pages in use from number `used` on
  for (int64_t j = used - below + static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x; j < p.n_moves; j += static_cast<int64_t>(gridDim.x) * kRowThreads)
    p.src[j] = p.dst[j] = -1;
}

__device__ __forceinline__ uint32_t in_use(const PoolParams& p, int64_t page0) {
  Counts<kTilePer> c;
  c.load(p.refs, p.n_pages, page0);
  uint32_t on = 0;
#pragma unroll
  for (int i = 0; i < kTilePer; ++i) on |= static_cast<uint32_t>(page0 + i < p.n_pages && c.v[i] > 0) << i;
  return on;
}
// Bits of the pages below number `used`.
__device__ __forceinline__ uint32_t bits_below(int64_t page0, int used) {
  const int64_t n = used - page0;
  return n <= 0 ? 0 : n >= kTilePer ? (1u << kTilePer) - 1 : (1u << n) - 1;
}

// Entries of the tables, kAt of a thread, `all` apart.
struct Entries {
  static constexpr int kAt = 4;
  int32_t page[kAt];
  __device__ void load(const PoolParams& p, int64_t i0, int64_t all) {
#pragma unroll
    for (int k = 0; k < kAt; ++k) page[k] = i0 + k * all < p.n_seqs * p.table_stride ? p.old_table[i0 + k * all] : -1;
  }
};

// Tables and counts follow the moves: part `at` of `all`, kAt entries and moves at
// a time, each step's reads together; `now` has the first entries.
__device__ __forceinline__ void follow_moves(const PoolParams& p, int64_t at, int64_t all, Entries& now) {
  const int32_t* map = p.scratch + pool_tiles(p.n_pages);
  const int64_t entries = p.n_seqs * p.table_stride, items = max(entries, p.n_moves);
  constexpr int kAt = Entries::kAt;
  for (int64_t i0 = at; i0 < items; i0 += kAt * all) {
    if (i0 != at) now.load(p, i0, all);
    int32_t j[kAt], from[kAt], to[kAt], refs[kAt];
#pragma unroll
    for (int k = 0; k < kAt; ++k) {
      const int64_t i = i0 + k * all;
      from[k] = i < p.n_moves ? p.src[i] : -1;
      to[k] = i < p.n_moves ? p.dst[i] : -1;
      j[k] = now.page[k] >= 0 && now.page[k] < p.n_pages ? map[now.page[k]] : -1;
    }
#pragma unroll
    for (int k = 0; k < kAt; ++k) {
      refs[k] = from[k] >= 0 ? p.refs[from[k]] : 0;
      if (j[k] >= 0) now.page[k] = p.dst[j[k]];
    }
#pragma unroll
    for (int k = 0; k < kAt; ++k) {
      if (i0 + k * all < entries) p.table[i0 + k * all] = now.page[k];
      if (from[k] >= 0) p.refs[to[k]] = refs[k], p.refs[from[k]] = 0;
    }
  }
}

// Of few pages every block of a cluster looks at all of them; the last part is
// the cluster's, too.
__global__ void __cluster_dims__(kFewBlocks) __launch_bounds__(kRowThreads) compact_few_kernel(const PoolParams p) {
  __shared__ int s_warp[32], s_tile[32];
  __shared__ unsigned short s_on[kFewTiles][kRowThreads];
  const int tiles = static_cast<int>(pool_tiles(p.n_pages)), me = blockIdx.x, lane = threadIdx.x & 31;
  Entries first;
  first.load(p, me * kRowThreads + threadIdx.x, kFewBlocks * kRowThreads);
  if (threadIdx.x < 32) s_tile[threadIdx.x] = 0;
  __syncthreads();
#pragma unroll 2
  for (int t = 0; t < tiles; ++t) {
    const uint32_t on = in_use(p, static_cast<int64_t>(t) * kPoolTile + threadIdx.x * kTilePer);
    s_on[t][threadIdx.x] = static_cast<unsigned short>(on);
    const int n = __reduce_add_sync(0xffffffffu, __popc(on));
    if (lane == 0) atomicAdd(&s_tile[t], n);
  }
  __syncthreads();
  const int used = __reduce_add_sync(0xffffffffu, s_tile[lane]), before = __reduce_add_sync(0xffffffffu, lane < me ? s_tile[lane] : 0);
  const int edge = used / kPoolTile;
  int below = edge < tiles ? __popc(s_on[edge][threadIdx.x] & bits_below(static_cast<int64_t>(edge) * kPoolTile + threadIdx.x * kTilePer, used)) : 0;
  block_sum<kRowThreads>(below, s_warp, below);
  below += __reduce_add_sync(0xffffffffu, lane < edge ? s_tile[lane] : 0);
  const uint32_t on = me < tiles ? s_on[me][threadIdx.x] : 0;
  int total;
  const int upto = before + block_sum<kRowThreads>(__popc(on), s_warp, total) - __popc(on);
  write_moves(p, static_cast<int64_t>(me) * kPoolTile + threadIdx.x * kTilePer, on, upto, used, below);
  cg::this_cluster().sync();
  follow_moves(p, me * kRowThreads + threadIdx.x, kFewBlocks * kRowThreads, first);
}

// Pages in use of a tile.
__global__ void __launch_bounds__(kRowThreads) compact_count_kernel(const PoolParams p) {
  __shared__ int s_warp[32];
  allow_next_kernel();
  int total;
  block_sum<kRowThreads>(__popc(in_use(p, static_cast<int64_t>(blockIdx.x) * kPoolTile + threadIdx.x * kTilePer)), s_warp, total);
  if (threadIdx.x == 0) p.scratch[blockIdx.x] = total;
}

__global__ void __launch_bounds__(kRowThreads) compact_moves_kernel(const PoolParams p) {
  __shared__ int s_warp[32];
  allow_next_kernel();
  const int64_t tiles = pool_tiles(p.n_pages), me = blockIdx.x, page0 = me * kPoolTile + threadIdx.x * kTilePer;
  const uint32_t on = in_use(p, page0);
  wait_for_last_kernel();
  // pages in use before this tile, and in all
  int before = 0, all = 0, used, below = 0, total;
  for (int64_t t = threadIdx.x; t < tiles; t += kRowThreads) {
    all += p.scratch[t];
    if (t < me) before += p.scratch[t];
  }
  block_sum<kRowThreads>(before, s_warp, before);
  block_sum<kRowThreads>(all, s_warp, used);
  const int64_t edge = used / kPoolTile;
  for (int64_t t = threadIdx.x; t < edge; t += kRowThreads) below += p.scratch[t];
  const int64_t edge0 = edge * kPoolTile + threadIdx.x * kTilePer;
  below += __popc(in_use(p, edge0) & bits_below(edge0, used));
  block_sum<kRowThreads>(below, s_warp, below);
  const int upto = before + block_sum<kRowThreads>(__popc(on), s_warp, total) - __popc(on);
  write_moves(p, page0, on, upto, used, below);
}

__global__ void __launch_bounds__(kRowThreads) compact_apply_kernel(const PoolParams p) {
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x, all = static_cast<int64_t>(gridDim.x) * kRowThreads;
  Entries first;
  first.load(p, at, all);  // (nothing before in this call writes them)
  wait_for_last_kernel();
  follow_moves(p, at, all, first);
}

// ---- copies: a block takes chunks of kCopyBytes of what is to be copied
constexpr int kCopyThreads = 256;
constexpr int kCopyUnits = 8;  // 16-byte units of a thread
constexpr int kCopyBytes = kCopyThreads * kCopyUnits * 16;
constexpr int kCopyBlocks = 4;    // on an SM
constexpr int kCopyWindow = 512;  // pairs that are looked at together

struct CopyPair {
  int from, to;
  uint32_t run;      // 16-byte units of each head: at most 2^13, of at most 2^10 heads
  uint64_t per_run;  // 2^40 / run, rounded up: u / run is u * per_run >> 40 for u below 2^23
};

__device__ __forceinline__ CopyPair copy_pair(const CopyPagesParams& p, int64_t i) {
  CopyPair c = {-1, -1, 0, 0};
  if (i >= p.n) return c;
  c.from = p.src[i], c.to = p.dst[i];
  // the blocks of the first tokens of each head
  const int blocks = p.tokens ? (min(max(p.tokens[i], 0), p.blocks * kKvBlockTokens) + kKvBlockTokens - 1) / kKvBlockTokens : p.blocks;
  if (c.from >= 0 && c.from < p.n_pages && c.to >= 0 && c.to < p.n_pages) c.run = static_cast<uint32_t>(blocks) * p.block_bytes / 16;
  if (c.run) c.per_run = (1ull << 40) / c.run + 1;
  return c;
}
__device__ __forceinline__ int64_t copy_chunks(const CopyPagesParams& p, const CopyPair& c) {
  return (static_cast<int64_t>(c.run) * p.heads + kCopyBytes / 16 - 1) / (kCopyBytes / 16);
}

__device__ __forceinline__ void copy_chunk(const CopyPagesParams& p, const CopyPair& c, int chunk) {
  const uint32_t gap = static_cast<uint32_t>(p.blocks) * p.block_bytes / 16 - c.run;  // units of a head that are not copied
  const uint32_t units = c.run * p.heads, u0 = chunk * (kCopyBytes / 16) + threadIdx.x;
  const uint4* s = reinterpret_cast<const uint4*>(p.pages + c.from * p.page_bytes);
  uint4* d = reinterpret_cast<uint4*>(p.pages + c.to * p.page_bytes);
  uint4 x[kCopyUnits];
  uint32_t at[kCopyUnits];
#pragma unroll
  for (int k = 0; k < kCopyUnits; ++k) {
    const uint32_t u = u0 + k * kCopyThreads;
    at[k] = u + static_cast<uint32_t>(u * c.per_run >> 40) * gap;
    if (u < units) x[k] = s[at[k]];
  }
#pragma unroll
  for (int k = 0; k < kCopyUnits; ++k)
    if (u0 + k * kCopyThreads < units) d[at[k]] = x[k];
}

// Every chunk of every pair in turn.
__global__ void __launch_bounds__(kCopyThreads, kCopyBlocks) copy_all_kernel(const CopyPagesParams p) {
  const int64_t chunks = (p.page_bytes + kCopyBytes - 1) / kCopyBytes, all = p.n * chunks;
  for (int64_t item = blockIdx.x; item < all; item += gridDim.x) {
    const int64_t i = div_small(item, chunks);
    const CopyPair c = copy_pair(p, i);
    if (c.run) copy_chunk(p, c, static_cast<int>(item - i * chunks));
  }
}

// Blocks take the chunks of the pairs that are to be copied in turn: those pairs
// are gathered first, kCopyWindow at a time, so that pairs without a page, or
// with few tokens, leave no block without work.
__global__ void __launch_bounds__(kCopyThreads, kCopyBlocks) copy_gathered_kernel(const CopyPagesParams p) {
  __shared__ CopyPair s_pair[kCopyWindow];
  __shared__ int64_t s_upto[kCopyWindow];  // chunks of the pairs up to and with this one
  __shared__ int s_warp[32];
  constexpr int kPer = kCopyWindow / kCopyThreads;
  int64_t done = 0;  // chunks of earlier windows
  for (int64_t w0 = 0; w0 < p.n; w0 += kCopyWindow) {
    CopyPair mine[kPer];
    int n = 0, pairs, total;
    int64_t chunks = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      mine[k] = copy_pair(p, w0 + threadIdx.x * kPer + k);
      if (mine[k].run) ++n, chunks += copy_chunks(p, mine[k]);
    }
    // (a page has at most 2^14 chunks)
    int at = block_sum<kCopyThreads>(n, s_warp, pairs) - n;
    int64_t upto = block_sum<kCopyThreads>(static_cast<int>(chunks), s_warp, total) - chunks;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (!mine[k].run) continue;
      upto += copy_chunks(p, mine[k]);
      s_pair[at] = mine[k], s_upto[at] = upto;
      ++at;
    }
    __syncthreads();
    // this block's: those with (done + index) % gridDim == blockIdx
    int64_t c = blockIdx.x - done % gridDim.x;
    if (c < 0) c += gridDim.x;
    for (; c < total; c += gridDim.x) {
      int lo = 0, hi = pairs - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s_upto[mid] <= c) lo = mid + 1;
        else hi = mid;
      }
      copy_chunk(p, s_pair[lo], static_cast<int>(c - (lo > 0 ? s_upto[lo - 1] : 0)));
    }
    done += total;
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_pool_reserve(const PoolParams& p, cudaStream_t s) {
  reserve_kernel<<<1, kGive, static_cast<unsigned>(p.n_seqs) * 4, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_pool_fork(const PoolParams& p, cudaStream_t s) {
  fork_kernel<<<static_cast<unsigned>(p.n_old + p.n_seqs), kForkThreads, static_cast<unsigned>(p.n_seqs) * 8, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_pool_release(const PoolParams& p, cudaStream_t s) {
  release_kernel<<<static_cast<unsigned>(p.n_seqs), kRowThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_pool_compact(const PoolParams& p, cudaStream_t s) {
  const unsigned tiles = static_cast<unsigned>((p.n_pages + kPoolTile - 1) / kPoolTile);
  const int64_t entries = p.n_seqs * p.table_stride;
  // Few pages and entries: all of it by a cluster of eight blocks, one launch (9001
  // pages, 16384 entries: 7.7 us on the device as with three kernels, a call 11.5
  // against 18.1; 200 pages, 4096 entries 4.6 against 6.8).  More: every tile has its
  // block (32768 pages: 8.1 us, 10.5 in a cluster), and tables have more than eight
  // (9001 pages, 262144 entries: 9.6 against 24.4).
  if (tiles <= kFewTiles && entries <= kFewEntries) {
    compact_few_kernel<<<kFewBlocks, kRowThreads, 0, s>>>(p);
    return cudaGetLastError();
  }
  compact_count_kernel<<<tiles, kRowThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_after(compact_moves_kernel, tiles, p, s, kRowThreads);
  if (e != cudaSuccess) return e;
  const int64_t items = entries > p.n_moves ? entries : p.n_moves;
  const int64_t blocks = (items + kRowThreads - 1) / kRowThreads;
  return launch_after(compact_apply_kernel, static_cast<unsigned>(blocks < 1 ? 1 : blocks < 1024 ? blocks : 1024), p, s, kRowThreads);
}

cudaError_t launch_copy_pages(const CopyPagesParams& p, cudaStream_t s) {
  int dev = 0, sms = 0;
  const cudaError_t found = current_device(&dev, &sms);
  if (found != cudaSuccess) return found;
  // Pages in part, as a fork has them, with pairs that are none between: gathered
  // (128 beams, 57 pages of 1 MB in part: 9.9 us against 12.4), but for chunks that
  // run all at once.  Whole pages, as a packing has them, one behind the other: as
  // they come (2200 of 9001 Q4_0 pages of 74 kB: 56 us, 5.8 TB/s read and written,
  // against 60).  Four blocks an SM, with 32 kB of loads each; of the second's 16 kB
  // chunks six blocks an SM take 58, a block for each 74.
  const int64_t items = p.n * ((p.page_bytes + kCopyBytes - 1) / kCopyBytes), most = kCopyBlocks * static_cast<int64_t>(sms);
  const unsigned grid = static_cast<unsigned>(items < most ? items : most);
  if (items <= most || !p.tokens) copy_all_kernel<<<grid, kCopyThreads, 0, s>>>(p);
  else copy_gathered_kernel<<<grid, kCopyThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace qgemv
