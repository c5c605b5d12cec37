// tree_work.cuh -- how the attention of drafted tokens is split over thread
// blocks, shared by its kernels.
//
// The work is a list of units -- UNIT cached tokens for one tile of ROWS rows
// -- ordered (sequence, head, row tile, position).  Each thread block takes an
// equal run of it; a run's part of one row tile is a segment.  A row tile
// costs more than its units (Q, the start and end of the softmax): it counts
// as `extra` units more, which come first and stand for no tokens, so that
// blocks whose sequences are short get fewer of them.  A row tile that
// one block covers is stored by it; the parts of a shared one go to the
// block's two workspace slots (0: it continues what an earlier block began,
// 1: it begins), and the join kernel adds them in order.
#pragma once

#include "kv_layout.cuh"

namespace qgemv {

constexpr int kMaxBlocks = 320;  // thread blocks of a call, at most
constexpr int kSlotRows = 64;    // rows of a workspace slot, at most
__host__ __device__ constexpr int64_t slot_floats(int D) { return static_cast<int64_t>(kSlotRows) * (D + 2); }

// `whole`: short contexts are not split; block b takes the row tiles b, b +
// grid, .. of the list whole, and there is nothing to join.
struct TreeArgs {
  TreeParams p;
  int G, page_shift, min_units, extra, grid, whole;
};

struct SeqWork {
  int64_t units;  // of one row tile
  int tiles;      // row tiles of a head
  int ctx, T;
};

template <int ROWS, int UNIT>
__device__ __forceinline__ SeqWork seq_work(const TreeArgs& a, int b) {
  const TreeParams& p = a.p;
  SeqWork s;
  const int64_t q0 = __ldg(p.cu_q + b);
  int64_t T = __ldg(p.cu_q + b + 1) - q0;
  if (q0 < 0 || T < 0) T = 0;
  T = min(T, min(static_cast<int64_t>(kMaxDrafts), p.n_q - q0));
  s.T = static_cast<int>(max(T, static_cast<int64_t>(0)));
  s.ctx = max(0, __ldg(p.ctx_lens + b));
  const int64_t n = min(static_cast<int64_t>(s.ctx) + s.T, p.table_stride << a.page_shift);
  s.units = max(static_cast<int64_t>(1), (n + UNIT - 1) / UNIT);
  s.tiles = (s.T * a.G + ROWS - 1) / ROWS;
  return s;
}

__device__ __forceinline__ int64_t warp_total(int64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ int64_t run_quota(const TreeArgs& a, int64_t total) {
  return max(static_cast<int64_t>(a.min_units), div_small(total + a.grid - 1, a.grid));
}

// The page table of a head of a sequence.
__device__ __forceinline__ const int32_t* table_row(const TreeParams& p, int seq, int head) {
  return p.table + (p.table_heads == 1 ? seq : static_cast<int64_t>(seq) * p.table_heads + head) * p.table_stride;
}

// A block's part of one row tile.
struct Segment {
  int seq, head, tile, ctx, T;
  int64_t u0, u1, units;  // units [u0, u1) of the row tile's `units`
  bool shared;
};

// The segments of this block, one after the other (a whole warp calls it).
template <int ROWS, int UNIT>
struct Cursor {
  int64_t cur, end, base;
  int seq;

  __device__ Cursor(const TreeArgs& a) {
    const int lane = threadIdx.x & 31, H = a.p.cache.kv_heads;
    const unsigned full = 0xffffffffu;
    auto cost_of = [&](int b) -> int64_t {
      if (b >= a.p.n_seqs) return 0;
      const SeqWork s = seq_work<ROWS, UNIT>(a, b);
      return (a.whole ? 1 : s.units + a.extra) * s.tiles * H;
    };
    auto scan = [&](int64_t x) {  // inclusive
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(full, x, o);
        if (lane >= o) x += y;
      }
      return x;
    };
    const int64_t mine0 = cost_of(lane), sum0 = scan(mine0);  // the first 32 sequences
    int64_t rest = 0;
    for (int b = 32 + lane; b < a.p.n_seqs; b += 32) rest += cost_of(b);
    int64_t total = __shfl_sync(full, sum0, 31);
    if (a.p.n_seqs > 32) total += warp_total(rest);
    if (a.whole) {
      cur = blockIdx.x;
      end = total;
    } else {
      const int64_t quota = run_quota(a, total);
      cur = quota * blockIdx.x;
      end = min(cur + quota, total);
    }
    seq = 0;
    base = 0;
    if (cur >= end) return;
    int64_t mine = mine0, sum = sum0;
    for (int b0 = 0;; b0 += 32) {
      if (b0 > 0) {
        mine = cost_of(b0 + lane);
        sum = scan(mine);
      }
      const unsigned past = __ballot_sync(full, base + sum > cur);
      if (past) {
        const int k = __ffs(past) - 1;
        seq = b0 + k;
        base += __shfl_sync(full, sum - mine, k);
        return;
      }
      base += __shfl_sync(full, sum, 31);
    }
  }

  __device__ bool next(const TreeArgs& a, Segment& s) {
    const int H = a.p.cache.kv_heads;
    while (cur < end) {
      const SeqWork w = seq_work<ROWS, UNIT>(a, seq);
      const int64_t in_seq = cur - base, cost = a.whole ? 1 : w.units + a.extra, per_seq = cost * w.tiles * H;
      if (in_seq >= per_seq) {
        base += per_seq;
        ++seq;
        continue;
      }
      const int64_t item = div_small(in_seq, cost);
      if (a.whole) {
        cur += a.grid;
        s.u0 = 0;
        s.u1 = w.units;
      } else {
        const int64_t v0 = in_seq - item * cost, v1 = min(cost, v0 + (end - cur));
        cur += v1 - v0;
        s.u0 = max(static_cast<int64_t>(0), v0 - a.extra);
        s.u1 = v1 - a.extra;
        if (s.u1 <= s.u0) continue;
      }
      s.seq = seq;
      s.ctx = w.ctx;
      s.T = w.T;
      s.units = w.units;
      s.head = static_cast<int>(div_small(item, w.tiles));
      s.tile = static_cast<int>(item - static_cast<int64_t>(s.head) * w.tiles);
      s.shared = s.u0 > 0 || s.u1 < w.units;
      return true;
    }
    return false;
  }
};

__device__ __forceinline__ float* tree_slot(const TreeParams& p, int block, bool begins, int D) {
  return reinterpret_cast<float*>(p.ws + kWsHeaderBytes) + (2 * block + (begins ? 1 : 0)) * slot_floats(D);
}

cudaError_t launch_tree_wide(const TreeArgs& a, int dev, cudaStream_t s);

}  // namespace qgemv
