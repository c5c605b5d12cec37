// attn_prompt.cu -- causal attention over packed prompts with grouped heads
// (qgemv_attn_prompt), on the fifth-generation tensor cores.
//
//   S = Q K^T,  P = exp2(S * scale * log2 e - m),  O = P V,  out = O / sum P
//
// Rows: the queries of a sequence and the G query heads of a key/value head,
// row = token * G + head, so that short prompts fill tiles and every K and V
// tile serves all of the heads that share it.  A piece is two row tiles of
// floor(128 / G) tokens of one key/value head; a block walks the keys in tiles
// of 128 up to the last one that the rows see.
//
// One block per SM takes the pieces one after the other from a counter, those
// with the most keys first within a sequence.  Where there are too few pieces
// to fill the GPU evenly so, each block takes an equal run of the list of all
// pieces' key tiles instead; the unnormalised results of pieces that runs
// share go to the workspace, and a second kernel joins them in order.
// A block's warps (12) run through the
// pieces on their own, held together by mbarriers only, so that one piece's
// start overlaps the end of the one before:
//   0-7    two softmax warpgroups, one for each row tile, a thread for each row
//   8      takes the pieces; issues the TMA loads of Q (as soon as the last
//          product with the one before is done), K and V (two stages each)
//   9      the MMAs
//   10-11  mend V tiles that hold masked positions
// Tensor memory, 512 columns: S0 S1 (128 each; P, 16-bit, replaces the first
// half of S), O0 O1.
//   * QK of row tile i for key tile j + 1 follows PV of tile j in issue order,
//     so P may lie over S, and a softmax warpgroup that sees S of tile j knows
//     that its PV of tile j - 1 is done: it rescales O itself, and only when
//     a row's maximum has grown by more than 2^8 since the reference m was
//     taken (P stays below 2^8, in range of fp16).  While one warpgroup takes
//     its exponentials the tensor cores work on the other row tile.
//   * A row's statistics live in its thread in fp32; no shuffles.
//   * Masked scores are replaced by -inf.  V rows that some row of the piece
//     must not see cannot be masked so (0 * NaN): in key tiles with masked
//     positions the mending warps zero what lies past the sequence and every
//     infinity and NaN, and note the first position of each per column; the
//     epilogue gives it to the rows that see it.
// What bounds it: both operands of Q K^T come from shared memory, whose
// bandwidth the products take whole, and the softmax warps need nearly as long
// for their exponentials (heads of 64: longer).  fp16, 64 heads of 128 over 8:
// one prompt of 16384 tokens 2.83 ms, 1553 TFLOP/s (0.83 of the library's dense
// bf16 product); one of 8192 0.73 ms (0.81); four packed ones of up to 4000,
// bf16, 0.29 ms (0.75).
//
// Every wait is bounded; on a timeout the block records the error, waits for
// its own copies and MMAs, frees tensor memory and returns.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kv_layout.cuh"
#include "per_device.h"
#include "tc_common.cuh"

namespace qgemv {
namespace {

constexpr int kThreads = 384;  // 12 warps
constexpr int kRowsPerBlock = 256;  // of a piece: two tiles of 128
constexpr int kKeys = 128;         // keys of a tile
constexpr int kChunk = 128 * 128;  // bytes of 128 rows of 64 values
constexpr int kErrPrompt = 16;
constexpr float kLazy = 8.f;  // log2 of the growth that makes O be rescaled

// Notes of infinite and NaN values: a copy for each of the two mending warps,
// which clears it before it uses it, of three pieces in turn.
constexpr int kNotes = 3;
constexpr int kItems = 4;  // ring of pieces

// Runs: a piece counts as this many key tiles more (its start and end), which
// come first; a run is that long at least.
constexpr int kStartTiles = 3;
constexpr int kMinRun = 4 + kStartTiles;
constexpr int kMaxPieces = 1024;  // of a call whose blocks take runs
constexpr double kJoinTiles = 10;  // what the second kernel takes, in key tiles

// The workspace of runs: two slots a block (0: it goes on with a piece, 1: it
// begins one that others go on with), each O [256][D], then m and l [256][2];
// then the first and the last block of each piece.
constexpr int kMaxBlocks = 152, kPartSlots = 2 * kMaxBlocks;
__host__ __device__ constexpr int64_t part_floats(int D) { return static_cast<int64_t>(kRowsPerBlock) * (D + 2); }
__device__ __forceinline__ float* part_slot(const PromptParams& p, int id, int D) {
  return reinterpret_cast<float*>(p.ws + kWsHeaderBytes) + id * part_floats(D);
}
__device__ __forceinline__ int* piece_blocks(const PromptParams& p, int piece, int D) {
  return reinterpret_cast<int*>(part_slot(p, kPartSlots, D)) + 2 * piece;
}

struct PromptArgs {
  PromptParams p;
  int G, tokens, n_slots;  // tokens of a row tile
};

// Barriers: full / empty pairs of the rings.  kBVf: a V tile has landed; kBFix:
// it is mended (or need not be).
enum { kBQ = 0, kBQe = 2, kBKf = 4, kBKe = 6, kBVf = 8, kBVe = 10, kBFix = 12, kBS = 14, kBP = 16, kBO = 18, kBNf = 20,
       kBNe = 23, kBIf = 26, kBIe = 30, kBDone = 34, kNBars = 35 };

// A piece: two row tiles of a sequence and head, and the key tiles t0 .. of
// them that this block takes.
struct Piece {
  int64_t q0, k0;      // first query and key of the sequence
  int tok0, nq;        // first token of the piece, tokens of the sequence
  int off, nk;         // query i sees the keys j <= i + off; keys
  int head;            // key/value head; -1: no more pieces
  int part;            // workspace slot of the results, -1: they are the piece's
  int all[2];          // key tiles that each row tile sees
  int t0, n[2], n_max; // key tiles: of each row tile, and the more of the two
  int first_masked;    // of those, the first with positions that some row of the piece does not see
  int mask_from;       // the first such position

  // keys that a token sees: 0 .. sees - 1
  __device__ int sees(int token) const { return max(0, min(nk, token + off + 1)); }

  __device__ int tiles() const { return max(all[0], all[1]); }

  // Pieces are numbered by slots of tokens, the last first, and heads within.
  // False: a slot without tokens.
  __device__ bool locate(const PromptArgs& a, int slot_from_last) {
    const PromptParams& p = a.p;
    const int step = 2 * a.tokens, slot = a.n_slots - 1 - slot_from_last;
    // The sequence of this slot: its pieces start at slot floor(cu / step) + b,
    // which leaves each sequence at least as many slots as it has pieces.
    int lo = 0, hi = p.n_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(p.cu_q + mid) / step + mid <= slot) lo = mid;
      else hi = mid - 1;
    }
    q0 = max(__ldg(p.cu_q + lo), 0);
    nq = static_cast<int>(min(static_cast<int64_t>(__ldg(p.cu_q + lo + 1)), p.n_q) - q0);
    const int64_t first = (slot - (q0 / step + lo)) * step;
    if (first < 0 || first >= nq) return false;
    tok0 = static_cast<int>(first);
    k0 = min(static_cast<int64_t>(max(__ldg(p.cu_k + lo), 0)), p.n_k);
    nk = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(__ldg(p.cu_k + lo + 1)), p.n_k) - k0));
    off = nk - nq;
    const int tok1 = tok0 + a.tokens;
    all[0] = (sees(min(tok1, nq) - 1) + kKeys - 1) / kKeys;
    all[1] = tok1 >= nq ? 0 : (sees(min(tok1 + a.tokens, nq) - 1) + kKeys - 1) / kKeys;
    mask_from = sees(tok0);
    return true;
  }

  __device__ void take(int of_head, int from, int to, int to_part) {
    head = of_head;
    part = to_part;
    t0 = from;
    n[0] = max(0, min(to, all[0]) - from);
    n[1] = max(0, min(to, all[1]) - from);
    n_max = max(n[0], n[1]);
    first_masked = max(0, mask_from / kKeys - from);
  }
};
static_assert(sizeof(Piece) * kItems <= 512, "room for the pieces");

// A block's run (a whole warp calls it).  The costs of 32 slots at a time are
// in the lanes.
struct Run {
  int64_t cur = 0, end = 0, base = 0;  // base: what comes before those slots
  int64_t cost = 0, sum = 0;           // of the lane's slot, all heads; sums up to it
  int s0 = 0;

  __device__ void costs(const PromptArgs& a) {
    const int lane = threadIdx.x & 31;
    Piece x;
    cost = s0 + lane < a.n_slots && x.locate(a, s0 + lane) ? static_cast<int64_t>(x.tiles() + kStartTiles) * a.p.kv_heads : 0;
    sum = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
  }

  __device__ void start(const PromptArgs& a) {
    int64_t total = 0;
    for (s0 = (a.n_slots - 1) / 32 * 32; s0 >= 0; s0 -= 32) {
      costs(a);
      total += __shfl_sync(0xffffffffu, sum, 31);
    }
    s0 = 0;  // the slots whose costs are there
    const int64_t quota = max(static_cast<int64_t>(kMinRun), div_small(total + gridDim.x - 1, gridDim.x));
    cur = quota * blockIdx.x;
    end = min(cur + quota, total);
  }

  // The next piece; false: the run ends.
  __device__ bool next(const PromptArgs& a, Piece& pc, int D) {
    const int lane = threadIdx.x & 31;
    while (cur < end) {
      const unsigned past = __ballot_sync(0xffffffffu, base + sum > cur);
      if (!past) {
        base += __shfl_sync(0xffffffffu, sum, 31);
        s0 += 32;
        costs(a);
        continue;
      }
      const int k = __ffs(past) - 1;
      const int64_t in = cur - base - __shfl_sync(0xffffffffu, sum - cost, k);
      pc.locate(a, s0 + k);
      const int64_t each = pc.tiles() + kStartTiles;
      const int head = static_cast<int>(div_small(in, each));
      const int64_t v0 = in - head * each, v1 = min(each, v0 + end - cur);
      cur += v1 - v0;
      const int from = static_cast<int>(max(static_cast<int64_t>(0), v0 - kStartTiles)), to = static_cast<int>(v1) - kStartTiles;
      // its first blocks may have nothing but a share of its start
      if (to <= from && !(pc.tiles() == 0 && v0 == 0)) continue;
      const bool first = from == 0, last = to >= pc.tiles() || pc.tiles() == 0;
      pc.take(head, from, max(to, 0), first && last ? -1 : static_cast<int>(2 * blockIdx.x) + (first ? 1 : 0));
      int* blocks = piece_blocks(a.p, (s0 + k) * a.p.kv_heads + head, D);
      if (lane == 0 && first) blocks[0] = blockIdx.x;
      if (lane == 0 && last) blocks[1] = blockIdx.x;
      return true;
    }
    return false;
  }
};

template <int D>
struct Smem {
  static constexpr int kTile = D / 64 * kChunk;  // 128 rows
  static constexpr int kQ = 0, kK = 2 * kTile, kV = 4 * kTile, kBars = 6 * kTile;
  static constexpr int kInts = kBars + 320;
  static constexpr int kPieces = kInts + 64;  // Piece[kItems]
  static constexpr int kBad = kPieces + 512;  // int[2][kNotes][3][D]
  static constexpr int kStage = kBad + 2 * kNotes * 3 * D * 4;  // of the epilogue: 32 rows x 64 bytes for each of 8 warps
  static constexpr int kBytes = kStage + 8 * 2048 + 1024;        // + alignment
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

template <int D, bool BF16, bool RUNS>
__global__ void __launch_bounds__(kThreads, 1)
prompt_kernel(const PromptArgs a, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
              const __grid_constant__ CUtensorMap vmap) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  using S = Smem<D>;
  const PromptParams& p = a.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBars);
  volatile int* s_int = reinterpret_cast<volatile int*>(smem + S::kInts);
  volatile int* s_abort = s_int;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + S::kInts) + 1;
  volatile int* s_anybad = s_int + 2;  // [2][kNotes]
  Piece* s_pieces = reinterpret_cast<Piece*>(smem + S::kPieces);
  int* s_bad = reinterpret_cast<int*>(smem + S::kBad);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const unsigned full = 0xffffffffu;
  const int G = a.G;
  allow_next_kernel();

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[kBQ + i], 1);
      mbar_init(&bars[kBQe + i], 1);
      mbar_init(&bars[kBKf + i], 1);
      mbar_init(&bars[kBKe + i], 1);
      mbar_init(&bars[kBVf + i], 1);
      mbar_init(&bars[kBVe + i], 1);
      mbar_init(&bars[kBFix + i], 64);
      mbar_init(&bars[kBS + i], 1);
      mbar_init(&bars[kBP + i], 128);
      mbar_init(&bars[kBO + i], 1);
    }
    for (int i = 0; i < kNotes; ++i) {
      mbar_init(&bars[kBNf + i], 64);
      mbar_init(&bars[kBNe + i], 256);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&bars[kBIf + i], 1);
      mbar_init(&bars[kBIe + i], 11);  // the other warps
    }
    mbar_init(&bars[kBDone], 1);
    fence_mbarrier_init();
    *s_abort = 0;
  }
  if (warp == 9) tmem_alloc_all(s_tmem);
  tcgen_before_sync();
  __syncthreads();
  tcgen_after_sync();
  const uint32_t tbase = *s_tmem;

  auto wait = [&](int bar, uint32_t parity) -> bool {
    if (mbar_try_wait(&bars[bar], parity)) return true;
    const unsigned long long t0 = global_timer_ns();
    while (!mbar_try_wait(&bars[bar], parity)) {
      if (*s_abort) return false;
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        atomicOr(reinterpret_cast<int*>(p.ws), kErrPrompt);
        *s_abort = 1;
        return false;
      }
    }
    return true;
  };
  // every lane waits; a lane whose wait ran out stops the warp
  auto wait_all = [&](int bar, uint32_t parity) { return __all_sync(full, wait(bar, parity)) != 0; };
  // parity of use n of a ring of k stages: of what fills it, of its being free again
  auto used = [](int n, int k) { return static_cast<uint32_t>((n / k) & 1); };
  auto freed = [](int n, int k) { return static_cast<uint32_t>(((n / k) - 1) & 1); };

  // The next piece, for the warps that are told (a whole warp calls it); false:
  // no more, or a wait ran out.
  int n_item = 0;
  auto next_piece = [&](Piece& pc) -> bool {
    const int st = n_item % kItems;
    if (!wait_all(kBIf + st, used(n_item, kItems))) return false;
    pc = s_pieces[st];
    ++n_item;
    return pc.head >= 0;
  };
  // its place may be used again
  auto release_piece = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[kBIe + (n_item - 1) % kItems]);
  };

  Piece pc;
  if (warp >= 8) {
    // 128 x 72 + 256 x 216 registers: the 384 x 168 of the launch.  The softmax
    // warps hold 128 scores each (88 and 208: packed prompts 302 us against 289)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 8) {
      // ---- pieces; K and V tiles
      int* counters = reinterpret_cast<int*>(p.ws) + 1;  // next piece, blocks that are done
      const int total = a.n_slots * p.kv_heads;
      const bool leader = elect_one();
      // the first piece is the block's number, the others come from the counter
      auto take = [&]() {
        int id = 0;
        if (lane == 0) id = static_cast<int>(gridDim.x) + atomicAdd(counters, 1);
        return __shfl_sync(full, id, 0);
      };
      int jt = 0, id = blockIdx.x, n_qi[2] = {0, 0};
      bool ok = true, more = true;
      Run run;
      if (RUNS) run.start(a);
      while (ok && more) {
        if (RUNS) {
          more = run.next(a, pc, D);
        } else {
          more = static_cast<unsigned>(id) < static_cast<unsigned>(total);  // (a workspace that was not set up ends here too)
          if (more && !pc.locate(a, id / p.kv_heads)) {
            id = take();
            continue;
          }
          if (more) pc.take(id % p.kv_heads, 0, pc.tiles(), -1);
        }
        const int st = n_item % kItems;
        if (n_item >= kItems) ok = wait_all(kBIe + st, freed(n_item, kItems));
        if (!ok) break;
        if (lane == 0) {
          if (more) s_pieces[st] = pc;
          else s_pieces[st].head = -1;
          mbar_arrive(&bars[kBIf + st]);
        }
        __syncwarp();
        ++n_item;
        if (!more) break;
        // the next piece is taken near this one's end: a block with a long one would
        // keep it waiting
        int ahead = !RUNS && pc.n_max == 0 ? take() : 0;
        for (int j = 0; ok && j < pc.n_max; ++j, ++jt) {
          if (!RUNS && j == max(0, pc.n_max - 2)) ahead = take();
          const int ks = jt & 1;
          auto load = [&](const CUtensorMap* map, int fullb, int empty, int base) -> bool {
            if (jt >= 2 && !wait_all(empty + ks, freed(jt, 2))) return false;
            if (leader) {
              mbar_arrive_expect_tx(&bars[fullb + ks], S::kTile);
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                tma_load_3d(smem + base + ks * S::kTile + c * kChunk, map, 64 * c, pc.head,
                            static_cast<int>(pc.k0) + (pc.t0 + j) * kKeys, &bars[fullb + ks]);
            }
            __syncwarp();
            return true;
          };
          ok = load(&kmap, kBKf, kBKe, S::kK);
          if (!ok) break;
          if (j == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (pc.n[i] == 0) continue;
              if (n_qi[i] > 0) ok = ok && wait_all(kBQe + i, (n_qi[i] - 1) & 1);
              if (!ok) continue;
              ++n_qi[i];
              if (leader) {
                // tokens past the sequence's end give rows that are not stored
                mbar_arrive_expect_tx(&bars[kBQ + i], D / 64 * a.tokens * G * 128);
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                  tma_load_3d(smem + S::kQ + i * S::kTile + c * kChunk, &qmap, 64 * c, pc.head * G,
                              static_cast<int>(pc.q0) + pc.tok0 + i * a.tokens, &bars[kBQ + i]);
              }
              __syncwarp();
            }
          }
          if (ok) ok = load(&vmap, kBVf, kBVe, S::kV);
          if (!ok) {  // this K tile is on its way: it must land before the block ends
            mbar_wait_bounded(&bars[kBKf + ks], used(jt, 2));
            break;
          }
        }
        id = ahead;
      }
      // copies in flight (after an abort) must land before the block ends
      for (int n = max(0, jt - 2); n < jt; ++n) {
        mbar_wait_bounded(&bars[kBKf + (n & 1)], used(n, 2));
        mbar_wait_bounded(&bars[kBVf + (n & 1)], used(n, 2));
      }
      for (int i = 0; i < 2; ++i)
        if (n_qi[i] > 0) mbar_wait_bounded(&bars[kBQ + i], (n_qi[i] - 1) & 1);
      if (!RUNS && lane == 0) {  // the last block leaves the counters as it found them
        __threadfence();
        if (atomicAdd(counters + 1, 1) == static_cast<int>(gridDim.x) - 1) {
          counters[0] = 0;
          counters[1] = 0;
        }
      }
    } else if (warp == 9) {
      // ---- MMAs
      const bool leader = elect_one();
      constexpr uint32_t id_qk = mma_idesc(BF16, false, false, kKeys), id_pv = mma_idesc(BF16, false, true, D);
      const uint32_t sq = smem_u32(smem + S::kQ), sk = smem_u32(smem + S::kK), sv = smem_u32(smem + S::kV);
      int jt = 0, n_qi[2] = {0, 0}, n_s[2] = {0, 0};
      bool ok = true;
      while (ok && next_piece(pc)) {
        release_piece();
        auto qk = [&](int i, int j) {
          const uint64_t da = sw128_desc(sq + i * S::kTile, 0, 1024);
          const uint64_t db = sw128_desc(sk + ((jt + j) & 1) * S::kTile, 0, 1024);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t o = ((k >> 2) * kChunk + (k & 3) * 32) >> 4;
            mma_ss(tbase + 128 * i, da + o, db + o, id_qk, k > 0, leader);
          }
          mma_commit(&bars[kBS + i], leader);
          if (j + 1 == pc.n[i]) mma_commit(&bars[kBQe + i], leader);
        };
        auto pv = [&](int i, int j) {
          const uint64_t db = sw128_desc(sv + ((jt + j) & 1) * S::kTile, kChunk, 1024);
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            mma_ts(tbase + 256 + 128 * i, tbase + 128 * i + 8 * k, db + ((k * 2048) >> 4), id_pv, j > 0 || k > 0, leader);
        };
        if (pc.n_max > 0) {
          ok = wait_all(kBKf + (jt & 1), used(jt, 2));
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (ok && pc.n[i] > 0) {
              ok = wait_all(kBQ + i, n_qi[i] & 1);
              ++n_qi[i];
              tcgen_after_sync();
              if (ok) qk(i, 0);
            }
          if (ok) mma_commit(&bars[kBKe + (jt & 1)], leader);
        }
        for (int j = 0; ok && j < pc.n_max; ++j) {
          const int x = jt + j;
          bool have_v = false, have_k = false;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (!ok) break;
            if (j >= pc.n[i]) continue;
            if (!have_v) ok = wait_all(kBFix + (x & 1), used(x, 2));
            have_v = true;
            if (ok) ok = wait_all(kBP + i, (n_s[i] + j) & 1);
            if (!ok) break;
            tcgen_after_sync();
            pv(i, j);
            if (j + 1 < pc.n[i]) {
              if (!have_k) ok = wait_all(kBKf + ((x + 1) & 1), used(x + 1, 2));
              have_k = true;
              if (ok) qk(i, j + 1);
            } else {
              mma_commit(&bars[kBO + i], leader);
            }
          }
          if (ok) {
            mma_commit(&bars[kBVe + (x & 1)], leader);
            if (have_k) mma_commit(&bars[kBKe + ((x + 1) & 1)], leader);
          }
        }
        jt += pc.n_max;
        n_s[0] += pc.n[0];
        n_s[1] += pc.n[1];
      }
      if (!ok) {  // MMAs in flight: let them finish before tensor memory is freed
        mma_commit(&bars[kBDone], leader);
        mbar_wait_bounded(&bars[kBDone], 0);
      }
    } else {
      // ---- V tiles with masked positions
      const int t = tid - 320;
      int jt = 0;
      bool ok = true;
      while (ok && next_piece(pc)) {
        release_piece();
        const int note = (n_item - 1) % kNotes;
        if (ok && n_item > kNotes) ok = wait_all(kBNe + note, freed(n_item - 1, kNotes));
        int* notes = s_bad + ((warp - 10) * kNotes + note) * 3 * D;
        if (pc.first_masked < pc.n_max)
          for (int x = lane; x < 3 * D; x += 32) notes[x] = 0x7fffffff;
        if (lane == 0) s_anybad[(warp - 10) * kNotes + note] = 0;
        __syncwarp();
        for (int j = 0; ok && j < pc.n_max; ++j, ++jt) {
          ok = wait_all(kBVf + (jt & 1), used(jt, 2));
          if (!ok) break;
          if (j >= pc.first_masked) {
            uint8_t* v = smem + S::kV + (jt & 1) * S::kTile;
            const int live = min(kKeys, pc.nk - (pc.t0 + j) * kKeys);  // positions of the tile inside the sequence
            constexpr uint32_t kExp = BF16 ? 0x7F807F80u : 0x7C007C00u, kOne = BF16 ? 0x00800080u : 0x04000400u;
            bool wrote = false;
            // rows from the first position that some row does not see
            const int r0 = max(0, pc.mask_from - (pc.t0 + j) * kKeys);
            constexpr int kAtOnce = 8;  // units of a thread in flight
            const int r1 = max(r0, live), units = (r1 - r0) * 8;
            for (int c = 0; c < D / 64; ++c) {
              uint8_t* vc = v + c * kChunk;
              for (int x0 = t; x0 < units; x0 += 64 * kAtOnce) {
                uint4 w[kAtOnce];
                uint32_t any = 0;
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                  // (past the end: the first unit again)
                  const int x = x0 + 64 * k < units ? x0 + 64 * k : x0;
                  w[k] = *reinterpret_cast<const uint4*>(vc + r0 * 128 + x * 16);
                }
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k)
                  any |= ((w[k].x & kExp) + kOne) | ((w[k].y & kExp) + kOne) | ((w[k].z & kExp) + kOne) | ((w[k].w & kExp) + kOne);
                if ((any & 0x80008000u) == 0) continue;
                for (int x = x0; x < units && x < x0 + 64 * kAtOnce; x += 64) {
                  const int r = r0 + (x >> 3), u = x & 7;
                  uint16_t* h = reinterpret_cast<uint16_t*>(vc + r0 * 128 + x * 16);
                  const int d0 = c * 64 + ((u ^ (r & 7)) << 3);
                  for (int e = 0; e < 8; ++e) {
                    const uint16_t y = h[e];
                    if ((y & (kExp & 0xffffu)) != (kExp & 0xffffu)) continue;
                    const int kind = (y & 0x7fff & ~(kExp & 0xffffu)) ? 0 : y >> 15 ? 2 : 1;
                    atomicMin(&notes[kind * D + d0 + e], (pc.t0 + j) * kKeys + r);
                    s_anybad[(warp - 10) * kNotes + note] = 1;
                    h[e] = 0;
                    wrote = true;
                  }
                }
              }
              for (int x = max(live, 0) * 8 + t; x < kKeys * 8; x += 64) {  // past the sequence
                *reinterpret_cast<uint4*>(vc + x * 16) = make_uint4(0u, 0u, 0u, 0u);
                wrote = true;
              }
            }
            if (wrote) fence_async_smem();
          }
          mbar_arrive(&bars[kBFix + (jt & 1)]);
        }
        mbar_arrive(&bars[kBNf + note]);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // ---- softmax warpgroup i, a thread for each row
    const int i = warp >> 2, wt = tid & 127;
    const uint32_t t_lane = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t t_s = tbase + t_lane + 128 * i, t_o = tbase + t_lane + 256 + 128 * i;
    const float sl = fmaxf(fabsf(p.scale) * kLog2e, 1.2e-38f);  // not 0: -inf * sl stays -inf
    const int tok_l = wt / G, head_l = wt - tok_l * G;  // this thread's row in its tile
    uint8_t* stage = smem + S::kStage + warp * 2048;
    int n_s = 0, n_o = 0;  // scores and results so far
    bool ok = true;
    while (ok && next_piece(pc)) {
      const int n = i == 0 ? pc.n[0] : pc.n[1], t0 = RUNS ? pc.t0 : 0;
      const int my_sees = pc.sees(min(pc.tok0 + i * a.tokens + tok_l, pc.nq - 1));
      const int all_see = pc.sees(pc.tok0 + i * a.tokens);  // what every row of the tile sees
      // A row that is no query of the piece (past the tile's tokens Q is what an
      // earlier call left there, past the sequence's another's) takes no part in
      // the warp's votes on the reference: no score passes +inf.  What it computes
      // is not stored.
      float m = wt < a.tokens * G && pc.tok0 + i * a.tokens + tok_l < pc.nq ? -INFINITY : INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j, ++n_s) {
        ok = wait_all(kBS + i, n_s & 1);
        if (!ok) break;
        tcgen_after_sync();
        uint32_t s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32 * c, s + 32 * c);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_wait_ld32(s + 32 * c);
        if (p.scale < 0.f) {  // the sign goes to the scores
#pragma unroll
          for (int c = 0; c < 128; ++c) s[c] ^= 0x80000000u;
        }
        if ((t0 + j + 1) * kKeys > all_see) {
          const int lim = my_sees - (t0 + j) * kKeys;
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c >= lim) s[c] = 0xff800000u;  // -inf
        }
        float top[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) top[c] = __uint_as_float(s[c]);
#pragma unroll
        for (int c = 4; c < 128; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            top[e] = c + e + 4 < 128 ? fmaxf(top[e], fmaxf(__uint_as_float(s[c + e]), __uint_as_float(s[c + e + 4])))
                                     : fmaxf(top[e], __uint_as_float(s[c + e]));
        const float mt = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * sl;
        if (__any_sync(full, mt > m + kLazy)) {
          const float mn = fmaxf(m, mt);
          const float f = m == -INFINITY ? 0.f : ex2(m - mn);
          l *= f;
          m = mn;
          if (j > 0) {
            const uint64_t f2 = pack2(f, f);
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(t_o + c, o);
              tmem_wait_ld32(o);
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                float x, y;
                unpack2(mul2(pack2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), f2), x, y);
                o[e] = __float_as_uint(x), o[e + 1] = __float_as_uint(y);
              }
              tmem_st32(t_o + c, o);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        const uint64_t sl2 = pack2(sl, sl), nm2 = pack2(-ref, -ref);
        uint64_t sum[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 128; c += 2) {
          float x, y;
          unpack2(fma2(pack2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sl2, nm2), x, y);
          x = ex2(x), y = ex2(y);
          sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], pack2(x, y));
          s[c >> 1] = cvt_pair<BF16>(x, y);
        }
        {
          float x, y;
          unpack2(add2(sum[0], sum[1]), x, y);
          l += x + y;
        }
        tmem_st32(t_s, s);
        tmem_st32(t_s + 32, s + 32);
        tmem_wait_store();
        tcgen_before_sync();
        mbar_arrive(&bars[kBP + i]);
      }
      // ---- epilogue
      if (!ok) break;
      if (n > 0) {
        ok = wait_all(kBO + i, n_o & 1);
        ++n_o;
      }
      const int note = (n_item - 1) % kNotes;
      ok = ok && wait_all(kBNf + note, used(n_item - 1, kNotes));
      if (!ok) break;
      tcgen_after_sync();
      // the piece, read again: its registers are scarce in the loop above
      const Piece& piece = s_pieces[(n_item - 1) % kItems];
      const int token = piece.tok0 + i * a.tokens + tok_l, part = RUNS ? piece.part : -1;
      const bool store = wt < a.tokens * G && token < piece.nq;
      const int64_t at = piece.q0 + token;  // row of q and out
      const int h = piece.head * G + head_l;
      const bool bad = s_anybad[note] != 0 || s_anybad[kNotes + note] != 0;
      const int* bad0 = s_bad + note * 3 * D;
      const int* bad1 = s_bad + (kNotes + note) * 3 * D;
      const bool use0 = s_anybad[note] != 0, use1 = s_anybad[kNotes + note] != 0;
      {
        const float inv = part >= 0 ? 1.f : l == 0.f ? 0.f : 1.f / l;
        T* out = static_cast<T*>(p.out.ptr);
        int64_t off8[4];  // of the rows this lane stores; -1: none
#pragma unroll
        for (int x = 0; x < 4; ++x)
          off8[x] = __shfl_sync(full, store ? at * p.out.token_stride + h * p.out.head_stride : -1, 8 * x + (lane >> 2));
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld32(t_o + c, o);
            tmem_wait_ld32(o);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(l == 0.f ? 0.f : __uint_as_float(o[e]) * inv);
          if (bad) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              auto seen = [&](int x) { return (use0 && bad0[x] < my_sees) || (use1 && bad1[x] < my_sees); };
              const bool nan = seen(c + e), up = seen(D + c + e), down = seen(2 * D + c + e);
              // added: O may hold infinities and NaN of other tiles, or of the scores
              if (nan || (up && down)) o[e] = 0x7fffffffu;
              else if (up) o[e] = __float_as_uint(__uint_as_float(o[e]) + INFINITY);
              else if (down) o[e] = __float_as_uint(__uint_as_float(o[e]) - INFINITY);
            }
          }
          // through shared memory, so that a store covers whole sectors: 32 rows of
          // 64 bytes (parts, in fp32: two halves of the columns)
          if (part >= 0) {
            float* to = part_slot(p, part, D) + (128 * i + 32 * (warp & 3)) * D + c;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
              for (int u = 0; u < 4; ++u)
                *reinterpret_cast<uint4*>(stage + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4)) =
                    make_uint4(o[16 * half + 4 * u], o[16 * half + 4 * u + 1], o[16 * half + 4 * u + 2], o[16 * half + 4 * u + 3]);
              __syncwarp();
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const int r = 8 * x + (lane >> 2), u = lane & 3;
                *reinterpret_cast<uint4*>(to + r * D + 16 * half + 4 * u) =
                    *reinterpret_cast<const uint4*>(stage + r * 64 + ((u ^ ((r >> 1) & 3)) << 4));
              }
              __syncwarp();
            }
          } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              uint4 w;
              w.x = cvt_pair<BF16>(__uint_as_float(o[8 * u]), __uint_as_float(o[8 * u + 1]));
              w.y = cvt_pair<BF16>(__uint_as_float(o[8 * u + 2]), __uint_as_float(o[8 * u + 3]));
              w.z = cvt_pair<BF16>(__uint_as_float(o[8 * u + 4]), __uint_as_float(o[8 * u + 5]));
              w.w = cvt_pair<BF16>(__uint_as_float(o[8 * u + 6]), __uint_as_float(o[8 * u + 7]));
              *reinterpret_cast<uint4*>(stage + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4)) = w;
            }
            __syncwarp();
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int r = 8 * x + (lane >> 2), u = lane & 3;
              const uint4 w = *reinterpret_cast<const uint4*>(stage + r * 64 + ((u ^ ((r >> 1) & 3)) << 4));
              if (off8[x] >= 0) *reinterpret_cast<uint4*>(out + off8[x] + c + 8 * u) = w;
            }
            __syncwarp();
          }
        }
        if (part >= 0)
          *reinterpret_cast<float2*>(part_slot(p, part, D) + kRowsPerBlock * D + 2 * (128 * i + wt)) = make_float2(m, l);
        else if (store && p.lse)
          p.lse[at * p.q_heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        tcgen_before_sync();
      }
      release_piece();
      mbar_arrive(&bars[kBNe + note]);
    }
  }
  __syncthreads();
  if (warp == 9) tmem_free_all(tbase);
}

// Adds the parts of a row: a warp for each.
template <int D, bool BF16>
__global__ void __launch_bounds__(128) prompt_join_kernel(const PromptArgs a) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  const PromptParams& p = a.p;
  const int lane = threadIdx.x & 31;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) >> 5;
  const int64_t token = div_small(row, p.q_heads);
  const int qh = static_cast<int>(row - token * p.q_heads), head = qh / a.G;
  int lo = 0, hi = p.n_seqs;  // the sequence: the first with cu[seq + 1] > token
  while (token < p.n_q && lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.cu_q + mid + 1) <= token) lo = mid + 1;
    else hi = mid;
  }
  const bool on = token < p.n_q && lo < p.n_seqs && __ldg(p.cu_q + lo) <= token;
  wait_for_last_kernel();  // every thread: what follows on the stream may rely on both kernels
  if (!on) return;
  const int64_t q0 = max(__ldg(p.cu_q + lo), 0);
  const int i = static_cast<int>(token - q0), in_piece = i % (2 * a.tokens);
  const int64_t slot = q0 / (2 * a.tokens) + lo + i / (2 * a.tokens);
  const int rr = 128 * (in_piece / a.tokens) + in_piece % a.tokens * a.G + qh - head * a.G;
  const int* blocks = piece_blocks(p, static_cast<int>((a.n_slots - 1 - slot) * p.kv_heads + head), D);
  const int b0 = max(0, blocks[0]), b1 = min(blocks[1], kMaxBlocks - 1);
  if (b0 >= b1) return;  // one block had it all
  const unsigned full = 0xffffffffu;
  float m = -INFINITY, l = 0.f, acc[D / 32];
#pragma unroll
  for (int c = 0; c < D / 32; ++c) acc[c] = 0.f;
  for (int c0 = b0; c0 <= b1; c0 += 32) {
    const int n = min(32, b1 - c0 + 1);
    // eight parts in flight at a time, the first beside their m and l
    float x[8][D / 32];
    auto fetch = [&](int k0) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k0 + k >= n) break;
        const float* part = part_slot(p, 2 * (c0 + k0 + k) + (c0 + k0 + k == b0 ? 1 : 0), D) + rr * D + lane * (D / 32);
        if constexpr (D == 128) *reinterpret_cast<float4*>(x[k]) = *reinterpret_cast<const float4*>(part);
        else *reinterpret_cast<float2*>(x[k]) = *reinterpret_cast<const float2*>(part);
      }
    };
    float2 ml = make_float2(-INFINITY, 0.f);
    const int mine = c0 + lane;
    if (mine <= b1)
      ml = *reinterpret_cast<const float2*>(part_slot(p, 2 * mine + (mine == b0 ? 1 : 0), D) + kRowsPerBlock * D + 2 * rr);
    fetch(0);
    float top = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(full, top, o));
    const float mn = fmaxf(m, top), ref = mn == -INFINITY ? 0.f : mn;
    const float g = m == -INFINITY ? 0.f : ex2(m - ref);
    const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - ref);
    m = mn;
    l *= g;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) acc[c] *= g;
    for (int k0 = 0; k0 < n; k0 += 8) {
      if (k0 > 0) fetch(k0);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k0 + k >= n) break;
        const float fk = __shfl_sync(full, f, k0 + k);
        l += __shfl_sync(full, ml.y, k0 + k) * fk;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) acc[c] += x[k][c] * fk;
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* out = static_cast<T*>(p.out.ptr) + token * p.out.token_stride + qh * p.out.head_stride + lane * (D / 32);
#pragma unroll
  for (int c = 0; c < D / 32; c += 2)
    *reinterpret_cast<uint32_t*>(out + c) = cvt_pair<BF16>(acc[c] * inv, acc[c + 1] * inv);
  if (p.lse && lane == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static std::atomic<EncodeFn> known{nullptr};  // of the driver, the same for every device
  EncodeFn fn = known.load(std::memory_order_relaxed);
  if (fn) return fn;
  void* f = nullptr;
  cudaDriverEntryPointQueryResult r;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
      r != cudaDriverEntryPointSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  fn = reinterpret_cast<EncodeFn>(f);
  known.store(fn, std::memory_order_relaxed);
  return fn;
}

// Map of rows [tokens][heads][D]: boxes of 64 values x box_heads x box_tokens.
cudaError_t make_map(CUtensorMap* map, const RowsIn& r, int D, int heads, int64_t tokens, bool bf16, int box_heads,
                     int box_tokens) {
  EncodeFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  // the stride of a dimension of one element is free; zero strides have no map
  const int64_t hs = heads > 1 ? r.head_stride : D, ts = tokens > 1 ? r.token_stride : static_cast<int64_t>(heads) * D;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(hs) * 2, static_cast<cuuint64_t>(ts) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_tokens)}, ones[3] = {1, 1, 1};
  const CUresult rc = fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                         const_cast<void*>(r.ptr), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return rc == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, bool BF16>
cudaError_t launch(const PromptParams& p, cudaStream_t s) {
  PromptArgs a;
  a.p = p;
  a.G = p.q_heads / p.kv_heads;
  a.tokens = 128 / a.G;
  a.n_slots = static_cast<int>(p.n_q / (2 * a.tokens)) + p.n_seqs;
  CUtensorMap qm = {}, km = {}, vm = {};
  if (p.n_k > 0) {  // without keys nothing is loaded
    cudaError_t e = make_map(&qm, p.q, D, p.q_heads, p.n_q, BF16, a.G, a.tokens);
    if (e == cudaSuccess) e = make_map(&km, p.k, D, p.kv_heads, p.n_k, BF16, 1, kKeys);
    if (e == cudaSuccess) e = make_map(&vm, p.v, D, p.kv_heads, p.n_k, BF16, 1, kKeys);
    if (e != cudaSuccess) return e;
  }
  int dev = 0, sms = 0;
  const cudaError_t found = current_device(&dev, &sms);
  if (found != cudaSuccess) return found;
  const int64_t pieces = static_cast<int64_t>(a.n_slots) * p.kv_heads;
  // Whole pieces, or runs: whichever makes the busiest block's share of the keys
  // less.  The lengths are known as averages only; either is right.  (Two chunks
  // of up to 300 tokens after 6000, 96 pieces: 67 us by runs, 81 whole; one of
  // 512 after 6000, 128 pieces: 93 by runs, 80 whole.)
  const double busy = std::ceil(static_cast<double>(p.n_q) / (2 * a.tokens) / p.n_seqs) * p.n_seqs * p.kv_heads;
  const double most = static_cast<double>(p.n_k) / p.n_seqs / kKeys;  // key tiles of a sequence's last piece
  const double mean = std::max(1.0, (p.n_k - 0.5 * p.n_q) / p.n_seqs / kKeys) + kStartTiles;
  const double whole = std::max(std::ceil(busy / sms) * mean, most + kStartTiles);
  const double runs = busy * mean / sms + kStartTiles + kJoinTiles;
  auto run = [&](auto by_runs, int64_t blocks) {
    constexpr bool RUNS = decltype(by_runs)::value;
    static std::atomic<uint64_t> set;
    const cudaError_t e = allow_shared_memory(set, dev, prompt_kernel<D, BF16, RUNS>, Smem<D>::kBytes);
    if (e != cudaSuccess) return e;
    prompt_kernel<D, BF16, RUNS>
        <<<static_cast<unsigned>(std::min<int64_t>(blocks, sms)), kThreads, Smem<D>::kBytes, s>>>(a, qm, km, vm);
    return cudaGetLastError();
  };
  if (pieces > kMaxPieces || runs >= whole) return run(std::false_type(), pieces);
  const cudaError_t e = run(std::true_type(), kMaxBlocks);
  if (e != cudaSuccess) return e;
  return launch_after(prompt_join_kernel<D, BF16>, static_cast<unsigned>((p.n_q * p.q_heads + 3) / 4), a, s);
}

}  // namespace

int64_t prompt_ws_bytes(int head_dim) { 
  return kPartSlots * part_floats(head_dim) * static_cast<int64_t>(sizeof(float)) + kMaxPieces * 2 * static_cast<int64_t>(sizeof(int));
}

cudaError_t launch_attn_prompt(const PromptParams& p, cudaStream_t s) {
  if (p.dtype == QGEMV_DT_F16) return p.head_dim == 64 ? launch<64, false>(p, s) : launch<128, false>(p, s);
  return p.head_dim == 64 ? launch<64, true>(p, s) : launch<128, true>(p, s);
}

}  // namespace qgemv
