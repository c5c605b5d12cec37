// attn_tree_wide.cu -- the attention of drafted tokens over the cache for row
// tiles of up to 64 rows (drafted tokens x heads of a group), on the
// fifth-generation tensor cores.
//
//   S^T = K Q^T   (128 keys x N rows)      O^T += V^T P^T   (d x N rows)
//
// Keys, not rows, lie along M = 128, so that few rows cost little (N is the
// number of rows, rounded up to 16) and a thread's key has its scales as two
// scalars.  A unit is 128 cached tokens (tree_work.cuh).
//
// Warps (28):
//   softmax (16)  four warpgroups, each for 16 of the rows, a thread for each
//          key: S^T from tensor memory, times the key's scale; p = exp2(s -
//          m_r) with a reference m_r for each row that all keys share, moved
//          (and O^T with it) only when some score passes it by 2^8 -- the four
//          warps agree on that by one reducing barrier; p * scale(v), rounded
//          to fp16, to shared memory
//   K (4)  codes to fp16 in the operands' swizzle, a thread for each token
//          (fp16 pages need none: their blocks are copied into place)
//   V (4)  likewise; in units that hold drafted tokens or end inside, whatever
//          must not meet a masked row's 0 is taken out of V (below)
//   copies of K and of V (bulk, from the pages), a warp for each, so that a V
//          that waits for its product holds up no K; MMAs; one that does nothing
// INT8 codes are exact in fp16.  fp16 values of drafted tokens may be infinite
// or NaN, and what lies past the sequence's end is whatever the page holds:
// both are zeroed in V, and the former noted by (drafted token, d) for the rows
// that see them.  Q4_0 does not come here: its groups' scales would take a
// product for each group of K and another rounding of V, and with them this
// kernel was slower than tiles of 24 or 32 rows by attn_tree.cu's (12 ragged
// sequences, 45 rows: 135 us against 84).
//
// Two sequences of up to 131000 fp16 tokens, 40 rows: 113 us, 0.87 of the copy
// bandwidth, start and join included; the chain of a unit (scores, maxima,
// barrier, P, product) is what is left.  Softmax warpgroups of 16 rows: a unit
// took 3300 cycles with one of 64 rows, 2900 with two of 32, 2500 with four.
//
// Every wait is bounded; on a timeout the block records the error, waits for
// its own copies and MMAs, frees tensor memory and returns.
#include <type_traits>

#include "per_device.h"
#include "tc_common.cuh"
#include "tree_work.cuh"

namespace qgemv {
namespace {

constexpr int kSoft = 4;                            // softmax warpgroups, each of kCols rows of the tile
constexpr int kConvWarp = 4 * kSoft;                // first of the decoding warps
constexpr int kLoadWarp = kConvWarp + 8, kMmaWarp = kLoadWarp + 1, kLoadVWarp = kLoadWarp + 2;
constexpr int kThreads = 32 * (kConvWarp + 12);
constexpr int kRows = 64;
constexpr int kCols = kRows / kSoft;
static_assert(kCols == 16, "half a warp's lanes a row, where l is summed");
constexpr int kKeys = 128;
constexpr int kBlocks = kKeys / kKvBlockTokens;  // cache blocks of a unit
constexpr int kErrWide = 64;
constexpr float kLazyW = 8.f;
constexpr float kNone = 1e30f;  // -m of a row that has seen nothing

// Notes of infinite and NaN values, of three segments in turn: when the first V
// of segment s is decoded, the product of two units before is done, so the
// softmax warpgroups have ended segment s - 3 at least, and the V warps clear
// its notes.
constexpr int kNotes = 3;

template <int FMT, int D>
struct Wide {
  using L = KvLayout<FMT, D>;
  static constexpr bool kF16 = FMT == QGEMV_KV_F16;
  static_assert(kF16 || FMT == QGEMV_KV_INT8, "format");
  static constexpr int kTile = kKeys * D * 2;  // a K or V operand
  static constexpr int kKs = kF16 ? 3 : 2, kVs = 2;
  // raw stages, half a unit of K or V codes each: the codes of a block as they
  // lie in it, K's with the block's scales after them
  static constexpr int kRawK = L::kV + L::kBlock - L::kKs, kRawV = L::kV;
  static constexpr int kHalf = kBlocks / 2 * (kRawK + kRawV);
  static constexpr int kRs = kF16 ? 0 : 3;
  static constexpr int kSBufs = 2;
  // shared memory
  static constexpr int kK = 0;
  static constexpr int kV = kK + kKs * kTile;
  static constexpr int kQ = kV + kVs * kTile;
  static constexpr int kP = kQ + kRows * D * 2;
  static constexpr int kRaw = kP + kKeys * 128;  // [kRs] stages of K, then of V
  static constexpr int kKsc = kRaw + kRs * kHalf;          // [kKs][128]
  static constexpr int kVsc = kKsc + (kF16 ? 0 : kKs * kKeys * 4);
  static constexpr int kM = kVsc + (kF16 ? 0 : kKs * kKeys * 4);  // float[64] -m, float[64] factors, float[4][64] x 2
  static constexpr int kRowOff = kM + 64 * 4 * 10;         // int64[64][2]: q and out offsets
  static constexpr int kRowMask = kRowOff + 64 * 16;       // uint64[64]
  static constexpr int kKeyMask = kRowMask + 64 * 8;       // uint32[kSoft][64]: a warpgroup's rows that see a drafted token
  static constexpr int kBad = kKeyMask + kSoft * 64 * 4;   // uint64[kNotes][3][D]
  static constexpr int kInts = kBad + (!kF16 ? 0 : kNotes * 3 * D * 8);
  static constexpr int kBars = kInts + 128;
  static constexpr int kBytes = kBars + 48 * 8 + 1024;  // + alignment
  static_assert(kBytes <= 227 * 1024, "shared memory");
  // tensor memory columns
  static constexpr int kOCol = kSBufs * kRows;
  static_assert(kOCol + kRows <= 512, "tensor memory");
};

// Barriers: index of the first of each kind (kRf, kRe: three of K, three of V).
struct Bars {
  static constexpr int kRf = 0, kRe = kRf + 6, kKf = kRe + 6, kKe = kKf + 3, kVl = kKe + 3, kVf = kVl + 2, kVe = kVf + 2,
                       kSf = kVe + 2, kSe = kSf + 2, kPf = kSe + 2, kPv = kPf + 1, kQf = kPv + 1, kDone = kQf + 1;
};

// OR of `pred` over the 128 threads of softmax warpgroup w.
__device__ __forceinline__ bool any_of_128(int w, bool pred) {
  __syncwarp();
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
               "bar.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(r)
               : "r"(pred ? 1u : 0u), "r"(1 + w)
               : "memory");
  return r != 0;
}

__device__ __forceinline__ float warp_max(float x) {
  int k = __float_as_int(x);
  k ^= (k >> 31) & 0x7fffffff;
  k = __reduce_max_sync(0xffffffffu, k);
  k ^= (k >> 31) & 0x7fffffff;
  return __int_as_float(k);
}

template <int FMT, int D>
__global__ void __launch_bounds__(kThreads, 1) tree_wide_kernel(const TreeArgs a) {
  using S = Wide<FMT, D>;
  using L = typename S::L;
  using B = Bars;
  const TreeParams& p = a.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBars);
  float* s_nm = reinterpret_cast<float*>(smem + S::kM);
  float* s_f = s_nm + 64;
  float* s_red = s_f + 64;  // [4][64]
  float* s_l = s_red + 256;
  int64_t* s_off = reinterpret_cast<int64_t*>(smem + S::kRowOff);
  uint64_t* s_rowmask = reinterpret_cast<uint64_t*>(smem + S::kRowMask);
  uint32_t* s_keymask = reinterpret_cast<uint32_t*>(smem + S::kKeyMask);
  unsigned long long* s_bad = reinterpret_cast<unsigned long long*>(smem + S::kBad);
  volatile int* s_int = reinterpret_cast<volatile int*>(smem + S::kInts);
  volatile int* s_abort = s_int;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + S::kInts) + 1;
  volatile int* s_anybad = s_int + 2;   // [kNotes]
  // blocks (bits) whose pages exist, of each half of a unit
  volatile int* s_valid = s_int + 6;    // [kKs][2]
  volatile int* s_vvalid = s_int + 12;  // [kVs], whole units (fp16)
  volatile int* s_rvalid = s_int + 14;  // [kRs]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const unsigned full = 0xffffffffu;
  allow_next_kernel();

  if (tid == 0) {
    for (int i = 0; i < 6; ++i) {
      mbar_init(&bars[B::kRf + i], 1);
      mbar_init(&bars[B::kRe + i], 64);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&bars[B::kKf + i], S::kF16 ? 1 : 128);
      mbar_init(&bars[B::kKe + i], 1 + 4 * kSoft);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[B::kVl + i], 1);
      mbar_init(&bars[B::kVf + i], 128);
      mbar_init(&bars[B::kVe + i], 1);
      mbar_init(&bars[B::kSf + i], 1);
      mbar_init(&bars[B::kSe + i], 128 * kSoft);
    }
    mbar_init(&bars[B::kPf], 128 * kSoft);
    mbar_init(&bars[B::kPv], 1);
    mbar_init(&bars[B::kQf], 128 * kSoft);
    mbar_init(&bars[B::kDone], 1);
    fence_mbarrier_init();
    *s_abort = 0;
    for (int i = 0; i < kNotes; ++i) s_anybad[i] = 0;
  }
  if (warp == kMmaWarp) tmem_alloc_all(s_tmem);
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
        atomicOr(reinterpret_cast<int*>(p.ws), kErrWide);
        *s_abort = 1;
        return false;
      }
    }
    return true;
  };
  // stage and parity of use n of a ring of `k` stages: the wait for what
  // fills it, and for its being free again
  auto used = [](int64_t n, int k) { return static_cast<uint32_t>((n / k) & 1); };
  auto freed = [](int64_t n, int k) { return static_cast<uint32_t>(((n / k) - 1) & 1); };

  int jt = 0;  // units so far: the same count in every warp
  Cursor<kRows, kKeys> work(a);
  Segment sg;

  if (warp < kConvWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 80;");
    // ------------------------------------------------------------ softmax --
    const int wg = warp >> 2, key = tid & 127, quarter = warp & 3;
    const int c0 = wg * kCols;  // first of this warpgroup's rows
    const uint32_t t_lane = static_cast<uint32_t>(32 * quarter) << 16;
    const float sl = p.scale * kLog2e;
    int n_seg = 0;
    // A wait that ran out sets `dead`; the four warps go on, and leave together
    // where they agree on it (a warp that left alone would hold up the others'
    // barriers).
    bool dead = false, left = false;
    while (!left && work.next(a, sg)) {
      const int R = sg.T * a.G, row0 = sg.tile * kRows, live = min(kRows, R - row0);
      const int ctx = sg.ctx, all = ctx + sg.T;
      const int64_t q0 = __ldg(p.cu_q + sg.seq);
      const bool drafts = sg.u1 * kKeys > ctx;  // drafted tokens among the keys
      // ---- this warpgroup's rows: Q, masks, references
      if (quarter == 0) {
        const int r = row0 + min(c0 + (lane & (kCols - 1)), live - 1), tok = r / a.G, h = sg.head * a.G + r - tok * a.G;
        const bool on = c0 + lane < live && lane < kCols;
        const uint64_t m = !on ? 0 : p.masks ? __ldg(reinterpret_cast<const unsigned long long*>(p.masks) + q0 + tok) : (~0ull >> (63 - tok));
        if (lane < kCols) {
          s_off[2 * (c0 + lane)] = (q0 + tok) * p.q.token_stride + h * p.q.head_stride;
          s_off[2 * (c0 + lane) + 1] = (q0 + tok) * p.out.token_stride + h * p.out.head_stride;
          s_rowmask[c0 + lane] = m;
          s_nm[c0 + lane] = kNone;
        }
        if (drafts)
          for (int i = 0; i < sg.T; ++i) {
            const unsigned bits = __ballot_sync(full, (m >> i) & 1);
            if (lane == 0) s_keymask[wg * kMaxDrafts + i] = bits;
          }
      }
      named_bar_sync(1 + wg, 128);
      {
        constexpr int U = D / 8;
        const __half* qb = static_cast<const __half*>(p.q.ptr);
#pragma unroll
        for (int it = 0; it < kCols * U / 128; ++it) {
          const int idx = it * 128 + key, r = c0 + idx / U, u = idx % U;
          uint4 w = make_uint4(0u, 0u, 0u, 0u);
          if (r < live) w = __ldg(reinterpret_cast<const uint4*>(qb + s_off[2 * r] + 8 * u));
          *reinterpret_cast<uint4*>(smem + S::kQ + (u >> 3) * (kRows * 128) + r * 128 + (((u & 7) ^ (r & 7)) << 4)) = w;
        }
        fence_async_smem();
        mbar_arrive(&bars[B::kQf]);
      }
      const bool busy = c0 < live;  // this warpgroup has rows

      uint64_t l2[kCols / 2];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) l2[i] = 0;
      const int n = static_cast<int>(sg.u1 - sg.u0);
      for (int j = 0; j < n; ++j, ++jt) {
        const int ks = jt % S::kKs, sb = jt % S::kSBufs;
        dead |= !wait(B::kKf + ks, used(jt, S::kKs)) || !wait(B::kSf + sb, used(jt, S::kSBufs));
        __syncwarp();
        tcgen_after_sync();
        if (!busy) {
          mbar_arrive(&bars[B::kSe + sb]);
          if (lane == 0) mbar_arrive(&bars[B::kKe + ks]);
          // not before the product of the unit before: S may be a unit ahead of
          // the other warpgroup's P, and this would count for that one
          if (jt > 0) dead |= !wait(B::kPv, (jt - 1) & 1);
          mbar_arrive(&bars[B::kPf]);
          if (any_of_128(wg, dead)) {
            left = true;
            break;
          }
          continue;
        }
        // ---- S of this key
        uint32_t raw[kCols];
        tmem_ld<kCols>(tbase + t_lane + sb * kRows + c0, raw);
        float f = sl, vs = 1.f, lv = 0.f;
        if constexpr (!S::kF16) {
          f *= reinterpret_cast<const float*>(smem + S::kKsc)[ks * kKeys + key];
          vs = reinterpret_cast<const float*>(smem + S::kVsc)[ks * kKeys + key];
          lv = __log2f(fmaxf(vs, 7.9e-31f));  // 2^-100
        }
        const bool there = (s_valid[2 * ks + (key >> 6)] >> ((key >> 4) & 3)) & 1;
        const int64_t pos = (sg.u0 + j) * kKeys + key;
        uint32_t vis = 0;  // the rows that see this key
        if (there) vis = pos < ctx ? ~0u : pos < all ? s_keymask[wg * kMaxDrafts + (pos - ctx)] : 0u;
        uint64_t x2[kCols / 2];
        const uint64_t f2 = pack2(f, f);
        tmem_wait_ld<kCols>(raw);
#pragma unroll
        for (int c = 0; c < kCols / 2; ++c)
          x2[c] = mul2(pack2(__uint_as_float(raw[2 * c]), __uint_as_float(raw[2 * c + 1])), f2);
        tcgen_before_sync();
        mbar_arrive(&bars[B::kSe + sb]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B::kKe + ks]);
        const bool some_masked = __any_sync(full, vis != ~0u);
        if (some_masked) {
#pragma unroll
          for (int i = 0; i < kCols / 2; ++i) {
            float x, y;
            unpack2(x2[i], x, y);
            if (!((vis >> (2 * i)) & 1)) x = -INFINITY;
            if (!((vis >> (2 * i + 1)) & 1)) y = -INFINITY;
            x2[i] = pack2(x, y);
          }
          if (vis == 0) vs = 0.f, lv = -100.f;
        }
        // ---- the rows' references
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < kCols / 4; ++i) {
          const ulonglong2 nm = *reinterpret_cast<const ulonglong2*>(s_nm + c0 + 4 * i);
          float x, y, z, w;
          unpack2(add2(x2[2 * i], nm.x), x, y);
          unpack2(add2(x2[2 * i + 1], nm.y), z, w);
          top[0] = fmaxf(top[0], fmaxf(x, y));
          top[1] = fmaxf(top[1], fmaxf(z, w));
        }
        if (any_of_128(wg, dead || fmaxf(top[0], top[1]) + lv > kLazyW)) {
          if (any_of_128(wg, dead)) {
            left = true;
            break;
          }
#pragma unroll
          for (int i = 0; i < kCols / 2; ++i) {
            float x, y;
            unpack2(x2[i], x, y);
            x = warp_max(x + lv);
            y = warp_max(y + lv);
            if (lane == i) *reinterpret_cast<float2*>(s_red + 64 * quarter + c0 + 2 * i) = make_float2(x, y);
          }
          named_bar_sync(1 + wg, 128);
          if (key < kCols) {
            const int r = c0 + key;
            const float m = -s_nm[r];
            const float mx = fmaxf(fmaxf(s_red[r], s_red[64 + r]), fmaxf(s_red[128 + r], s_red[192 + r]));
            const float mn = fmaxf(m, mx);
            s_f[r] = m == -kNone ? 0.f : ex2(m - mn);
            s_nm[r] = -mn;
          }
          named_bar_sync(1 + wg, 128);
#pragma unroll
          for (int i = 0; i < kCols / 4; ++i) {
            const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(s_f + c0 + 4 * i);
            l2[2 * i] = mul2(l2[2 * i], f.x);
            l2[2 * i + 1] = mul2(l2[2 * i + 1], f.y);
          }
          if (j > 0) {  // O^T of the units before: this thread's d
            dead |= !wait(B::kPv, (jt - 1) & 1);
            __syncwarp();
            tcgen_after_sync();
            uint32_t o[kCols];
            tmem_ld<kCols>(tbase + t_lane + S::kOCol + c0, o);
            tmem_wait_ld<kCols>(o);
#pragma unroll
            for (int c = 0; c < kCols / 2; ++c) {
              float x, y;
              unpack2(mul2(pack2(__uint_as_float(o[2 * c]), __uint_as_float(o[2 * c + 1])),
                           reinterpret_cast<const uint64_t*>(s_f + c0)[c]),
                      x, y);
              o[2 * c] = __float_as_uint(x), o[2 * c + 1] = __float_as_uint(y);
            }
            tmem_st<kCols>(tbase + t_lane + S::kOCol + c0, o);
            tmem_wait_store();
          }
        }
        // ---- P
        uint32_t w2[kCols / 2];
        const uint64_t vs2 = pack2(vs, vs);
#pragma unroll
        for (int i = 0; i < kCols / 4; ++i) {
          const ulonglong2 nm = *reinterpret_cast<const ulonglong2*>(s_nm + c0 + 4 * i);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x, y;
            unpack2(add2(x2[2 * i + e], e ? nm.y : nm.x), x, y);
            x = ex2(x), y = ex2(y);
            const uint64_t pp = pack2(x, y);
            l2[2 * i + e] = add2(l2[2 * i + e], pp);
            if constexpr (!S::kF16) {
              unpack2(mul2(pp, vs2), x, y);
              if (some_masked) {  // 0 where masked, whatever the scale holds
                if (!((vis >> (4 * i + 2 * e)) & 1)) x = 0.f;
                if (!((vis >> (4 * i + 2 * e + 1)) & 1)) y = 0.f;
              }
            }
            w2[2 * i + e] = cvt_pair<false>(x, y);
          }
        }
        if (jt > 0) dead |= !wait(B::kPv, (jt - 1) & 1);  // the product before has read P
#pragma unroll
        for (int u = 0; u < kCols / 8; ++u)
          *reinterpret_cast<uint4*>(smem + S::kP + key * 128 + (((c0 / 8 + u) ^ (key & 7)) << 4)) =
              make_uint4(w2[4 * u], w2[4 * u + 1], w2[4 * u + 2], w2[4 * u + 3]);
        fence_async_smem();
        tcgen_before_sync();
        mbar_arrive(&bars[B::kPf]);
      }
      if (left) break;
      // ---- the segment's end: l over the keys, O^T
      dead |= !wait(B::kPv, (jt - 1) & 1);
      if (any_of_128(wg, dead)) break;
      tcgen_after_sync();
      float* slot = tree_slot(p, blockIdx.x, sg.u0 == 0, D);
      const int bb = n_seg % kNotes;
      const bool bad = S::kF16 && s_anybad[bb] != 0;
      if (busy) {
        {
          // Each step halves the rows a lane holds: lanes 2i and 2i + 1 end with
          // half of the keys of row i each.
          float l[kCols];
#pragma unroll
          for (int i = 0; i < kCols / 2; ++i) unpack2(l2[i], l[2 * i], l[2 * i + 1]);
#pragma unroll
          for (int o = 16, h = kCols / 2; h > 0; o >>= 1, h >>= 1) {
#pragma unroll
            for (int i = 0; i < h; ++i) {
              const bool up = lane & o;
              const float give = up ? l[i] : l[i + h], keep = up ? l[i + h] : l[i];
              l[i] = keep + __shfl_xor_sync(full, give, o);
            }
          }
          l[0] += __shfl_xor_sync(full, l[0], 1);
          if (!(lane & 1)) s_l[64 * quarter + c0 + (lane >> 1)] = l[0];
        }
        named_bar_sync(1 + wg, 128);
        if (key < kCols) {
          const int r = c0 + key;
          const float l = (s_l[r] + s_l[64 + r]) + (s_l[128 + r] + s_l[192 + r]);
          const float nm = s_nm[r], m = nm == kNone ? -INFINITY : -nm;
          s_f[r] = sg.shared ? 1.f : l == 0.f ? 0.f : 1.f / l;
          if (sg.shared) {
            *reinterpret_cast<float2*>(slot + kSlotRows * D + 2 * r) = make_float2(m, l);
          } else if (p.lse && r < live) {
            const int rr = row0 + r, tok = rr / a.G;
            p.lse[(q0 + tok) * p.q_heads + sg.head * a.G + rr - tok * a.G] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
          }
        }
        named_bar_sync(1 + wg, 128);
        uint32_t o[kCols];
        tmem_ld<kCols>(tbase + t_lane + S::kOCol + c0, o);
        tmem_wait_ld<kCols>(o);
        __half* outb = static_cast<__half*>(p.out.ptr);
        if (key < D) {
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            const int r = c0 + c;
            if (r < live) {
              float x = __uint_as_float(o[c]) * s_f[r];
              if (S::kF16 && bad) {
                const unsigned long long* bd = s_bad + bb * 3 * D + key;
                const uint64_t rm = s_rowmask[r];
                const bool nan = bd[0] & rm, up = bd[D] & rm, down = bd[2 * D] & rm;
                if (nan || (up && down)) x = __int_as_float(0x7fffffff);
                else if (up) x += INFINITY;
                else if (down) x -= INFINITY;
              }
              if (sg.shared) slot[r * D + key] = x;
              else outb[s_off[2 * r + 1] + key] = __float2half_rn(x);
            }
          }
        }
        tcgen_before_sync();
      }
      named_bar_sync(1 + wg, 128);
      ++n_seg;
    }
  } else if (warp < kLoadWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    // ----------------------------------------------- codes to operands ----
    const int key = tid & 127, half = key >> 6;
    const bool is_v = warp >= kConvWarp + 4;
    int n_seg = 0;
    // As for the softmax: a wait that ran out sets `dead`, the warps of V leave
    // together, at a segment's start.
    bool dead = false;
    while (!(S::kF16 && !is_v) && !(dead && !is_v) && work.next(a, sg)) {
      const int n = static_cast<int>(sg.u1 - sg.u0), ctx = sg.ctx, all = ctx + sg.T;
      const int bb = n_seg % kNotes;
      bool left = false;
      auto start_notes = [&]() {
        left = any_of_128(kSoft, dead);
        if constexpr (S::kF16) {
          if (left) return;
          for (int i = key; i < 3 * D; i += 128) s_bad[bb * 3 * D + i] = 0;
          if (key == 0) s_anybad[bb] = 0;
          named_bar_sync(1 + kSoft, 128);
        }
      };
      for (int j = 0; j < n; ++j, ++jt) {
        const int64_t pos = (sg.u0 + j) * kKeys + key;
        const int ks = jt % S::kKs, vst = jt % S::kVs;
        uint8_t* dst = smem + (is_v ? S::kV + vst * S::kTile : S::kK + ks * S::kTile) + key * 128;
        auto note = [&](int d, int kind) {  // a drafted token's value that is infinite or NaN
          atomicOr(&s_bad[(bb * 3 + kind) * D + d], 1ull << (pos - ctx));
          s_anybad[bb] = 1;
        };
        if constexpr (S::kF16) {
          dead |= !wait(B::kVl + vst, used(jt, S::kVs));
          __syncwarp();
          if (j == 0) start_notes();
          if (left) break;
          const int valid = s_vvalid[vst];
          if ((sg.u0 + j + 1) * kKeys > ctx || valid != (1 << kBlocks) - 1) {
            const bool on = ((valid >> (key >> 4)) & 1) && pos < all;
#pragma unroll 2
            for (int u = 0; u < D / 8; ++u) {
              uint4* at = reinterpret_cast<uint4*>(dst + (u >> 3) * (kKeys * 128) + (((u & 7) ^ (key & 7)) << 4));
              if (!on) {
                *at = make_uint4(0u, 0u, 0u, 0u);
              } else if (pos >= ctx) {
                const uint4 w = *at;
                const uint32_t e = (((w.x & 0x7C007C00u) + 0x04000400u) | ((w.y & 0x7C007C00u) + 0x04000400u) |
                                    ((w.z & 0x7C007C00u) + 0x04000400u) | ((w.w & 0x7C007C00u) + 0x04000400u)) & 0x80008000u;
                if (e) {
                  uint16_t* hw = reinterpret_cast<uint16_t*>(at);
                  for (int i = 0; i < 8; ++i) {
                    const uint32_t x = hw[i];
                    if ((x & 0x7C00u) != 0x7C00u) continue;
                    note(8 * u + i, (x & 0x3FFu) ? 0 : x >> 15 ? 2 : 1);
                    hw[i] = 0;
                  }
                }
              }
            }
            fence_async_smem();
          }
          mbar_arrive(&bars[B::kVf + vst]);
        } else {
          const int64_t rt = 2ll * jt + half;
          const int rs = static_cast<int>(rt % S::kRs), rb = rs + (is_v ? 3 : 0);
          dead |= !wait(B::kRf + rb, used(rt, S::kRs));
          if (is_v && jt >= S::kVs) dead |= !wait(B::kVe + vst, freed(jt, S::kVs));
          if (!is_v && jt >= S::kKs) dead |= !wait(B::kKe + ks, freed(jt, S::kKs));
          __syncwarp();
          if (is_v && j == 0) start_notes();
          if (left) break;
          const int tok = key & 15;
          const int nb = rs * (kBlocks / 2) + ((key >> 4) & 3);  // block of the ring
          const uint8_t* blk = is_v ? smem + S::kRaw + S::kRs * (kBlocks / 2) * S::kRawK + nb * S::kRawV : smem + S::kRaw + nb * S::kRawK;
          // 16-byte unit U of the row: chunk U >> 3, swizzled
          auto put = [&](int U, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
            *reinterpret_cast<uint4*>(dst + (U >> 3) * (kKeys * 128) + (((U & 7) ^ (key & 7)) << 4)) = make_uint4(w0, w1, w2, w3);
          };
          constexpr int N = D / 16;
          // which unit first: eight neighbouring lanes read eight (d = 64:
          // four) different ones
          const int turn = is_v ? (lane & (N - 1)) ^ ((D == 128 ? 2 * ((lane >> 1) & 3) : 0)) : lane & (N - 1);
#pragma unroll
          for (int u = 0; u < N; ++u) {
            const int unit = is_v ? u ^ turn : (u + turn) & (N - 1);
            const uint4 c = lds128(blk + (is_v ? L::v_off(tok, 16 * unit) - L::kV : L::k_off(tok, 16 * unit)));
            put(2 * unit, i8_pair<0x4140>(c.x), i8_pair<0x4342>(c.x), i8_pair<0x4140>(c.y), i8_pair<0x4342>(c.y));
            put(2 * unit + 1, i8_pair<0x4140>(c.z), i8_pair<0x4342>(c.z), i8_pair<0x4140>(c.w), i8_pair<0x4342>(c.w));
          }
          if (!is_v) {
            reinterpret_cast<float*>(smem + S::kKsc)[ks * kKeys + key] = reinterpret_cast<const float*>(blk + L::kV)[tok];
            reinterpret_cast<float*>(smem + S::kVsc)[ks * kKeys + key] = reinterpret_cast<const float*>(blk + L::kV + L::kVs - L::kKs)[tok];
          }
          if (!is_v && (key & 63) == 0) s_valid[2 * ks + half] = s_rvalid[rs];
          fence_async_smem();
          mbar_arrive(&bars[is_v ? B::kVf + vst : B::kKf + ks]);
          mbar_arrive(&bars[B::kRe + rb]);
        }
      }
      if (left) break;
      ++n_seg;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == kLoadWarp || warp == kLoadVWarp) {
      // -------------------------------------------------------- copies ----
      const bool is_v = warp == kLoadVWarp;
      bool ok = true;
      int n_raw = 0;  // stages filled (half units; fp16: units)
      while (ok && work.next(a, sg)) {
        const int n = static_cast<int>(sg.u1 - sg.u0);
        const int64_t n_pos = static_cast<int64_t>(sg.ctx) + sg.T;
        // lane b < 8: the page of block b of a unit, looked up a unit ahead
        auto page_of = [&](int j) -> int64_t {
          const int64_t pos = (sg.u0 + j) * kKeys + kKvBlockTokens * (lane & 7);
          const int64_t pi = pos >> a.page_shift;
          if (j >= n || pos >= n_pos || pi >= p.table_stride) return -1;
          const int64_t pg = __ldg(p.table + sg.seq * p.table_stride + pi);
          return pg < p.cache.n_pages ? pg : -1;
        };
        int64_t ahead = page_of(0);
        for (int j = 0; ok && j < n; ++j) {
          const int64_t page = ahead;
          ahead = page_of(j + 1);
          const int64_t pos = (sg.u0 + j) * kKeys + kKvBlockTokens * (lane & 7);
          const unsigned valid = __ballot_sync(full, page >= 0) & 0xffu;
          const uint8_t* src = page >= 0 ? kv_block<FMT, D>(p.cache, page, sg.head,
                                                            static_cast<int>(pos & (p.cache.page_tokens - 1)) / kKvBlockTokens)
                                         : nullptr;
          if constexpr (S::kF16) {  // into place
            const int stages = is_v ? S::kVs : S::kKs, st = n_raw % stages;
            const int filled = (is_v ? B::kVl : B::kKf) + st;
            ok = __all_sync(full, n_raw < stages || wait((is_v ? B::kVe : B::kKe) + st, freed(n_raw, stages))) != 0;
            if (!ok) break;
            if (lane == 0) {
              if (is_v) {
                s_vvalid[st] = static_cast<int>(valid);
              } else {
                s_valid[2 * st] = static_cast<int>(valid & 15u);
                s_valid[2 * st + 1] = static_cast<int>(valid >> 4);
              }
              mbar_arrive_expect_tx(&bars[filled], static_cast<uint32_t>(__popc(valid)) * L::kV);
            }
            __syncwarp();
            if (lane < 8 && src) {
              uint8_t* dst = smem + (is_v ? S::kV : S::kK) + st * S::kTile + lane * 2048;
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                bulk_load(dst + c * (kKeys * 128), src + (is_v ? L::kV : 0) + c * 2048, 2048, &bars[filled]);
            }
            ++n_raw;
          } else {
            for (int h = 0; h < 2; ++h, ++n_raw) {
              const int rs = n_raw % S::kRs, rb = rs + (is_v ? 3 : 0);
              ok = __all_sync(full, n_raw < S::kRs || wait(B::kRe + rb, freed(n_raw, S::kRs))) != 0;
              if (!ok) break;
              const unsigned here = (valid >> (4 * h)) & 15u;
              if (lane == 0) {
                if (!is_v) s_rvalid[rs] = static_cast<int>(here);
                mbar_arrive_expect_tx(&bars[B::kRf + rb], __popc(here) * (is_v ? S::kRawV : S::kRawK));
              }
              __syncwarp();
              if ((lane >> 2) == h && src) {
                const int nb = rs * (kBlocks / 2) + (lane & 3);
                if (is_v) {
                  bulk_load(smem + S::kRaw + S::kRs * (kBlocks / 2) * S::kRawK + nb * S::kRawV, src + L::kV, S::kRawV, &bars[B::kRf + rb]);
                } else {
                  uint8_t* dst = smem + S::kRaw + nb * S::kRawK;
                  bulk_load(dst, src, L::kV, &bars[B::kRf + rb]);
                  bulk_load(dst + L::kV, src + L::kKs, L::kBlock - L::kKs, &bars[B::kRf + rb]);
                }
              }
            }
          }
        }
      }
      // copies in flight (after an abort) must land before the block ends
      {
        const int stages = !S::kF16 ? S::kRs : is_v ? S::kVs : S::kKs;
        const int filled = !S::kF16 ? B::kRf + (is_v ? 3 : 0) : is_v ? B::kVl : B::kKf;
        for (int x = max(0, n_raw - stages); x < n_raw; ++x) mbar_wait_bounded(&bars[filled + x % stages], used(x, stages));
      }
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------- MMAs ----
      const bool leader = elect_one();
      int n_seg = 0;
      bool ok = true;
      const uint32_t sk = smem_u32(smem + S::kK), sv = smem_u32(smem + S::kV), sq = smem_u32(smem + S::kQ),
                     sp = smem_u32(smem + S::kP);
      // every lane waits; a lane whose wait ran out stops them all
      auto wait_all = [&](int bar, uint32_t parity) { return __all_sync(full, wait(bar, parity)) != 0; };
      while (ok && work.next(a, sg)) {
        const int n = static_cast<int>(sg.u1 - sg.u0);
        const int live = min(kRows, sg.T * a.G - sg.tile * kRows), N = (live + 15) & ~15;
        const uint32_t id_qk = mma_idesc(false, false, false, N), id_pv = mma_idesc(false, true, true, N);
        auto qk = [&](int x) {
          const int ks = x % S::kKs, sb = x % S::kSBufs;
          tcgen_after_sync();
          const uint64_t da = sw128_desc(sk + ks * S::kTile, 0, 1024), db = sw128_desc(sq, 0, 1024);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t oa = ((k >> 2) * (kKeys * 128) + (k & 3) * 32) >> 4;
            const uint32_t ob = ((k >> 2) * (kRows * 128) + (k & 3) * 32) >> 4;
            mma_ss(tbase + sb * kRows, da + oa, db + ob, id_qk, k > 0, leader);
          }
          mma_commit(&bars[B::kSf + sb], leader);
          mma_commit(&bars[B::kKe + ks], leader);
        };
        auto pv = [&](int x) {
          const int vst = x % S::kVs;
          tcgen_after_sync();
          const uint64_t da = sw128_desc(sv + vst * S::kTile, kKeys * 128, 1024), db = sw128_desc(sp, 0, 1024);
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            mma_ss(tbase + S::kOCol, da + ((k * 2048) >> 4), db + ((k * 2048) >> 4), id_pv, x > jt || k > 0, leader);
          mma_commit(&bars[B::kPv], leader);
          mma_commit(&bars[B::kVe + vst], leader);
        };
        auto now = [&](int bar, uint32_t parity) { return __all_sync(full, mbar_test(&bars[bar], parity)) != 0; };
        ok = wait_all(B::kQf, n_seg & 1);
        // S runs ahead of P V by one unit; whichever is ready goes first, so that a late K does not hold up a V that waits.
        unsigned long long t0 = global_timer_ns();
        for (int x = jt, y = jt; ok && y < jt + n;) {
          bool went = false;
          if (x < jt + n && x <= y + 1 && now(B::kKf + x % S::kKs, used(x, S::kKs)) &&
              (x < S::kSBufs || now(B::kSe + x % S::kSBufs, freed(x, S::kSBufs)))) {
            qk(x++);
            went = true;
          }
          if (y < x && now(B::kPf, y & 1) && now(B::kVf + y % S::kVs, used(y, S::kVs))) {
            pv(y++);
            went = true;
          }
          if (went) {
            t0 = global_timer_ns();
          } else if (__any_sync(full, *s_abort != 0 || global_timer_ns() - t0 > kWaitLimitNs)) {
            if (leader && *s_abort == 0) atomicOr(reinterpret_cast<int*>(p.ws), kErrWide);
            *s_abort = 1;
            ok = false;
          }
        }
        jt += n;
        ++n_seg;
      }
      if (!ok) {  // MMAs in flight: let them finish before tensor memory is freed
        mma_commit(&bars[B::kDone], leader);
        mbar_wait_bounded(&bars[B::kDone], 0);
      }
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) tmem_free_all(tbase);
}

template <int FMT, int D>
cudaError_t launch(const TreeArgs& a, int dev, cudaStream_t s) {
  using S = Wide<FMT, D>;
  static std::atomic<uint64_t> set;
  const cudaError_t e = allow_shared_memory(set, dev, tree_wide_kernel<FMT, D>, S::kBytes);
  if (e != cudaSuccess) return e;
  tree_wide_kernel<FMT, D><<<a.grid, kThreads, S::kBytes, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_wide(const TreeArgs& a, int dev, cudaStream_t s) {
  auto by_dim = [&](auto fmt) {
    constexpr int F = decltype(fmt)::value;
    return a.p.cache.head_dim == 64 ? launch<F, 64>(a, dev, s) : launch<F, 128>(a, dev, s);
  };
  switch (a.p.cache.format) {
    case QGEMV_KV_F16: return by_dim(std::integral_constant<int, QGEMV_KV_F16>());
    default: return by_dim(std::integral_constant<int, QGEMV_KV_INT8>());
  }
}

}  // namespace qgemv
