// attn_tree.cu -- attention of drafted tokens over the paged key/value cache
// (qgemv_attn_tree).
//
// Rows of a sequence and key/value head: row = token * G + head of the group.
// tree_kernel takes them in tiles of 8, 16, 24 or 32, by mma.sync; many rows
// of the fp16 and INT8 formats go to attn_tree_wide.cu.  A unit is a block of
// 16 cached tokens (tree_work.cuh); within a thread block's segment a warp
// takes every W-th unit:
//
//   copy      one bulk copy into the warp's own ring of shared-memory stages
//   S' = K Q' mma.m16n8k16, the unit's tokens its 16 rows and 8 query rows its
//             columns, so that the common eight rows (one token of a group of
//             8 heads) fill an instruction.  K straight from the block's
//             layout: stored bytes and nibbles are fp16 subnormals as they
//             stand (code + offset, times 2^-24), and the sums start at
//             -offset times the row's sum of q, so that a code pair costs one
//             instruction; the scales of the tokens (Q4_0: of each group, on
//             partial sums) go to S in fp32.  The sums are thus of the size of
//             offset * |sum q|, and their fp32 error with them: at most about
//             2^-23 max|k| sum|q| (measured on keys with one value that is not
//             0: 2^-26, INT8, and 2^-24, Q4_0), which is more than that of the
//             products alone where most of k is small
//   softmax   base 2, an own reference m for each warp and row that moves only
//             when a score passes it by 2^8: without a move no shuffle is
//             needed.  m is taken over s + log2(scale of v), because what is
//             rounded to fp16 is p * scale(v), the factor of v's codes: it
//             stays in [0, 2^8] whatever the scales are
//   O' += V' P' the same instruction, 16 values of the head its rows.  P'
//             is the scores' registers, transposed 8 x 8 between lanes.  V's
//             codes are exact in fp16 (their offsets are taken off first: here
//             sums run over all keys, and would not stay small beside the
//             offsets' share)
//
// A warp's O, m and l live in its registers.  At the end of a segment the
// warps' results are added in warp order through shared memory.
//
// Two sequences of 224000 tokens together, one token of 64 heads over 8: fp16
// 139 us (the bytes' floor 137), INT8 84 (71), Q4_0 69 (39).  fp16 and INT8
// stream at the copy bandwidth, with about 12 us of start, join and gap around
// it; Q4_0 is held up by instruction issue (decoding V, the products' scales).
// With the rows, not the tokens, along the products' 16 rows, half of an
// instruction was empty at 8 rows: INT8 88 us (Q4_0 of 252000 tokens 110
// against 76).
#include <algorithm>

#include "per_device.h"
#include "tc_common.cuh"
#include "tree_work.cuh"

namespace qgemv {
namespace {

constexpr int kNarrowRows = 32;  // rows of a pass, at most
constexpr int64_t kWholeTokens = 768;
constexpr int kErrTree = 32;
constexpr float kLazyT = 8.f;
constexpr int kRingBytes = 100 * 1024;
constexpr int kBlocksPerSm = 2;  // one's start and end of a row tile beside the other's stream

// c += a . b: 16 x 16 . 16 x 8, fp16 in, fp32 sums.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// c = a . b + z, z for columns 2 t and 2 t + 1
__device__ __forceinline__ void mma16816_from(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1, float z0, float z1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
               : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
               : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(z0), "f"(z1));
}
// c = a . b
__device__ __forceinline__ void mma16816_first(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
               : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(0.f));
}

// The transpose of an 8 x 8 matrix of 16-bit values, lane (g, t) holding row g, columns 2t and 2t + 1.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Per format: words of K and V of a lane, and the fp16 pairs in them.
template <int FMT, int D>
struct Codes;

template <int D>
struct Codes<QGEMV_KV_F16, D> {
  using L = KvLayout<QGEMV_KV_F16, D>;
  static constexpr int kKw = D / 8;
  static constexpr int kQ2 = 8;  // from the first pair of an operand's k to the second
  __device__ static int q_at(int ks, int t) { return 16 * ks + 2 * t; }
  __device__ static int out_at(int nb, int n) { return 8 * nb + n; }
  // ldmatrix: lane l gives the address of row l & 7 of matrix l >> 3
  __device__ static void load_k(const uint8_t* b, int tok, int lane, uint32_t (&w)[kKw]) {
    tok += (lane & 7) - (lane >> 2);  // of the eight tokens, this lane's row
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                   : "r"(smem_u32(b + L::k_off(tok, 64 * i + 16 * (lane >> 3)))));
  }
  __device__ static void k_frag(const uint32_t (&w)[kKw], int ks, uint32_t& b0, uint32_t& b1) {
    b0 = w[2 * ks], b1 = w[2 * ks + 1];
  }
  // matrices: tokens 0-7 and 8-15 of columns 16i .., then of 16i + 8 ..
  __device__ static void load_v(const uint8_t* b, int, int lane, uint32_t (&w)[4 * (D / 16)]) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
      asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                   : "r"(smem_u32(b + L::v_off(lane & 15, 32 * i + 16 * (lane >> 4)))));
  }
  __device__ static void v_frag(const uint32_t (&w)[4 * (D / 16)], int nb, uint32_t& b0, uint32_t& b1) {
    b0 = w[2 * nb], b1 = w[2 * nb + 1];
  }
};

template <int D>
struct Codes<QGEMV_KV_INT8, D> {
  using L = KvLayout<QGEMV_KV_INT8, D>;
  static constexpr int kKw = D / 16;
  static constexpr int kQ2 = 2;
  static constexpr uint32_t kOff0 = 0x80808080u, kOff1 = 0x80808080u;  // -128 * 2^-24
  __device__ static int q_at(int ks, int t) { return 64 * (ks >> 2) + 16 * t + 4 * (ks & 3); }
  __device__ static int out_at(int nb, int n) { return D / 8 * n + nb; }
  __device__ static void load_k(const uint8_t* b, int tok, int lane, uint32_t (&w)[kKw]) {
    const int t = lane & 3;
#pragma unroll
    for (int h = 0; h < D / 64; ++h) *reinterpret_cast<uint4*>(&w[4 * h]) = lds128(b + L::k_off(tok, 64 * h + 16 * t));
  }
  __device__ static void k_frag(const uint32_t (&w)[kKw], int ks, uint32_t& b0, uint32_t& b1) {
    b0 = prmt(w[ks], 0u, 0x4140), b1 = prmt(w[ks], 0u, 0x4342);
  }
  // V: [token][word]
  __device__ static void load_v(const uint8_t* b, int g, int lane, uint32_t (&w)[4 * (D / 32)]) {
    const int t = lane & 3;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint8_t* at = b + L::v_off(2 * t + (k & 1) + 8 * (k >> 1), D / 8 * g);
      if constexpr (D == 128) *reinterpret_cast<uint4*>(&w[4 * k]) = lds128(at);
      else *reinterpret_cast<uint2*>(&w[2 * k]) = *reinterpret_cast<const uint2*>(at);
    }
  }
  __device__ static void v_frag(const uint32_t (&w)[4 * (D / 32)], int nb, uint32_t& b0, uint32_t& b1) {
    constexpr int P = D / 32;
    const int e = nb >> 2, c = nb & 3;
    const uint32_t x = prmt(w[e], w[P + e], c & 2 ? 0x7362u : 0x5140u);
    const uint32_t y = prmt(w[2 * P + e], w[3 * P + e], c & 2 ? 0x7362u : 0x5140u);
    b0 = c & 1 ? i8_pair<0x4342>(x) : i8_pair<0x4140>(x);
    b1 = c & 1 ? i8_pair<0x4342>(y) : i8_pair<0x4140>(y);
  }
};

template <int D>
struct Codes<QGEMV_KV_Q4_0, D> {
  using L = KvLayout<QGEMV_KV_Q4_0, D>;
  static constexpr int kKw = D / 32;
  static constexpr int kQ2 = 2;
  static constexpr uint32_t kOff0 = 0x80088008u, kOff1 = 0x80808080u;  // -8 * 2^-24, and 16 times that
  __device__ static int q_at(int ks, int t) { return 32 * (ks >> 1) + 8 * t + 4 * (ks & 1); }
  __device__ static int out_at(int nb, int n) { return 32 * (nb >> 2) + 4 * n + (nb & 3); }
  __device__ static void load_k(const uint8_t* b, int tok, int lane, uint32_t (&w)[kKw]) {
    const uint8_t* at = b + L::k_off(tok, D / 8 * (lane & 3));
    if constexpr (D == 128) *reinterpret_cast<uint4*>(w) = lds128(at);
    else *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(at);
  }
  __device__ static void k_frag(const uint32_t (&w)[kKw], int ks, uint32_t& b0, uint32_t& b1) {
    const uint32_t x = ks & 1 ? w[ks >> 1] >> 8 : w[ks >> 1];
    b0 = x & 0x000F000Fu, b1 = x & 0x00F000F0u;  // the latter times 16
  }
  // V: [token][group pair]
  __device__ static void load_v(const uint8_t* b, int g, int lane, uint32_t (&w)[4 * (D / 64)]) {
    const int t = lane & 3;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint8_t* at = b + L::v_off(2 * t + (k & 1) + 8 * (k >> 1), D / 16 * g);
      if constexpr (D == 128) *reinterpret_cast<uint2*>(&w[2 * k]) = *reinterpret_cast<const uint2*>(at);
      else w[k] = *reinterpret_cast<const uint32_t*>(at);
    }
  }
  __device__ static void v_frag(const uint32_t (&w)[4 * (D / 64)], int nb, uint32_t& b0, uint32_t& b1) {
    constexpr int P = D / 64;
    const int grp = nb >> 2, e = grp >> 1;
    const uint32_t sel = grp & 1 ? 0x7632u : 0x5410u;
    const uint32_t x = prmt(w[e], w[P + e], sel), y = prmt(w[2 * P + e], w[3 * P + e], sel);
    switch (nb & 3) {
      case 0: b0 = q4_pair<0>(x), b1 = q4_pair<0>(y); break;
      case 1: b0 = q4_pair<1>(x), b1 = q4_pair<1>(y); break;
      case 2: b0 = q4_pair<2>(x), b1 = q4_pair<2>(y); break;
      default: b0 = q4_pair<3>(x), b1 = q4_pair<3>(y);
    }
  }
};

// Q4_0 scales of a token's groups, from `at`.
template <int D>
__device__ __forceinline__ void load_scales(const uint8_t* at, __half2 (&sc)[D / 64]) {
  if constexpr (D == 128) *reinterpret_cast<uint2*>(sc) = *reinterpret_cast<const uint2*>(at);
  else *reinterpret_cast<uint32_t*>(sc) = *reinterpret_cast<const uint32_t*>(at);
}

// Magnitude bits of a pair of fp16, the larger.
__device__ __forceinline__ uint32_t top_half(uint32_t w) { return max(w & 0x7fffu, (w >> 16) & 0x7fffu); }
// A pair of fp16 times f, in fp32, rounded to fp16.
__device__ __forceinline__ uint32_t scaled_pair(uint32_t w, float f) {
  return half_pair(h2f(w & 0xffffu) * f, h2f(w >> 16) * f);
}

// Shape of a kernel: W warps, NT tiles of 8 rows.
template <int FMT, int D, int NT>
struct TreeShape {
  using L = KvLayout<FMT, D>;
  static constexpr int kWarps = NT > 2 || FMT == QGEMV_KV_F16 ? 4 : NT == 2 && D == 128 ? 6 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kRows = 8 * NT;
  static constexpr int kFitting = kRingBytes / (kWarps * L::kBlock);
  static constexpr int kStages = kFitting > 6 ? 6 : kFitting;
  static constexpr int kRing = kWarps * kStages * L::kBlock;
  static constexpr int kPitch = D + 4;  // of a row of the warps' O: four rows' stores meet no bank twice
  static constexpr int kMerge = kWarps * kRows * kPitch * 4 + kRows * D * 2;  // the warps' O, then the rows as fp16
  static constexpr int kRegion = kRing > kMerge ? kRing : kMerge;
  static constexpr int kQ = (kRegion + 127) / 128 * 128;        // Q fragments
  static constexpr int kOffs = kQ + NT * (D / 16) * 256;        // the sums' starts, [group, INT8: all][row]
  static constexpr int kMl = kOffs + kRows * (FMT == QGEMV_KV_Q4_0 ? 16 : FMT == QGEMV_KV_INT8 ? 4 : 0);  // m, l of each warp and row
  static constexpr int kMask = kMl + kWarps * kRows * 8;        // mask words of the rows
  static constexpr int kBars = kMask + kRows * 8;
  static constexpr int kBytes = kBars + kWarps * kStages * 8 + 16;
};

template <int FMT, int D, int NT>
__global__ void __launch_bounds__(TreeShape<FMT, D, NT>::kThreads, kBlocksPerSm) tree_kernel(const TreeArgs a) {
  using Sh = TreeShape<FMT, D, NT>;
  using L = KvLayout<FMT, D>;
  using C = Codes<FMT, D>;
  constexpr int W = Sh::kWarps, NS = Sh::kStages, KS = D / 16, MB = D / 16;
  const TreeParams& p = a.p;
  extern __shared__ __align__(128) uint8_t smem[];
  uint4* s_q = reinterpret_cast<uint4*>(smem + Sh::kQ);  // [8 rows][two steps of k][lane]
  float* s_offs = reinterpret_cast<float*>(smem + Sh::kOffs);
  float2* s_ml = reinterpret_cast<float2*>(smem + Sh::kMl);
  uint64_t* s_mask = reinterpret_cast<uint64_t*>(smem + Sh::kMask);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sh::kBars);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const unsigned full = 0xffffffffu;

  allow_next_kernel();
  Cursor<Sh::kRows, kKvBlockTokens> work(a);
  uint64_t* my_bars = bars + warp * NS;
  uint8_t* my_ring = smem + warp * NS * L::kBlock;
  if (lane < NS) mbar_init(&my_bars[lane], 1);
  fence_mbarrier_init();
  __syncwarp();
  int ring_at = 0;           // stage of the next unit, and the
  uint32_t ring_parity = 0;  // parity of its landing

  Segment sg;
  while (work.next(a, sg)) {
    const int64_t u0 = sg.u0, u1 = sg.u1;
    const int seq = sg.seq, head = sg.head;
    const int R = sg.T * a.G, row0 = sg.tile * Sh::kRows;
    const int64_t q0 = p.cu_q[seq];
    const int ctx = sg.ctx, all = ctx + sg.T;
    const int32_t* table = table_row(p, seq, head);

    // ---- this warp's units: u0 + warp + W * k
    const int n_mine = static_cast<int>((u1 - u0 - warp + W - 1) / W);
    unsigned long long src_of = 0;  // lane l: the block of unit 32 * floor(k / 32) + l, 0 if its page is missing
    uint32_t have = 0;              // stages with a unit whose page exists
    auto prefetch = [&](int k, int st) {
      if ((k & 31) == 0) {
        const int64_t u = u0 + warp + static_cast<int64_t>(W) * (k + lane);
        const int64_t pi = (u * kKvBlockTokens) >> a.page_shift;
        src_of = 0;
        if (k + lane < n_mine && pi < p.table_stride) {
          const int page = __ldg(table + pi);
          if (page >= 0 && page < p.cache.n_pages)
            src_of = reinterpret_cast<unsigned long long>(
                kv_block<FMT, D>(p.cache, page, head, static_cast<int>(u & ((p.cache.page_tokens >> 4) - 1))));
        }
      }
      const unsigned long long src = __shfl_sync(full, src_of, k & 31);
      have = src ? have | 1u << st : have & ~(1u << st);
      if (lane == 0) {
        if (src) {
          mbar_arrive_expect_tx(&my_bars[st], L::kBlock);
          bulk_load(my_ring + st * L::kBlock, reinterpret_cast<const void*>(src), L::kBlock, &my_bars[st]);
        } else {
          mbar_arrive(&my_bars[st]);
        }
      }
    };
    // the ring goes on where the segment before left it
    auto stage_of = [&](int k) { return (ring_at + k) % NS; };
    // ---- Q fragments and masks of the row tile: loaded ahead of the first
    // copies' page lookups, stored after
    constexpr int kQAll = NT * KS / 2 * 32, kQPer = (kQAll + Sh::kThreads - 1) / Sh::kThreads;
    uint4 qf[kQPer];
#pragma unroll
    for (int x = 0; x < kQPer; ++x) {
      const int i = tid + x * Sh::kThreads;
      const int ln = i & 31, ks = 2 * ((i >> 5) % (KS / 2)), r = row0 + 8 * (i / (16 * KS)) + (ln >> 2);
      qf[x] = make_uint4(0u, 0u, 0u, 0u);
      if (r < R && i < kQAll) {
        const int tok = r / a.G;
        const __half* q = static_cast<const __half*>(p.q.ptr) + (q0 + tok) * p.q.token_stride +
                          (head * a.G + r - tok * a.G) * p.q.head_stride;
        auto at = [&](int d) { return __ldg(reinterpret_cast<const unsigned*>(q + d)); };
        const int d0 = C::q_at(ks, ln & 3), d1 = C::q_at(ks + 1, ln & 3);
        qf[x] = make_uint4(at(d0), at(d0 + C::kQ2), at(d1), at(d1 + C::kQ2));
      }
    }
    uint64_t row_mask = 0;
    if (tid < Sh::kRows && row0 + tid < R) {
      const int tok = (row0 + tid) / a.G;
      row_mask = p.masks ? p.masks[q0 + tok] : (~0ull >> (63 - tok));
    }
    for (int k = 0; k < NS && k < n_mine; ++k) prefetch(k, stage_of(k));
    // (codes as subnormals are 2^-24 of their values)
    float sl = p.scale * kLog2e * (FMT == QGEMV_KV_F16 ? 1.f : 16777216.f);
    if constexpr (FMT == QGEMV_KV_Q4_0) {
      // Half of the codes come times 16 (k_frag), so their q is divided by it.  The
      // tile's q are brought to 2^15 .. 2^16 by a power of 2 first, which the
      // scores' factor takes back: none loses bits but those below 2^-24 of the
      // largest.  (Codes shifted into place instead: two sequences of 224000
      // tokens, one row, 71.1 us against 69; a power for each row: 12 ragged ones
      // of 45 rows 84.8 against 83.8.)
      uint32_t* s_top = reinterpret_cast<uint32_t*>(s_offs);  // of each warp, until the sums' starts
      uint32_t top = 0;
#pragma unroll
      for (int x = 0; x < kQPer; ++x)
        top = max(top, max(max(top_half(qf[x].x), top_half(qf[x].y)), max(top_half(qf[x].z), top_half(qf[x].w))));
      top = __reduce_max_sync(full, top);
      if (lane == 0) s_top[warp] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < W; ++w) top = max(top, s_top[w]);
      // (zeros, infinities and NaN stay as they are)
      const int e = top == 0 || top >= 0x7C00u ? 0 : 15 - (static_cast<int>(__float_as_uint(h2f(top)) >> 23) - 127);
      const float f = __int_as_float((127 + e) << 23);
#pragma unroll
      for (int x = 0; x < kQPer; ++x) {
        qf[x].x = scaled_pair(qf[x].x, f), qf[x].z = scaled_pair(qf[x].z, f);
        qf[x].y = scaled_pair(qf[x].y, f * 0.0625f), qf[x].w = scaled_pair(qf[x].w, f * 0.0625f);
      }
      sl *= __int_as_float((127 - e) << 23);
    }
#pragma unroll
    for (int x = 0; x < kQPer; ++x)
      if (tid + x * Sh::kThreads < kQAll) s_q[tid + x * Sh::kThreads] = qf[x];
    if (tid < Sh::kRows) s_mask[tid] = row_mask;
    __syncthreads();

    // where the sums of S start: -offset * sum of q, by a product with constants
    if constexpr (FMT != QGEMV_KV_F16) {
      if (warp == 0) {
        const uint4 off = make_uint4(C::kOff0, C::kOff0, C::kOff1, C::kOff1);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          float c[4];
#pragma unroll
          for (int kp = 0; kp < KS / 2; ++kp) {
            const uint4 qb = s_q[(i * (KS / 2) + kp) * 32 + lane];
            if (kp == 0 || FMT == QGEMV_KV_Q4_0) mma16816_first(c, off, qb.x, qb.y);
            else mma16816(c, off, qb.x, qb.y);
            mma16816(c, off, qb.z, qb.w);
            const int grp = FMT == QGEMV_KV_Q4_0 ? kp : 0;
            if (g == 0 && (FMT == QGEMV_KV_Q4_0 || kp == KS / 2 - 1))
              *reinterpret_cast<float2*>(s_offs + grp * Sh::kRows + 8 * i + 2 * t) = make_float2(c[0], c[1]);
          }
        }
      }
      __syncthreads();
    }

    float o[NT][MB][4], m[NT][2], l[NT][2];  // values 16 b + g, + 8; rows 2t and 2t + 1 of each tile
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int n = 0; n < MB; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[i][n][c] = 0.f;
      m[i][0] = m[i][1] = -INFINITY;
      l[i][0] = l[i][1] = 0.f;
    }

    for (int k = 0; k < n_mine; ++k) {
      const int st = ring_at;
      const bool landed = mbar_wait_bounded(&my_bars[st], ring_parity);
      if (!__all_sync(full, landed)) {
        // Give up: record it, and let the copies in flight land (or their waits
        // run out too) before the ring is used for anything else.
        if (lane == 0) atomicOr(reinterpret_cast<int*>(p.ws), kErrTree);
        for (int x = 1; x < NS && k + x < n_mine; ++x)
          mbar_wait_bounded(&my_bars[(st + x) % NS], st + x < NS ? ring_parity : ring_parity ^ 1u);
        break;
      }
      if ((have >> st) & 1) {
        const uint8_t* blk = my_ring + st * L::kBlock;
        const int64_t pos0 = (u0 + warp + static_cast<int64_t>(W) * k) * kKvBlockTokens;
        const bool edge = pos0 + kKvBlockTokens > ctx;  // some positions are drafted, or past the end
        // ---- S: tokens g and g + 8 of the block, rows 2t and 2t + 1 of each tile
        float s[NT][4];
        {
          uint32_t kw[2][C::kKw];
          C::load_k(blk, g, lane, kw[0]);
          C::load_k(blk, 8 + g, lane, kw[1]);
          auto k_codes = [&](int ks) {
            uint4 r;
            C::k_frag(kw[0], ks, r.x, r.z);
            C::k_frag(kw[1], ks, r.y, r.w);
            return r;
          };
          if constexpr (FMT == QGEMV_KV_Q4_0) {
            // sums of each group, times the tokens' scales of the group
            alignas(8) __half2 ksc[2][D / 64];
            load_scales<D>(blk + L::kKs + g * (D / 16), ksc[0]);
            load_scales<D>(blk + L::kKs + (8 + g) * (D / 16), ksc[1]);
#pragma unroll
            for (int grp = 0; grp < D / 32; ++grp) {
              const uint4 k0 = k_codes(2 * grp), k1 = k_codes(2 * grp + 1);
              const float f0 = grp & 1 ? __high2float(ksc[0][grp >> 1]) : __low2float(ksc[0][grp >> 1]);
              const float f1 = grp & 1 ? __high2float(ksc[1][grp >> 1]) : __low2float(ksc[1][grp >> 1]);
#pragma unroll
              for (int i = 0; i < NT; ++i) {
                const uint4 qb = s_q[(i * (KS / 2) + grp) * 32 + lane];
                float part[4];
                const float2 from = *reinterpret_cast<const float2*>(s_offs + grp * Sh::kRows + 8 * i + 2 * t);
                mma16816_from(part, k0, qb.x, qb.y, from.x, from.y);
                mma16816(part, k1, qb.z, qb.w);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint64_t x = pack2(part[2 * h], part[2 * h + 1]), f = h ? pack2(f1, f1) : pack2(f0, f0);
                  unpack2(grp == 0 ? mul2(x, f) : fma2(x, f, pack2(s[i][2 * h], s[i][2 * h + 1])), s[i][2 * h], s[i][2 * h + 1]);
                }
              }
            }
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
              for (int h = 0; h < 2; ++h) unpack2(mul2(pack2(s[i][2 * h], s[i][2 * h + 1]), pack2(sl, sl)), s[i][2 * h], s[i][2 * h + 1]);
          } else {
#pragma unroll
            for (int kp = 0; kp < KS / 2; ++kp) {
              const uint4 k0 = k_codes(2 * kp), k1 = k_codes(2 * kp + 1);
#pragma unroll
              for (int i = 0; i < NT; ++i) {
                const uint4 qb = s_q[(i * (KS / 2) + kp) * 32 + lane];
                if (kp > 0) {
                  mma16816(s[i], k0, qb.x, qb.y);
                } else if (FMT == QGEMV_KV_INT8) {
                  const float2 from = *reinterpret_cast<const float2*>(s_offs + 8 * i + 2 * t);
                  mma16816_from(s[i], k0, qb.x, qb.y, from.x, from.y);
                } else {
                  mma16816_first(s[i], k0, qb.x, qb.y);
                }
                mma16816(s[i], k1, qb.z, qb.w);
              }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float ksc = sl;
              if constexpr (FMT == QGEMV_KV_INT8) ksc *= *reinterpret_cast<const float*>(blk + L::kKs + 4 * (8 * h + g));
#pragma unroll
              for (int i = 0; i < NT; ++i) unpack2(mul2(pack2(s[i][2 * h], s[i][2 * h + 1]), pack2(ksc, ksc)), s[i][2 * h], s[i][2 * h + 1]);
            }
          }
        }
        if (edge) {
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int64_t pos = pos0 + g + 8 * (c >> 1);
              const bool on = pos < ctx || (pos < all && ((s_mask[8 * i + 2 * t + (c & 1)] >> (pos - ctx)) & 1));
              if (!on) s[i][c] = -INFINITY;
            }
        }
        // ---- scales of V and the reference
        float vs[2][FMT == QGEMV_KV_Q4_0 ? D / 32 : 1], lv[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (FMT == QGEMV_KV_Q4_0) {
            alignas(8) __half2 vsc[D / 64];
            load_scales<D>(blk + L::kVs + (8 * h + g) * (D / 16), vsc);
            __half2 top = __habs2(vsc[0]);
            if constexpr (D == 128) top = __hmax2(top, __habs2(vsc[1]));
            lv[h] = lg2(fmaxf(fmaxf(__low2float(top), __high2float(top)), 7.9e-31f));  // 2^-100
#pragma unroll
            for (int x = 0; x < D / 32; ++x) vs[h][x] = x & 1 ? __high2float(vsc[x >> 1]) : __low2float(vsc[x >> 1]);
          } else if constexpr (FMT == QGEMV_KV_INT8) {
            vs[h][0] = *reinterpret_cast<const float*>(blk + L::kVs + 4 * (8 * h + g));
            lv[h] = lg2(fmaxf(vs[h][0], 7.9e-31f));
          } else {
            vs[h][0] = 1.f;
            lv[h] = 0.f;
          }
        }
        bool grow = false;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x, y;
            unpack2(add2(pack2(s[i][2 * h], s[i][2 * h + 1]), pack2(lv[h], lv[h])), x, y);
            grow |= x > m[i][0] + kLazyT || y > m[i][1] + kLazyT;
          }
        if (__any_sync(full, grow)) {
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float top = fmaxf(s[i][h] + lv[0], s[i][2 + h] + lv[1]);
#pragma unroll
              for (int x = 4; x < 32; x *= 2) top = fmaxf(top, __shfl_xor_sync(full, top, x));
              const float mn = fmaxf(m[i][h], top);
              const float f = m[i][h] == -INFINITY ? 0.f : ex2(m[i][h] - mn);
              m[i][h] = mn;
              l[i][h] *= f;
#pragma unroll
              for (int n = 0; n < MB; ++n) o[i][n][h] *= f, o[i][n][2 + h] *= f;
            }
        }
        // ---- P (in place of S); l takes p itself
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint64_t less = pack2(m[i][0] == -INFINITY ? 0.f : -m[i][0], m[i][1] == -INFINITY ? 0.f : -m[i][1]);
            float x, y;
            unpack2(add2(pack2(s[i][2 * h], s[i][2 * h + 1]), less), x, y);
            s[i][2 * h] = ex2(x), s[i][2 * h + 1] = ex2(y);
            unpack2(add2(pack2(l[i][0], l[i][1]), pack2(s[i][2 * h], s[i][2 * h + 1])), l[i][0], l[i][1]);
          }
        // p * scale(v).  Where a masked token's scale is infinite or NaN (past the
        // end it may be anything) the product is 0 all the same; a seen token's is
        // NaN, however small its p.
        uint32_t hidden = 0;  // bits [tile][c]: masked for the row; bit 31 where some lane's token is such a one
        if (FMT != QGEMV_KV_F16 && edge) {
          bool odd = false;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int x = 0; x < (FMT == QGEMV_KV_Q4_0 ? D / 32 : 1); ++x) odd |= !(fabsf(vs[h][x]) < INFINITY);
          if (__any_sync(full, odd)) {
            hidden = 1u << 31;
            for (int x = 0; x < 4 * NT; ++x) {
              const int64_t pos = pos0 + g + 8 * ((x >> 1) & 1);
              const bool on = pos < ctx || (pos < all && ((s_mask[8 * (x >> 2) + 2 * t + (x & 1)] >> (pos - ctx)) & 1));
              if (!on) hidden |= 1u << x;
            }
          }
        }
        // as the second operand: lane (g, t) row g, tokens 2t, 2t + 1 and 8 more
        auto weights = [&](int i, int x) -> uint2 {
          float w[4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint64_t pp = pack2(s[i][2 * h], s[i][2 * h + 1]);
            if (FMT != QGEMV_KV_F16) pp = mul2(pp, pack2(vs[h][x], vs[h][x]));
            unpack2(pp, w[2 * h], w[2 * h + 1]);
          }
          if (hidden) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if ((hidden >> (4 * i + c)) & 1) w[c] = 0.f;
          }
          return make_uint2(transpose8(half_pair(w[0], w[1])), transpose8(half_pair(w[2], w[3])));
        };
        // ---- O, its values the rows of the product
        uint32_t vw[4 * L::kRow / 32];
        C::load_v(blk, g, lane, vw);
        auto v_codes = [&](int n) {
          uint4 r;
          C::v_frag(vw, 2 * n, r.x, r.z);
          C::v_frag(vw, 2 * n + 1, r.y, r.w);
          return r;
        };
        uint2 pb[NT];
        if constexpr (FMT == QGEMV_KV_Q4_0) {
#pragma unroll
          for (int grp = 0; grp < D / 32; ++grp) {
#pragma unroll
            for (int i = 0; i < NT; ++i) pb[i] = weights(i, grp);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const uint4 v = v_codes(2 * grp + n);
#pragma unroll
              for (int i = 0; i < NT; ++i) mma16816(o[i][2 * grp + n], v, pb[i].x, pb[i].y);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < NT; ++i) pb[i] = weights(i, 0);
          if (FMT == QGEMV_KV_F16 && edge) {
            // fp16 values of positions past the end are whatever the page
            // holds: zero.  Infinities and NaN of drafted tokens reach the rows
            // that see them through a product of 0s and 1s instead.
            const uint32_t k01 = (pos0 + 2 * t < all ? 0xffffu : 0u) | (pos0 + 2 * t + 1 < all ? 0xffff0000u : 0u);
            const uint32_t k23 = (pos0 + 2 * t + 8 < all ? 0xffffu : 0u) | (pos0 + 2 * t + 9 < all ? 0xffff0000u : 0u);
#pragma unroll
            for (int n = 0; n < MB; ++n) {
              uint4 v = v_codes(n);
              v.x &= k01, v.y &= k01, v.z &= k23, v.w &= k23;
              auto bad = [](uint32_t x) { return ((x & 0x7C007C00u) + 0x04000400u) & 0x80008000u; };
              if (__any_sync(full, (bad(v.x) | bad(v.y) | bad(v.z) | bad(v.w)) != 0)) {
                for (int kind = 0; kind < 3; ++kind) {  // NaN, +inf, -inf
                  auto is = [&](uint32_t b) {
                    uint32_t r = 0;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                      const uint32_t x = (b >> (16 * h)) & 0xffffu;
                      const bool on = kind == 0 ? (x & 0x7fffu) > 0x7C00u : x == (kind == 1 ? 0x7C00u : 0xFC00u);
                      if (on) r |= 0x3C00u << (16 * h);
                    }
                    return r;
                  };
                  const uint4 which = make_uint4(is(v.x), is(v.y), is(v.z), is(v.w));
#pragma unroll
                  for (int i = 0; i < NT; ++i) {
                    auto sees = [&](int nb) {
                      uint32_t r = 0;
#pragma unroll
                      for (int e = 0; e < 2; ++e) {
                        const int64_t pos = pos0 + 8 * nb + 2 * t + e;
                        if (pos < ctx || (pos < all && ((s_mask[8 * i + g] >> (pos - ctx)) & 1))) r |= 0x3C00u << (16 * e);
                      }
                      return r;
                    };
                    float cnt[4];
                    mma16816_first(cnt, which, sees(0), sees(1));
                    const float val = __int_as_float(kind == 0 ? 0x7fffffff : kind == 1 ? 0x7f800000 : 0xff800000);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                      if (cnt[c] > 0.f) o[i][n][c] += val;
                  }
                }
                auto finite = [&](uint32_t x) {
                  if (bad(x) & 0x8000u) x &= 0xffff0000u;
                  if (bad(x) & 0x80000000u) x &= 0xffffu;
                  return x;
                };
                v = make_uint4(finite(v.x), finite(v.y), finite(v.z), finite(v.w));
              }
#pragma unroll
              for (int i = 0; i < NT; ++i) mma16816(o[i][n], v, pb[i].x, pb[i].y);
            }
          } else {
#pragma unroll
            for (int n = 0; n < MB; ++n) {
              const uint4 v = v_codes(n);
#pragma unroll
              for (int i = 0; i < NT; ++i) mma16816(o[i][n], v, pb[i].x, pb[i].y);
            }
          }
        }
      }
      __syncwarp();
      if (k + NS < n_mine) prefetch(k + NS, st);
      ring_at = st + 1 == NS ? 0 : st + 1;
      ring_parity ^= st + 1 == NS ? 1u : 0u;
    }

    // ---- the warps' results, in warp order
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int x = 4; x < 32; x *= 2) l[i][h] += __shfl_xor_sync(full, l[i][h], x);
    __syncthreads();  // every ring is empty
    float* s_o = reinterpret_cast<float*>(smem);  // [warp][row][value, as the products order them]
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int n = 0; n < MB; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          s_o[(warp * Sh::kRows + 8 * i + 2 * t + (c & 1)) * Sh::kPitch + 16 * n + 8 * (c >> 1) + g] = o[i][n][c];
      if (g == 0) {
        s_ml[warp * Sh::kRows + 8 * i + 2 * t] = make_float2(m[i][0], l[i][0]);
        s_ml[warp * Sh::kRows + 8 * i + 2 * t + 1] = make_float2(m[i][1], l[i][1]);
      }
    }
    __syncthreads();

    // four values of a row each
    constexpr int kVec = Sh::kRows * D / 4;
    constexpr int kPer = (kVec + Sh::kThreads - 1) / Sh::kThreads;
    float4 acc[kPer];
    float mm[kPer], ll[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      ll[j] = 0.f;
    }
    auto row_of = [&](int v) { return v / (D / 4); };
    auto to = [&](auto* dst, int v, float x, float y, float z, float w) {
      const int n = (v % (D / 4)) / 2, n0 = 4 * (v & 1);
      using T = std::remove_reference_t<decltype(*dst)>;
      dst[C::out_at(n, n0)] = static_cast<T>(x);
      dst[C::out_at(n, n0 + 1)] = static_cast<T>(y);
      dst[C::out_at(n, n0 + 2)] = static_cast<T>(z);
      dst[C::out_at(n, n0 + 3)] = static_cast<T>(w);
    };
    auto add = [&](int j, float pm, float pl, const float4& x, float top) {
      const float f = pm == -INFINITY ? 0.f : ex2(pm - top);
      ll[j] += pl * f;
      // a part with nothing adds nothing (its O is 0, and f too)
      acc[j].x += x.x * f, acc[j].y += x.y * f, acc[j].z += x.z * f, acc[j].w += x.w * f;
    };
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int v = tid + j * Sh::kThreads, row = row_of(v);
      if (v >= kVec) continue;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < W; ++w) top = fmaxf(top, s_ml[w * Sh::kRows + row].x);
      mm[j] = top;
      const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float2 ml = s_ml[w * Sh::kRows + row];
        add(j, ml.x, ml.y, *reinterpret_cast<const float4*>(s_o + (w * Sh::kRows + row) * Sh::kPitch + 4 * (v % (D / 4))), ref);
      }
    }

    if (sg.shared) {
      float* mine = tree_slot(p, blockIdx.x, u0 == 0, D);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int v = tid + j * Sh::kThreads, row = row_of(v);
        if (v >= kVec || row0 + row >= R) continue;
        to(mine + row * D, v, acc[j].x, acc[j].y, acc[j].z, acc[j].w);
        if (v % (D / 4) == 0) *reinterpret_cast<float2*>(mine + kSlotRows * D + 2 * row) = make_float2(mm[j], ll[j]);
      }
    } else {
      __half* s_out = reinterpret_cast<__half*>(smem + W * Sh::kRows * Sh::kPitch * 4);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int v = tid + j * Sh::kThreads, row = row_of(v);
        if (v >= kVec) continue;
        const float inv = ll[j] == 0.f ? 0.f : 1.f / ll[j];
        to(s_out + row * D, v, acc[j].x * inv, acc[j].y * inv, acc[j].z * inv, acc[j].w * inv);
        const int64_t r = row0 + row;
        if (p.lse && r < R && v % (D / 4) == 0) {
          const int tok = static_cast<int>(r) / a.G;
          p.lse[(q0 + tok) * p.q_heads + head * a.G + r - tok * a.G] = ll[j] == 0.f ? -INFINITY : (mm[j] + log2f(ll[j])) * kLn2;
        }
      }
      __syncthreads();
      for (int i = tid; i < Sh::kRows * D / 8; i += Sh::kThreads) {
        const int row = i / (D / 8), u = i % (D / 8), r = row0 + row;
        if (r < R) {
          const int tok = r / a.G;
          __half* out = static_cast<__half*>(p.out.ptr) + (q0 + tok) * p.out.token_stride +
                        (head * a.G + r - tok * a.G) * p.out.head_stride;
          *reinterpret_cast<uint4*>(out + 8 * u) = *reinterpret_cast<const uint4*>(s_out + row * D + 8 * u);
        }
      }
    }
    fence_async_smem();  // the ring is written by copies again
    __syncthreads();
  }
}

// Adds the parts of the rows that several blocks share: a warp for each row.
template <int ROWS, int UNIT, int D>
__global__ void __launch_bounds__(128) tree_join_kernel(const TreeArgs a) {
  const TreeParams& p = a.p;
  const int lane = threadIdx.x & 31, H = p.cache.kv_heads;
  const unsigned full = 0xffffffffu;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) >> 5;
  // Every thread waits for the main kernel, those with nothing to do too: what
  // follows this kernel on the stream may rely on both.
  auto leave = [] { wait_for_last_kernel(); };
  if (row >= p.n_q * p.q_heads) return leave();
  const int64_t token = row / p.q_heads;
  const int qh = static_cast<int>(row - token * p.q_heads), head = qh / a.G;
  // its sequence, and the units before it
  int64_t total = 0, base = 0;
  int seq = 0;
  for (int b = lane; b < p.n_seqs; b += 32) {
    const SeqWork s = seq_work<ROWS, UNIT>(a, b);
    const int64_t w = (s.units + a.extra) * s.tiles * H;
    total += w;
    if (__ldg(p.cu_q + b + 1) <= token) base += w, ++seq;
  }
  total = warp_total(total);
  base = warp_total(base);
  seq = static_cast<int>(warp_total(seq));
  if (seq >= p.n_seqs) return leave();
  const SeqWork s = seq_work<ROWS, UNIT>(a, seq);
  const int64_t i = token - __ldg(p.cu_q + seq);
  if (i < 0 || i >= s.T) return leave();
  const int64_t quota = run_quota(a, total);
  const int r = static_cast<int>(i) * a.G + qh - head * a.G;
  const int64_t first = base + (static_cast<int64_t>(head) * s.tiles + r / ROWS) * (s.units + a.extra) + a.extra;
  wait_for_last_kernel();
  const int b0 = static_cast<int>(div_small(first, quota)), b1 = static_cast<int>(div_small(first + s.units - 1, quota));
  if (b0 == b1) return;  // one block had it all
  float m = -INFINITY, l = 0.f, acc[D / 32];
#pragma unroll
  for (int c = 0; c < D / 32; ++c) acc[c] = 0.f;
  for (int c0 = b0; c0 <= b1; c0 += 32) {
    const int n = min(32, b1 - c0 + 1);
    // sixteen parts in flight at a time, the first beside their m and l
    float x[16][D / 32];
    auto fetch = [&](int k0) {
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        if (k0 + k >= n) break;
        const float* part = tree_slot(p, c0 + k0 + k, c0 + k0 + k == b0, D) + (r % ROWS) * D + lane * (D / 32);
        if constexpr (D == 128) *reinterpret_cast<float4*>(x[k]) = *reinterpret_cast<const float4*>(part);
        else *reinterpret_cast<float2*>(x[k]) = *reinterpret_cast<const float2*>(part);
      }
    };
    float2 ml = make_float2(-INFINITY, 0.f);
    const int mine = c0 + lane;
    if (mine <= b1)
      ml = *reinterpret_cast<const float2*>(tree_slot(p, mine, mine == b0, D) + kSlotRows * D + 2 * (r % ROWS));
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
    for (int k0 = 0; k0 < n; k0 += 16) {
      if (k0 > 0) fetch(k0);
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        if (k0 + k >= n) break;
        const float fk = __shfl_sync(full, f, k0 + k);
        l += __shfl_sync(full, ml.y, k0 + k) * fk;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) acc[c] += x[k][c] * fk;
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  __half* out = static_cast<__half*>(p.out.ptr) + token * p.out.token_stride + qh * p.out.head_stride + lane * (D / 32);
#pragma unroll
  for (int c = 0; c < D / 32; c += 2)
    *reinterpret_cast<uint32_t*>(out + c) = half_pair(acc[c] * inv, acc[c + 1] * inv);
  if (p.lse && lane == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <int FMT, int D, int NT>
cudaError_t launch(const TreeArgs& a, int dev, cudaStream_t s) {
  using Sh = TreeShape<FMT, D, NT>;
  static_assert(Sh::kStages >= 2 && Sh::kBytes <= 113 * 1024, "shared memory of a block");
  static std::atomic<uint64_t> set;
  const cudaError_t e = allow_shared_memory(set, dev, tree_kernel<FMT, D, NT>, Sh::kBytes);
  if (e != cudaSuccess) return e;
  tree_kernel<FMT, D, NT><<<a.grid, Sh::kThreads, Sh::kBytes, s>>>(a);
  return cudaGetLastError();
}

template <int ROWS, int UNIT>
cudaError_t launch_join(const TreeArgs& a, cudaStream_t s) {
  const int64_t rows = a.p.n_q * a.p.q_heads;
  const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
  return a.p.cache.head_dim == 64 ? launch_after(tree_join_kernel<ROWS, UNIT, 64>, grid, a, s)
                                  : launch_after(tree_join_kernel<ROWS, UNIT, 128>, grid, a, s);
}

}  // namespace

int64_t tree_ws_bytes(int head_dim) {
  return 2 * kMaxBlocks * slot_floats(head_dim) * static_cast<int64_t>(sizeof(float));
}

cudaError_t launch_attn_tree(const TreeParams& p, cudaStream_t s) {
  int dev = 0, sms = 0;
  const cudaError_t found = current_device(&dev, &sms);
  if (found != cudaSuccess) return found;
  TreeArgs a;
  a.p = p;
  a.G = p.q_heads / p.cache.kv_heads;
  a.page_shift = 0;
  while ((1 << a.page_shift) < p.cache.page_tokens) ++a.page_shift;
  a.grid = sms < kMaxBlocks ? sms : kMaxBlocks;
  // (hints may be 0: one token is the least that a call has)
  const int64_t rows = std::max<int64_t>(1, p.max_new) * a.G;
  // Up to 32 rows this file's kernel is faster on the whole (two sequences of up
  // to 131000 tokens, INT8: 8 rows 84 us against 146, 32 rows 120 against 152;
  // fp16 of 32 rows 152 against 149).  Beyond it needs several tiles and passes
  // over the cache.  fp16: the wide kernel is faster from there (those
  // sequences, 40 rows: 113 us against 133; 64 rows: 148 against 230).  INT8,
  // whose codes the wide kernel has to write out as fp16 first: two passes are
  // no slower on the whole (64 rows: 16 sequences of up to 16000 tokens 82 us
  // against 92, two of 131000 176 against 164), but for contexts that are not
  // split (one of up to 700: 20 against 18).
  // Contexts of up to kWholeTokens positions (as the caller bounds them) are
  // not split: a second kernel would take longer than the split saves (one
  // sequence and token, INT8: 700 positions 9.3 us against 10.3 split, 1000
  // positions 11.1 against 10.7).
  a.whole = static_cast<int64_t>(p.max_ctx) + p.max_new <= kWholeTokens;
  const int narrow = p.cache.format == QGEMV_KV_INT8 && !a.whole ? 2 * kNarrowRows : kNarrowRows;
  if (rows > narrow && p.cache.format != QGEMV_KV_Q4_0) {
    a.extra = 4;  // a row tile's start and end: about four units of 128 tokens
    a.min_units = 2 + a.extra;
    const cudaError_t e = launch_tree_wide(a, dev, s);
    return e != cudaSuccess || a.whole ? e : launch_join<64, 128>(a, s);
  }
  // Two blocks per SM, so that one's starts and ends of row tiles run beside
  // the other's stream: 64 ragged INT8 sequences of up to 4000 tokens 49 us
  // against 70 with one of twice the warps (many row tiles); a few long sequences lose up to 3%.
  a.grid = std::min(kBlocksPerSm * sms, kMaxBlocks);
  a.extra = 32;  // a row tile's start and end: about 32 units of 16 tokens (those 64 sequences: 64 us at 16, 49 at 32)
  a.min_units = 10 + a.extra;  // a block's share, at least (one sequence of 1500 tokens: 10.9 us, with 16 11.3)
  auto by_rows = [&](auto fmt, auto d) {
    constexpr int F = decltype(fmt)::value, D = decltype(d)::value;
    auto run = [&](auto nt) {
      constexpr int NT = decltype(nt)::value;
      const cudaError_t e = launch<F, D, NT>(a, dev, s);
      return e != cudaSuccess || a.whole ? e : launch_join<8 * NT, kKvBlockTokens>(a, s);
    };
    // the smallest tiles that take the rows in as few passes over the cache
    const int64_t tiles = (rows + kNarrowRows - 1) / kNarrowRows, each = (rows + tiles - 1) / tiles;
    if (each <= 8) return run(std::integral_constant<int, 1>());
    if (each <= 16) return run(std::integral_constant<int, 2>());
    if (each <= 24) return run(std::integral_constant<int, 3>());
    return run(std::integral_constant<int, 4>());
  };
  auto by_dim = [&](auto fmt) {
    return p.cache.head_dim == 64 ? by_rows(fmt, std::integral_constant<int, 64>())
                                  : by_rows(fmt, std::integral_constant<int, 128>());
  };
  switch (p.cache.format) {
    case QGEMV_KV_F16: return by_dim(std::integral_constant<int, QGEMV_KV_F16>());
    case QGEMV_KV_INT8: return by_dim(std::integral_constant<int, QGEMV_KV_INT8>());
    default: return by_dim(std::integral_constant<int, QGEMV_KV_Q4_0>());
  }
}

}  // namespace qgemv
