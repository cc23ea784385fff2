// fp8_paged_decode, fp8_block_decode: attention of the decode tokens over the 8-bit K/V cache, all
// pages of a sequence or the blocks (pages) that each token lists.
//
//   l_i = scale q . K_i,  out = sum_i softmax(l)_i V_i,  lse = ln sum_i exp(l_i)
//
// over the visible tokens i, K_i = 2^Ek code, V_i = 2^Ev code with one E for 32 tokens and a head.
//
// Bound: HBM, 256 bytes a cached token and KV head, while a tile has up to 32 rows (query heads of
// one KV head, for all decode tokens of the sequence); the tensor pipe above.
//
// Work.  A tile is 8 NT M rows of one KV head of one owner (a sequence; with block lists a token),
// a unit 32 cached tokens of it.  All units of all tiles form one list, cut into equal ranges, one
// a CTA, and those into one for each group of M warps.  A group's units come through a ring of
// shared-memory stages by tensor copies (TMA, 128-byte swizzle), sent for by four warps of their own
// (it would take a quarter of a computing warp's time); warps of different groups never wait for one
// another before the end.  So the ragged lengths of a batch balance to within a unit.  256 ragged
// contexts, 0.92 GB of pages, take 157 us as a graph: 5.9 TB/s with start, ends and joins.
//
// A unit in a warp (8 NT rows, everything in registers between the two products; tokens, then dims
// are the 16-row side of mma m16n8k16, so keys and values are widened once for all rows):
//   S^T = K q^T: E4M3 codes widen to f16 exactly, q (bf16, scaled by a power of two) too, so products
//     are exact and sums fp32.  The k index of the fragments is a permutation of the head's dims that
//     lets a lane read 32 consecutive bytes of a key; with the swizzle no two lanes of a
//     quarter-warp meet in a bank.
//   p = 2^((S g - m) f + 8), scale log2(e) 2^Ek = f g with f in [1, 2) and g a power of two: S g is
//     exact, and so is its difference to a near reference m, however large the logits are (a fused
//     multiply-add of S and the whole factor against a rounded product is off by 2^8 at logits of 9e7).
//     m moves only where a row's largest logit lies 2^7 above it, so a unit costs one vote and no
//     reduction.  z sums p in fp32; P is f16 (11 bits: 2^-12 of a weight; weights down to 2^-16 of the
//     largest keep all of them).
//   O^T += V^T P^T: weights of two rows are transposed in registers (movmatrix, 8 x 8); a pair of
//     tokens' bytes is put side by side by byte permutes and widened to f16x2, exact.  O is kept in
//     units of 2^Er, the largest 2^Ev met: 2^(Ev - Er) goes into the exponent of p (and out of z).
//     The product of a unit with Ev more than 6 below Er is scaled in fp32 before it is added.
// Such units, and those where some row does not see all 32 tokens (a sequence's end), take a second form
// of the step: scores are masked, and values that no row sees, and NaN codes, are kept from the product
// (clean() below).  Where Ev lies 2^30 above the first unit's, or 2^60 below Er and the sums have become
// small against Er, O gets a unit for which it and the product both stay fp32 numbers, by what the rows
// hold and what they give weight (renorm() below): a row keeps its sum beside blocks of any scale that it
// does not see, or gives no weight.  Batches of which a third of the blocks have scales 2^20 below the
// others take 210 us for 157, of scales 2^119 below 231.
// mma.sync, as scores become weights without leaving the registers: the tensor memory path (tcgen05)
// computes 128-row tiles from shared memory, and scores and weights would go through tensor and shared
// memory, with a wait each, for tiles that have 1 to 128 rows.
//
// Ranges cut tiles.  A group keeps the tile it ends in until all groups of the CTA are done; then
// pieces of the same tile are joined in shared memory.  Pieces of a tile in several CTAs go to the
// workspace and are joined by a second kernel, in the order of the list: results repeat bit for bit.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include <cuda.h>
#include <cudaTypedefs.h>  // PFN_cuTensorMapEncodeTiled

#include "fp8_kv.cuh"

namespace mx4 {

namespace {

constexpr int kWarps = 8;                        // that compute; four more bring the units
constexpr int kThreads = (kWarps + 4) * 32;
// Registers: 384 threads of 168 at the start, then 128 of 40 and 256 of 232 (the same 64512).
constexpr int kLoadRegs = 40, kComputeRegs = 232;
// Three columns of queries do not fit the registers beside O: they are read from shared memory, which
// leaves two stages a warp.
constexpr bool q_shared(int NT) { return NT == 3; }
constexpr int stages_of(int NT) { return q_shared(NT) ? 16 : 24; }  // of all groups of a CTA
constexpr int kStepBytes = 2 * kSub * kFp8Row;   // K rows, V rows of a unit
constexpr int kMaxOwners = 2048;                 // sequences of a launch (their prefix sums)
constexpr int kRecRow = kHeadDim + 4;            // floats of a row in shared memory: O, m, z, Er
constexpr int kFold = 6;                         // V scales this far below Er go into the weights
constexpr int kNoScale = -1000;                  // Er before the first unit
constexpr int kSpan = 30;                        // Er may grow by 2^kSpan beyond the first before renorm()
constexpr int kFar = 60;                         // V scales this far below Er need it too, where sums
constexpr float kHold = 40.f;                    // may have gone down by more than 2^kHold against Er
constexpr int kTop = 100;                        // it leaves numbers up to 2^kTop
constexpr int kMost = 29;                        // a unit's product is below 2^kMost: 32 weights of 2^15, 448
constexpr float kNoRef = -FLT_MAX;               // m before the first logit: no logit lies below it
constexpr float kUp = 8.f;                       // weights are 2^kUp at the reference
constexpr float kLazy = 7.f;                     // a weight may grow by 2^kLazy before m moves
constexpr int64_t kMinUnits = 8;                 // of a CTA: one for each group of one warp

// Shared memory, in bytes: stages | queries | barriers | sums | seg | jobs | units | Er |
// prefix sums.
template <int NT>
struct Layout {
  static constexpr int kQOff = stages_of(NT) * kStepBytes;  // [warp][NT][4][32 lanes] of 16 bytes
  static constexpr int kBarOff = kQOff + (q_shared(NT) ? kWarps * NT * 2048 : 0);
  static constexpr int kSumOff = kBarOff + 2 * stages_of(NT) * 8;
  static constexpr int kSegOff = kSumOff + 16 * 8;       // [group]: last tile, first tile if it began before
  static constexpr int kJobOff = kSegOff + kWarps * 8;   // tiles whose pieces are joined
  static constexpr int kUnitOff = kJobOff + (kWarps + 2) * 16;  // [group][64]: units looked up ahead
  static constexpr int kErOff = kUnitOff + kWarps * 64 * 16;  // [warp][8 NT]: Er of rows, where they differ
  static constexpr int kPrefOff = kErOff + kWarps * 8 * NT * 4;
  static constexpr int kBytes = kPrefOff + kMaxOwners * 8 + 1024;  // 1024: the stages' alignment
  static_assert(kUnitOff % 16 == 0 && kJobOff % 16 == 0 && kBytes <= 232448, "shared memory");
};

// Division of numbers below 2^31 by d >= 1: (mulhi(x, mul) + x) >> shift.
struct Div {
  uint32_t mul, shift, d;
  explicit Div(uint32_t v = 1) : d(v) {
    shift = 0;
    while ((1ull << shift) < v) ++shift;
    mul = (uint32_t)((((1ull << shift) - v) << 32) / v + 1);
  }
  __device__ __forceinline__ int operator()(uint32_t x) const { return (int)((__umulhi(x, mul) + x) >> shift); }
};

struct DecodeArgs {
  CUtensorMap kmap, vmap;
  const uint16_t* q;        // bf16 [T, H, 128]
  const uint8_t* ks;        // e8m0 [P, Hkv, 4]
  const uint8_t* vs;
  const int32_t* table;     // [B, W]
  int64_t W;
  const int32_t* seq_lens;  // [B]
  const int32_t* idx;       // [T, kb] (block lists) or null
  int kb;
  int64_t num_pages;
  int B, Q, H, Hkv, G;
  int R, TR, RT;            // rows of an owner and KV head, of a tile, tiles they take
  Div by_hr, by_rt, by_g, by_q, by_n;  // tiles of an owner, tiles of a head, G, Q, units of a list
  bool negative;            // |scale| log2(e) = fm 2^fe (1, and a zero's exponent, where that is 0)
  float fm, lazy, fl;       // fm in [1, 2), kLazy / fm, fm ln 2
  int fe;
  uint16_t* out;
  float* lse;
  float* rec;               // pieces: [CTA][0: of a tile begun before, 1: begun here][TR][128], m z Er
  float* scratch;           // [CTA][8 warps][8 NT][128], m z Er: tiles that a group ended but did not begin
  int32_t* meta;            // [CTA][2]: the tile that begins here and ends in a later CTA (-1: none), that CTA
  uint32_t* status;
};

// The list of units: how many a CTA takes, and where a group's range lies.
struct Cut {
  int64_t U, per;
  __device__ __forceinline__ int64_t lo(int64_t cta) const { return min(U, cta * per); }
  __device__ __forceinline__ int64_t group_lo(int64_t cta, int gi, int n) const {
    const int64_t a = lo(cta);
    return a + (lo(cta + 1) - a) * gi / n;
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D = A B + C, not volatile: the compiler may order products by their operands.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at));
  return v;
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {  // i known at compile time
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

__device__ __forceinline__ void sts128(uint32_t at, int4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// An 8 x 8 matrix of halves, row lane / 4 in the lanes: its transpose alike.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// (the pages leave L2 first: 256 ragged contexts 159 us for 164, 64 sequences of 20 rows 167 for 182)
__device__ __forceinline__ void tensor_copy(uint32_t dst, const CUtensorMap* map, int row, int head,
                                            int page, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%2, %3, %4, %5}], [%6], %7;\n" ::"r"(dst),
      "l"(map), "r"(0), "r"(row), "r"(head), "r"(page), "r"(bar), "l"(policy)
      : "memory");
}

// A warp's part of a tile: 8 NT rows.  Lane (g, c) = (lane / 4, lane % 4) holds, of rows 8 t + 2 c + e
// (e = 0, 1), dims 16 g .. 16 g + 15 of O: o[j][t][e] dim 16 g + 2 j, o[j][t][2 + e] dim 16 g + 2 j + 1.
template <int NT>
struct Rows {
  static constexpr bool QS = q_shared(NT);
  uint32_t qb[QS ? 1 : NT][8][2];     // row 8 t + g, dims 32 c + 4 j + {0, 1}, + {2, 3}
  uint32_t qs;                        // QS: where the lane's are, two j's together, 512 bytes apart
  float o[8][NT][4];
  float m[NT][2], z[NT][2];            // reference (a score in units of g), sum
  int fe[NT][2];                       // g = 2^(fe + Ek)
  int er;                              // O is in units of 2^er
  int cap;                             // the largest scale byte that needs no renorm(); -1: rows have Er of
  uint32_t er_at;                      // their own, here
  float hold;                          // what a row's sum has gone down by against er, at most (log2)

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j][t][0] = o[j][t][1] = o[j][t][2] = o[j][t][3] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[t][e] = kNoRef;
        z[t][e] = 0.f;
      }
    }
    er = kNoScale;
    cap = 254;
    hold = 0.f;
  }
  __device__ __forceinline__ int row_er(int r) const {
    int x = er;
    if (cap < 0) asm volatile("ld.shared.s32 %0, [%1];" : "=r"(x) : "r"(er_at + r * 4) : "memory");
    return x;
  }

  // q rows -> f16 fragments, scaled so that a row's largest element lies in [2^14, 2^15) (exact, but
  // for elements 2^-29 of it; rows whose largest is below 2^-86 lose bits).  v: 32 dims of row 8 t + g.
  __device__ __forceinline__ void set_q(const uint4 (&v)[NT][4], const DecodeArgs& a, int lane) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      uint32_t am = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t w = word(v[t][i >> 2], i & 3);
        am = max(am, max((w << 17) >> 1, w & 0x7FFF0000u));
      }
      am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
      am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
      const int sigma = am == 0u ? 0 : min(100, max(-113, 14 - ((int)(am >> 23) - 127)));
      const float up = __uint_as_float((uint32_t)(127 + sigma) << 23) * (a.negative ? -1.f : 1.f);
#pragma unroll
      for (int e = 0; e < 2; ++e) fe[t][e] = __shfl_sync(0xFFFFFFFFu, a.fe - sigma, (2 * (lane & 3) + e) * 4);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        uint32_t x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = word(v[t][j >> 1], i);
          x[i] = half2_bits(bf16_bits_to_float(w & 0xFFFFu) * up, bf16_bits_to_float(w >> 16) * up);
        }
        if constexpr (QS) {
          sts128(qs + (t * 4 + j / 2) * 512, make_int4(x[0], x[1], x[2], x[3]));
        } else {
          qb[t][j][0] = x[0], qb[t][j][1] = x[1], qb[t][j + 1][0] = x[2], qb[t][j + 1][1] = x[3];
        }
      }
    }
  }

  // One unit: 32 tokens from position tb on, K rows at ka and V rows at va (shared memory), scale
  // bytes kb and vb.  General: some row does not see all of them, or Ev is far below er, or NaN;
  // lim(row of the warp) is then a row's last visible token, max_lim the last that any sees.
  template <bool General, class Lim>
  __device__ __forceinline__ void step(uint32_t ka, uint32_t va, int kb, int vb, int tb, int lane, Lim lim,
                                       int max_lim, const DecodeArgs& a) {
    const int g = lane >> 2, c = lane & 3;
    float s[2][NT][4];  // tokens 16 i + g (rows 2 c, 2 c + 1), then 16 i + g + 8
    constexpr int kI = QS ? 2 : 1;  // 16 tokens at a time, or all: queries are then read once
#pragma unroll
    for (int i0 = 0; i0 < 2; i0 += kI) {
      uint4 x[kI][2][2];
#pragma unroll
      for (int i = 0; i < kI; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t at = ka + (16 * (i0 + i) + 8 * h + g) * kFp8Row;
          x[i][h][0] = lds128(at + (((2 * c) ^ g) << 4));
          x[i][h][1] = lds128(at + (((2 * c + 1) ^ g) << 4));
        }
      uint4 q[NT];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (QS)
          if (j % 2 == 0)
#pragma unroll
            for (int t = 0; t < NT; ++t) q[t] = lds128(qs + (t * 4 + j / 2) * 512);
#pragma unroll
        for (int i = 0; i < kI; ++i) {
          uint32_t k[4];
          e4m3x4_f16x2(word(x[i][0][j >> 2], j & 3), k[0], k[2]);
          e4m3x4_f16x2(word(x[i][1][j >> 2], j & 3), k[1], k[3]);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint32_t b0 = QS ? word(q[t], 2 * (j & 1)) : qb[QS ? 0 : t][j][0];
            const uint32_t b1 = QS ? word(q[t], 2 * (j & 1) + 1) : qb[QS ? 0 : t][j][1];
            if (j == 0) mma0(s[i0 + i][t], k, b0, b1); else mma(s[i0 + i][t], k, b0, b1);
          }
        }
      }
    }
    // factors stay normal numbers (a score of 0 is a logit of 0 whatever the scales) or NaN
    float gk[NT][2], top[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        gk[t][e] = __int_as_float(kb == 255 ? 0x7FC00000 : min(max(fe[t][e] + kb, 1), 254) << 23);
    if constexpr (General) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int rel = lim(8 * t + 2 * c + e) - tb;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (8 * i + g > rel) s[i >> 1][t][2 * (i & 1) + e] = -INFINITY;
          if (rel < 0) gk[t][e] = FLT_MIN;  // no NaN from a scale that the row does not see
        }
    }
    bool above = false;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        top[t][e] = fmaxf(fmaxf(s[0][t][e], s[0][t][2 + e]), fmaxf(s[1][t][e], s[1][t][2 + e])) * gk[t][e];
        above |= top[t][e] - m[t][e] > a.lazy;
      }
    if (__any_sync(0xFFFFFFFFu, above)) {
      float most = 0.f;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = top[t][e];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
          if (x - m[t][e] > a.lazy) {
            const float by = (x - m[t][e]) * a.fm, down = ex2(-by);
            if (m[t][e] != kNoRef) most = fmaxf(most, by);
            m[t][e] = x;
            z[t][e] *= down;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              o[j][t][e] *= down;
              o[j][t][2 + e] *= down;
            }
          }
        }
      most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
      hold += fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
    }
    const bool far = General && vb != 255 && (vb > cap || (vb - 127 < er - kFar && hold > kHold));
    if (vb - 127 > er && vb != 255 && !far) {  // O to the new unit (nothing is in it before the first)
      const float down = er == kNoScale ? 0.f : ex2((float)(er - vb + 127));
      hold = er == kNoScale ? 0.f : hold + (float)(vb - 127 - er);
      if (er == kNoScale) cap = min(254, vb + kSpan);
      er = vb - 127;
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][t][e] *= down;
    }
    const int fold = General ? 0 : vb - 127 - er;
    const float up = kUp + (float)fold, back = __int_as_float((127 - fold) << 23);
    uint32_t p[4][NT];  // tokens 8 i + 2 c, + 1 of row 8 t + g
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float w[2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[e][i] = ex2(fmaf(fmaf(s[i >> 1][t][2 * (i & 1) + e], gk[t][e], -m[t][e]), a.fm, up));
        z[t][e] = fmaf((w[e][0] + w[e][1]) + (w[e][2] + w[e][3]), back, z[t][e]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i][t] = transpose8(half2_bits(w[0][i], w[1][i]));
    }
    float ev[General ? NT : 1][2];  // 2^(Ev - Er); 0 for rows that see none: a scale of NaN is not theirs
    if constexpr (General) {
      if (far) renorm(p, vb - 127, lane, lim);
      const float all = vb == 255 ? e8m0_to_float(255) : ex2(fminf((float)(vb - 127 - er), 127.f));
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) ev[t][e] = lim(8 * t + 2 * c + e) < tb ? 0.f : all;
      if (cap < 0 && vb != 255) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (lim(8 * t + 2 * c + e) >= tb) ev[t][e] = ex2(fminf((float)(vb - 127 - row_er(8 * t + 2 * c + e)), 127.f));
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint4 y[4];  // tokens 16 k + 2 c + {0, 1, 8, 9}, dims 16 g .. 16 g + 15
#pragma unroll
      for (int i = 0; i < 4; ++i)
        y[i] = lds128(va + (16 * k + 2 * c + (i & 1) + 8 * (i >> 1)) * kFp8Row + ((g ^ (2 * c + (i & 1))) << 4));
      if constexpr (General) clean(y, 16 * k + 2 * c, tb, c, lim, max_lim);
      if constexpr (!General) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t v[4];
          values(y, j, v);
#pragma unroll
          for (int t = 0; t < NT; ++t) mma(o[j][t], v, p[2 * k][t], p[2 * k + 1][t]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t v[4];
          values(y, j, v);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float x[4];
            mma0(x, v, p[2 * k][t], p[2 * k + 1][t]);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][t][e] = fmaf(ev[t][e & 1], x[e], o[j][t][e]);
          }
        }
      }
    }
  }

  // O to a unit in which it, and the product to come of weights p and values of scale 2^ev, is below
  // 2^(kTop + 1): the least such unit, so that what is far smaller stays too.  One for all rows where
  // theirs lie within 2^90, else one each; rows without weight here do not count the product, and
  // those that see nothing at all (lim) count for nothing.
  template <class Lim>
  __device__ __forceinline__ void renorm(const uint32_t (&p)[4][NT], int ev, int lane, Lim lim) {
    const int c = lane & 3;
    int want[NT][2], most = kNoScale, least = 1 << 20, held = 1 << 20;  // held: sums are 2^held at least
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      uint32_t any = p[0][t] | p[1][t] | p[2][t] | p[3][t];  // of row 8 t + g
      any |= __shfl_xor_sync(0xFFFFFFFFu, any, 1);
      any |= __shfl_xor_sync(0xFFFFFFFFu, any, 2);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool weight = __shfl_sync(0xFFFFFFFFu, any, (2 * c + e) * 4) != 0u;
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, fmaxf(fabsf(o[j][t][e]), fabsf(o[j][t][2 + e])));
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        int x = kNoScale;
        if (lim(8 * t + 2 * c + e) >= 0) {
          if (top > 0.f) {  // (kNoScale / 2: below any result)
            x = max(row_er(8 * t + 2 * c + e) + (int)(__float_as_uint(top) >> 23) - 127 - kTop, kNoScale / 2);
            held = min(held, x + kTop);
          } else if (weight) {
            held = min(held, ev - 33);  // a weight of 2^-24 and a code of 2^-9
          }
          if (weight) x = max(x, ev + kMost - kTop);
          if (x != kNoScale) least = min(least, x);
        }
        want[t][e] = x;
        most = max(most, x);
      }
    }
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    least = __reduce_min_sync(0xFFFFFFFFu, least);
    held = __reduce_min_sync(0xFFFFFFFFu, held);
    const bool same = most - least <= 90;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (same) want[t][e] = most;
        const int r = 8 * t + 2 * c + e, old = row_er(r);
        const int up = old == kNoScale || want[t][e] == kNoScale ? 0 : min(252, max(-252, old - want[t][e]));
        const float f0 = __int_as_float((127 + up / 2) << 23), f1 = __int_as_float((127 + up - up / 2) << 23);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[j][t][e] = o[j][t][e] * f0 * f1;
          o[j][t][2 + e] = o[j][t][2 + e] * f0 * f1;
        }
      }
    __syncwarp();
    if (!same && lane < 4)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          asm volatile("st.shared.s32 [%0], %1;" ::"r"(er_at + (8 * t + 2 * c + e) * 4), "r"(want[t][e]) : "memory");
    __syncwarp();
    er = most;
    hold = (float)(most - held);
    // (sums of 2^10 and more may go down by 2^101 before the next time)
    cap = !same ? -1 : most == kNoScale ? 254 : min(254, most + 127 + kTop - kMost + kSpan);
  }

  // Dims 2 j, 2 j + 1 of the lane's as f16: tokens 2 c, 2 c + 1 of the four, then 2 c + 8, 2 c + 9.
  __device__ __forceinline__ void values(const uint4 (&y)[4], int j, uint32_t (&v)[4]) const {
    const uint32_t sel = (j & 1) ? 0x7362 : 0x5140;
    e4m3x4_f16x2(__byte_perm(word(y[0], j >> 1), word(y[1], j >> 1), sel), v[0], v[1]);
    e4m3x4_f16x2(__byte_perm(word(y[2], j >> 1), word(y[3], j >> 1), sel), v[2], v[3]);
  }

  // V rows of a tail (tokens r0 + {0, 1, 8, 9} of the unit): those that no row of the warp sees become
  // zeros (they may hold anything), and so do NaN codes, whose weight of 0 would carry them to rows
  // that do not see them; O of the rows that do becomes NaN here (a row sees a prefix of the tokens,
  // so the first NaN of a dim decides).
  template <class Lim>
  __device__ __forceinline__ void clean(uint4 (&y)[4], int r0, int tb, int c, Lim lim, int max_lim) {
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (tb + r0 + (i & 1) + 8 * (i >> 1) > max_lim) y[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) any |= ((word(y[i], j) & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    }
    if (!__any_sync(0xFFFFFFFFu, any != 0)) return;
#pragma unroll
    for (int d = 0; d < 16; ++d) {
      int first = 32;
#pragma unroll
      for (int i = 3; i >= 0; --i)
        if (((word(y[i], d >> 2) >> (8 * (d & 3))) & 0x7F) == 0x7F) first = r0 + (i & 1) + 8 * (i >> 1);
      first = min(first, __shfl_xor_sync(0xFFFFFFFFu, first, 1));
      first = min(first, __shfl_xor_sync(0xFFFFFFFFu, first, 2));
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (first < 32 && tb + first <= lim(8 * t + 2 * c + e)) o[d >> 1][t][2 * (d & 1) + e] = __uint_as_float(0x7FC00000u);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i].x = drop_nan(y[i].x);
      y[i].y = drop_nan(y[i].y);
      y[i].z = drop_nan(y[i].z);
      y[i].w = drop_nan(y[i].w);
    }
  }
  static __device__ __forceinline__ uint32_t drop_nan(uint32_t w) {
    const uint32_t n = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    return w & ~((n >> 7) * 0xFFu);
  }

  __device__ __forceinline__ void sum_z() {  // over the lanes of a row
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) z[t][e] += __shfl_xor_sync(0xFFFFFFFFu, z[t][e], d);
  }
  // rows of the warp: O to p (row_floats a row), reference, sum and unit to mz (mz_floats a row)
  __device__ __forceinline__ void put(float* p, int row_floats, float* mz, int mz_floats, int lane) const {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * t + 2 * c + e;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(p + r * row_floats + 16 * g + 4 * i) =
              make_float4(o[2 * i][t][e], o[2 * i][t][2 + e], o[2 * i + 1][t][e], o[2 * i + 1][t][2 + e]);
        if (g == 0) *reinterpret_cast<float4*>(mz + r * mz_floats) = make_float4(m[t][e], z[t][e], (float)row_er(r), 0.f);
      }
  }
};

// A finished row from O (units 2^(m - kUp + er)), m and z: O / z first, then its unit (2^er / z may lie
// below fp32's range where the result does not), and the lse.
struct Finish {
  float inv, unit, rest;
  __device__ __forceinline__ Finish(float z, float er) {
    const int e = (int)er, e0 = min(max(e, -126), 127), e1 = max(e - e0, -126);
    inv = z == 0.f ? 0.f : 1.f / z;
    unit = __int_as_float((e0 + 127) << 23);
    rest = __int_as_float((e1 + 127) << 23);
  }
  __device__ __forceinline__ float operator()(float o) const { return o * inv * unit * rest; }
};
__device__ __forceinline__ float row_lse(const DecodeArgs& a, float m, float z) {
  return z == 0.f ? -INFINITY : fmaf(m, a.fl, (log2f(z) - kUp) * 0.69314718f);
}

struct Tile {
  int owner, head, rt;
};
__device__ __forceinline__ Tile tile_of(const DecodeArgs& a, int tile) {
  Tile t;
  t.owner = a.by_hr(tile);
  const int r = tile - t.owner * (int)a.by_hr.d;
  t.head = a.by_rt(r);
  t.rt = r - t.head * a.RT;
  return t;
}

// Row r of a tile's owner: the decode token and query head it is.
template <bool Lists>
__device__ __forceinline__ int64_t row_of(const DecodeArgs& a, const Tile& t, int r) {
  const int j = Lists ? 0 : a.by_g(r);
  const int64_t tok = Lists ? t.owner : (int64_t)t.owner * a.Q + j;
  return tok * a.H + t.head * a.G + (r - j * a.G);
}

// A row's sum of pieces, mz = (m, z, er, -) of each.
struct Joined {
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float z = 0.f, m = kNoRef, er = kNoScale;
  // All pieces, before the first is added.  er: the largest of theirs, each less what its weights go
  // down by, so that a large unit without weight takes nothing from the others.
  __device__ __forceinline__ void see(float x, float unit, float fm) {
    const float top = fmaxf(m, x);
    er = fmaxf(er + (m - top) * fm, unit + (x - top) * fm);
    m = top;
  }
  __device__ __forceinline__ void see(float4 mz, float fm) { see(mz.x, mz.z, fm); }
  __device__ __forceinline__ void seen() { er = rintf(fmaxf(er, (float)kNoScale)); }  // a whole power of two
  __device__ __forceinline__ void add(float4 v, float4 mz, float fm) {
    const float d = (mz.x - m) * fm, fo = ex2(0.5f * (d + (mz.z - er)));  // twice: large sums of small units
    z = fmaf(ex2(d), mz.y, z);
    acc.x = fmaf(fo, fo * v.x, acc.x);
    acc.y = fmaf(fo, fo * v.y, acc.y);
    acc.z = fmaf(fo, fo * v.z, acc.z);
    acc.w = fmaf(fo, fo * v.w, acc.w);
  }
};
template <bool Lists>
__device__ __forceinline__ void put_row(const DecodeArgs& a, const Tile& t, int row, const Joined& j, int lane) {
  const Finish f(j.z, j.er);
  const int64_t at = row_of<Lists>(a, t, row);
  *reinterpret_cast<uint2*>(a.out + at * kHeadDim + 4 * lane) =
      make_uint2(bf16x2_bits(f(j.acc.x), f(j.acc.y)), bf16x2_bits(f(j.acc.z), f(j.acc.w)));
  if (a.lse && lane == 0) a.lse[at] = row_lse(a, j.m, j.z);
}

// The owner that unit u belongs to: pref sums the owners' units, HR tiles each.
__device__ __forceinline__ int owner_of(const int64_t* pref, int B, int HR, int64_t u) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pref[mid] * HR > u) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Unit u: its tile, first token, KV head and the table's entry (-2 where the unit is skipped).
struct Look {
  int tile, tb, head, page;
};
template <bool Lists>
__device__ __forceinline__ Look look_up(const DecodeArgs& a, const int64_t* pref, int HR, int64_t u) {
  Look r{0, 0, 0, -2};
  int owner;
  if (Lists) {
    const uint32_t n = a.kb * kPageSubs;
    r.tile = (u >> 31) ? (int)(u / n) : a.by_n((uint32_t)u);
    const int i = (int)(u - (int64_t)r.tile * n);
    const Tile t = tile_of(a, r.tile);
    owner = a.by_q(t.owner);
    r.head = t.head;
    const int b = a.idx[(int64_t)t.owner * a.kb + i / kPageSubs];
    const int64_t L = a.seq_lens[owner];
    const int64_t p = L - a.Q + (t.owner - owner * a.Q);
    if (b < 0 || L < 0 || L > a.W * kPageTokens) return r;
    if (p < 0 || b > p / kPageTokens) {
      flag(a.status, MX4_STATUS_BAD_INDEX);
      return r;
    }
    r.tb = b * kPageTokens + (i % kPageSubs) * kSub;
    if (r.tb > p) return r;
  } else {
    owner = owner_of(pref, a.B, HR, u);
    const int64_t before = owner ? pref[owner - 1] : 0;
    const uint32_t n = (uint32_t)(pref[owner] - before), v = (uint32_t)(u - before * HR);  // < 2^28
    const uint32_t in = v / n;
    r.tile = owner * HR + (int)in;
    r.head = a.by_rt(in);
    r.tb = (int)(v - in * n) * kSub;
  }
  r.page = a.table[(int64_t)owner * a.W + r.tb / kPageTokens];
  if (r.page < 0 || r.page >= a.num_pages) {
    flag(a.status, MX4_STATUS_BAD_PAGE);
    r.page = -2;
  }
  return r;
}

// K's and V's scale of a looked-up unit; (0, 0) where it is skipped.
__device__ __forceinline__ int2 scales_of(const DecodeArgs& a, const Look& l) {
  if (l.page < 0) return make_int2(0, 0);
  const int64_t at = ((int64_t)l.page * a.Hkv + l.head) * kPageSubs + (l.tb % kPageTokens) / kSub;
  return make_int2(a.ks[at], a.vs[at]);
}

// The barrier's transactions, ahead of the arrival.
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_done(uint32_t bar, uint32_t parity) {  // does not wait
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0u;
}
__device__ __forceinline__ void compute_sync() {  // the computing warps
  asm volatile("bar.sync 1, %0;\n" ::"n"(kWarps * 32) : "memory");
}

// One warp brings the units of one or two groups: looks them up 32 at a time, a lane each, keeps them
// in a ring of 64 for the group to read (tile, first token, page or -2, scales and head), and sends
// for a unit's rows as soon as its stage is free.
template <int NT, bool Lists, int NG, int S>
__device__ __forceinline__ void load_units(const DecodeArgs& a, const Cut& cut, const int64_t* pref, int HR,
                                           uint32_t base_at, int which, int lane) {
  using Lay = Layout<NT>;
  constexpr int GP = NG > 4 ? 2 : 1;
  if (which >= NG) return;
  int64_t u0[GP];
  int n[GP], next[GP];
  auto full = [&](int j) { return base_at + Lay::kBarOff + (which + 4 * j) * S * 8; };
  auto units = [&](int j) { return base_at + Lay::kUnitOff + (which + 4 * j) * 1024; };
  auto send = [&](int j, int st, int page, int tb, int head) {
    const uint64_t policy = read_once();
    const uint32_t bar = full(j) + st * 8, dst = base_at + ((which + 4 * j) * S + st) * kStepBytes;
    tensor_copy(dst, &a.kmap, tb % kPageTokens, head, page, bar, policy);
    tensor_copy(dst + kSub * kFp8Row, &a.vmap, tb % kPageTokens, head, page, bar, policy);
  };
#pragma unroll
  for (int j = 0; j < GP; ++j) {
    u0[j] = cut.group_lo(blockIdx.x, which + 4 * j, NG);
    n[j] = (int)(cut.group_lo(blockIdx.x, which + 4 * j + 1, NG) - u0[j]);
    next[j] = min(S, n[j]);
    Look l{0, 0, 0, -2};
    if (lane < n[j]) l = look_up<Lists>(a, pref, HR, u0[j] + lane);
    // The scales are asked for ahead of the rows (behind the rows of all SMs they came 3 us later); the
    // arrival, which the group waits for, follows when they are there.
    const int2 sc = scales_of(a, l);
    if (lane < next[j] && l.page >= 0) {
      mbar_expect_tx(full(j) + lane * 8, kStepBytes);
      send(j, lane, l.page, l.tb, l.head);
    }
    sts128(units(j) + lane * 16, make_int4(l.tile, l.tb, l.page, sc.x | (sc.y << 8) | (l.head << 16)));
    __syncwarp();
    if (lane < next[j]) mbar_arrive(full(j) + lane * 8);
  }
  uint32_t idle = 0;
  for (bool more = true; more;) {
    more = false;
    bool did = false;
#pragma unroll
    for (int j = 0; j < GP; ++j) {
      const int k = next[j];
      if (k >= n[j]) continue;
      more = true;
      const int st = k % S;
      if (!__all_sync(0xFFFFFFFFu, mbar_done(full(j) + (stages_of(NT) + st) * 8, (k / S - 1) & 1))) continue;
      if ((k & 31) == 0) {  // the next 32
        Look l{0, 0, 0, -2};
        if (k + lane < n[j]) l = look_up<Lists>(a, pref, HR, u0[j] + k + lane);
        const int2 sc = scales_of(a, l);
        sts128(units(j) + ((k + lane) & 63) * 16, make_int4(l.tile, l.tb, l.page, sc.x | (sc.y << 8) | (l.head << 16)));
        __syncwarp();
      }
      if (lane == 0) {
        const uint4 x = lds128(units(j) + (k & 63) * 16);
        const uint32_t bar = full(j) + st * 8;
        if ((int)x.z >= 0) {
          mbar_arrive_expect_tx(bar, kStepBytes);
          send(j, st, (int)x.z, (int)x.y, (int)x.w >> 16);
        } else {
          mbar_arrive(bar);
        }
      }
      __syncwarp();
      next[j] = k + 1;
      did = true;
    }
    idle = did ? 0 : idle + 1;
    if (more && !did) {
      if (idle > kWaitPolls) {
        if (lane == 0) flag(a.status, MX4_STATUS_TIMEOUT);
        break;
      }
      __nanosleep(32);
    }
  }
  // copies in flight land before the CTA can end
#pragma unroll
  for (int j = 0; j < GP; ++j)
    for (int k = max(0, next[j] - S); k < next[j]; ++k) mbar_wait(full(j) + k % S * 8, (k / S) & 1);
}

// ---------------------------------------------------------------------------

template <int M, int NT, bool Lists>
__global__ void __launch_bounds__(kThreads, 1) fp8_decode_kernel(const __grid_constant__ DecodeArgs a) {
  using Lay = Layout<NT>;
  constexpr int kStages = stages_of(NT), NG = kWarps / M, S = kStages / NG;  // groups, stages of a group
  constexpr int WR = 8 * NT, TR = M * WR;           // rows of a warp, of a tile
  static_assert(S < 32, "the ring of looked-up units holds 64");
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* const sm = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base_at = smem_addr(sm);
  int64_t* const sums = reinterpret_cast<int64_t*>(sm + Lay::kSumOff);
  int2* const seg = reinterpret_cast<int2*>(sm + Lay::kSegOff);
  int4* const jobs = reinterpret_cast<int4*>(sm + Lay::kJobOff);  // [0].x: how many
  int64_t* const pref = reinterpret_cast<int64_t*>(sm + Lay::kPrefOff);
  if (tid < kStages) {
    mbar_init(base_at + Lay::kBarOff + tid * 8, 1);
    mbar_init(base_at + Lay::kBarOff + (kStages + tid) * 8, M);
    fence_barrier_init();
  }
  pdl_wait();
  pdl_launch_dependents();

  // ---- units of the owners before each one
  const int HR = a.Hkv * a.RT;
  auto seq_units = [&](int s) {
    const int L = a.seq_lens[s];
    const bool ok = L >= 0 && L <= a.W * kPageTokens;
    if (!ok && blockIdx.x == 0) flag(a.status, MX4_STATUS_BAD_LEN);
    return ok ? (L + kSub - 1) / kSub : 0;
  };
  Cut cut;
  if (Lists) {
    if (blockIdx.x == 0)
      for (int s = tid; s < a.B; s += kThreads) seq_units(s);
    cut.U = (int64_t)a.B * a.Q * HR * a.kb * kPageSubs;
    __syncthreads();
  } else {
    const int per = (a.B + kThreads - 1) / kThreads;
    const int s0 = min(a.B, tid * per), s1 = min(a.B, s0 + per);
    int64_t sum = 0;
    for (int s = s0; s < s1; ++s) sum += seq_units(s);
    int64_t inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, inc, d);
      if (lane >= d) inc += y;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int64_t before = inc - sum;
    for (int w = 0; w < warp; ++w) before += sums[w];
    for (int s = s0; s < s1; ++s) {
      before += seq_units(s);
      pref[s] = before;
    }
    __syncthreads();
    cut.U = pref[a.B - 1] * HR;
  }
  cut.per = max((cut.U + gridDim.x - 1) / gridDim.x, (int64_t)kMinUnits);

  // ---- owners without units: their rows are empty
  for (int64_t t = blockIdx.x; !Lists && t < (int64_t)a.B * a.Q; t += gridDim.x) {
    const int s = (int)(t / a.Q);
    if (pref[s] != (s ? pref[s - 1] : 0)) continue;
    for (int i = tid; i < a.H * kHeadDim / 8; i += kThreads)
      reinterpret_cast<uint4*>(a.out + t * a.H * kHeadDim)[i] = make_uint4(0, 0, 0, 0);
    if (a.lse)
      for (int i = tid; i < a.H; i += kThreads) a.lse[t * a.H + i] = -INFINITY;
  }

  if (warp >= kWarps) {
    // ================= units of groups warp - 8 and, with eight groups, warp - 4
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
    load_units<NT, Lists, NG, S>(a, cut, pref, HR, base_at, warp - kWarps, lane);
    return;
  }
  // ================= computing
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kComputeRegs));
  const int group = warp / M, wig = warp % M;
  const uint32_t full = base_at + Lay::kBarOff + group * S * 8, empty = full + kStages * 8;
  const uint32_t ring = base_at + group * S * kStepBytes, units = base_at + Lay::kUnitOff + group * 1024;
  const int64_t u0 = cut.group_lo(blockIdx.x, group, NG);
  const int n = (int)(cut.group_lo(blockIdx.x, group + 1, NG) - u0);

  Rows<NT> w;
  w.qs = base_at + Lay::kQOff + warp * NT * 2048 + lane * 16;
  w.er_at = base_at + Lay::kErOff + warp * WR * 4;
  int tile_id = -1, min_lim = 0;  // of the warp's rows: the least last visible token
  bool active = false;            // this warp has rows of the tile
  uint4 q_raw[NT][4];
  auto begin_tile = [&]() {  // its queries on their way
    const Tile tile = tile_of(a, tile_id);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = tile.rt * TR + wig * WR + 8 * t + (lane >> 2);
      const bool real = r < a.R;
      const uint4* const p =
          reinterpret_cast<const uint4*>(a.q + (real ? row_of<Lists>(a, tile, r) : 0) * kHeadDim) + 4 * (lane & 3);
#pragma unroll
      for (int i = 0; i < 4; ++i) q_raw[t][i] = real ? p[i] : make_uint4(0, 0, 0, 0);
    }
  };
  auto base_of = [&](const Tile& tile) {  // position of the owner's first decode token
    const int s = Lists ? a.by_q(tile.owner) : tile.owner;
    return a.seq_lens[s] - a.Q + (Lists ? tile.owner - s * a.Q : 0);
  };
  auto set_tile = [&]() {
    const Tile tile = tile_of(a, tile_id);
    const int r0 = tile.rt * TR + wig * WR;
    active = r0 < a.R;
    min_lim = base_of(tile) + (Lists ? 0 : a.by_g(r0));
    w.set_q(q_raw, a, lane);
    w.clear();
  };

  int head_id = -1;
  bool dead = false, fresh = false;  // fresh: the tile begins in this range
  if (n > 0) {
    int64_t x0;
    if (Lists) {
      const uint32_t per = a.kb * kPageSubs;
      tile_id = (u0 >> 31) ? (int)(u0 / per) : a.by_n((uint32_t)u0);
      x0 = (int64_t)tile_id * per;
    } else {
      const int owner = owner_of(pref, a.B, HR, u0);
      const int64_t before = owner ? pref[owner - 1] : 0;
      const uint32_t per = (uint32_t)(pref[owner] - before), in = (uint32_t)(u0 - before * HR) / per;
      tile_id = owner * HR + (int)in;
      x0 = before * HR + (int64_t)in * per;
    }
    fresh = u0 == x0;
    begin_tile();
    set_tile();
  }
  // the first row of the CTA in scratch memory
  const int64_t cta_row = (int64_t)blockIdx.x * kWarps * WR;
  float4* const scratchmz = reinterpret_cast<float4*>(a.scratch + (int64_t)gridDim.x * kWarps * WR * kHeadDim);
  float4* const recmz = reinterpret_cast<float4*>(a.rec + 2 * (int64_t)gridDim.x * TR * kHeadDim);

  auto write_out = [&]() {
    const Tile tile = tile_of(a, tile_id);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = tile.rt * TR + wig * WR + 8 * t + 2 * (lane & 3) + e;
        if (r >= a.R) continue;
        const int64_t at = row_of<Lists>(a, tile, r);
        const Finish f(w.z[t][e], (float)w.row_er(8 * t + 2 * (lane & 3) + e));
        uint4* const p = reinterpret_cast<uint4*>(a.out + at * kHeadDim + 16 * (lane >> 2));
#pragma unroll
        for (int i = 0; i < 2; ++i)
          p[i] = make_uint4(bf16x2_bits(f(w.o[4 * i][t][e]), f(w.o[4 * i][t][2 + e])),
                            bf16x2_bits(f(w.o[4 * i + 1][t][e]), f(w.o[4 * i + 1][t][2 + e])),
                            bf16x2_bits(f(w.o[4 * i + 2][t][e]), f(w.o[4 * i + 2][t][2 + e])),
                            bf16x2_bits(f(w.o[4 * i + 3][t][e]), f(w.o[4 * i + 3][t][2 + e])));
        if (a.lse && lane < 4) a.lse[at] = row_lse(a, w.m[t][e], w.z[t][e]);
      }
  };

  for (int k = 0, st = 0, phase = 0; k < n; ++k) {
    dead = !__all_sync(0xFFFFFFFFu, mbar_wait(full + st * 8, phase));
    if (dead) break;
    const uint4 uu = lds128(units + (k & 63) * 16);
    const int4 u = make_int4(uu.x, uu.y, uu.z, uu.w);
    if (u.x != tile_id) {  // the tile in front ends inside this range: it is whole, or its last piece
      w.sum_z();
      if (fresh) {
        if (active) write_out();
      } else {
        head_id = tile_id;
        const int64_t row = cta_row + warp * WR;
        w.put(a.scratch + row * kHeadDim, kHeadDim, reinterpret_cast<float*>(scratchmz + row), 4, lane);
      }
      fresh = true;
      tile_id = u.x;
      begin_tile();
      set_tile();
    }
    if (u.z >= 0 && active) {
      const uint32_t ka = ring + st * kStepBytes, va = ka + kSub * kFp8Row;
      const int kb = u.w & 0xFF, vb = (u.w >> 8) & 0xFF;
      if (u.y + kSub - 1 <= min_lim && vb >= w.er + 127 - kFold && vb <= w.cap) {  // (255 is above it)
        w.template step<false>(ka, va, kb, vb, u.y, lane, 0, 0, a);
      } else {
        const Tile tile = tile_of(a, tile_id);
        const int base = base_of(tile), r0 = tile.rt * TR + wig * WR;
        auto lim = [&](int r) { return r0 + r >= a.R ? -1 : Lists ? base : base + a.by_g(r0 + r); };
        w.template step<true>(ka, va, kb, vb, u.y, lane, lim, lim(min(WR, a.R - r0) - 1), a);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty + st * 8);
    if (++st == S) {
      st = 0;
      phase ^= 1;
    }
  }
  if (dead && lane == 0) flag(a.status, MX4_STATUS_TIMEOUT);

  // ---- pieces: each group's last tile is in registers, a tile that it ended inside its range but
  // did not begin in the scratch memory.  Pieces of one tile are joined, in the order of the units.
  if (wig == 0 && lane == 0) seg[group] = make_int2(n > 0 ? tile_id : -1, head_id);
  if (n > 0) w.sum_z();
  compute_sync();  // all stages are read
  float* const mine = reinterpret_cast<float*>(sm) + warp * WR * kRecRow;
  w.put(mine, kRecRow, mine + kHeadDim, kRecRow, lane);
  if (warp == 0) {
    // Lane g has group g.  A job: tile, first and last group with it, the group behind whose first
    // tile it is (or -1), and where the sum goes: 2 the result, else the CTA's piece in rec.
    const int2 sg = lane < NG ? seg[lane] : make_int2(-1, -1);
    const uint32_t some = __ballot_sync(0xFFFFFFFFu, sg.x >= 0);
    const uint32_t below = some & ((1u << lane) - 1);
    const int prev = below ? 31 - __clz(below) : -1;
    const int prev_id = __shfl_sync(0xFFFFFFFFu, sg.x, max(prev, 0));
    const bool lead = sg.x >= 0 && (prev < 0 || prev_id != sg.x);
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, sg.x);
    const int end = 31 - __clz(same);
    const uint32_t above = some & ~((2u << end) - 1);
    const int next = above ? __ffs(above) - 1 : -1;
    const int next_head = __shfl_sync(0xFFFFFFFFu, sg.y, max(next, 0));
    const bool ends = next >= 0 && next_head == sg.x;  // the tile ends in the group behind
    int to = 2, id = sg.x, until = -1;
    if (lead) {
      const int owner = a.by_hr(sg.x);
      int64_t x0, x1;  // the tile's units
      if (Lists) {
        x0 = (int64_t)sg.x * a.kb * kPageSubs;
        x1 = x0 + a.kb * kPageSubs;
      } else {
        const int64_t before = owner ? pref[owner - 1] : 0, units = pref[owner] - before;
        x0 = before * HR + (sg.x - owner * HR) * units;
        x1 = x0 + units;
      }
      const int64_t lo = cut.lo(blockIdx.x), hi = cut.lo(blockIdx.x + 1);
      to = x0 < lo ? 0 : x1 > hi ? 1 : 2;
      if (to == 1) until = (int)((x1 - 1) / cut.per);
    }
    const bool head = prev < 0 && sg.x >= 0 && sg.y >= 0;  // the end of a tile that began in a CTA before
    const uint32_t leads = __ballot_sync(0xFFFFFFFFu, lead), heads = __ballot_sync(0xFFFFFFFFu, head);
    const int at = 1 + __popc(leads & ((1u << lane) - 1)) + (heads ? 1 : 0);
    if (lead) jobs[at] = make_int4(id, lane | (end << 8), ends ? next : -1, to);
    if (head) jobs[1] = make_int4(sg.y, 1 | (0 << 8), lane, 0);
    if (lane == 0) jobs[0].x = __popc(leads) + (heads ? 1 : 0);
    const uint32_t open = __ballot_sync(0xFFFFFFFFu, lead && to == 1);  // at most one
    if (open ? lane == __ffs(open) - 1 : lane == 0) {  // the second kernel joins it with the next CTAs'
      a.meta[2 * blockIdx.x] = open ? id : -1;
      a.meta[2 * blockIdx.x + 1] = until;
    }
  }
  compute_sync();
  constexpr int kRows = 4;  // rows at a time: their loads are in flight together
  const int items = jobs[0].x * (TR / kRows);
  for (int i = warp; i < items; i += kWarps) {
    const int4 job = jobs[1 + i / (TR / kRows)];
    const int r0 = i % (TR / kRows) * kRows, g0 = job.y & 255, g1 = job.y >> 8, tail = job.z;
    const Tile t = tile_of(a, job.x);
    const float* const p = reinterpret_cast<const float*>(sm) + r0 * kRecRow;
    const int64_t tr = cta_row + tail * TR + r0;
    Joined j[kRows];
    float4 tail_mz[kRows], tail_o[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      tail_mz[r] = tail >= 0 ? __ldcg(scratchmz + tr + r) : make_float4(kNoRef, 0.f, kNoScale, 0.f);
      tail_o[r] = tail >= 0 ? __ldcg(reinterpret_cast<const float4*>(a.scratch + (tr + r) * kHeadDim) + lane)
                            : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int x = g0; x <= g1; ++x)  // (a group without units between them has none of the tile)
      if (seg[x].x == job.x)
#pragma unroll
        for (int r = 0; r < kRows; ++r)
          j[r].see(*reinterpret_cast<const float4*>(p + (x * TR + r) * kRecRow + kHeadDim), a.fm);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      j[r].see(tail_mz[r], a.fm);
      j[r].seen();
    }
    for (int x = g0; x <= g1; ++x)
      if (seg[x].x == job.x)
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const float* const y = p + (x * TR + r) * kRecRow;
          j[r].add(*reinterpret_cast<const float4*>(y + 4 * lane), *reinterpret_cast<const float4*>(y + kHeadDim), a.fm);
        }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      j[r].add(tail_o[r], tail_mz[r], a.fm);
      const int row = t.rt * TR + r0 + r;
      if (row >= a.R) continue;
      if (job.w == 2) {
        put_row<Lists>(a, t, row, j[r], lane);
      } else {
        const int64_t at = (2 * (int64_t)blockIdx.x + job.w) * TR + r0 + r;
        *reinterpret_cast<float4*>(a.rec + at * kHeadDim + 4 * lane) = j[r].acc;
        if (lane == 0) recmz[at] = make_float4(j[r].m, j[r].z, j[r].er, 0.f);
      }
    }
  }
}

// Joins the pieces of the tiles that begin in CTA blockIdx.x of the first kernel and end in another:
// two rows a CTA, four warps each.
template <bool Lists>
__global__ void __launch_bounds__(256) fp8_join_kernel(const __grid_constant__ DecodeArgs a, int ctas) {
  __shared__ float4 acc_s[8][32];
  __shared__ float z_s[8];
  pdl_launch_dependents();
  pdl_wait();
  const int id = a.meta[2 * blockIdx.x];
  if (id < 0) return;
  const int last = a.meta[2 * blockIdx.x + 1];
  const Tile t = tile_of(a, id);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp & 3;
  const int r = 2 * blockIdx.y + (warp >> 2), row = t.rt * a.TR + r;
  const float4* const recmz = reinterpret_cast<const float4*>(a.rec + 2 * (int64_t)ctas * a.TR * kHeadDim);
  auto slot = [&](int x) {  // CTA x's piece: its last tile's, or the one that it began in
    return (2 * (int64_t)x + (x == (int)blockIdx.x ? 1 : 0)) * a.TR + r;
  };
  Joined j;
  if (row < a.R) {
    for (int x = blockIdx.x + lane; x <= last; x += 32) j.see(recmz[slot(x)], a.fm);
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      const float x = __shfl_xor_sync(0xFFFFFFFFu, j.m, d);
      j.see(x, __shfl_xor_sync(0xFFFFFFFFu, j.er, d), a.fm);
    }
    j.seen();
#pragma unroll 8
    for (int x = blockIdx.x + part; x <= last; x += 4)
      j.add(*reinterpret_cast<const float4*>(a.rec + slot(x) * kHeadDim + 4 * lane), recmz[slot(x)], a.fm);
  }
  acc_s[warp][lane] = j.acc;
  if (lane == 0) z_s[warp] = j.z;
  __syncthreads();
  if (part != 0 || row >= a.R) return;
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    const float4 v = acc_s[warp + i][lane];
    j.z += z_s[warp + i];
    j.acc.x += v.x;
    j.acc.y += v.y;
    j.acc.z += v.z;
    j.acc.w += v.w;
  }
  put_row<Lists>(a, t, row, j, lane);
}

cudaError_t kv_map(const uint8_t* pages, int64_t page_stride, int64_t head_stride, int64_t num_pages,
                   int Hkv, CUtensorMap* tm) {
  static PFN_cuTensorMapEncodeTiled_v12000 enc = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[4] = {kFp8Row, kPageTokens, (cuuint64_t)Hkv, (cuuint64_t)num_pages};
  const cuuint64_t strides[3] = {kFp8Row, (cuuint64_t)(Hkv > 1 ? head_stride : kFp8Page),
                                 (cuuint64_t)page_stride};
  const cuuint32_t box[4] = {kFp8Row, kSub, 1, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const CUresult r = enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(pages), dims,
                         strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Warps of a group and 8-row columns of a warp: the fewest that hold all rows of an owner and KV
// head.  Three columns a warp at most: q, O and a unit's scores fill the registers.  128 rows a tile
// at most.
struct Shape {
  int M, NT;
};
Shape shape_of(int rows) {
  if (rows <= 24) return {1, (rows + 7) / 8};
  if (rows <= 48) return {2, rows <= 32 ? 2 : 3};
  if (rows <= 96) return {4, rows <= 64 ? 2 : 3};
  return {8, 2};
}

// Workspace: pieces for the second kernel [2 CTAs][TR][128], their m, z, Er [2 CTAs][TR][4],
// scratch of the groups [CTAs][8][8 NT] alike, meta [CTAs][2].
size_t piece_floats(Shape s, int ctas) { return (size_t)ctas * 2 * 8 * s.NT * s.M * kRecRow; }
size_t scratch_floats(Shape s, int ctas) { return (size_t)ctas * kWarps * 8 * s.NT * kRecRow; }

template <int M, int NT, bool Lists>
cudaError_t launch(DecodeArgs a, int64_t B, int num_sms, cudaStream_t stream) {
  auto kern = fp8_decode_kernel<M, NT, Lists>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<NT>::kBytes);
  if (e != cudaSuccess) return e;
  a.TR = 8 * NT * M;
  a.RT = (a.R + a.TR - 1) / a.TR;
  a.by_hr = Div(a.Hkv * a.RT);
  a.by_rt = Div(a.RT);
  a.by_g = Div(a.G);
  a.by_q = Div(a.Q);
  a.by_n = Div(Lists ? a.kb * kPageSubs : 1);
  a.scratch = a.rec + piece_floats({M, NT}, num_sms);
  a.meta = reinterpret_cast<int32_t*>(a.scratch + scratch_floats({M, NT}, num_sms));
  const DecodeArgs all = a;
  const int64_t step = Lists ? B : kMaxOwners;  // lists take no prefix sums
  for (int64_t b0 = 0; b0 < B; b0 += step) {
    a = all;
    a.B = (int)std::min<int64_t>(step, B - b0);
    a.q += b0 * a.Q * a.H * kHeadDim;
    a.out += b0 * a.Q * a.H * kHeadDim;
    if (a.lse) a.lse += b0 * a.Q * a.H;
    a.table += b0 * a.W;
    a.seq_lens += b0;
    e = launch_pdl(kern, dim3(num_sms), dim3(kThreads), Layout<NT>::kBytes, stream, a);
    if (e != cudaSuccess) return e;
    e = launch_pdl(fp8_join_kernel<Lists>, dim3(num_sms, a.TR / 2), dim3(256), 0, stream, a, num_sms);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <bool Lists>
cudaError_t launch_shape(const DecodeArgs& a, int64_t B, int num_sms, cudaStream_t stream) {
  const Shape s = shape_of(a.R);
  switch (s.M * 8 + s.NT) {
    case 8 + 1: return launch<1, 1, Lists>(a, B, num_sms, stream);
    case 8 + 2: return launch<1, 2, Lists>(a, B, num_sms, stream);
    case 8 + 3: return launch<1, 3, Lists>(a, B, num_sms, stream);
    case 16 + 2: return launch<2, 2, Lists>(a, B, num_sms, stream);
    case 16 + 3: return launch<2, 3, Lists>(a, B, num_sms, stream);
    case 32 + 2: return launch<4, 2, Lists>(a, B, num_sms, stream);
    case 32 + 3: return launch<4, 3, Lists>(a, B, num_sms, stream);
    default: return launch<8, 2, Lists>(a, B, num_sms, stream);
  }
}

}  // namespace

size_t fp8_decode_workspace_bytes(int rows, int num_sms) { 
  const Shape s = shape_of(rows);
  return (piece_floats(s, num_sms) + scratch_floats(s, num_sms)) * 4 + (size_t)num_sms * 2 * sizeof(int32_t);
}

cudaError_t launch_fp8_decode(const uint16_t* q, int64_t B, int Q, int H, int Hkv,
                              const uint8_t* k_pages, const uint8_t* v_pages, const uint8_t* k_scales,
                              const uint8_t* v_scales, int64_t page_stride, int64_t head_stride,
                              int64_t num_pages, const int32_t* block_table, int64_t bt_width,
                              const int32_t* seq_lens, const int32_t* block_idx, int kb, float scale,
                              uint16_t* out, float* lse, void* ws, uint32_t* status, int num_sms,
                              cudaStream_t stream) {
  DecodeArgs a{};
  cudaError_t e = kv_map(k_pages, page_stride, head_stride, num_pages, Hkv, &a.kmap);
  if (e == cudaSuccess) e = kv_map(v_pages, page_stride, head_stride, num_pages, Hkv, &a.vmap);
  if (e != cudaSuccess) return e;
  a.q = q;
  a.ks = k_scales;
  a.vs = v_scales;
  a.table = block_table;
  a.W = bt_width;
  a.seq_lens = seq_lens;
  a.idx = block_idx;
  a.kb = kb;
  a.num_pages = num_pages;
  a.Q = Q;
  a.H = H;
  a.Hkv = Hkv;
  a.G = H / Hkv;
  a.R = block_idx ? a.G : Q * a.G;
  a.negative = scale < 0.f;
  const double factor = std::fabs((double)scale) * 1.4426950408889634;
  a.fe = factor == 0.0 ? -4096 : std::ilogb(factor);
  a.fm = factor == 0.0 ? 1.f : (float)std::scalbn(factor, -a.fe);
  a.lazy = kLazy / a.fm;
  a.fl = (float)((factor == 0.0 ? 1.0 : std::scalbn(factor, -a.fe)) * 0.6931471805599453);
  a.out = out;
  a.lse = lse;
  a.rec = static_cast<float*>(ws);
  a.status = status;
  return block_idx ? launch_shape<true>(a, B, num_sms, stream) : launch_shape<false>(a, B, num_sms, stream);
}

}  // namespace mx4
